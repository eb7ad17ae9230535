"""Paged caches and packed prompts at the edges of what their definitions allow."""
import ctypes
import functools
import math
import os
import re
import subprocess
import time

import pytest
import torch

from long_context_token_b200 import build, hs2

from _paged_ref import Pool, TYPES, attend, check, quantise
from test_paged import DEV, L, P, _kv, cache_of, check_prompts, check_step, cu_of, same  # noqa: F401 (L is a fixture)


# ---------------------------------------------------------------- the host's checks (CPU)
@pytest.mark.parametrize("scale,code", [(3e38, 1), (2.36e38, 1), (-0.0, 1), (2.3e38, 3), (1e-45, 3)])
def test_scales_that_float32_cannot_hold_in_log2_units_are_refused(L, scale, code):  # noqa: F811
    """(A workspace that is too small, the last check, keeps the good ones from running.)"""
    kv = _kv()
    assert L.hs2_paged_attn(P, 0, 16, 2048, 128, ctypes.byref(kv), scale, P, P, P, 16, None) == code
    p = hs2.Packed(P, P, P, P, P, 1024, 128, 256, 128, 10, 20, 2, 8, 2, 128, 0)
    assert L.hs2_packed_attn(ctypes.byref(p), scale, P, P, P, 16, None) == code


def test_step_kernels_are_built_with_the_registers_that_they_share_out(tmp_path):
    """Their warps take and give back registers of those that the block was launched with."""
    source = os.path.join(build.CSRC, "paged_attn.cu")
    text = open(source).read()
    launch, consumers, producers = map(int, re.search(
        r"kLaunchRegs = (\d+), kConsumerRegs = (\d+), kProducerRegs = (\d+);", text).groups())
    assert 256 * consumers + 128 * producers <= 384 * launch
    flags = [f for f in build.NVCC_FLAGS if f not in ("-lineinfo", "--threads", "0")]
    out = subprocess.run([build.nvcc(), *flags, "-I", os.path.join(build.ROOT, "include"), "-Xptxas", "-v",
                          "-cubin", "-o", str(tmp_path / "step.cubin"), source], capture_output=True, text=True)
    assert out.returncode == 0, out.stderr
    used = re.findall(r"Compiling entry function '\w*paged_attn_kernel\w*'.*?Used (\d+) registers", out.stderr, re.S)
    assert len(used) == 32 and set(map(int, used)) == {launch}


# ---------------------------------------------------------------- on the GPU

def half(dtype):
    return torch.finfo(dtype).eps / 2


def bound(o, w_abs_v, mag, n, out_type, weight_type, lost=0.0):
    """How far a result may be from its definition: a float32 logit is off by at most
    e = 160 * 2^-24 of `mag` (the largest sum |q_i k_i| * scale) + 1, which moves a weight and the
    sum of the weights by at most 2.1 e each; a weight is rounded once; the products of 16 keys
    at a time enter the sum one after another, each addition off by at most 2^-23 of what it has
    (the weights' own sum the same); the quotient's two roundings and the result's own.  `lost`:
    what roundings of weights below the normal numbers of their type may add up to."""
    e = 160 * 2.0 ** -24 * (mag + 1)
    rel = half(weight_type) + 4.2 * e + 2 * (n / 16 + 8) * 2.0 ** -23
    own = half(out_type) * (o.abs() + rel * w_abs_v + lost) + torch.finfo(out_type).smallest_normal * half(out_type)
    return rel * w_abs_v + lost + own


@pytest.mark.gpu
def test_read_counts_its_rows_on_the_stream_it_is_given():
    """The offsets are written on the stream that the read is given, behind other work there."""
    lens = [130, 7]
    pool = Pool(lens, 2, 64, 16, "f16", seed=50)
    cache = cache_of(pool)
    ws = hs2.paged_workspace(cache)
    want = cu_of(lens).to(DEV)
    cu = torch.zeros_like(want)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)  # about 50 ms
        cu.copy_(want)
    k, v = hs2.paged_kv_read(cache, cu, ws, stream=s)
    torch.cuda.synchronize()
    assert hs2.check_device_status(ws) == 0
    assert k.shape == v.shape == (137, 2, 64)
    for i, got in enumerate((k, v)):
        assert same(got, torch.cat([pool.rows(b, 0, n)[i] for b, n in enumerate(lens)]).half())


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("h_q", [2, 16, 40])
def test_step_of_a_query_with_an_infinity_over_codes(d, h_q):
    """Logits that are all -inf give zeros and -inf, ones of both signs NaN; a finite element
    beside the infinity, however large, changes neither, and no other head sees them."""
    pool = Pool([700, 40], 1, d, 16, "fp8", seed=51)
    pg, r = pool.at(0, 0, 700)
    pool.k[pg, :, r, 9] = 0x38  # 1.0
    q = torch.randn(2, h_q, d, generator=torch.Generator().manual_seed(52)).to(torch.bfloat16)
    q[0, 0, 9] = q[1, 1, 9] = -math.inf
    q[0, 0, 3] = 3e38
    cache = cache_of(pool)
    ws = hs2.paged_workspace(cache, h_q)
    out, lse = (x.cpu() for x in hs2.paged_attn(q.to(DEV), cache, ws))
    assert hs2.check_device_status(ws) == 0
    assert bool((out[0, 0] == 0).all()) and bool(lse[0, 0] == -math.inf)
    assert bool(torch.isnan(out[1, 1]).all()) and bool(torch.isnan(lse[1, 1]))
    scale = float(torch.tensor(1 / math.sqrt(d), dtype=torch.float32))
    for b, n in enumerate(pool.lens):
        k, v = pool.rows(b, 0, n)
        for h in range(h_q):
            if (b, h) not in ((0, 0), (1, 1)):
                ref = attend(q[b, h:h + 1].double(), k[:, 0], v[:, 0], scale, torch.tensor([n]))
                check(out[b, h:h + 1], lse[b, h:h + 1], ref, torch.bfloat16, torch.float16, n)


def sinks(n, d, h_kv, h_q, gap, every, dtype, seed):
    """Rows of n keys of which one, or one of `every`, has a logit `gap` above all others'
    (which are 0) and a V of zeros: the result is what the others add up to.  sm_scale is 1."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randn(1, h_q, d, generator=g)
    q[..., 0] = 1.0
    k = torch.zeros(n, h_kv, d)
    v = torch.rand(n, h_kv, d, generator=g) * 1000 + 500
    at = torch.arange(0, n, every or n)
    k[at, :, 0] = gap
    v[at] = 0
    return q.to(dtype), k.to(dtype), v.to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d,h_q,h_kv,gap,every", [(128, 4, 2, 18.5, None), (128, 4, 1, 18.5, 7),
                                                  (64, 16, 16, 17.0, 5), (64, 34, 2, 12.0, None)])
def test_small_weights_of_long_contexts_count(dtype, d, h_q, h_kv, gap, every):
    """Weights down to 2^-27 of the largest.  A float16 weight below 2^-14 is off by at most
    2^-25, and the largest lies in [2^7, 2^15]: 2^-32 of it.  The step over pages, and queries
    after a prefix (one and two tiles per work item)."""
    n, dt = 50001, TYPES[dtype]
    q, k, v = sinks(n, d, h_kv, h_q, gap, every, dt, seed=53)
    g = h_q // h_kv

    def hold(out, lse, n):
        for h in range(h_kv):
            hs = slice(h * g, (h + 1) * g)
            vv = v[:n, h].double()
            o, z, a, mag = attend(q[0, hs].double(), k[:n, h].double(), vv, 1.0, torch.full((g,), n))
            lost = 2.0 ** -32 * torch.exp(gap - z)[:, None] * vv.sum(0) if dtype == "f16" else 0.0
            assert bool(((out[hs].cpu().double() - o).abs() <= bound(o, a, mag, n, dt, dt, lost)).all())
            assert bool(((lse[hs].cpu().double() - z).abs() <= 1e-3).all())

    cache = cache_of(Pool([n], h_kv, d, 64, dtype, seed=54, empty=True))
    ws, pws = hs2.paged_workspace(cache, h_q), hs2.packed_workspace(DEV)
    kd, vd = k.to(DEV), v.to(DEV)
    hs2.paged_kv_write(kd, vd, cache, ws)
    out, lse = hs2.paged_attn(q.to(DEV), cache, ws, 1.0)
    hold(out[0], lse[0], n)
    # (the last of three queries sees all keys)
    out, lse = hs2.packed_attn(q.to(DEV).repeat(3, 1, 1), kd, vd, cu_of([3]).to(DEV), cu_of([n]).to(DEV), pws, 1.0)
    hold(out[2], lse[2], n)
    reps, short = 150, 3001  # the same keys for many sequences: more work items than SMs
    cu = torch.arange(reps + 1, dtype=torch.int32, device=DEV)
    out, lse = hs2.packed_attn(q.to(DEV).repeat(reps, 1, 1), kd[:short].repeat(reps, 1, 1),
                               vd[:short].repeat(reps, 1, 1), cu, cu * short, pws, 1.0)
    for b in (0, reps - 1):
        hold(out[b], lse[b], short)
    assert hs2.check_device_status(ws) == 0 and hs2.check_device_status(pws) == 0


def check_codes(pool, q, out, lse, scale, what=""):
    """Results over an FP8 pool.  A weight times its V scale is off by half a step of float16,
    or by 2^-32 of the largest such product over rows of V that are not all zeros."""
    g = q.shape[1] // pool.h_kv
    for b, n in enumerate(pool.lens):
        k, v = pool.rows(b, 0, n)
        pg, r = pool.at(b, 0, n)
        for h in range(pool.h_kv):
            hs = slice(h * g, (h + 1) * g)
            qq = q[b, hs].double()
            o, z, a, mag = attend(qq, k[:, h], v[:, h], scale, torch.full((g,), n))
            w = torch.exp((qq @ k[:, h].T) * scale - z[:, None])  # [g, n]
            vs = pool.v_scale[pg, h, r].double()
            codes = pool.v[pg, h, r].view(torch.float8_e4m3fn).double().abs()
            live = codes.amax(-1) > 0
            top = (w * vs * live).amax(-1) if n else torch.zeros(g).double()
            lost = 2.0 ** -32 * top[:, None] * codes.sum(0)
            lim = bound(o, a, mag, n, q.dtype, torch.float16, lost)
            off = (out[b, hs].cpu().double() - o).abs()
            assert bool((off <= lim).all()), f"{what} sequence {b}, head {h}: {(off / lim).max().item()} of the bound"
            # the weights' float32 sum, and the logits' own error
            far = 4.2 * 160 * 2.0 ** -24 * (mag + 1) + (n / 16 + 8) * 2.0 ** -23 + 2.0 ** -20 * (1 + z.abs())
            assert bool(((lse[b, hs].cpu().double() - z).abs() <= far).all()), what


@pytest.mark.gpu
@pytest.mark.parametrize("d,h_q,h_kv", [(128, 8, 1), (64, 4, 2), (128, 32, 1)])
@pytest.mark.parametrize("gap", [12.8, 13.5, 25.0, 40.0])
def test_zero_rows_of_v_take_nothing_from_the_others(d, h_q, h_kv, gap):
    """The library's own write gives a row of zeros the scale 1, a hundred times an ordinary
    row's.  Such a row under a dominant logit (a sink) leaves the other keys their weights:
    one in a cut sequence, some in whole ones, and a sequence that has no other rows."""
    lens = [100000, 300, 33, 5000]
    pool = Pool(lens, h_kv, d, 32, "fp8", seed=55, empty=True)
    g = torch.Generator().manual_seed(56)
    t = sum(lens)
    k, v = (torch.randn(t, h_kv, d, generator=g) for _ in range(2))
    k[..., 0] = 0
    zero = [0, 100000 + 20, 100000 + 299] + list(range(100300, 100333)) + list(range(100333, 105333, 7))
    k[zero] = 0
    k[zero, :, 0] = gap / 2
    v[zero] = 0
    q = torch.randn(len(lens), h_q, d, generator=g) * 0.03
    q[..., 0] = 2.0
    q, k, v = (x.to(torch.bfloat16) for x in (q, k, v))
    cache = cache_of(pool)
    ws = hs2.paged_workspace(cache, h_q)
    hs2.paged_kv_write(k.to(DEV), v.to(DEV), cache, ws, cu_new=cu_of(lens).to(DEV))
    pool.k, pool.v, pool.k_scale, pool.v_scale = (x.cpu() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale))
    assert bool((pool.v_scale[pool.at(0, 0, 1)[0], :, pool.at(0, 0, 1)[1]] == 1).all())
    out, lse = hs2.paged_attn(q.to(DEV), cache, ws, 1.0)
    assert hs2.check_device_status(ws) == 0
    check_codes(pool, q, out, lse, 1.0, f"gap {gap}")
    assert bool((out[2] == 0).all())
    # negative zeros are zeros
    cache.v[(cache.v == 0)] = 0x80
    out2, lse2 = hs2.paged_attn(q.to(DEV), cache, ws, 1.0)
    assert same(lse2, lse.cpu()) and torch.equal(out2, out)


@pytest.mark.gpu
@pytest.mark.parametrize("d,h_q,h_kv", [(128, 8, 1), (64, 34, 2)])
def test_scales_of_v_mixed_within_a_sequence(d, h_q, h_kv):
    """V scales over 2^-20 .. 2^20 within each sequence, under flat and under steep logits, and
    a row of small codes with a large scale beside rows of large codes with small ones."""
    for flat in (True, False):
        pool = Pool([60000, 333, 32], h_kv, d, 16, "fp8", seed=57)
        g = torch.Generator().manual_seed(58)
        for b, n in enumerate(pool.lens):
            pg, r = pool.at(b, 0, n)
            pool.v_scale[pg, :, r] = 2.0 ** (40 * torch.rand(n, h_kv, generator=g) - 20)
            if b == 0:  # most rows' scales are 2^-27 of some that are zero except in their first elements
                pool.v_scale[pg, :, r] = 2.0 ** -27
                pool.v[pg, :, r] = 0x7E  # 448
                one, row = pg[5::32], r[5::32]
                pool.v_scale[one, :, row] = 1.0
                pool.v[one, :, row] = 0
                pool.v[one, :, row, :3] = 0x38
        q = torch.randn(3, h_q, d, generator=g).to(torch.bfloat16) * (0.0 if flat else 1.0)
        cache = cache_of(pool)
        ws = hs2.paged_workspace(cache, h_q)
        out, lse = hs2.paged_attn(q.to(DEV), cache, ws)
        assert hs2.check_device_status(ws) == 0
        check_codes(pool, q, out, lse, float(torch.tensor(1 / math.sqrt(d), dtype=torch.float32)), f"flat {flat}")


CUT = [  # (h_q, h_kv, d, lengths) whose sequences are cut into many parts, joined at once or in groups
    (16, 1, 128, [131072] * 2), (3, 1, 64, [90001, 1, 100000]), (64, 1, 128, [120011, 3]),
    (128, 1, 64, [70001]), (20, 1, 128, [150000]), (4, 4, 64, [9001, 77, 0, 12345]), (8, 2, 128, [40000, 1333]),
]
BLOCK = 97  # keys in a row with the same V


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "f16", "fp8"])
@pytest.mark.parametrize("h_q,h_kv,d,lens", CUT)
def test_every_part_of_a_cut_sequence_counts_once(kv, h_q, h_kv, d, lens):
    """Each V row is 1 in one element, which moves with the key and the head.  Under equal
    logits every sum is a whole number that float32 holds, so a result is the count of its
    keys over their number, rounded; a lost, doubled or misplaced part of a sequence moves
    many elements by a tenth.  Under random logits the results stay sums of positive terms,
    held by their relative error alone."""
    pool = Pool(lens, h_kv, d, 32, kv, seed=59)
    for b, n in enumerate(lens):
        if n == 0:
            continue
        pg, r = pool.at(b, 0, n)
        at = (torch.arange(n)[:, None] // BLOCK + 5 * torch.arange(h_kv) + b) % d  # [n, h_kv]
        hot = torch.nn.functional.one_hot(at, d)
        if kv == "fp8":
            pool.v[pg, :, r] = (hot * 0x38).to(torch.uint8)
            pool.v_scale[pg, :, r] = 1.0
        else:
            pool.v[pg, :, r] = hot.to(pool.v.dtype)
    cache = cache_of(pool)
    ws = hs2.paged_workspace(cache, h_q)
    qt = torch.float16 if kv == "f16" else torch.bfloat16
    wt = torch.float16 if kv == "fp8" else qt
    scale = float(torch.tensor(1 / math.sqrt(d), dtype=torch.float32))
    g = h_q // h_kv
    for flat in (True, False):
        q = torch.randn(len(lens), h_q, d, generator=torch.Generator().manual_seed(60)).to(qt) * (0.0 if flat else 1.0)
        out, lse = (x.cpu().double() for x in hs2.paged_attn(q.to(DEV), cache, ws))
        assert hs2.check_device_status(ws) == 0
        for b, n in enumerate(lens):
            if n == 0:
                assert bool((out[b] == 0).all())
                continue
            k, v = pool.rows(b, 0, n)
            for h in range(h_kv):
                hs = slice(h * g, (h + 1) * g)
                if flat:  # a reciprocal, a product and a rounding to 16 bits
                    want = v[:, h].sum(0).expand(g, d) / n
                    lim = (half(qt) + 2.0 ** -22) * want + 2.0 ** -25
                    assert bool(((lse[b, hs] - math.log(n)).abs() < 1e-5).all())
                else:
                    want, z, _, mag = attend(q[b, hs].double(), k[:, h], v[:, h], scale, torch.full((g,), n))
                    lim = bound(want, want, mag, n, qt, wt, n * 2.0 ** -32 if wt == torch.float16 else 0.0)
                    assert bool((lim < 0.02 * want + 1e-4).all())  # a part is a hundredth of a sequence, at least
                off = (out[b, hs] - want).abs()
                assert bool((off <= lim).all()), f"sequence {b}, head {h}, flat {flat}"


def positive(n, d, dtype, shape, seed, dead=0):
    """Queries, keys and a V of positive elements on the device, and the definition's results in
    float64.  shape "even": logits of order 1; "rising", "falling": by 40 along the keys; the
    first `dead` keys have logits of -inf."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = torch.randn(4, d, device=DEV, generator=g)
    k = torch.randn(n, d, device=DEV, generator=g)
    v = (torch.rand(n, d, device=DEV, generator=g) + 0.5).to(dtype)
    q[:, 0] = 1.0
    k[:, 0] = torch.linspace(-20, 20, n, device=DEV) * {"even": 0, "rising": 1, "falling": -1}[shape] * math.sqrt(d)
    q, k = q.to(dtype), k.to(dtype)
    k[:dead, 0] = -math.inf
    return q, k, v


def long_reference(q, k, v):
    scale = float(torch.tensor(1 / math.sqrt(q.shape[1]), dtype=torch.float32))
    x = (q.double() @ k.double().T) * scale
    z = torch.logsumexp(x, -1)
    mag = float((q.abs().double() @ k.nan_to_num(neginf=0.0).abs().double().T).max()) * scale
    return torch.exp(x - z[:, None]) @ v.double(), z, mag


def hold_long(out, lse, ref, dtype, weight_type, drained, n, what):
    """The sums of positive terms.  The tensor cores cut what they add: each of 16 products by
    less than 2^-25 of the sum so far and the sum by less than 2^-23 of it, over `drained` keys;
    what they have summed is then added in float32 (half a unit of 2^-23 each time)."""
    o, z, mag = ref
    cut = drained / 16 * (2.0 ** -21 + 2.0 ** -23) + (n / drained + 8) * 2.0 ** -24
    rel = half(weight_type) + 4.2 * 160 * 2.0 ** -24 * (mag + 1) + cut + half(dtype)
    off = ((out.double() - o) / o).abs().max().item()
    assert off <= rel * (1 + 2.0 ** -8), f"{what}: off by {off}, {off / rel} of the bound"
    assert float((lse.double() - z).abs().max()) <= 4.2 * 160 * 2.0 ** -24 * (mag + 1) + 2.0 ** -14, what


@pytest.mark.gpu
@pytest.mark.parametrize("tiles", [1, 2])
@pytest.mark.parametrize("dtype,d,n,shape,dead", [
    ("f16", 64, 2 ** 20, "even", 0), ("f16", 128, 2 ** 20 - 77, "even", 0), ("bf16", 64, 2 ** 22, "even", 0),
    ("bf16", 128, 300000, "rising", 0), ("f16", 64, 300001, "falling", 0), ("f16", 128, 200000, "even", 50000),
    ("bf16", 64, 16384 + 1, "even", 0), ("f16", 128, 2 * 16384, "even", 0)])
def test_prompt_sums_over_long_sequences(dtype, d, n, shape, dead, tiles):
    """A query behind up to 2^22 keys, in items of one and (among many empty sequences) two tiles."""
    q, k, v = positive(n, d, TYPES[dtype], shape, 61, dead)
    ref = long_reference(q, k, v)
    batch = 1 if tiles == 1 else 200
    cu_q, cu_k = (torch.tensor([0] * (batch // 2) + [m] * (batch - batch // 2 + 1), dtype=torch.int32, device=DEV)
                  for m in (1, n))
    cu_q[0] = cu_k[0] = 0
    ws = hs2.packed_workspace(DEV)
    out, lse = hs2.packed_attn(q[None], k[:, None], v[:, None], cu_q, cu_k, ws)
    assert hs2.check_device_status(ws) == 0
    hold_long(out[0], lse[0], ref, TYPES[dtype], TYPES[dtype], 16384, n, f"{shape}, {tiles} tiles")


@pytest.mark.gpu
@pytest.mark.parametrize("kv,d,group,n,shape,dead", [
    ("f16", 64, 128, 2 ** 20, "even", 0), ("fp8", 64, 100, 2 ** 20, "even", 0), ("bf16", 128, 40, 2 ** 19, "rising", 0),
    ("f16", 128, 20, 2 ** 18, "falling", 0), ("f16", 64, 4, 2 ** 20, "even", 0), ("f16", 64, 12, 2 ** 19, "even", 0),
    ("f16", 64, 128, 100000, "even", 30000)])
def test_step_sums_over_long_sequences(kv, d, group, n, shape, dead):
    """160 sequences on the same pages, so that a CTA takes about a whole one."""
    dt, batch, page = (torch.bfloat16 if kv == "bf16" else torch.float16), 160, 64
    q, k, v = positive(n, d, dt, shape, 62, dead)
    num = -(-n // page)
    shape4 = (num, 1, page, d)
    scales = ()
    if kv == "fp8":
        kc, ks = quantise(k.cpu())
        vc, vs = quantise(v.cpu())
        pools = [torch.zeros(shape4, dtype=torch.uint8, device=DEV) for _ in range(2)]
        scales = [torch.zeros(shape4[:3], device=DEV) for _ in range(2)]
        for p, s, c, x in zip(pools, scales, (kc, vc), (ks, vs)):
            p.view(-1, d)[:n], s.view(-1)[:n] = c.to(DEV), x.to(DEV)
        k, v = ((c.view(torch.float8_e4m3fn).double() * x.double()[:, None]).to(DEV) for c, x in ((kc, ks), (vc, vs)))
    else:
        pools = [torch.zeros(shape4, dtype=dt, device=DEV) for _ in range(2)]
        for p, x in zip(pools, (k, v)):
            p.view(-1, d)[:n] = x
    ref = long_reference(q, k, v)
    pages = torch.arange(num, dtype=torch.int32, device=DEV).repeat(batch, 1)
    lens = torch.full((batch,), n, dtype=torch.int32, device=DEV)
    cache = hs2.PagedCache(*pools, pages, lens, *scales)
    ws = hs2.paged_workspace(cache, group)
    heads = q.repeat(group // 4, 1)[None].repeat(batch, 1, 1)
    out, lse = hs2.paged_attn(heads, cache, ws)
    assert hs2.check_device_status(ws) == 0
    for b in (0, 1, batch // 2, batch - 1):
        for h in range(0, group, 4):
            hold_long(out[b, h:h + 4], lse[b, h:h + 4], ref, dt, torch.float16 if kv == "fp8" else dt, 16384, n,
                      f"{shape}, sequence {b}, head {h}")


@pytest.mark.gpu
@pytest.mark.parametrize("batch", [1, 200])  # one and two tiles per work item
def test_a_sequence_that_one_block_walks_for_a_second(batch):
    """2^26 keys, the most of a sequence (rows 16 bytes apart, so that they fit): no wait gives
    up.  Equal logits and a V of ones: sums of 16384 keys are exact, and so are their sums.  Four
    times as many are refused; the first 2^26 still give the same."""
    n, d = 2 ** 28, 64
    k = torch.zeros(8 * n + d, dtype=torch.bfloat16, device=DEV).as_strided((n, 1, d), (8, d, 1))
    v = torch.ones(8 * n + d, dtype=torch.bfloat16, device=DEV).as_strided((n, 1, d), (8, d, 1))
    q = torch.randn(1, 1, d, device=DEV).to(torch.bfloat16)
    ws = hs2.packed_workspace(DEV)
    for m, code in ((2 ** 26, 0), (n, 7)):
        cu_q, cu_k = (torch.tensor([0] + [x] * batch, dtype=torch.int32, device=DEV) for x in (1, m))
        out, lse = hs2.packed_attn(q, k, v, cu_q, cu_k, ws)
        assert hs2.check_device_status(ws) == code
        assert bool((out == 1).all()) and abs(lse.item() - math.log(2 ** 26)) < 1e-4


@pytest.mark.gpu
def test_waits_that_run_out_are_reported_and_end():
    """With no loads issued, every warp that waits for one gives up once and the kernels wind
    down: partial results and counters too, so that the calls after them need only a clean
    status.  (Prompts in items of one and of two tiles, a step in parts and in groups of them.)"""
    lib = hs2.lib()
    step = Pool([40000, 300, 0], 1, 128, 32, "bf16", seed=63)
    q = torch.randn(3, 16, 128, generator=torch.Generator().manual_seed(64)).to(torch.bfloat16)
    cache = cache_of(step)
    ws, pws = hs2.paged_workspace(cache, 16), hs2.packed_workspace(DEV)
    prompts = []
    for heads, lens in (((4, 2), [300, 1]), ((40, 40), [300, 70, 0, 129])):
        x = torch.randn(sum(lens), heads[0] + 2 * heads[1], 64, generator=torch.Generator().manual_seed(65)).half()
        prompts.append((x[:, :heads[0]], x[:, heads[0]:sum(heads)], x[:, sum(heads):], lens))

    def prompt(a, k, v, lens):
        return hs2.packed_attn(a.to(DEV), k.to(DEV), v.to(DEV), cu_of(lens).to(DEV), workspace=pws)

    calls = [(ws, lambda: hs2.paged_attn(q.to(DEV), cache, ws))] + \
        [(pws, functools.partial(prompt, *p)) for p in prompts]
    for w, call in calls:
        lib.hs2_debug_stall_waits(1)
        try:
            begin = time.monotonic()
            call()
            torch.cuda.synchronize()
            took = time.monotonic() - begin
        finally:
            lib.hs2_debug_stall_waits(0)
        assert hs2.check_device_status(w) == 5
        assert took < 12, f"{took} s to give up"
        assert hs2.check_device_status(w) == 0
        w.zero_()
    check_step(step, q, *calls[0][1]())
    for (a, k, v, lens), (w, call) in zip(prompts, calls[1:]):
        out, lse = call()
        check_prompts(a, k, v, lens, lens, out, lse)
    assert hs2.check_device_status(ws) == 0 and hs2.check_device_status(pws) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d,h_q,h_kv", [("f16", 64, 2, 1), ("bf16", 128, 6, 2), ("f16", 128, 7, 7)])
def test_prompts_longer_than_one_sum(dtype, d, h_q, h_kv):
    """Whole prompts of more keys than are summed at once: the queries around the first ones that
    see 16384 and 32768 keys, whose two tiles leave the sum at different steps, and the last."""
    lens = [33000, 16385, 300]
    t, dt = sum(lens), TYPES[dtype]
    g = torch.Generator(device=DEV).manual_seed(66)
    q, k = (torch.randn(t, h, d, device=DEV, generator=g).to(dt) for h in (h_q, h_kv))
    v = (torch.rand(t, h_kv, d, device=DEV, generator=g) + 0.5).to(dt)
    ws = hs2.packed_workspace(DEV)
    out, lse = hs2.packed_attn(q, k, v, cu_of(lens).to(DEV), workspace=ws)
    assert hs2.check_device_status(ws) == 0
    scale = float(torch.tensor(1 / math.sqrt(d), dtype=torch.float32))
    at = 0
    for n in lens:
        for lo in (0, 16200, 16384, 32700, n - 130):
            hi = min(lo + 140, n)
            if lo >= hi or lo < 0:
                continue
            rows, seen = slice(at + lo, at + hi), torch.arange(lo, hi, device=DEV)[:, None]
            for h in range(h_q):
                qq, kk, vv = q[rows, h].double(), k[at:at + hi, h * h_kv // h_q].double(), v[at:at + hi, h * h_kv // h_q].double()
                x = torch.where(torch.arange(hi, device=DEV) <= seen, (qq @ kk.T) * scale, -math.inf)
                z = torch.logsumexp(x, -1)
                ref = torch.exp(x - z[:, None]) @ vv, z, float((qq.abs() @ kk.abs().T).max()) * scale
                hold_long(out[rows, h], lse[rows, h], ref, dt, dt, 16384, n, f"prompt of {n}, from {lo}, head {h}")
        at += n
