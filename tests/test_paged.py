"""Paged caches and packed prompts: every operator against its float64 definition, the
refusals, and a run of them together.  GPU tests except for the host's checks."""
import ctypes
import math

import pytest
import torch

from long_context_token_b200 import build, hs2

from _paged_ref import Pool, TYPES, attend, check, quantise

DEV = "cuda:0"


# ---------------------------------------------------------------- the host's checks (CPU)
@pytest.fixture(scope="module")
def L():
    build.build()
    return hs2.lib()


P = 1 << 20  # an aligned address that no host check dereferences


def _kv(**kw):
    f = dict(k=P, v=P, k_scale=None, v_scale=None, pages=P, lens=P, page_stride=8 * 16 * 128,
             head_stride=16 * 128, row_stride=128, scale_page_stride=128, scale_head_stride=16,
             scale_row_stride=1, batch=2, max_pages=4, num_pages=9, page_size=16, n_kv_heads=8,
             head_dim=128, dtype=0)
    f.update(kw)
    return hs2.PagedKV(**f)


BAD_CACHES = [
    (dict(k=None), 1), (dict(pages=None), 1), (dict(lens=None), 1),
    (dict(k=P + 8), 1),                                # misaligned rows
    (dict(row_stride=132), 1), (dict(head_stride=-128), 1),  # not whole 16 bytes; negative
    (dict(row_stride=64), 1),                          # rows overlap
    (dict(batch=0), 1), (dict(max_pages=0), 1), (dict(num_pages=0), 1), (dict(n_kv_heads=0), 1),
    (dict(k_scale=P, v_scale=P), 1),                   # a 16-bit cache with scales
    (dict(dtype=1), 1), (dict(dtype=1, k_scale=P), 1),  # FP8 without its scales
    (dict(dtype=1, k_scale=P + 2, v_scale=P), 1),
    (dict(dtype=3), 2), (dict(head_dim=96), 2), (dict(page_size=4), 2), (dict(page_size=24), 2),
    (dict(page_size=512), 2), (dict(batch=65536), 2), (dict(max_pages=1 << 27), 2),
]


@pytest.mark.parametrize("change,code", BAD_CACHES)
def test_every_paged_call_refuses_a_bad_cache(L, change, code):
    kv = ctypes.byref(_kv(**change))
    big = 1 << 40
    assert L.hs2_paged_workspace_bytes(kv, 16) == 0
    assert L.hs2_paged_kv_write(P, P, 0, 1024, 128, 2, P, kv, P, big, None) == code
    assert L.hs2_paged_kv_read(kv, P, None, 2, P, P, 0, 1024, 128, P, big, None) == code
    assert L.hs2_paged_attn(P, 0, 16, 2048, 128, kv, 0.1, P, P, P, big, None) == code


def test_paged_workspace_sizes(L):
    kv = ctypes.byref(_kv())
    assert 4 <= L.hs2_paged_workspace_bytes(kv, 0) <= 512
    # the same for every batch and page table: one workspace serves calls of any sizes
    other = ctypes.byref(_kv(batch=3000, max_pages=70))
    assert L.hs2_paged_workspace_bytes(other, 64) == L.hs2_paged_workspace_bytes(kv, 64)
    # two partial results of 8 heads x (128 + 2) floats for each of at least 148 CTAs
    assert L.hs2_paged_workspace_bytes(kv, 64) >= 2 * 148 * 8 * 130 * 4
    assert L.hs2_paged_workspace_bytes(kv, 12) == 0       # not a multiple of 8 heads
    assert L.hs2_paged_workspace_bytes(kv, 8 * 129) == 0  # a group above 128
    assert L.hs2_paged_workspace_bytes(kv, -8) == 0


@pytest.mark.parametrize("args,code", [
    (dict(k=None), 1), (dict(k=P + 2), 1), (dict(dtype=2), 1), (dict(dtype=1), 2),
    (dict(ts=1028), 1), (dict(n=-1), 1), (dict(n=3, cu=None), 1), (dict(ws=None), 1),
    (dict(ws_bytes=16), 3), (dict(n=(1 << 31) - 1), 2),
])
def test_write_and_read_refuse_bad_arguments(L, args, code):
    a = dict(k=P, dtype=0, ts=1024, n=2, cu=P, ws=P, ws_bytes=1 << 20)
    a.update(args)
    kv = ctypes.byref(_kv())
    assert L.hs2_paged_kv_write(a["k"], P, a["dtype"], a["ts"], 128, a["n"], a["cu"], kv, a["ws"],
                                a["ws_bytes"], None) == code
    assert L.hs2_paged_kv_read(kv, a["cu"], None, a["n"], a["k"], P, a["dtype"], a["ts"], 128,
                               a["ws"], a["ws_bytes"], None) == code


@pytest.mark.parametrize("heads", [1, 2, 8])
def test_row_counts_that_do_not_round_up_are_refused(L, heads):
    """Counts are rounded up to whole blocks of up to a thousand rows in 32 bits."""
    n = ((1 << 31) - 1000) // heads
    kv = ctypes.byref(_kv(n_kv_heads=heads))
    assert L.hs2_paged_kv_write(P, P, 0, 0, 128, n, P, kv, P, 1 << 20, None) == 2
    assert L.hs2_paged_kv_read(kv, P, None, n, P, P, 0, 1024, 128, P, 1 << 20, None) == 2
    f = dict(q=P, k=P, v=P, cu_q=P, cu_k=P, q_token_stride=1024, q_head_stride=128, kv_token_stride=8,
             kv_head_stride=8, n_q=10, n_k=10, batch=2, h_q=heads, n_kv_heads=heads, head_dim=128, dtype=0)
    for k in ("n_q", "n_k"):
        a = hs2.Packed(**dict(f, **{k: n}))
        assert L.hs2_packed_attn(ctypes.byref(a), 0.1, P, P, P, 1 << 20, None) == 2


def test_nothing_to_move_is_no_error(L):
    kv = ctypes.byref(_kv())
    assert L.hs2_paged_kv_write(None, None, 0, 1024, 128, 0, P, kv, P, 4096, None) == 0
    assert L.hs2_paged_kv_read(kv, P, None, 0, None, None, 0, 1024, 128, P, 4096, None) == 0


@pytest.mark.parametrize("args,code", [
    (dict(q=None), 1), (dict(q=P + 8), 1), (dict(out=None), 1), (dict(dtype=2), 1),
    (dict(dtype=1), 2), (dict(h_q=12), 2), (dict(h_q=0), 2), (dict(qs=2050), 1),
    (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=math.inf), 1),
    (dict(scale=math.nan), 1), (dict(lse=P + 2), 1), (dict(ws_bytes=4096), 3),
])
def test_paged_attn_refuses_bad_arguments(L, args, code):
    a = dict(q=P, dtype=0, h_q=16, qs=2048, scale=0.1, out=P, lse=P, ws_bytes=1 << 40)
    a.update(args)
    assert L.hs2_paged_attn(a["q"], a["dtype"], a["h_q"], a["qs"], 128, ctypes.byref(_kv()),
                            a["scale"], a["out"], a["lse"], P, a["ws_bytes"], None) == code


@pytest.mark.parametrize("args,code", [
    (dict(cu_q=None), 1), (dict(cu_k=None), 1), (dict(q=None), 1), (dict(k=None), 1),
    (dict(v=P + 4), 1), (dict(head_dim=32), 2), (dict(dtype=1), 2), (dict(dtype=5), 2),
    (dict(h_q=7), 2), (dict(h_q=2 * 129), 2), (dict(batch=0), 1), (dict(batch=65536), 2),
    (dict(n_q=-1), 1), (dict(n_q=1 << 30), 2), (dict(q_token_stride=1025), 1),
    (dict(kv_head_stride=-128), 1), (dict(scale=math.nan), 1), (dict(ws_bytes=16), 3),
    (dict(out=P + 8), 1),
])
def test_packed_attn_refuses_bad_arguments(L, args, code):
    f = dict(q=P, k=P, v=P, cu_q=P, cu_k=P, q_token_stride=1024, q_head_stride=128,
             kv_token_stride=256, kv_head_stride=128, n_q=10, n_k=20, batch=2, h_q=8, n_kv_heads=2,
             head_dim=128, dtype=0)
    o = dict(scale=0.1, ws_bytes=1 << 20, out=P)
    for k, v in args.items():
        (o if k in o else f)[k] = v
    p = hs2.Packed(**f)
    assert L.hs2_packed_attn(ctypes.byref(p), o["scale"], o["out"], P, P, o["ws_bytes"], None) == code


def test_no_queries_is_no_error(L):
    p = hs2.Packed(P, P, P, P, P, 1024, 128, 256, 128, 0, 20, 2, 8, 2, 128, 0)
    assert L.hs2_packed_attn(ctypes.byref(p), 0.1, None, None, P, 4096, None) == 0


# ---------------------------------------------------------------- helpers
def cu_of(lens):
    return torch.tensor([0] + list(torch.tensor(lens).cumsum(0)), dtype=torch.int32)


def cache_of(pool):
    return hs2.PagedCache(*pool.to(DEV))


def bits(t):
    return t.contiguous().view(torch.uint8 if t.element_size() == 1 else
                               torch.int16 if t.element_size() == 2 else torch.int32)


def same(got, want):
    return torch.equal(bits(got.cpu()), bits(want))


# ---------------------------------------------------------------- writing and reading back
NEW = [  # lengths after the write, new tokens of each
    ([1], [1]),
    ([5, 0, 17, 64, 33, 1], [5, 0, 16, 1, 0, 1]),
    ([200, 31, 129], [70, 31, 100]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,new", NEW)
@pytest.mark.parametrize("kv,src", [("bf16", "bf16"), ("f16", "f16"), ("fp8", "bf16"), ("fp8", "f16")])
@pytest.mark.parametrize("h_kv,d,page,layout", [(1, 128, 16, "hnd"), (3, 64, 8, "nhd"), (8, 128, 64, "nhd"),
                                                (5, 64, 256, "hnd")])
def test_write_and_read(lens, new, kv, src, h_kv, d, page, layout):
    pool = Pool(lens, h_kv, d, page, kv, layout, seed=1, empty=True)
    g = torch.Generator().manual_seed(2)
    t = sum(new)
    pad = 3  # rows behind the last sequence
    fused = torch.randn(t + pad, 2 * h_kv + 1, d, generator=g)
    fused[t // 2, 0] = 0  # a zero row: scale 1
    fused[0, h_kv] *= 1000
    fused[t:] = math.nan
    fused = fused.to(TYPES[src]).to(DEV)
    k_new, v_new = fused[:, :h_kv], fused[:, h_kv:2 * h_kv]  # views of a wider projection
    cache = cache_of(pool)
    ws = hs2.paged_workspace(cache)
    cu = cu_of(new).to(DEV)
    hs2.paged_kv_write(k_new, v_new, cache, ws, cu_new=cu)
    assert hs2.check_device_status(ws) == 0
    at = 0
    for b, n in enumerate(new):
        pg, r = pool.at(b, lens[b] - n, lens[b])
        for x, p, s in ((k_new, pool.k, pool.k_scale), (v_new, pool.v, pool.v_scale)):
            rows = x[at:at + n].cpu()
            if kv == "fp8":
                p[pg, :, r], s[pg, :, r] = quantise(rows)
            else:
                p[pg, :, r] = rows
        at += n
    want = pool.to("cpu")
    assert same(cache.k, want[0]) and same(cache.v, want[1])  # the rest untouched, bit for bit
    if kv == "fp8":
        assert same(cache.k_scale, want[4]) and same(cache.v_scale, want[5])
    # read the new rows back from their own start, into tensors with rows behind
    start = torch.tensor([a - n for a, n in zip(lens, new)], dtype=torch.int32, device=DEV)
    dt = TYPES[src]
    k_out, v_out = (torch.full((t + pad, h_kv, d), 7.0, dtype=dt, device=DEV) for _ in range(2))
    hs2.paged_kv_read(cache, cu, ws, start=start, k_out=k_out, v_out=v_out)
    assert hs2.check_device_status(ws) == 0
    assert bool((k_out[t:] == 7).all()) and bool((v_out[t:] == 7).all())
    wants = [pool.rows(b, lens[b] - n, lens[b]) for b, n in enumerate(new)]
    for i, got in enumerate((k_out, v_out)):
        # code * scale is within one float32 rounding of the product; rounding that to 16 bits
        # lands on the neighbour only where the exact product is at a tie: a step then
        w = torch.cat([x[i] for x in wants])
        if kv == "fp8":
            off = (got[:t].cpu().double() - w).abs()
            lim = w.abs() * torch.finfo(dt).eps / 2 * (1 + 2.0 ** -10) + torch.finfo(dt).smallest_normal
            assert bool((off <= lim).all())
        else:
            assert same(got[:t], w.to(dt))


@pytest.mark.gpu
@pytest.mark.parametrize("src", ["bf16", "f16"])
def test_quotients_at_the_middle_between_codes(src):
    """Rows of every 16-bit mantissa against maxima of every mantissa and many sizes: quotients
    at and next to ties, below the normal codes, and scales near the ends of float32."""
    dt = TYPES[src]
    bits = 7 if src == "bf16" else 10
    mant = 1 + torch.arange(2 ** bits) / 2.0 ** bits
    rows = []
    g = torch.Generator().manual_seed(19)
    for e in ([-126, -110, -60, -51, -40, 0, 100, 127] if src == "bf16" else [-14, -8, 0, 15]):
        for _ in range(40):
            top = mant[torch.randint(2 ** bits, (1,), generator=g)] * 2.0 ** e
            shift = torch.randint(0, 18, (128,), generator=g)
            x = mant[torch.randint(2 ** bits, (128,), generator=g)].double() * 2.0 ** (e - 1 - shift.double())
            x[5] = top
            x[6] = -top / 2
            x[7] = 0
            rows.append((x * torch.where(torch.rand(128, generator=g) < 0.5, -1.0, 1.0)).to(dt))
    x = torch.stack(rows)[:, None]
    n = x.shape[0]
    pool = Pool([n], 1, 128, 64, "fp8", seed=20, empty=True)
    cache = cache_of(pool)
    ws = hs2.paged_workspace(cache)
    hs2.paged_kv_write(x.to(DEV), x.flip(0).contiguous().to(DEV), cache, ws)
    pg, r = pool.at(0, 0, n)
    for got, scale, want in ((cache.k, cache.k_scale, x), (cache.v, cache.v_scale, x.flip(0))):
        codes, s = quantise(want)
        assert same(scale.cpu()[pg, :, r], s)
        assert torch.equal(got.cpu()[pg, :, r], codes)


@pytest.mark.gpu
@pytest.mark.parametrize("src", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128])
def test_write_of_infinities_and_nan(src, d):
    """The scale of a row ignores its NaN; codes are the IEEE quotients: x / inf is 0."""
    x = torch.randn(6, 1, d, generator=torch.Generator().manual_seed(48)).to(TYPES[src])
    x[1, 0, 5], x[2, 0, 60] = math.inf, -math.inf
    x[3, 0, 7] = math.nan
    x[4, 0, 0], x[4, 0, 50] = math.inf, math.nan
    x[5] = math.nan
    f = x[:, 0].float()
    amax = f.abs().nan_to_num(0.0, posinf=math.inf).amax(-1)
    s = torch.where(amax > 0, amax / torch.full_like(amax, 448.0), torch.ones_like(amax))
    y = f / s[:, None]
    codes = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    cache = cache_of(Pool([6], 1, d, 8, "fp8", empty=True))
    hs2.paged_kv_write(x.to(DEV), x.to(DEV), cache, hs2.paged_workspace(cache))
    pg = int(cache.pages[0, 0])
    for got, scale in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        assert same(scale[pg, 0, :6], s)
        got = got[pg, 0, :6].cpu()
        nan = torch.isnan(y)
        assert bool(((got & 0x7F) == 0x7F)[nan].all()) and torch.equal(got[~nan], codes[~nan])


@pytest.mark.gpu
def test_uniform_write_is_the_packed_one():
    lens, n = [40, 9, 1024], 3
    a, b = (Pool(lens, 2, 128, 32, "fp8", seed=3, empty=True) for _ in range(2))
    x = torch.randn(2, 9, 2, 128, device=DEV).to(torch.bfloat16)
    ca, cb = cache_of(a), cache_of(b)
    ws = hs2.paged_workspace(ca)
    hs2.paged_kv_write(x[0], x[1], ca, ws)
    hs2.paged_kv_write(x[0], x[1], cb, ws, cu_new=cu_of([n] * 3).to(DEV))
    assert same(ca.k, cb.k.cpu()) and same(ca.v_scale, cb.v_scale.cpu())
    with pytest.raises(hs2.Hs2Error):
        hs2.paged_kv_write(x[0, :4], x[1, :4], ca, ws)  # 4 tokens for 3 sequences


@pytest.mark.gpu
def test_moves_report_bad_lengths_and_pages_and_touch_nothing():
    pool = Pool([40, 20, 33], 2, 64, 16, "f16", seed=4)
    cache = cache_of(pool)
    ws = hs2.paged_workspace(cache)
    before = cache.k.clone()
    x = torch.randn(6, 2, 64, device=DEV).to(torch.float16)
    cache.lens.copy_(torch.tensor([1, -1, 100], dtype=torch.int32))  # too short; negative; too long
    hs2.paged_kv_write(x, x, cache, ws)
    assert hs2.check_device_status(ws) == 7
    assert same(cache.k, before.cpu())
    cache.lens.copy_(torch.tensor([40, 20, 33], dtype=torch.int32))
    good = cache.pages.clone()
    cache.pages[0, 2], cache.pages[1, 1], cache.pages[2, 2] = -1, pool.num_pages, 1 << 30
    hs2.paged_kv_write(x, x, cache, ws)
    assert hs2.check_device_status(ws) == 6
    k, v = hs2.paged_kv_read(cache, cu_of([40, 20, 33]).to(DEV), ws)
    assert hs2.check_device_status(ws) == 6
    assert bool((k[32:40] == 0).all()) and bool((k[40:56] != 0).any())
    cache.pages.copy_(good)
    k, v = hs2.paged_kv_read(cache, cu_of([40, 21, 33]).to(DEV), ws)  # one past the second
    assert hs2.check_device_status(ws) == 7
    assert bool((k[60] == 0).all()) and bool(torch.isfinite(k).all())


# ---------------------------------------------------------------- one new token per sequence
def run_step(pool, h_q, qtype, strided=False, seed=5, scale=None, **kw):
    B, d = len(pool.lens), pool.d
    g = torch.Generator().manual_seed(seed)
    wide = torch.randn(B, h_q + 3, d, generator=g).to(TYPES[qtype])
    q = wide[:, 2:2 + h_q] if strided else wide[:, 2:2 + h_q].contiguous()
    cache = cache_of(pool)
    ws = hs2.paged_workspace(cache, h_q)
    qd = wide.to(DEV)[:, 2:2 + h_q] if strided else q.to(DEV)
    out, lse = hs2.paged_attn(qd, cache, ws, scale, **kw)
    assert hs2.check_device_status(ws) == 0
    check_step(pool, q, out, lse, scale)
    out2, lse2 = hs2.paged_attn(qd, cache, ws, scale)  # the workspace is as it was
    assert same(out2, out.cpu()) and same(lse2, lse.cpu())
    return cache, ws, qd, out, lse


def check_step(pool, q, out, lse, scale=None):
    B, h_q, d = q.shape
    g = h_q // pool.h_kv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    scale = float(torch.tensor(scale, dtype=torch.float32))
    out, lse = out.cpu(), lse.cpu()
    # FP8: weights are rounded to float16, whichever type the queries have
    wt = torch.float16 if pool.kv == "fp8" else q.dtype
    for b, n in enumerate(pool.lens):
        k, v = pool.rows(b, 0, n)
        for h in range(pool.h_kv):
            hs = slice(h * g, (h + 1) * g)
            ref = attend(q[b, hs].double(), k[:, h], v[:, h], scale, torch.full((g,), n))
            check(out[b, hs], lse[b, hs], ref, q.dtype, wt, n, f"sequence {b} ({n}), head {h}")


TYPE_PAIRS = [("bf16", "bf16"), ("f16", "f16"), ("fp8", "bf16"), ("fp8", "f16")]


@pytest.mark.gpu
@pytest.mark.parametrize("kv,qtype", TYPE_PAIRS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("h_q,h_kv", [(1, 1), (16, 1), (14, 2), (8, 8), (17, 1), (64, 2), (80, 1), (128, 1)])
def test_step_heads(kv, qtype, d, h_q, h_kv):
    run_step(Pool([0, 1, 63, 300, 64, 129], h_kv, d, 16, kv, "nhd", seed=6), h_q, qtype, strided=True)


@pytest.mark.gpu
@pytest.mark.parametrize("kv,qtype", [("bf16", "bf16"), ("fp8", "bf16")])
@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
def test_step_pages_and_lengths(kv, qtype, page):
    """Lengths around the pages' and tiles' edges, table rows wider than any sequence."""
    lens = [1, page - 1, page, page + 1, 15, 16, 17, 127, 128, 129, 0, 511, 2 * page + 3, 1000]
    run_step(Pool(lens, 2, 128, page, kv, seed=7, max_pages=1024), 8, qtype)


@pytest.mark.gpu
@pytest.mark.parametrize("kv,d,h_q,h_kv,lens", [
    ("bf16", 128, 16, 1, [40000]),          # one sequence over the whole GPU
    ("bf16", 128, 16, 1, [131072] * 2),     # dozens of tiles for each CTA: the ring goes round
    ("f16", 128, 3, 1, [90001, 1, 100000]),
    ("fp8", 64, 16, 1, [200000, 131]),
    ("fp8", 128, 20, 1, [150000]),
    ("fp8", 128, 64, 1, [20011, 3]),
    ("f16", 64, 4, 4, [9001, 77, 0, 12345]),
    ("bf16", 128, 8, 2, [300] * 200),       # more sequences than SMs
    ("fp8", 64, 12, 4, [17, 0, 900, 65, 1] * 30),
])
def test_step_split_and_joined(kv, d, h_q, h_kv, lens):
    run_step(Pool(lens, h_kv, d, 32, kv, seed=8), h_q, "f16" if kv == "f16" else "bf16")


@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_step_large_and_peaked_logits(kv):
    """Logits of several hundred, rising and falling along the keys, and one key that takes all."""
    pool = Pool([700, 700, 130], 1, 128, 64, kv, seed=9)
    ramp = torch.linspace(0, 6, 700)
    for b, r in ((0, ramp), (1, ramp.flip(0))):
        pg, row = pool.at(b, 0, 700)
        if kv == "fp8":
            pool.k_scale[pg, :, row] *= r[:, None] * 20
        else:
            pool.k[pg, :, row] *= r[:, None, None].to(pool.k.dtype)
    run_step(pool, 16, "bf16", scale=1.0)


def inf_logits(q, k):
    """Makes q . k -inf for the rows k (every other element of theirs is finite)."""
    q[..., 0] = 1.0
    k[..., 0] = -math.inf


@pytest.mark.gpu
@pytest.mark.parametrize("kv,h_q,h_kv", [("bf16", 2, 1), ("f16", 16, 1), ("f16", 64, 1), ("bf16", 8, 8)])
def test_step_logits_of_minus_infinity(kv, h_q, h_kv):
    """Keys with a logit of -inf have no weight, in whatever parts a sequence is cut; a row of
    only such keys gives zeros and -inf, as one without keys."""
    lens, dead = [30000, 40, 30000, 200, 0], [20000, 40, 30000, 150, 0]
    pool = Pool(lens, h_kv, 64, 16, kv, seed=41)
    q = torch.randn(len(lens), h_q, 64, generator=torch.Generator().manual_seed(42)).to(TYPES[kv])
    for b, n in enumerate(dead):
        pg, r = pool.at(b, 0, n)
        rows = pool.k[pg, :, r]
        inf_logits(q, rows)
        pool.k[pg, :, r] = rows
    cache = cache_of(pool)
    ws = hs2.paged_workspace(cache, h_q)
    out, lse = (x.cpu() for x in hs2.paged_attn(q.to(DEV), cache, ws))
    assert hs2.check_device_status(ws) == 0
    g, scale = h_q // h_kv, float(torch.tensor(0.125))
    for b, n in enumerate(lens):
        k, v = pool.rows(b, dead[b], n)  # the others are as if they were not there
        for h in range(h_kv):
            hs = slice(h * g, (h + 1) * g)
            ref = attend(q[b, hs].double(), k[:, h], v[:, h], scale, torch.full((g,), n - dead[b]))
            check(out[b, hs], lse[b, hs], ref, q.dtype, q.dtype, n, f"sequence {b}, head {h}")


@pytest.mark.gpu
@pytest.mark.parametrize("kv,value", [("bf16", math.nan), ("f16", math.nan), ("fp8", math.nan),
                                      ("bf16", math.inf), ("f16", math.inf)])
def test_step_keeps_nan(kv, value):
    """A NaN or +inf logit makes its sequence's results NaN, the lse included, and no other's."""
    pool = Pool([30000, 50, 60, 20000], 1, 128, 32, kv, seed=43)
    for b, at in ((0, 17001), (1, 31)):
        pg, r = pool.at(b, at, at + 1)
        pool.k[pg, 0, r, 5] = 0x7F if kv == "fp8" else value
    cache = cache_of(pool)
    ws = hs2.paged_workspace(cache, 16)
    qt = torch.float16 if kv == "f16" else torch.bfloat16
    q = torch.randn(4, 16, 128, generator=torch.Generator().manual_seed(44)).to(qt)
    q[..., 5] = 1.0
    out, lse = hs2.paged_attn(q.to(DEV), cache, ws)
    for b, bad in enumerate((True, True, False, False)):
        assert bool((torch.isnan(out[b]) == bad).all()) and bool((torch.isnan(lse[b]) == bad).all())


@pytest.mark.gpu
def test_step_scales_of_all_sizes():
    """FP8 rows of V whose scales span 2^-40 .. 2^40 and 0: each weight is held relative to
    the largest weight times scale."""
    pool = Pool([513], 2, 128, 16, "fp8", seed=10)
    pg, row = pool.at(0, 0, 513)
    for power in (-40, 40):
        pool.v_scale[pg, :, row] = 2.0 ** power * (1 + torch.rand(513, 2))
        cache, ws, q, out, lse = None, None, None, None, None
        g = torch.Generator().manual_seed(11)
        q = torch.randn(1, 8, 128, generator=g).to(torch.bfloat16)
        cache = cache_of(pool)
        ws = hs2.paged_workspace(cache, 8)
        out, lse = hs2.paged_attn(q.to(DEV), cache, ws)
        k, v = pool.rows(0, 0, 513)
        for h in range(2):
            o, z, a, mag = attend(q[0, 4 * h:4 * h + 4].double(), k[:, h], v[:, h],
                                  float(torch.tensor(1 / math.sqrt(128.0))), torch.full((4,), 513))
            f = 2.0 ** -power  # the bound is for values of order 1
            check(out.cpu()[0, 4 * h:4 * h + 4].double() * f, lse.cpu()[0, 4 * h:4 * h + 4],
                  (o * f, z, a * f, mag), torch.bfloat16, torch.float16, 513)
    pool.v_scale[pg, :, row] = 0.0
    cache = cache_of(pool)
    out, lse = hs2.paged_attn(q.to(DEV), cache, hs2.paged_workspace(cache, 8))
    assert bool((out == 0).all()) and bool(torch.isfinite(lse).all())


@pytest.mark.gpu
def test_step_reports_bad_lengths_and_pages():
    pool = Pool([100, 60, 33], 2, 128, 16, "bf16", seed=12)
    for t in (pool.k, pool.v):
        t.nan_to_num_(0.5)
    cache, ws, q, out, lse = run_step(pool, 4, "bf16")
    cache.pages[1, 3] = pool.num_pages
    out2, lse2 = hs2.paged_attn(q, cache, ws)
    assert hs2.check_device_status(ws) == 6
    assert same(out2[0], out[0].cpu()) and same(out2[2], out[2].cpu())  # the others unharmed
    cache.pages[1, 3] = 0
    cache.lens[0], cache.lens[2] = -5, 10 ** 9
    out2, lse2 = hs2.paged_attn(q, cache, ws)
    assert hs2.check_device_status(ws) in (6, 7)
    assert bool((out2[0] == 0).all()) and bool((lse2[0] == -math.inf).all())


# ---------------------------------------------------------------- packed prompts
def run_prompts(lq, lk, h_q, h_kv, d, dtype, pad_q=0, pad_k=0, fused=None, scale=None, seed=13):
    g = torch.Generator().manual_seed(seed)
    dt = TYPES[dtype]
    tq, tk = sum(lq), sum(lk)
    fused = lq == lk if fused is None else fused
    if fused:
        x = torch.randn(tq + pad_q, h_q + 2 * h_kv, d, generator=g).to(dt)
        x[tq:] = math.nan
        dev = x.to(DEV)
        cut = (slice(0, h_q), slice(h_q, h_q + h_kv), slice(h_q + h_kv, None))
        q, k, v = (x[:, c] for c in cut)
        qd, kd, vd = (dev[:, c] for c in cut)
    else:
        q, k, v = (torch.randn(n, h, d, generator=g).to(dt)
                   for n, h in ((tq + pad_q, h_q), (tk + pad_k, h_kv), (tk + pad_k, h_kv)))
        q[tq:], k[tk:], v[tk:] = math.nan, math.nan, math.nan
        qd, kd, vd = q.to(DEV), k.to(DEV), v.to(DEV)
    cu_q, cu_k = cu_of(lq).to(DEV), cu_of(lk).to(DEV)
    ws = hs2.packed_workspace(DEV)
    out = torch.full((tq + pad_q, h_q, d), 7.0, dtype=dt, device=DEV)
    lse = torch.full((tq + pad_q, h_q), 7.0, device=DEV)
    hs2.packed_attn(qd, kd, vd, cu_q, cu_k, ws, scale, out=out, lse=lse)
    assert hs2.check_device_status(ws) == 0
    assert bool((out[tq:] == 7).all()) and bool((lse[tq:] == 7).all())  # rows behind: left
    check_prompts(q, k, v, lq, lk, out, lse, scale)
    out2, lse2 = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
    hs2.packed_attn(qd, kd, vd, cu_q, cu_k, ws, scale, out=out2, lse=lse2)
    assert same(out2, out.cpu()) and same(lse2, lse.cpu())


def check_prompts(q, k, v, lq, lk, out, lse, scale=None):
    d, g = q.shape[2], q.shape[1] // k.shape[1]
    scale = float(torch.tensor(1.0 / math.sqrt(d) if scale is None else scale, dtype=torch.float32))
    out, lse = out.cpu(), lse.cpu()
    a = c = 0
    for n, m in zip(lq, lk):
        visible = torch.arange(m - n + 1, m + 1)
        for h in range(q.shape[1]):
            ref = attend(q[a:a + n, h].double(), k[c:c + m, h // g].double(), v[c:c + m, h // g].double(),
                         scale, visible)
            check(out[a:a + n, h], lse[a:a + n, h], ref, q.dtype, q.dtype, m, f"prompt of {n} on {m}, head {h}")
        a, c = a + n, c + m


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("h_q,h_kv", [(1, 1), (4, 4), (8, 2), (7, 1), (6, 2), (16, 1), (80, 1)])
def test_prompt_heads(dtype, d, h_q, h_kv):
    run_prompts([1, 130, 0, 37, 64], [1, 130, 0, 37, 64], h_q, h_kv, d, dtype, pad_q=5)


@pytest.mark.gpu
@pytest.mark.parametrize("lens", [[1], [2], [127, 128, 129], [255, 256, 257], [16] * 40, [1] * 70,
                                  [0, 0, 300, 0], [1025, 3, 700]])
def test_prompt_lengths(lens):
    run_prompts(lens, lens, 4, 2, 128, "bf16", pad_q=1)


@pytest.mark.gpu
@pytest.mark.parametrize("d,dtype", [(64, "f16"), (128, "bf16")])
@pytest.mark.parametrize("lq,lk", [
    ([1, 1, 1], [1000, 129, 1]),               # single tokens after long prefixes
    ([40, 200, 3], [240, 200, 800]),
    ([50, 0, 20, 9], [20, 30, 0, 9]),          # more queries than keys: the first see nothing
    ([300], [0]), ([64], [63]),
])
def test_prompt_prefixes(d, dtype, lq, lk):
    run_prompts(lq, lk, 6, 2, d, dtype, pad_q=4, pad_k=9, fused=False)


@pytest.mark.gpu
@pytest.mark.parametrize("d,dtype", [(64, "f16"), (128, "bf16")])
@pytest.mark.parametrize("h_q,h_kv,lq,lk", [
    # enough work for two tiles per work item: both full, the second short, empty or ahead
    (16, 16, [513, 3, 300, 256, 129, 128, 127, 1], None),
    (32, 8, [65, 700, 64, 0, 1, 33], None),
    (14, 2, [1300, 36, 18, 19], None),          # 18 tokens x 7 heads a tile
    (40, 8, [300, 50, 500], [900, 20, 700]),    # prefixes, and queries that see nothing
    (32, 16, [1] * 30, list(range(1, 600, 20))),
    (16, 16, [200, 64, 320], [200, 0, 320]),
])
def test_prompt_two_tiles(d, dtype, h_q, h_kv, lq, lk):
    run_prompts(lq, lk or lq, h_q, h_kv, d, dtype, pad_q=3, pad_k=0 if lk is None else 4,
                fused=lk is None)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("h_q,h_kv", [(4, 2), (16, 16)])
def test_prompt_large_logits(dtype, h_q, h_kv):
    run_prompts([400, 150, 300], [400, 150, 300], h_q, h_kv, 128, dtype, scale=3.0)


@pytest.mark.gpu
@pytest.mark.parametrize("h_q,h_kv", [(2, 1), (16, 16)])
def test_prompt_rising_logits(h_q, h_kv):
    """Keys whose logits rise along the prompt: the softmax reference moves in every step and
    the outputs so far are rescaled each time."""
    n, d = 700, 64
    g = torch.Generator().manual_seed(25)
    q = (torch.randn(n, h_q, d, generator=g) * 0.1 + 1).half()
    k = torch.randn(n, h_kv, d, generator=g) * 0.1 + torch.linspace(-3, 6, n)[:, None, None]
    v = torch.randn(n, h_kv, d, generator=g).half()
    k = k.half()
    ws = hs2.packed_workspace(DEV)
    out, lse = hs2.packed_attn(q.to(DEV), k.to(DEV), v.to(DEV), cu_of([n]).to(DEV), workspace=ws)
    assert hs2.check_device_status(ws) == 0
    check_prompts(q, k, v, [n], [n], out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("heads", [(4, 2, 2), (40, 40, 40)])  # one and two tiles per work item
def test_prompt_garbage_stays_in_its_sequence(heads):
    """Infinities and NaN in one sequence's rows, and in rows no sequence owns, reach no other."""
    lens = [100, 61, 130]
    g = torch.Generator().manual_seed(14)
    q, k, v = (torch.randn(300, h, 64, generator=g).to(torch.bfloat16).to(DEV) for h in heads)
    cu = cu_of(lens).to(DEV)
    ws = hs2.packed_workspace(DEV)
    clean, _ = hs2.packed_attn(q, k, v, cu, workspace=ws)
    for x in (k, v):
        x[100:161] = math.nan
        x[110] = math.inf
        x[291:] = -math.inf
    out, _ = hs2.packed_attn(q, k, v, cu, workspace=ws)
    for rows in (slice(0, 100), slice(161, 291)):
        assert same(out[rows], clean[rows].cpu())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("h_q,h_kv", [(4, 2), (40, 40)])  # one and two tiles per work item
def test_prompt_logits_of_minus_infinity(dtype, h_q, h_kv):
    """Keys with a logit of -inf have no weight; a row of only such keys gives zeros and -inf."""
    n, dead, d = 300, 140, 64
    g = torch.Generator().manual_seed(45)
    q, k, v = (torch.randn(n, h, d, generator=g).to(TYPES[dtype]) for h in (h_q, h_kv, h_kv))
    inf_logits(q, k[:dead])
    ws = hs2.packed_workspace(DEV)
    out, lse = hs2.packed_attn(q.to(DEV), k.to(DEV), v.to(DEV), cu_of([n]).to(DEV), workspace=ws)
    assert hs2.check_device_status(ws) == 0
    assert bool((out[:dead] == 0).all()) and bool((lse[:dead] == -math.inf).all())
    check_prompts(q[dead:], k[dead:], v[dead:], [n - dead], [n - dead], out[dead:], lse[dead:])


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64)])
@pytest.mark.parametrize("h_q,h_kv", [(4, 2), (40, 40)])
@pytest.mark.parametrize("at", [0, 3, 14, 79, 142, 270])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_prompt_keeps_nan(dtype, d, h_q, h_kv, at, value):
    """A NaN or +inf logit makes the results NaN of the queries that see its key, whichever key
    it is, and of no query before it."""
    n = 300
    g = torch.Generator().manual_seed(46)
    q, k, v = (torch.randn(n, h, d, generator=g).to(TYPES[dtype]) for h in (h_q, h_kv, h_kv))
    q[..., 0] = 1.0
    cu, ws = cu_of([n]).to(DEV), hs2.packed_workspace(DEV)
    clean, clean_lse = hs2.packed_attn(q.to(DEV), k.to(DEV), v.to(DEV), cu, workspace=ws)
    k[at, :, 0] = value
    out, lse = hs2.packed_attn(q.to(DEV), k.to(DEV), v.to(DEV), cu, workspace=ws)
    assert hs2.check_device_status(ws) == 0
    assert same(out[:at], clean[:at].cpu()) and same(lse[:at], clean_lse[:at].cpu())
    assert bool(torch.isnan(out[at:]).all()) and bool(torch.isnan(lse[at:]).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("h_q,h_kv", [(4, 2), (40, 40)])
def test_prompt_large_values_behind_the_mask(dtype, h_q, h_kv):
    """The largest finite V behind a query's mask adds nothing to it."""
    n, d = 300, 128
    g = torch.Generator().manual_seed(47)
    q, k, v = (torch.randn(n, h, d, generator=g).to(TYPES[dtype]).to(DEV) for h in (h_q, h_kv, h_kv))
    cu, ws = cu_of([n]).to(DEV), hs2.packed_workspace(DEV)
    clean, clean_lse = hs2.packed_attn(q, k, v, cu, workspace=ws)
    for at in (1, 70, 200):
        big = v.clone()
        big[at:] = torch.finfo(v.dtype).max
        out, lse = hs2.packed_attn(q, k, big, cu, workspace=ws)
        assert same(out[:at], clean[:at].cpu()) and same(lse, clean_lse.cpu())


@pytest.mark.gpu
def test_prompt_reports_bad_offsets():
    q, k = torch.ones(64, 2, 64, device=DEV).half(), torch.ones(64, 1, 64, device=DEV).half()
    ws = hs2.packed_workspace(DEV)
    for cu_q, cu_k in (([0, 30, 65], [0, 30, 64]), ([0, 40, 64], [0, 70, 64]),
                       ([0, 64, 20], [0, 64, 64]), ([0, 10, 64], [-5, 10, 64])):
        cu_q, cu_k = (torch.tensor(c, dtype=torch.int32, device=DEV) for c in (cu_q, cu_k))
        hs2.packed_attn(q, k, k, cu_q, cu_k, ws)
        assert hs2.check_device_status(ws) == 7


# ---------------------------------------------------------------- together, and how they are called
@pytest.mark.gpu
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_a_served_batch(kv):
    """Prompts in, their rows into the pages, a second chunk after its cached prefix, then
    decode steps captured once as a graph and replayed with growing lengths."""
    h_q, h_kv, d, page = 8, 2, 128, 16
    first, second, steps = [70, 1, 33], [20, 64, 5], 3
    total = [a + b + steps for a, b in zip(first, second)]
    pool = Pool(total, h_kv, d, page, kv, seed=15, empty=True)
    cache = cache_of(pool)
    ws, pws = hs2.paged_workspace(cache, h_q), hs2.packed_workspace(DEV)
    g = torch.Generator().manual_seed(16)

    def proj(n):
        return torch.randn(n, h_q + 2 * h_kv, d, generator=g).to(torch.bfloat16)

    def cached(b, lo, rows):  # what the cache holds of these rows from position lo on
        k, v = rows[:, h_q:h_q + h_kv], rows[:, h_q + h_kv:]
        if kv == "fp8":
            return tuple((c.view(torch.float8_e4m3fn).double() * s.double()[..., None])
                         for c, s in (quantise(k), quantise(v)))
        return k.double(), v.double()

    have = [(torch.zeros(0, h_kv, d).double(),) * 2 for _ in first]
    lens = [0] * 3
    for chunk in (first, second):
        x = proj(sum(chunk))
        xd = x.to(DEV)
        q, k, v = xd[:, :h_q], xd[:, h_q:h_q + h_kv], xd[:, h_q + h_kv:]
        cu = cu_of(chunk).to(DEV)
        before = list(lens)
        lens = [a + b for a, b in zip(lens, chunk)]
        cache.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        hs2.paged_kv_write(k, v, cache, ws, cu_new=cu)
        cu_k = cu_of(lens).to(DEV)
        kk, vv = hs2.paged_kv_read(cache, cu_k, ws)  # prefix and chunk, as the cache holds them
        out, lse = hs2.packed_attn(q, kk, vv, cu, cu_k, pws)
        at = 0
        for b, n in enumerate(chunk):
            new = cached(b, before[b], x[at:at + n])
            have[b] = tuple(torch.cat([o, w]) for o, w in zip(have[b], new))
            at += n
        check_prompts(x[:, :h_q], kk.cpu(), vv.cpu(), chunk, lens, out, lse)
    # decode
    xs = [proj(3) for _ in range(steps)]
    x = xs[0].to(DEV).clone()
    out = torch.empty(3, h_q, d, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(3, h_q, device=DEV)

    def step():
        cache.lens.add_(1)
        hs2.paged_kv_write(x[:, h_q:h_q + h_kv], x[:, h_q + h_kv:], cache, ws)
        hs2.paged_attn(x[:, :h_q], cache, ws, out=out, lse=lse)

    step()  # warm-up outside the capture; its slot is written again by the first replay
    cache.lens.sub_(1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(steps):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        for b in range(3):
            new = cached(b, lens[b] + i, xs[i][b:b + 1])
            have[b] = tuple(torch.cat([o, w]) for o, w in zip(have[b], new))
            for h in range(h_kv):
                hs = slice(4 * h, 4 * h + 4)
                n = have[b][0].shape[0]
                ref = attend(xs[i][b, hs].double(), have[b][0][:, h], have[b][1][:, h],
                             float(torch.tensor(1 / math.sqrt(128.0))), torch.full((4,), n))
                check(out.cpu()[b, hs], lse.cpu()[b, hs], ref, torch.bfloat16,
                      torch.float16 if kv == "fp8" else torch.bfloat16, n, f"step {i}")
    assert hs2.check_device_status(ws) == 0 and hs2.check_device_status(pws) == 0


@pytest.mark.gpu
def test_on_another_stream_and_without_workspaces():
    pool = Pool([130, 7], 2, 64, 16, "f16", seed=17)
    cache, ws, q, out, lse = run_step(pool, 6, "f16")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out2, lse2 = hs2.paged_attn(q, cache, stream=s)
    k, v = hs2.paged_kv_read(cache, cu_of([130, 7]).to(DEV), ws, n_tokens=137, stream=s)
    torch.cuda.synchronize()
    assert same(out2, out.cpu()) and same(lse2, lse.cpu())
    qs = torch.randn(137, 6, 64, device=DEV).half()
    cu = cu_of([130, 7]).to(DEV)
    a = hs2.packed_attn(qs, k, v, cu)
    s.wait_stream(torch.cuda.current_stream())
    b = hs2.packed_attn(qs, k, v, cu, stream=s)
    torch.cuda.synchronize()
    assert same(a[0], b[0].cpu()) and same(a[1], b[1].cpu())


@pytest.mark.gpu
def test_offsets_past_32_bits_in_the_pages():
    """A pool of 4.7 GB per tensor whose last pages are in use: every operator on them."""
    n, page, lens = 290000, 64, [130, 64, 1]
    pool = Pool(lens, 1, 128, page, "bf16", seed=26)
    small = pool.k, pool.v, pool.pages.clone()
    far = torch.tensor([0, n - 1, 140000, n - 7, 200000, 131071, 131072, n - 2], dtype=torch.int32)
    k, v = (torch.empty(n, 1, page, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    for at in range(pool.num_pages):
        k[far[at]], v[far[at]] = small[0][at].to(DEV), small[1][at].to(DEV)
    used = pool.pages >= 0
    pages = torch.where(used, far[pool.pages.clamp(min=0).long()], pool.pages)
    cache = hs2.PagedCache(k, v, pages.to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV))
    ws = hs2.paged_workspace(cache, 4)
    q = torch.randn(3, 4, 128, generator=torch.Generator().manual_seed(27)).to(torch.bfloat16)
    out, lse = hs2.paged_attn(q.to(DEV), cache, ws)
    check_step(pool, q, out, lse)
    rows = hs2.paged_kv_read(cache, cu_of(lens).to(DEV), ws)
    for i, got in enumerate(rows):
        assert same(got, torch.cat([pool.rows(b, 0, m)[i] for b, m in enumerate(lens)]).to(torch.bfloat16))
    x = torch.randn(3, 1, 128, device=DEV).to(torch.bfloat16)
    hs2.paged_kv_write(x, x + 1, cache, ws)  # the last row of each
    again = hs2.paged_kv_read(cache, cu_of([1] * 3).to(DEV), ws,
                              start=cache.lens - 1, n_tokens=3)
    assert same(again[0], x.cpu()) and same(again[1], (x + 1).cpu())
    assert hs2.check_device_status(ws) == 0


@pytest.mark.gpu
def test_offsets_past_32_bits_in_the_prompts():
    """150000 tokens of 128 heads of 128: 2.4e9 elements of q and out."""
    h, d, n, m = 128, 128, 150000, 50
    q = torch.empty(n, h, d, dtype=torch.float16, device=DEV)
    for a in range(0, n, 10000):
        q[a:a + 10000].normal_()
    k, v = (torch.randn(n, 1, d, device=DEV).half() for _ in range(2))
    cu = torch.arange(0, n + 1, m, dtype=torch.int32, device=DEV)
    ws = hs2.packed_workspace(DEV)
    out, lse = hs2.packed_attn(q, k, v, cu, workspace=ws)
    assert hs2.check_device_status(ws) == 0
    for a in (0, 131050, n - m):  # 131072 tokens of 128 x 128: 2^31 elements
        s = slice(a, a + m)
        check_prompts(q[s, ::37].cpu(), k[s].cpu(), v[s].cpu(), [m], [m], out[s, ::37], lse[s, ::37])


@pytest.mark.gpu
def test_two_calls_at_once():
    """Decode and prompts on two streams, each with its own workspace, over and over."""
    pool = Pool([3000, 1, 777, 2000], 4, 128, 32, "fp8", seed=28)
    cache, ws, q, out, lse = run_step(pool, 16, "bf16")
    g = torch.Generator().manual_seed(29)
    x = torch.randn(1500, 24, 64, generator=g).half().to(DEV)
    cu, pws = cu_of([700, 0, 800]).to(DEV), hs2.packed_workspace(DEV)
    args = (x[:, :16], x[:, 16:20], x[:, 20:], cu)
    want = hs2.packed_attn(*args, workspace=pws)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(30):
        got.append(hs2.paged_attn(q, cache, ws, stream=streams[0])
                   + hs2.packed_attn(*args, workspace=pws, stream=streams[1]))
    torch.cuda.synchronize()
    for o, z, po, pz in got:
        assert same(o, out.cpu()) and same(z, lse.cpu())
        assert same(po, want[0].cpu()) and same(pz, want[1].cpu())
    assert hs2.check_device_status(ws) == 0 and hs2.check_device_status(pws) == 0


@pytest.mark.gpu
def test_one_workspace_for_calls_of_all_shapes():
    """Batches, groups and operators that change from call to call on the same workspace."""
    pools = [(Pool(lens, h_kv, d, 16, kv, seed=21), h_q) for lens, h_kv, d, kv, h_q in (
        ([9000], 1, 128, "bf16", 16), ([5, 0, 700] * 40, 4, 128, "bf16", 8),
        ([3000, 1, 2500], 2, 64, "f16", 14), ([40000], 1, 128, "fp8", 16))]
    ws = max((hs2.paged_workspace(cache_of(p), h) for p, h in pools), key=torch.numel)
    g = torch.Generator().manual_seed(22)
    x = torch.randn(300, 6, 64, generator=g).half().to(DEV)
    cu = cu_of([100, 200]).to(DEV)
    want = hs2.packed_attn(x[:, :4], x[:, 4:5], x[:, 5:], cu)[0]
    for pool, h_q in pools + pools[::-1]:
        q = torch.randn(len(pool.lens), h_q, pool.d, generator=g)
        q = q.to(torch.float16 if pool.kv == "f16" else torch.bfloat16)
        out, lse = hs2.paged_attn(q.to(DEV), cache_of(pool), ws)
        check_step(pool, q, out, lse)
        assert same(hs2.packed_attn(x[:, :4], x[:, 4:5], x[:, 5:], cu, workspace=ws)[0], want.cpu())
    assert hs2.check_device_status(ws) == 0


@pytest.mark.gpu
def test_first_calls_inside_a_capture():
    """Every operator captured in a graph without having run before in these forms."""
    pool = Pool([50, 3], 1, 64, 8, "fp8", seed=23)
    cache = cache_of(pool)
    ws, pws = hs2.paged_workspace(cache, 2), hs2.packed_workspace(DEV)
    g = torch.Generator().manual_seed(24)
    q = torch.randn(2, 2, 64, generator=g).half()
    x = torch.randn(53, 2, 64, generator=g).half().to(DEV)
    qd, cu = q.to(DEV), cu_of([50, 3]).to(DEV)
    out, lse = torch.empty_like(qd), torch.empty(2, 2, device=DEV)
    k, v = torch.empty(53, 1, 64, device=DEV).half(), torch.empty(53, 1, 64, device=DEV).half()
    po, pl = torch.empty_like(x), torch.empty(53, 2, device=DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hs2.paged_kv_write(x[:2, :1], x[2:4, :1], cache, ws)  # the last row of each, again
        hs2.paged_kv_read(cache, cu, ws, k_out=k, v_out=v)
        hs2.paged_attn(qd, cache, ws, out=out, lse=lse)
        hs2.packed_attn(x, k, v, cu, workspace=pws, out=po, lse=pl)
    for b, n in enumerate(pool.lens):
        pg, r = pool.at(b, n - 1, n)
        pool.k[pg, :, r], pool.k_scale[pg, :, r] = quantise(x[b:b + 1, :1].cpu())
        pool.v[pg, :, r], pool.v_scale[pg, :, r] = quantise(x[2 + b:3 + b, :1].cpu())
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        check_step(pool, q, out, lse)
        check_prompts(x.cpu(), k.cpu(), v.cpu(), [50, 3], [50, 3], po, pl)
    assert hs2.check_device_status(ws) == 0 and hs2.check_device_status(pws) == 0


@pytest.mark.gpu
def test_calls_refuse_bad_tensors():
    pool = Pool([20, 30], 2, 64, 16, "f16", seed=18)
    k, v, pages, lens, _, _ = pool.to(DEV)
    cache = hs2.PagedCache(k, v, pages, lens)
    ws = hs2.paged_workspace(cache, 4)
    q = torch.zeros(2, 4, 64, device=DEV).half()
    rows = torch.zeros(2, 2, 64, device=DEV).half()
    for bad in (lambda: hs2.PagedCache(k.cpu(), v, pages, lens),
                lambda: hs2.PagedCache(k, v.transpose(1, 2).contiguous().transpose(1, 2), pages, lens),
                lambda: hs2.PagedCache(k, v, pages.long(), lens),
                lambda: hs2.PagedCache(k, v, pages, lens[:1]),
                lambda: hs2.PagedCache(k, v, pages, lens, lens.float(), lens.float()),
                lambda: hs2.PagedCache(k.float(), v.float(), pages, lens),
                lambda: hs2.paged_attn(q[:1], cache, ws),
                lambda: hs2.paged_attn(q.bfloat16(), cache, ws),
                lambda: hs2.paged_attn(q, cache, ws, out=torch.zeros(2, 4, 64, device=DEV)),
                lambda: hs2.paged_attn(q, cache, ws.cpu()),
                lambda: hs2.paged_attn(q, cache, ws.float()),
                lambda: hs2.paged_kv_write(rows.float(), rows.float(), cache, ws),
                lambda: hs2.paged_kv_write(rows, rows[:1], cache, ws),
                lambda: hs2.paged_kv_write(rows, rows, cache, ws, cu_new=lens),
                lambda: hs2.paged_kv_read(cache, lens, ws),
                lambda: hs2.packed_attn(q, rows, rows.bfloat16(), lens),
                lambda: hs2.packed_attn(q, rows, rows, lens[:1]),
                lambda: hs2.packed_attn(q, rows, rows, lens.cpu())):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: hs2.paged_attn(q[:, :3].contiguous(), cache, ws),
                lambda: hs2.paged_attn(q, cache, ws[:256]),
                lambda: hs2.paged_attn(q, cache, ws, sm_scale=0.0),
                lambda: hs2.packed_attn(q[:, :3].contiguous(), rows, rows, lens)):
        with pytest.raises(hs2.Hs2Error):
            bad()
