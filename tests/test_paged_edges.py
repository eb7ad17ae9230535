"""Paged caches and packed prompts at the edges of what their definitions allow."""
import math

import pytest
import torch

from long_context_token_b200 import hs2

from _paged_ref import Pool, attend, check
from test_paged import DEV, cache_of, cu_of, same


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
