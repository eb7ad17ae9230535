"""Paged caches and packed prompts at the edges of what their definitions allow."""
import torch

import pytest

from long_context_token_b200 import hs2

from _paged_ref import Pool
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
