"""Waits of the token probabilities and of the page copies that run out, without
a GPU fault: the test build makes the threads that walk a row, or the lane that
stores, wait first on a barrier that nothing completes, with the bound shortened
to 1 ms. The kernel sets the timeout bit, lets its copies land and returns; the
next call is right."""
import pytest
import torch

import paged_kv_cache_60_gb300 as da

from gpu_util import debug_build_library

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tlib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return debug_build_library()


class Stalled:
    def __init__(self, lib):
        self.lib = lib

    def __enter__(self):
        assert self.lib.decode_attn_debug_wait_limit(1000000) == 0
        assert self.lib.decode_attn_debug_stall(1) == 0

    def __exit__(self, *exc):
        torch.cuda.synchronize()
        self.lib.decode_attn_debug_stall(0)
        self.lib.decode_attn_debug_wait_limit(0)


@pytest.mark.parametrize("rows,V", [(1, 500001), (300, 20000), (200, 128256)])
def test_streaming_row_whose_wait_runs_out(tlib, rows, V):
    """One row a cluster, and rows with fewer and with more pieces than the ring has slots."""
    g = torch.Generator(device="cuda").manual_seed(5)
    logits = torch.randn(rows, 1, V, device="cuda", generator=g)
    want, probs = torch.empty_like(logits), torch.empty_like(logits)
    error = torch.zeros(1, dtype=torch.int32, device="cuda")
    da.token_probs(logits, want)
    with Stalled(tlib):
        da.token_probs(logits, probs, device_error=error, lib=tlib)
    assert error.item() == da.DA_DEV_TIMEOUT
    error.zero_()
    da.token_probs(logits, probs, device_error=error, lib=tlib)
    assert error.item() == 0 and torch.equal(probs, want)


@pytest.mark.parametrize("copies", [1, 40, 6000])
def test_copies_whose_wait_runs_out(tlib, copies):
    H, D, P = 2, 64, 16
    desc = da.Desc.make(B=1, H_kv=H, G=8, D_qk=D, D_v=D, s_q=1, page_size=P, kv_dtype=da.KV_BF16, num_pages=2 * copies, max_pages_per_seq=1)
    g = torch.Generator(device="cuda").manual_seed(6)
    k, v = (torch.randn(2 * copies, P, H, D, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    k0, v0 = k.clone(), v.clone()
    pairs = torch.stack([torch.arange(copies), torch.arange(copies) + copies], 1).to(torch.int32).cuda()
    error = torch.zeros(1, dtype=torch.int32, device="cuda")
    with Stalled(tlib):
        da.copy_pages(desc, pairs, k, v, device_error=error, lib=tlib)
    assert error.item() == da.DA_DEV_TIMEOUT
    assert torch.equal(k, k0) and torch.equal(v, v0)  # every piece was given up
    error.zero_()
    da.copy_pages(desc, pairs, k, v, device_error=error, lib=tlib)
    assert error.item() == 0
    for x, x0 in ((k, k0), (v, v0)):
        assert torch.equal(x[copies:], x0[:copies]) and torch.equal(x[:copies], x0[:copies])
