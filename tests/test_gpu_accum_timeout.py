"""Waits of the weight accumulation that run out, without a GPU fault: as for the
attention kernels, the test build makes the warps that sum wait first on a
barrier that nothing completes, with the bound shortened to 1 ms. The kernel
sets the timeout bit, lets its copies land and returns; the weights of the
chunks given up stay, and the next call is right. With few chunks the copies
have all been issued before anyone gives up; with many the copying warp gives up
too."""
import pytest
import torch

import paged_kv_cache_60_gb300 as da
from workloads import KV_BF16, KV_FP8, KV_MLA656

from gpu_util import debug_build_library
from test_gpu_accum import Step, _spec

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tlib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    return debug_build_library()


def _accum(tlib, s, weights):
    d = s.dw
    da.accum_weights(s.desc, d.q, d.k_pool, d.k_scale, d.block_table, d.cache_seqlens, s.meta, s.lse, weights, lib=tlib)
    torch.cuda.synchronize()


def _stalled_then_right(tlib, spec):
    s = Step(spec, nan_fresh=False)
    want = s.run()                                # the product build
    weights = s.weights.cuda()
    assert tlib.decode_attn_debug_wait_limit(1000000) == 0
    assert tlib.decode_attn_debug_stall(1) == 0
    try:
        _accum(tlib, s, weights)
    finally:
        tlib.decode_attn_debug_stall(0)
        tlib.decode_attn_debug_wait_limit(0)
    assert da.get_error(s.meta) & da.DA_DEV_TIMEOUT
    assert torch.equal(weights.cpu(), s.weights)  # every chunk was given up
    da.sched_meta(s.desc, s.dw.cache_seqlens, s.meta)
    _accum(tlib, s, weights)
    assert da.get_error(s.meta) == 0
    assert torch.equal(weights.view(torch.int32), want.view(torch.int32))
    s.check(weights)


@pytest.mark.parametrize("kv,H,D,s_q", [(KV_BF16, 2, 128, 1), (KV_BF16, 4, 64, 1), (KV_FP8, 4, 128, 1), (KV_FP8, 2, 128, 3)])
@pytest.mark.parametrize("lens,splits", [([90, 30], 1), ([9000, 4000], 1)])
def test_wait_that_runs_out_and_the_call_after_it(tlib, kv, H, D, s_q, lens, splits):
    _stalled_then_right(tlib, _spec(kv, 2, H, D, 32, lens, s_q, splits, seed=91))


@pytest.mark.parametrize("s_q", [1, 2])
@pytest.mark.parametrize("lens,splits", [([90, 30], 1), ([5000, 2500], 1), ([700, 1, 333], 0)])
def test_latent_wait_that_runs_out_and_the_call_after_it(tlib, lens, splits, s_q):
    """The products that have been issued end before the tensor memory is given back."""
    _stalled_then_right(tlib, _spec(KV_MLA656, len(lens), 1, 576, 32, lens, s_q, splits, seed=92))
