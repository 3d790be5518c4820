"""A wait of the attention call that runs out in parts of a few chunks: all of
their copies have been issued before a consumer gives up, and they land before
the CTA ends. Test build, 1 ms; the next call matches the oracle."""
import pytest
import torch

import oracle
import paged_kv_cache_60_gb300 as da
from workloads import KV_BF16, KV_FP8, WorkloadSpec, make_workload

from gpu_util import LSE_TOL, OUT_TOL, DeviceWorkload, debug_build_library, make_desc, max_err

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tlib():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    oracle.build_oracle()
    return debug_build_library()


@pytest.mark.parametrize("kv,D,s_q", [(KV_BF16, 128, 1), (KV_BF16, 64, 1), (KV_FP8, 128, 1), (KV_BF16, 128, 2)])
@pytest.mark.parametrize("lengths,splits", [([5, 64, 130, 0], 1), ([200, 90, 1, 129], 0)])
def test_parts_whose_copies_are_all_issued(tlib, kv, D, s_q, lengths, splits):
    spec = WorkloadSpec(name="t", B=4, H_kv=2, G=8, D_qk=D, D_v=D, page_size=16, kv_dtype=kv, lengths=lengths, splits=splits, seed=53,
                        s_q=s_q)
    w = make_workload(spec)
    dw, desc = DeviceWorkload(w), make_desc(w)
    rows = (4, 16) if s_q == 1 else (4, s_q, 16)

    def call():
        meta = torch.empty(da.sched_meta_bytes(desc), dtype=torch.uint8, device="cuda")
        out, lse = torch.zeros(*rows, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(*rows, device="cuda")
        da.sched_meta(desc, dw.cache_seqlens, meta, lib=tlib)
        da.fwd(desc, dw.q, dw.k_pool, dw.v_pool, dw.k_scale, dw.v_scale, dw.block_table, dw.cache_seqlens, meta, out, lse, lib=tlib)
        torch.cuda.synchronize()
        return out, lse, da.get_error(meta)

    assert tlib.decode_attn_debug_wait_limit(1000000) == 0
    assert tlib.decode_attn_debug_stall(1) == 0
    try:
        assert call()[2] & da.DA_DEV_TIMEOUT
    finally:
        tlib.decode_attn_debug_stall(0)
        tlib.decode_attn_debug_wait_limit(0)
    out, lse, err = call()
    assert err == 0
    e_out, e_lse = max_err(out, lse, *(oracle.attend(w) if s_q == 1 else oracle.attend_multi(w)))
    assert e_out <= OUT_TOL and e_lse <= LSE_TOL, (e_out, e_lse)
