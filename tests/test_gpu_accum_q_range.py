"""The e4m3 accumulation multiplies with q as f16, as the attention call does:
values below 2^-14 lose bits, and the weights are those of the rounded q, whose
lse the attention call gave. A bf16 value above 65504 is infinite there."""
import math

import pytest
import torch

import paged_kv_cache_60_gb300 as da
from workloads import KV_FP8

from gpu_util import ensure_built, run
from test_gpu_accum import Step, _spec

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_built()


@pytest.mark.parametrize("s_q", [1, 2, 4])
def test_small_queries(s_q):
    s = Step(_spec(KV_FP8, 2, 2, 128, 16, [90, 41], s_q, 0, seed=95))
    down = 2.0 ** -19                                   # six of the eight significant bits are left, and fewer
    s.dw.q.mul_(down)
    s.dw.k_scale.mul_(1 / down)
    s.w.k_scale = s.dw.k_scale.cpu()
    s.w.q = s.dw.q.cpu().half().float()
    assert not torch.equal(s.w.q, s.dw.q.cpu().float())
    s.out, s.lse, s.meta, s.desc = run(s.w, dw=s.dw)
    got = s.run()
    s.check(got)
    assert da.get_error(s.meta) == 0


def test_queries_beyond_f16():
    """An infinite query value reaches its own KV head's weights only, as it does the attention's rows."""
    s = Step(_spec(KV_FP8, 1, 2, 128, 16, [70], 1, 0, seed=96))
    s.dw.q[0, 3, 5] = 70000.0                           # a query head of KV head 0
    s.out, s.lse, s.meta, s.desc = run(s.w, dw=s.dw)
    assert not torch.isfinite(s.lse[0, 3]) and torch.isfinite(s.lse[0, 8:]).all()
    got = s.run().cpu()
    for t in range(70):
        v = got[int(s.w.block_table[0, t // 16]), :, t % 16]
        assert math.isfinite(float(v[1]))
    assert torch.isnan(got[s.w.block_table[0, :4].long(), 0]).any()
