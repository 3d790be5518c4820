"""The scales of the block formats in the attention calls of the binding, on the
device: the per-head format's are refused before anything is launched, the right
ones taken, on other streams than the default one too."""
import pytest
import torch

import paged_kv_cache_60_gb300 as da

from gpu_util import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ensure_built()


def _state(kv, P=16, H=2, pages=12, cols=4):
    g = torch.Generator(device="cuda").manual_seed(1)
    desc = da.Desc.make(B=2, H_kv=H, G=8, D_qk=128, D_v=128, page_size=P, max_pages_per_seq=cols, num_pages=pages, kv_dtype=kv)
    x = torch.randn(64, H * 128, device="cuda", generator=g).to(torch.bfloat16)
    pools = [torch.zeros(pages, P, H, 128, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.full((pages, H, P // 16), 7.0, device="cuda") for _ in range(2)]
    table = torch.randperm(pages, device="cuda", generator=g)[:2 * cols].view(2, cols).int()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    da.append_block(desc, x[:50], x[14:], i32([0, 0]), table, *pools, *scales, token_starts=i32([0, 33, 50]))
    q = torch.randn(2, 8 * H, 128, device="cuda", generator=g).to(torch.bfloat16)
    return desc, q, pools, scales, table, i32([33, 17]), [torch.full((2, 8 * H, 128), 9.0, dtype=torch.bfloat16, device="cuda"),
                                                          torch.full((2, 8 * H), 9.0, device="cuda")]


@pytest.mark.parametrize("kv", [da.KV_FP8_BLOCK, da.KV_INT8_BLOCK])
def test_refused_and_taken(kv):
    desc, q, pools, scales, table, lens, out = _state(kv)
    meta = torch.empty(da.sched_meta_bytes(desc), dtype=torch.uint8, device="cuda")
    da.sched_meta(desc, lens, meta)
    for bad in (torch.ones(2, device="cuda"), scales[0][:-1].contiguous(), scales[0].cpu(), scales[0].half(), scales[0][:1].expand(12, 2, 1)):
        for ks, vs in ((bad, scales[1]), (scales[0], bad)):
            with pytest.raises(da.DecodeAttnError, match="scales"):
                da.fwd(desc, q, *pools, ks, vs, table, lens, meta, *out)
            with pytest.raises(da.DecodeAttnError, match="scales"):
                da.fwd_static_scratch(desc, q, *pools, ks, vs, table, lens, *out)
    torch.cuda.synchronize()
    assert (out[0] == 9).all() and (out[1] == 9).all()
    with pytest.raises(da.DecodeAttnError):
        da.fwd(desc, q, *pools, None, scales[1], table, lens, meta, *out)
    da.fwd(desc, q, *pools, *scales, table, lens, meta, *out)
    want = [t.clone() for t in out]
    assert torch.isfinite(want[1]).all() and not (want[0] == 9).any()
    # without scratch of the caller's, on the default stream (the first call, which prepares the buffer) and on another
    for stream in (None, torch.cuda.Stream()):
        for t in out:
            t.zero_()
        torch.cuda.synchronize()
        if stream is None:
            da.fwd_static_scratch(desc, q, *pools, *scales, table, lens, *out)
        else:
            with torch.cuda.stream(stream):               # the current stream is what the binding takes
                da.fwd_static_scratch(desc, q, *pools, *scales, table, lens, *out)
            stream.synchronize()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
