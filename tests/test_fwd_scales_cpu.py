"""The scales that the attention calls are given with the block formats, without a
GPU: a tensor that the kernel would read past the end of, of another type or
layout, or on another device, is refused before the library is called."""
import pytest
import torch

import paged_kv_cache_60_gb300 as da


class Library:
    """Counts the calls of the attention entry points, and does nothing."""

    def __init__(self):
        self.calls = 0

    def _call(self, *args):
        self.calls += 1
        return 0

    decode_attn_fwd = decode_attn_fwd_ex = _call


class StaticScratch(Library):
    def __init__(self):
        super().__init__()

        def f(*args):
            return self._call(*args)
        f.restype = f.argtypes = None
        self.decode_attn_fwd_static_scratch = f


def _desc(**kw):
    base = dict(B=4, H_kv=2, G=8, D_qk=128, D_v=128, page_size=64, max_pages_per_seq=10, num_pages=40, kv_dtype=da.KV_FP8_BLOCK, splits=0, num_sms=152)
    return da.Desc.make(**{**base, **kw})


def _calls(monkeypatch):
    """Each attention call of the binding as f(desc, k_scale, v_scale), with the library that it reaches."""
    t = torch.zeros(8)
    lib, scratch = Library(), StaticScratch()
    monkeypatch.setattr(da, "load_library", lambda: scratch)
    return [(lambda d, k, v: da.fwd(d, t, t, t, k, v, t, t, t, t, t, stream=0, lib=lib), lib),
            (lambda d, k, v: da.fwd(d, t, t, t, k, v, t, t, t, t, t, stream=0, sinks=t, lib=lib), lib),
            (lambda d, k, v: da.fwd_static_scratch(d, t, t, t, k, v, t, t, t, t, stream=0), scratch)]


GOOD = torch.zeros(40, 2, 4)
BAD = [torch.zeros(2), torch.zeros(40, 2, 3), torch.zeros(39, 2, 4), torch.zeros(40, 2, 4, dtype=torch.bfloat16),
       torch.zeros(40, 2, 8)[:, :, ::2], torch.zeros(1, 2, 4).expand(40, 2, 4), torch.zeros(0)]  # (another device: test_gpu_fwd_scales.py)


@pytest.mark.parametrize("kv", [da.KV_FP8_BLOCK, da.KV_INT8_BLOCK])
@pytest.mark.parametrize("bad", range(len(BAD)))
def test_scales_of_another_size_type_or_place(monkeypatch, kv, bad):
    for call, lib in _calls(monkeypatch):
        for k, v in ((BAD[bad], GOOD), (GOOD, BAD[bad])):
            with pytest.raises(da.DecodeAttnError, match="scale"):
                call(_desc(kv_dtype=kv), k, v)
        assert lib.calls == 0


def test_the_right_ones_and_other_formats(monkeypatch):
    for n, (call, lib) in enumerate(_calls(monkeypatch)):
        before = lib.calls
        call(_desc(), GOOD, GOOD)
        call(_desc(), GOOD.view(80, 4), GOOD.view(-1))    # the same bytes
        call(_desc(), None, GOOD)                         # the library's own check refuses a missing one
        call(_desc(kv_dtype=da.KV_FP8), torch.zeros(2), torch.zeros(2))
        call(_desc(kv_dtype=da.KV_BF16), None, None)
        assert lib.calls == before + 5, n
