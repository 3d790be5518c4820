"""How the binding hands addresses and streams to decode_attn_fwd_static_scratch,
without a GPU: a stand-in of the C function with the same types receives all 64
bits of them."""
import ctypes

import pytest
import torch

import paged_kv_cache_60_gb300 as da
from paged_kv_cache_60_gb300 import build as dabuild


def test_the_functions_types_are_declared():
    dabuild.build()
    lib = da.load_library()
    t = torch.zeros(8)
    with pytest.raises(da.DecodeAttnError):                # refused before anything is launched
        da.fwd_static_scratch(da.Desc.make(B=0, H_kv=1, G=8, D_qk=64, D_v=64, page_size=16, max_pages_per_seq=1, num_pages=1, kv_dtype=da.KV_BF16),
                              t, t, t, None, None, t, t, t, t, stream=0)
    f = lib.decode_attn_fwd_static_scratch
    assert f.argtypes is not None and len(f.argtypes) == 11 and f.argtypes[1:] == [ctypes.c_void_p] * 10


def test_a_streams_handle_arrives_whole(monkeypatch):
    got = []
    P = ctypes.c_void_p

    class Library:
        # a foreign function without declared types, as a library's attribute is at first
        pass
    callback = ctypes.CFUNCTYPE(ctypes.c_int, P, P, P, P, P, P, P, P, P, P, P)(lambda *a: got.append(a) or 0)
    prototype = ctypes.CDLL(None).abs.__class__            # (its declared types can be set and are empty)
    f = prototype(ctypes.cast(callback, P).value)
    f.argtypes = None
    lib = Library()
    lib.decode_attn_fwd_static_scratch = f
    monkeypatch.setattr(da, "load_library", lambda: lib)
    t = torch.zeros(8)
    d = da.Desc.make(B=1, H_kv=1, G=8, D_qk=64, D_v=64, page_size=16, max_pages_per_seq=1, num_pages=1, kv_dtype=da.KV_BF16)
    handle = 0x7F12_3456_89AB_CDE0
    monkeypatch.setattr(da, "_stream", lambda stream, dev=None: handle)   # as the current stream's handle comes
    da.fwd_static_scratch(d, t, t, t, None, None, t, t, t, t)
    assert got[0][10] == handle and got[0][1] == t.data_ptr() and got[0][4] is None
