"""Host-side checks of the operators around decode attention, without a GPU:
the C entry points refuse bad arguments with the documented codes before any
launch, and the Python binding refuses tensors that are not what the call
reads."""
import ctypes

import pytest
import torch

import paged_kv_cache_60_gb300 as da
from paged_kv_cache_60_gb300 import build as dabuild

P = ctypes.c_void_p
G = P(0x100000)          # a well-aligned address that nothing may read


@pytest.fixture(scope="module")
def lib():
    dabuild.build()
    return da.load_library()


def _desc(**kw):
    base = dict(B=4, H_kv=2, G=8, D_qk=128, D_v=128, page_size=16, max_pages_per_seq=10, num_pages=40,
                kv_dtype=da.KV_BF16, splits=0, num_sms=152)
    base.update(kw)
    return da.Desc.make(**base)


def _latent(**kw):
    return _desc(**{**dict(kv_dtype=da.KV_MLA656, H_kv=1, G=128, D_qk=576, D_v=512), **kw})


def _rope(rot=128, sections=(64,), **kw):
    return da.Rope.make(rot, sections, **kw)


def test_rope_append_refusals(lib):
    def call(d, r=None, n=4, q=G, qs=0, k=P(0x300000), ks=0, v=P(0x400000), vs=0, freq=G, at=G, req=G, pos=G, bt=G, out=P(0x900000), kp=G, vp=G,
             sk=None, sv=None, err=None):
        return lib.decode_attn_rope_append(ctypes.byref(d), ctypes.byref(r or _rope()), n, q, qs, k, ks, v, vs, freq, at, req,
                                           pos, bt, out, kp, vp, sk, sv, err, None)
    d = _desc()
    for name in ("q", "k", "v", "freq", "at", "pos", "bt", "out", "kp", "vp"):
        assert call(d, **{name: None}) == -1, name
        off = 8 if name in ("q", "k", "v", "out", "kp", "vp") else 2
        assert call(d, **{name: P(0x900000 + off)}) == -4, name
    assert call(d, req=P(0x100002)) == -4 and call(d, err=P(0x100002)) == -4
    assert call(d, n=-1) == -2 and call(d, n=(1 << 30) + 1) == -2
    assert call(d, n=0) == 0 and call(d, n=0, q=None, out=None) == 0          # nothing to do
    assert call(d, req=None, n=5) == -2                                       # not B * s_q tokens
    for bad in (_rope(8, (4,)), _rope(24, (12,)), _rope(144, (72,)), _rope(64, (30,)), _rope(64, (40, -8)),
                da.Rope(64, 0, (ctypes.c_int32 * 4)(32, 0, 0, 0), 0, 0), da.Rope(64, 5, (ctypes.c_int32 * 4)(32, 0, 0, 0), 0, 0),
                da.Rope(64, 1, (ctypes.c_int32 * 4)(16, 16, 0, 0), 0, 0)):
        assert call(d, bad) == -2
    assert call(d, qs=2 * 8 * 128 - 8) == -2 and call(d, qs=2 * 8 * 128 + 4) == -2
    assert call(d, ks=128) == -2 and call(d, vs=2 * 128 + 1) == -2
    assert call(_desc(G=0)) == -2 and call(_desc(D_qk=100, D_v=100)) == -3 and call(_desc(D_qk=128, D_v=64)) == -3
    assert call(_desc(kv_dtype=9)) == -3
    assert call(_desc(kv_dtype=da.KV_FP8)) == -8 and call(_desc(kv_dtype=da.KV_FP8), sk=G, sv=P(0x100002)) == -4
    # q_out is q row for row, or apart from it
    assert call(d, out=P(0x100000 + 2 * 128)) == -3 and call(d, out=G, qs=2 * 8 * 128 * 2) == -3
    assert call(d, out=P(0x300000 - 0x1000)) == -3 and call(d, out=P(0x400000 + 2 * 4 * 256 - 16)) == -3
    m = _latent()
    assert call(m, _rope(64, (32,))) == -3                                    # no v_new
    assert call(m, _rope(128, (64,)), v=None, vp=None) == -2                  # more than the 64 RoPE values
    assert call(m, _rope(64, (32,)), v=None, vp=P(0x200000)) == -3
    assert lib.decode_attn_rope_append(ctypes.byref(d), None, 4, *[G, 0] * 3, *[G] * 8, None, None, None, None) == -1


def test_accum_weights_refusals(lib):
    def call(d, q=G, k=G, sk=None, bt=G, sl=G, meta=G, n=None, lse=G, acc=None, wl=None, decay=1.0, w=G):
        size = n if n is not None else da.sched_meta_bytes(d)
        return lib.decode_attn_accum_weights(ctypes.byref(d), q, k, sk, bt, sl, meta, size, lse, acc, wl, decay, w, None)
    d = _desc()
    for name in ("q", "k", "bt", "sl", "meta", "lse", "w"):
        assert call(d, **{name: None}) == -1, name
        assert call(d, **{name: P(0x100008)}) == -4, name
    assert call(d, acc=P(0x100002)) == -4 and call(d, wl=P(0x100001)) == -4
    assert call(d, n=da.sched_meta_bytes(d) - 16) == -6
    for decay in (-0.5, float("inf"), float("nan")):
        assert call(d, decay=decay) == -2
    assert call(_desc(window=64)) == -3
    assert call(_desc(kv_dtype=da.KV_FP8)) == -8
    assert call(_desc(D_qk=96, D_v=96), n=1 << 30) == -3 and call(_desc(s_q=5), n=1 << 30) == -3
    assert call(_desc(num_pages=1 << 28), n=1 << 30) == -2
    assert call(_latent(num_sms=2, topk=64), n=1 << 30) == -3                 # sparse decode
    long = [_latent(num_sms=2, B=1, page_size=64, max_pages_per_seq=(1 << 25) - k) for k in (2, 5)]
    assert call(long[0], q=None) == -2 and call(long[1], q=None) == -1        # token indices end below 2^31 - 256


def test_evict_refusals(lib):
    def call(d, budget=100, first=4, last=8, sl=G, bt=G, dt=P(0x200000), kp=G, vp=G, w=G, kept=G, new=P(0x300000), err=None):
        return lib.decode_attn_evict(ctypes.byref(d), budget, first, last, sl, bt, dt, kp, vp, w, kept, new, err, None)
    d = _desc()
    for name in ("sl", "bt", "dt", "kp", "vp", "w", "kept", "new"):
        assert call(d, **{name: None}) == -1, name
        assert call(d, **{name: P(0x700008 if name in ("kp", "vp") else 0x700002)}) == -4, name
    assert call(d, err=P(0x100002)) == -4
    for bad in (dict(budget=0), dict(budget=161), dict(first=-1), dict(last=-1), dict(first=50, last=51)):
        assert call(d, **bad) == -2, bad
    assert call(d, dt=G) == -3 and call(d, new=G) == -3                       # the tables, or the lengths, are one
    assert call(_desc(kv_dtype=da.KV_FP8, D_qk=72, D_v=72)) == -3             # rows of 16-byte vectors
    assert call(_desc(D_qk=100, D_v=100)) == -3
    assert call(_latent(), vp=P(0x400000)) == -3
    assert call(_desc(B=1, max_pages_per_seq=(1 << 26) + 1)) == -2            # over 2^30 tokens a request
    assert call(_desc(B=1 << 22, H_kv=256, max_pages_per_seq=10)) == -2


def test_verify_drafts_refusals(lib):
    def call(B=2, K=3, V=100, kind=0, p=G, ps=0, q=G, qs=0, x=G, u=G, sl=None, a=G, out=G, new=None, err=None):
        return lib.decode_attn_verify_drafts(B, K, V, kind, p, ps, q, qs, x, u, sl, a, out, new, err, None)
    for name in ("p", "x", "u", "a", "out"):
        assert call(**{name: None}) == -1, name
        assert call(**{name: P(0x100002)}) == -4, name
    assert call(kind=1, p=P(0x100001)) == -4 and call(kind=2, q=P(0x100003)) == -4
    assert call(sl=G) == -1 and call(new=G) == -1                             # lengths: both or neither
    assert call(sl=G, new=P(0x100002)) == -4
    for bad in (dict(B=0), dict(K=-1), dict(K=64), dict(V=0), dict(V=1 << 20), dict(ps=99), dict(qs=99), dict(ps=-1)):
        assert call(**bad) == -2, bad
    assert call(kind=3) == -3 and call(kind=-1) == -3


def test_binding_refuses_host_tensors_and_shapes():
    d = _desc()
    z = torch.zeros
    i32 = torch.int32
    with pytest.raises(da.DecodeAttnError):
        da.verify_drafts(z(2, 4, 10), z(2, 3, 10), z(2, 3, dtype=i32), z(2, 4), z(2, dtype=i32), z(2, 4, dtype=i32))
    with pytest.raises(da.DecodeAttnError):
        da.verify_drafts(z(2, 10), None, None, z(2, 1), z(2, dtype=i32), z(2, 1, dtype=i32))
    with pytest.raises(da.DecodeAttnError):
        da.evict(d, 4, z(4, dtype=i32), z(4, 10, dtype=i32), z(4, 10, dtype=i32), z(1), z(1), z(1), z(1), z(1))
    with pytest.raises(da.DecodeAttnError):
        da.accum_weights(d, z(4, 16, 128), z(1), None, z(1), z(1), z(1), z(4, 16), z(1))
    with pytest.raises(da.DecodeAttnError):
        da.rope_append(d, _rope(), z(4, 2048), z(4, 256), z(4, 256), z(64), z(1, 4), z(4, dtype=i32), z(4, 10), z(4, 2048), z(1), z(1))
    with pytest.raises(da.DecodeAttnError):
        da.Rope.make(64, [8, 8, 8, 4, 4])
