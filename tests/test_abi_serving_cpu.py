"""Host-side checks of the cache with scales per block, the page operators and
the token probabilities, without a GPU: the C entry points refuse bad arguments
with the documented codes before any launch, and the Python binding refuses
tensors that are not what the call reads."""
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
    base = dict(B=4, H_kv=2, G=8, D_qk=128, D_v=128, page_size=16, max_pages_per_seq=10, num_pages=40, kv_dtype=da.KV_FP8_BLOCK,
                splits=0, num_sms=152)
    return da.Desc.make(**{**base, **kw})


BLOCKS = [da.KV_FP8_BLOCK, da.KV_INT8_BLOCK]


@pytest.mark.parametrize("kv", BLOCKS)
def test_block_formats_in_the_attention_calls(lib, kv):
    n = ctypes.c_size_t(0)

    def rc(**kw):
        return lib.decode_attn_sched_meta_bytes(ctypes.byref(_desc(kv_dtype=kv, **kw)), ctypes.byref(n))
    assert rc() == 0 and rc(s_q=4) == 0 and rc(window=64) == 0 and rc(page_size=192) == 0
    assert rc(s_q=5) == -3 and rc(page_size=8) == -3 and rc(D_qk=64, D_v=64) == -3 and rc(topk=8) == -3 and rc(G=4) == -3
    d = _desc(kv_dtype=kv)
    size = da.sched_meta_bytes(d)

    def fwd(ks, vs):
        return lib.decode_attn_fwd(ctypes.byref(d), G, G, G, ks, vs, G, G, G, size, G, G, None)
    assert fwd(None, G) == -8 and fwd(G, None) == -8 and fwd(P(0x100002), G) == -4
    # the operators that do not know the format refuse it
    assert lib.decode_attn_append_kv(ctypes.byref(d), G, G, 0, G, G, G, G, G, G, None, None) == -3
    r = da.Rope.make(128)
    assert lib.decode_attn_rope_append(ctypes.byref(d), ctypes.byref(r), 4, G, 0, G, 0, G, 0, G, G, G, G, G, P(0x900000), G, G, G, G, None,
                                       None) == -3
    assert lib.decode_attn_accum_weights(ctypes.byref(d), G, G, G, G, G, G, size, G, None, None, 1.0, G, None) == -3
    assert lib.decode_attn_evict(ctypes.byref(d), 10, 0, 0, G, G, P(0x200000), G, G, G, G, P(0x300000), None, None) == -3


@pytest.mark.parametrize("kv", BLOCKS)
def test_append_block_refusals(lib, kv):
    def call(d, n=4, k=G, ks=0, v=G, vs=0, starts=G, pos=G, bt=G, kp=G, vp=G, sk=G, sv=G, err=None):
        return lib.decode_attn_append_block(ctypes.byref(d), n, k, ks, v, vs, starts, pos, bt, kp, vp, sk, sv, err, None)
    d = _desc(kv_dtype=kv)
    for name in ("k", "v", "pos", "bt", "kp", "vp"):
        assert call(d, **{name: None}) == -1, name
        assert call(d, **{name: P(0x100008 if name in ("k", "v", "kp", "vp") else 0x100002)}) == -4, name
    for name in ("sk", "sv"):
        assert call(d, **{name: None}) == -8 and call(d, **{name: P(0x100002)}) == -4
    assert call(d, starts=P(0x100001)) == -4 and call(d, err=P(0x100002)) == -4
    assert call(d, n=-1) == -2 and call(d, n=(1 << 30) + 1) == -2
    assert call(d, n=0) == 0 and call(d, n=0, k=None, sk=None) == 0             # nothing to do
    assert call(d, starts=None, n=5) == -2                                      # not B * s_q tokens
    assert call(d, ks=248) == -2 and call(d, vs=260) == -2
    for bad in (dict(B=0), dict(H_kv=0), dict(H_kv=4097), dict(page_size=0), dict(num_pages=0), dict(max_pages_per_seq=1 << 28), dict(s_q=65)):
        assert call(_desc(kv_dtype=kv, **bad)) == -2, bad
    for bad in (dict(D_qk=64, D_v=64), dict(D_v=64), dict(page_size=8), dict(page_size=24), dict(kv_dtype=da.KV_BF16), dict(kv_dtype=da.KV_FP8)):
        assert call(_desc(**{**dict(kv_dtype=kv), **bad})) == -3, bad
    assert lib.decode_attn_append_block(None, 4, *[G, 0] * 2, *[G] * 7, None, None) == -1


def test_page_operator_refusals(lib):
    d = _desc(kv_dtype=99, G=0, D_qk=0)              # the format does not matter to the tables
    Q = [P(0x100000 * i) for i in range(1, 12)]

    def args(names, kw):
        return [kw.get(n, Q[i]) for i, n in enumerate(names)]

    def fork(d, **kw):
        return lib.decode_attn_fork_pages(ctypes.byref(d), *args(("par", "sl", "bt", "held", "refs", "nbt", "nheld", "nsl"), kw), kw.get("err"), None)

    def free(d, **kw):
        return lib.decode_attn_free_pages(ctypes.byref(d), *args(("done", "sl", "bt", "held", "refs"), kw), kw.get("err"), None)

    def reserve(d, **kw):
        return lib.decode_attn_reserve_pages(ctypes.byref(d), *args(("new", "sl", "bt", "held", "refs", "copies", "missing"), kw), kw.get("err"), None)

    def compact(d, **kw):
        return lib.decode_attn_compact_pages(ctypes.byref(d), *args(("bt", "held", "refs", "nbt", "nrefs", "page", "copies", "counts"), kw),
                                             kw.get("err"), None)
    calls = {fork: "par sl bt held refs nbt nheld nsl", free: "done sl bt held refs", reserve: "sl bt held refs copies missing",
             compact: "bt held refs nbt nrefs page copies counts"}
    for call, names in calls.items():
        for name in names.split():
            assert call(d, **{name: None}) == -1, (call, name)
            assert call(d, **{name: P(0x900002)}) == -4, (call, name)
        assert call(d, err=P(0x100001)) == -4
        for bad in (dict(B=0), dict(B=8193), dict(page_size=0), dict(num_pages=0), dict(num_pages=(1 << 23) + 1), dict(max_pages_per_seq=0),
                    dict(max_pages_per_seq=1 << 28), dict(B=8000, max_pages_per_seq=1 << 20, page_size=1)):
            assert call(_desc(**bad)) == -2, (call, bad)
    assert reserve(d, new=P(0x100002)) == -4 and reserve(_desc(s_q=65)) == -2
    assert reserve(d, copies=P(0x600004)) == -4 and compact(d, copies=P(0x600004)) == -4      # pairs
    assert fork(d, nbt=Q[2]) == -3 and fork(d, nheld=Q[3]) == -3 and fork(d, nsl=Q[1]) == -3
    assert compact(d, nbt=Q[0]) == -3 and compact(d, nrefs=Q[2]) == -3 and compact(d, page=Q[2]) == -3
    assert lib.decode_attn_free_pages(None, *Q[:5], None, None) == -1


def test_copy_pages_refusals(lib):
    def call(d, n=4, c=G, nc=None, kp=G, vp=G, ks=G, vs=G, w=None, err=None):
        return lib.decode_attn_copy_pages(ctypes.byref(d), n, c, nc, kp, vp, ks, vs, w, err, None)
    d = _desc()
    for name in ("c", "kp", "vp"):
        assert call(d, **{name: None}) == -1 and call(d, **{name: P(0x100002)}) == -4, name
    for name in ("ks", "vs"):
        assert call(d, **{name: None}) == -8 and call(d, **{name: P(0x100002)}) == -4, name
    for name in ("nc", "w", "err"):
        assert call(d, **{name: P(0x100002)}) == -4, name
    assert call(d, n=0, c=None, kp=None) == 0 and call(d, n=-1) == -2 and call(d, n=(1 << 30) + 1) == -2
    assert call(_desc(kv_dtype=9)) == -3 and call(_desc(page_size=8)) == -3 and call(_desc(D_v=64)) == -3
    assert call(_desc(kv_dtype=da.KV_BF16, D_qk=2, D_v=2, H_kv=1, page_size=3)) == -3          # 12 bytes a page
    assert call(_desc(kv_dtype=da.KV_BF16, H_kv=0)) == -2 and call(_desc(D_qk=5000, D_v=5000)) == -2
    m = _desc(kv_dtype=da.KV_MLA656, H_kv=1, G=128, D_qk=576, D_v=512)
    assert call(m, vp=P(0x200000)) == -3 and call(_desc(kv_dtype=da.KV_MLA656)) == -3


def test_token_probs_refusals(lib):
    def call(B=2, K=3, V=100, lt=0, x=G, ls=0, pt=0, y=P(0x900000), ps=0, err=None, **rules):
        r = da.TokenRules(**{k: (v.value if isinstance(v, P) else v) for k, v in rules.items()})
        return lib.decode_attn_token_probs(B, K, V, lt, x, ls, pt, y, ps, ctypes.byref(r), err, None)
    assert call(x=None) == -1 and call(y=None) == -1
    assert call(x=P(0x100002)) == -4 and call(lt=1, x=P(0x100001)) == -4 and call(pt=2, y=P(0x900001)) == -4 and call(err=P(0x100002)) == -4
    for bad in (dict(B=0), dict(B=(1 << 20) + 1), dict(K=-1), dict(K=64), dict(V=0), dict(V=(1 << 19) - 6), dict(ls=99), dict(ps=99), dict(ls=-1),
                dict(history=G, history_lens=G, history_cols=0), dict(bias_starts=G, n_bias=-1), dict(allowed=G, allowed_stride=3)):
        assert call(**bad) == -2, bad
    for bad in (dict(lt=3), dict(pt=-1)):
        assert call(**bad) == -3
    assert call(history=G, history_cols=5) == -1 and call(bias_starts=G, n_bias=2, bias_tokens=G) == -1
    for name in ("temperature", "repetition", "frequency", "presence", "history_lens", "prompt_lens", "draft_tokens", "bias_starts", "allowed"):
        assert call(**{name: P(0x100002)}) == -4, name
    # the probabilities are the logits' own rows, or apart from them
    assert call(y=P(0x100000 + 400)) == -3 and call(y=G, pt=1) == -3 and call(y=G, ps=200) == -3 and call(y=P(0x100000 - 16)) == -3


def test_binding_refuses_host_tensors_and_shapes():
    z, i32 = torch.zeros, torch.int32
    d = _desc()
    with pytest.raises(da.DecodeAttnError):
        da.append_block(d, z(4, 256), z(4, 256), z(4, dtype=i32), z(4, 10, dtype=i32), z(1), z(1), z(40, 2, 1), z(40, 2, 1))
    b, t, r = z(4, dtype=i32), z(4, 10, dtype=i32), z(40, dtype=i32)
    for call in (lambda: da.fork_pages(d, b, b, t, b, r, t, b, b), lambda: da.free_pages(d, b, b, t, b, r),
                 lambda: da.reserve_pages(d, b, t, b, r, z(4, 2, dtype=i32), z(1, dtype=i32)),
                 lambda: da.compact_pages(d, t, b, r, t, r, r, z(20, 2, dtype=i32), z(2, dtype=i32)),
                 lambda: da.copy_pages(d, z(4, 2, dtype=i32), z(1), z(1), z(40, 2, 1), z(40, 2, 1))):
        with pytest.raises(da.DecodeAttnError):
            call()
    for bad in (dict(logits=z(2, 10)), dict(history=z(2, 5, dtype=i32)), dict(history=z(3, 5, dtype=i32), history_lens=z(2, dtype=i32)), dict()):
        with pytest.raises(da.DecodeAttnError):
            da.token_probs(**{**dict(logits=z(2, 1, 10), probs=z(2, 1, 10)), **bad})
