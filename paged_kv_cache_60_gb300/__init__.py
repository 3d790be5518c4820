"""Paged-KV decode attention for GB300 (sm_103a).

A thin Python binding over the C ABI in include/decode_attn.h. The entry
points keep the C names without the ``decode_attn_`` prefix; each one only
marshals arguments (tensor data pointers, the current CUDA stream) and calls
the shared library, which runs every step in its own CUDA kernels. There is no
fallback: if the library is missing or was built for another machine, the
import raises.

    desc = Desc.make(B=..., H_kv=..., G=..., D_qk=..., D_v=..., page_size=...,
                     max_pages_per_seq=..., num_pages=..., kv_dtype=KV_BF16)
    meta = torch.empty(sched_meta_bytes(desc), dtype=torch.uint8, device="cuda")
    sched_meta(desc, cache_seqlens, meta)
    fwd(desc, q, k_pool, v_pool, k_scale, v_scale, block_table, cache_seqlens, meta, out, lse)

Around the step: append_kv and rope_append write new tokens, verify_drafts
accepts a chain of drafts, accum_weights gathers the attention weight of cached
tokens and evict keeps the heaviest. All but append_kv check every
tensor's dtype, shape, strides and device and raise DecodeAttnError.
"""
import ctypes
import os

from . import build as _build_mod

KV_BF16 = 0
KV_FP8 = 1
KV_MLA656 = 2

PROB_F32 = 0
PROB_BF16 = 1
PROB_F16 = 2

DA_OK = 0
DA_ERR_NULL = -1
DA_ERR_DIMS = -2
DA_ERR_UNSUPPORTED = -3
DA_ERR_ALIGN = -4
DA_ERR_SPLITS = -5
DA_ERR_META_SIZE = -6
DA_ERR_CUDA = -7
DA_ERR_SCALE = -8

DA_DEV_BAD_PAGE = 1
DA_DEV_SEQ_TOO_LONG = 2
DA_DEV_NEG_LEN = 4
DA_DEV_TIMEOUT = 8
DA_DEV_META_MISMATCH = 16
DA_DEV_BAD_TOKEN = 32
DA_DEV_BAD_PROBS = 64
DA_DEV_BAD_REQUEST = 128

LIB_PATH = _build_mod.LIB_PATH


class Desc(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H_kv", ctypes.c_int32), ("G", ctypes.c_int32),
                ("D_qk", ctypes.c_int32), ("D_v", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("max_pages_per_seq", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("kv_dtype", ctypes.c_int32), ("splits", ctypes.c_int32), ("num_sms", ctypes.c_int32),
                ("softmax_scale", ctypes.c_float), ("s_q", ctypes.c_int32), ("window", ctypes.c_int32),
                ("topk", ctypes.c_int32)]

    @classmethod
    def make(cls, B, H_kv, G, D_qk, D_v, page_size, max_pages_per_seq, num_pages, kv_dtype=KV_BF16,
             splits=0, num_sms=0, softmax_scale=0.0, s_q=1, window=0, topk=0):
        return cls(B, H_kv, G, D_qk, D_v, page_size, max_pages_per_seq, num_pages, kv_dtype, splits,
                   num_sms, softmax_scale, s_q, window, topk)


class LaunchOpts(ctypes.Structure):
    _fields_ = [("use_pdl", ctypes.c_int32), ("main_begin", ctypes.c_void_p), ("main_end", ctypes.c_void_p),
                ("sinks", ctypes.c_void_p), ("indices", ctypes.c_void_p)]


class Rope(ctypes.Structure):
    """Rotary positions with one or several axes (da_rope in the header)."""
    _fields_ = [("rot_dim", ctypes.c_int32), ("n_axes", ctypes.c_int32), ("sections", ctypes.c_int32 * 4),
                ("interleaved", ctypes.c_int32), ("adjacent", ctypes.c_int32)]

    @classmethod
    def make(cls, rot_dim, sections=None, interleaved=False, adjacent=False):
        """``sections``: pairs per axis (default: one axis with all of them)."""
        sections = [rot_dim // 2] if sections is None else [int(x) for x in sections]
        if not 1 <= len(sections) <= 4:
            raise DecodeAttnError("1 to 4 axes are supported")
        return cls(rot_dim, len(sections), (ctypes.c_int32 * 4)(*sections), int(interleaved), int(adjacent))


class DecodeAttnError(RuntimeError):
    pass


_libs = {}


def load_library(path: str = LIB_PATH):
    """Load the shared library (raises if it has not been built). Each path is
    loaded once; the default path is the one every entry point below uses
    unless it is given another handle (``lib=``)."""
    if path in _libs:
        return _libs[path]
    if not os.path.exists(path):
        raise DecodeAttnError(f"CUDA library not built: {path} (run paged_kv_cache_60_gb300/build.py)")
    lib = ctypes.CDLL(path)
    P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    DP = ctypes.POINTER(Desc)
    lib.decode_attn_sched_meta_bytes.argtypes = [DP, ctypes.POINTER(SZ)]
    lib.decode_attn_meta_offsets.argtypes = [DP, ctypes.POINTER(SZ)]
    lib.decode_attn_num_parts.argtypes = [DP, ctypes.POINTER(I32)]
    lib.decode_attn_sched_meta.argtypes = [DP, P, P, SZ, P]
    lib.decode_attn_fwd.argtypes = [DP, P, P, P, P, P, P, P, P, SZ, P, P, P]
    lib.decode_attn_fwd_ex.argtypes = [DP, P, P, P, P, P, P, P, P, SZ, P, P, ctypes.POINTER(LaunchOpts), P]
    lib.decode_attn_get_error.argtypes = [P, ctypes.POINTER(I32), P]
    lib.decode_attn_append_kv.argtypes = [DP, P, P, ctypes.c_int64, P, P, P, P, P, P, P, P]
    I64, F32 = ctypes.c_int64, ctypes.c_float
    lib.decode_attn_rope_append.argtypes = [DP, ctypes.POINTER(Rope), I32, P, I64, P, I64, P, I64, P, P, P, P, P, P,
                                            P, P, P, P, P, P]
    lib.decode_attn_accum_weights.argtypes = [DP, P, P, P, P, P, P, SZ, P, P, P, F32, P, P]
    lib.decode_attn_evict.argtypes = [DP, I32, I32, I32, P, P, P, P, P, P, P, P, P, P]
    lib.decode_attn_verify_drafts.argtypes = [I32, I32, I32, I32, P, I64, P, I64, P, P, P, P, P, P, P, P]
    lib.decode_attn_strerror.argtypes = [ctypes.c_int]
    lib.decode_attn_strerror.restype = ctypes.c_char_p
    for f in ("decode_attn_sched_meta_bytes", "decode_attn_meta_offsets", "decode_attn_num_parts",
              "decode_attn_sched_meta", "decode_attn_fwd", "decode_attn_fwd_ex", "decode_attn_get_error",
              "decode_attn_append_kv", "decode_attn_rope_append", "decode_attn_accum_weights", "decode_attn_evict",
              "decode_attn_verify_drafts"):
        getattr(lib, f).restype = ctypes.c_int
    _libs[path] = lib
    return lib


def strerror(code: int) -> str:
    return load_library().decode_attn_strerror(int(code)).decode()


def _check(rc: int):
    if rc != DA_OK:
        raise DecodeAttnError(f"decode_attn error {rc}: {strerror(rc)}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream, dev=None):
    """The stream's handle; None: the current stream (of device ``dev``, if the caller has looked it up)."""
    import torch
    if stream is None:
        # the handle alone: building a Stream object costs more than a small call's launch
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None and (dev is not None or torch.cuda.is_initialized()):
            return raw(torch.cuda.current_device() if dev is None else dev) or None
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def sched_meta_bytes(desc: Desc) -> int:
    n = ctypes.c_size_t(0)
    _check(load_library().decode_attn_sched_meta_bytes(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def meta_offsets(desc: Desc):
    offs = (ctypes.c_size_t * 8)()
    _check(load_library().decode_attn_meta_offsets(ctypes.byref(desc), offs))
    return list(offs)


def num_parts(desc: Desc) -> int:
    n = ctypes.c_int32(0)
    _check(load_library().decode_attn_num_parts(ctypes.byref(desc), ctypes.byref(n)))
    return n.value


def sched_meta(desc: Desc, cache_seqlens, meta, stream=None, lib=None):
    _check((lib or load_library()).decode_attn_sched_meta(ctypes.byref(desc), _ptr(cache_seqlens), _ptr(meta),
                                                 meta.numel() * meta.element_size(), _stream(stream)))


def fwd(desc: Desc, q, k_pool, v_pool, k_scale, v_scale, block_table, cache_seqlens, meta, out, lse,
        stream=None, use_pdl=True, main_begin=None, main_end=None, sinks=None, indices=None, lib=None):
    lib = lib or load_library()
    args = (ctypes.byref(desc), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(k_scale), _ptr(v_scale),
            _ptr(block_table), _ptr(cache_seqlens), _ptr(meta), meta.numel() * meta.element_size(),
            _ptr(out), _ptr(lse))
    if use_pdl and main_begin is None and main_end is None and sinks is None and indices is None:
        _check(lib.decode_attn_fwd(*args, _stream(stream)))
    else:
        def ev(e):
            if e is None:
                return None
            if not e.cuda_event:     # torch creates events lazily, at their first record
                e.record()
            return ctypes.c_void_p(e.cuda_event)
        opts = LaunchOpts(1 if use_pdl else 0, ev(main_begin), ev(main_end),
                          None if sinks is None else ctypes.c_void_p(sinks.data_ptr()),
                          None if indices is None else ctypes.c_void_p(indices.data_ptr()))
        _check(lib.decode_attn_fwd_ex(*args, ctypes.byref(opts), _stream(stream)))


def fwd_static_scratch(desc: Desc, q, k_pool, v_pool, k_scale, v_scale, block_table, cache_seqlens, out, lse,
                       stream=None):
    """sched_meta + fwd without any caller scratch, for callers that cannot
    allocate device memory; see decode_attn_fwd_static_scratch in the header
    (fixed 16 MiB library buffer, first call per device before any capture,
    overlapping calls race)."""
    lib = load_library()
    f = lib.decode_attn_fwd_static_scratch
    if f.restype is not ctypes.c_int:
        P = ctypes.c_void_p
        f.argtypes = [ctypes.POINTER(Desc), P, P, P, P, P, P, P, P, P, P]
        f.restype = ctypes.c_int
    _check(f(ctypes.byref(desc), _ptr(q), _ptr(k_pool), _ptr(v_pool), _ptr(k_scale), _ptr(v_scale),
             _ptr(block_table), _ptr(cache_seqlens), _ptr(out), _ptr(lse), _stream(stream)))


def append_kv(desc: Desc, k_new, v_new, positions, block_table, k_pool, v_pool, k_scale=None, v_scale=None,
              device_error=None, new_row_stride=0, stream=None, lib=None):
    """Write each request's new token (bf16 rows of k_new / v_new, v_new None
    for the 656-byte token) into slot positions[b] % page_size of page
    block_table[b][positions[b] // page_size], quantising for e4m3 pools;
    see decode_attn_append_kv in the header. ``device_error``: optional
    device int32 tensor that receives the error bits."""
    _check((lib or load_library()).decode_attn_append_kv(
        ctypes.byref(desc), _ptr(k_new), _ptr(v_new), int(new_row_stride), _ptr(positions), _ptr(block_table),
        _ptr(k_pool), _ptr(v_pool), _ptr(k_scale), _ptr(v_scale), _ptr(device_error), _stream(stream)))


def _device():
    """The current CUDA device's index (one that no tensor has, before CUDA is in use)."""
    import torch
    return torch.cuda.current_device() if torch.cuda.is_initialized() else -2


def _need(dev, name, t, dtype, shape=None):
    """A contiguous tensor of this dtype (and shape) on device ``dev``; its address."""
    if t.dtype is dtype and t.get_device() == dev and t.is_contiguous() and (shape is None or t.shape == shape):
        return t.data_ptr()
    want = "" if shape is None else f" of shape {tuple(shape)}"
    raise DecodeAttnError(f"{name}: want a contiguous {dtype} tensor{want} on the current CUDA device, "
                          f"got {t.dtype} {tuple(t.shape)} on {t.device}, strides {t.stride()}")


def _opt(dev, name, t, dtype, shape=None):
    return None if t is None else _need(dev, name, t, dtype, shape)


def _rows(dev, name, t, dtype, n, width):
    """n rows of `width` contiguous values; their address and the distance between rows."""
    d = t.dim()
    if not (t.dtype is dtype and t.get_device() == dev and d in (2, 3) and t.shape[0] == n and t.numel() == n * width
            and t.stride(d - 1) == 1 and (d == 2 or t.stride(1) == t.shape[2]) and (n < 2 or t.stride(0) >= width)):
        raise DecodeAttnError(f"{name}: want a {dtype} tensor of {n} rows of {width} contiguous values on the current "
                              f"CUDA device, got {t.dtype} {tuple(t.shape)} on {t.device}, strides {t.stride()}")
    return t.data_ptr(), (t.stride(0) if n > 1 else width)


def _pool(dev, name, t, desc):
    """A pool of this desc, given by its bytes ([num_pages][page_size][H_kv][row]); its address."""
    row = 656 if desc.kv_dtype == KV_MLA656 else desc.D_qk * (2 if desc.kv_dtype == KV_BF16 else 1)
    if not (t.get_device() == dev and t.is_contiguous()
            and t.numel() * t.element_size() == desc.num_pages * desc.page_size * desc.H_kv * row):
        raise DecodeAttnError(f"{name}: not a pool of this desc on the current CUDA device "
                              f"({t.dtype} {tuple(t.shape)} on {t.device}, strides {t.stride()})")
    return t.data_ptr()


def rope_append(desc: Desc, rope: Rope, q, k_new, v_new, inv_freq, rope_positions, positions, block_table, q_out,
                k_pool, v_pool, k_scale=None, v_scale=None, requests=None, device_error=None, stream=None, lib=None):
    """Rotate the new tokens' q and K by their positions (one or several axes)
    and write K and V into the pool, any number of tokens per request; see
    decode_attn_rope_append in the header. ``q`` [N, H_q * D] (or [N, H_q, D]),
    ``k_new`` and ``v_new`` [N, H_kv * D] (v_new None and k_new [N, 576] for the
    656-byte token) may be column slices of one projection output;
    ``rope_positions`` int32 [n_axes, N], ``positions`` and ``requests`` int32
    [N]. ``q_out`` bf16 [N, H_q, D] may be ``q``."""
    import torch
    bf16, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    dev, n, D, heads = _device(), positions.numel(), desc.D_qk, (desc.H_kv,)
    q_len, kv_len = desc.H_kv * desc.G * D, desc.H_kv * D
    qp, qs = _rows(dev, "q", q, bf16, n, q_len)
    kp, ks = _rows(dev, "k_new", k_new, bf16, n, kv_len)
    vp, vs = (None, 0) if v_new is None else _rows(dev, "v_new", v_new, bf16, n, kv_len)
    if q_out.numel() != n * q_len:
        raise DecodeAttnError(f"q_out: want {n} rows of {q_len} values, got {tuple(q_out.shape)}")
    _check((lib or load_library()).decode_attn_rope_append(
        ctypes.byref(desc), ctypes.byref(rope), n, qp, qs, kp, ks, vp, vs,
        _need(dev, "inv_freq", inv_freq, f32, (rope.rot_dim // 2,)),
        _need(dev, "rope_positions", rope_positions, i32, (rope.n_axes, n)),
        _opt(dev, "requests", requests, i32, (n,)), _need(dev, "positions", positions, i32),
        _need(dev, "block_table", block_table, i32, (desc.B, desc.max_pages_per_seq)),
        _need(dev, "q_out", q_out, bf16), _pool(dev, "k_pool", k_pool, desc),
        None if v_pool is None else _pool(dev, "v_pool", v_pool, desc), _opt(dev, "k_scale", k_scale, f32, heads),
        _opt(dev, "v_scale", v_scale, f32, heads), _opt(dev, "device_error", device_error, i32), _stream(stream, dev)))


def accum_weights(desc: Desc, q, k_pool, k_scale, block_table, cache_seqlens, meta, lse, weights, num_accepted=None,
                  weighted_lens=None, decay=1.0, stream=None, lib=None):
    """Add the softmax weights of the step's attention call to ``weights`` (fp32
    [num_pages, H_kv, page_size]); q, block_table, cache_seqlens, meta and lse are
    that call's. ``num_accepted`` int32 [B]: query tokens 0..a of a verified chain
    count; ``weighted_lens`` int32 [B]: tokens past it start from 0. See
    decode_attn_accum_weights in the header."""
    import torch
    i32, f32 = torch.int32, torch.float32
    dev, B = _device(), desc.B
    rows = B * max(1, desc.s_q) * desc.H_kv * desc.G
    if q.numel() != rows * desc.D_qk or lse.numel() != rows:
        raise DecodeAttnError(f"q {tuple(q.shape)} and lse {tuple(lse.shape)} are not of this desc")
    _check((lib or load_library()).decode_attn_accum_weights(
        ctypes.byref(desc), _need(dev, "q", q, torch.bfloat16), _pool(dev, "k_pool", k_pool, desc),
        _opt(dev, "k_scale", k_scale, f32, (desc.H_kv,)),
        _need(dev, "block_table", block_table, i32, (B, desc.max_pages_per_seq)),
        _need(dev, "cache_seqlens", cache_seqlens, i32, (B,)), _need(dev, "meta", meta, meta.dtype),
        meta.numel() * meta.element_size(), _need(dev, "lse", lse, f32),
        _opt(dev, "num_accepted", num_accepted, i32, (B,)), _opt(dev, "weighted_lens", weighted_lens, i32, (B,)),
        decay, _need(dev, "weights", weights, f32, (desc.num_pages, desc.H_kv, desc.page_size)), _stream(stream, dev)))


def evict(desc: Desc, budget, cache_seqlens, block_table, dst_block_table, k_pool, v_pool, weights, kept, new_seqlens,
          keep_first=0, keep_last=0, device_error=None, stream=None, lib=None):
    """Cut every request's cache to ``budget`` tokens per KV head (the first
    ``keep_first``, the last ``keep_last`` and the heaviest between them by
    ``weights``), copied in their order to the pages of ``dst_block_table``;
    ``kept`` int32 [B, H_kv, budget] gets their positions, ``new_seqlens`` the
    lengths. See decode_attn_evict in the header."""
    import torch
    i32, dev, B = torch.int32, _device(), desc.B
    table = (B, desc.max_pages_per_seq)
    _check((lib or load_library()).decode_attn_evict(
        ctypes.byref(desc), budget, keep_first, keep_last, _need(dev, "cache_seqlens", cache_seqlens, i32, (B,)),
        _need(dev, "block_table", block_table, i32, table), _need(dev, "dst_block_table", dst_block_table, i32, table),
        _pool(dev, "k_pool", k_pool, desc), None if v_pool is None else _pool(dev, "v_pool", v_pool, desc),
        _need(dev, "weights", weights, torch.float32, (desc.num_pages, desc.H_kv, desc.page_size)),
        _need(dev, "kept", kept, i32, (B, desc.H_kv, budget)), _need(dev, "new_seqlens", new_seqlens, i32, (B,)),
        _opt(dev, "device_error", device_error, i32), _stream(stream, dev)))


def _prob_rows(dev, name, t, dtype, shape):
    """Probabilities [B, rows, V], the rows evenly spaced; their address and the distance between rows."""
    B, rows, V = shape
    step = V if t.dim() != 3 or B * rows < 2 else t.stride(1) if rows > 1 else t.stride(0)
    if not (t.dtype is dtype and t.get_device() == dev and t.shape == shape and (V == 1 or t.stride(2) == 1)
            and step >= V and (B == 1 or rows == 1 or t.stride(0) == rows * step)):
        raise DecodeAttnError(f"{name}: want a {dtype} tensor of shape {shape} with evenly spaced rows on the current "
                              f"CUDA device, got {t.dtype} {tuple(t.shape)} on {t.device}, strides {t.stride()}")
    return t.data_ptr(), step


def verify_drafts(target_probs, draft_probs, draft_tokens, uniform, num_accepted, out_tokens, cache_seqlens=None,
                  new_seqlens=None, device_error=None, stream=None, lib=None):
    """Accept or refuse the drafts of every request and draw its next token:
    ``target_probs`` [B, K + 1, V], ``draft_probs`` [B, K, V] of the same dtype
    (None: certain drafts), ``draft_tokens`` int32 [B, K] (None for K = 0),
    ``uniform`` fp32 [B, K + 1]; ``num_accepted`` int32 [B], ``out_tokens`` int32
    [B, K + 1] and, with ``cache_seqlens``, ``new_seqlens`` int32 [B] are written.
    See decode_attn_verify_drafts in the header."""
    import torch
    i32, dev, dtype = torch.int32, _device(), target_probs.dtype
    if target_probs.dim() != 3 or target_probs.shape[1] < 1:
        raise DecodeAttnError(f"target_probs: want [B, K + 1, V], got {tuple(target_probs.shape)}")
    B, rows, V = target_probs.shape
    K = rows - 1
    kind = {torch.float32: PROB_F32, torch.bfloat16: PROB_BF16, torch.float16: PROB_F16}.get(dtype, -1)
    tp, ts = _prob_rows(dev, "target_probs", target_probs, dtype, (B, rows, V))
    dp, ds = None, 0
    if draft_probs is not None and K > 0:
        dp, ds = _prob_rows(dev, "draft_probs", draft_probs, dtype, (B, K, V))
    _check((lib or load_library()).decode_attn_verify_drafts(
        B, K, V, kind, tp, ts, dp, ds, _opt(dev, "draft_tokens", draft_tokens, i32, (B, K)),
        _need(dev, "uniform", uniform, torch.float32, (B, rows)), _opt(dev, "cache_seqlens", cache_seqlens, i32, (B,)),
        _need(dev, "num_accepted", num_accepted, i32, (B,)), _need(dev, "out_tokens", out_tokens, i32, (B, rows)),
        _opt(dev, "new_seqlens", new_seqlens, i32, (B,)), _opt(dev, "device_error", device_error, i32),
        _stream(stream, dev)))


def get_error(meta, stream=None) -> int:
    e = ctypes.c_int32(0)
    _check(load_library().decode_attn_get_error(_ptr(meta), ctypes.byref(e), _stream(stream)))
    return e.value


__all__ = ["Desc", "LaunchOpts", "DecodeAttnError", "load_library", "strerror", "sched_meta_bytes",
           "meta_offsets", "num_parts", "sched_meta", "fwd", "fwd_static_scratch", "append_kv", "rope_append",
           "accum_weights", "evict", "verify_drafts", "get_error", "Rope", "KV_BF16", "KV_FP8", "KV_MLA656", "PROB_F32",
           "PROB_BF16", "PROB_F16"]
