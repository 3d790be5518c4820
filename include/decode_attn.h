/*
 * decode_attn.h -- C ABI of the paged-KV decode attention library (GB300, sm_103a).
 *
 * The operation (XQA page "TensorRT-LLM 源码完全拆解(二十九)", section
 * "先把 decode 注意力的约束写清楚"): one new query token per request. For request
 * b, KV head h and the G query heads h*G+g that share it,
 *
 *     out[b, h*G+g, :] = softmax(sigma * q[b, h*G+g, :] . K_{b,h}^T) V_{b,h}
 *     lse[b, h*G+g]    = ln sum_t exp(sigma * q . k_t)           (natural log)
 *
 * where K_{b,h}, V_{b,h} are the first L_b = cache_seqlens[b] tokens of the
 * request, gathered through block_table from a pool of fixed-size pages
 * (XQA page, section "Hopper:一次 TMA 只搬一个页", "VLLM layout").
 *
 * The work is split along the sequence into split-KV partials, each with its
 * own lse, and a combine step merges them (XQA page, section "归约怎么记";
 * FlashMLA page "FlashMLA 注意力内核源码走读", sections "调度" and
 * "合并与性能账本"). The call sequence follows FlashMLA's two-call shape:
 *
 *     decode_attn_sched_meta(...)   once per change of cache_seqlens (reusable)
 *     decode_attn_fwd(...)          every decode step / layer
 *
 * Memory: the caller allocates every buffer. The library never allocates,
 * never synchronises inside decode_attn_fwd, and keeps no per-call state
 * outside the sched_meta buffer. All pointers below are DEVICE pointers unless
 * noted; all must be 16-byte aligned.
 *
 * Errors: every entry point returns DA_OK (0) or a negative DA_ERR_* code,
 * detected on the host before anything is launched. Errors that only the
 * device can see (a block-table entry outside the pool, a length beyond
 * max_pages_per_seq * page_size, a pipeline wait that ran out of time) set
 * bits in an error word inside sched_meta; the kernels skip the offending
 * work and never trap. Read the word with decode_attn_get_error.
 *
 * Determinism: identical inputs give bitwise identical out and lse (fixed
 * reduction order, no floating-point atomics).
 */
#ifndef DECODE_ATTN_H
#define DECODE_ATTN_H

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* KV cache formats. */
typedef enum {
    /* k_pool, v_pool: bf16 [num_pages][page_size][H_kv][D], D = D_qk = D_v. */
    DA_KV_BF16 = 0,
    /* k_pool, v_pool: float8 e4m3 bytes [num_pages][page_size][H_kv][D];
     * element value = e4m3 * k_scale[h] (resp. v_scale[h]), one fp32 scale per
     * (KV head, tensor) -- the per-tensor KV scale of the XQA page, section
     * "Hopper 路径上 V 不做显式反量化". */
    DA_KV_FP8_PER_TENSOR = 1,
    /* k_pool: 656-byte tokens [num_pages][page_size][1][656] (FlashMLA page,
     * section "数据加载"): 512 e4m3, 4 fp32 scales (one per 128 values), 64 bf16
     * RoPE values. K = the 576 dequantised values, V = the first 512. v_pool
     * must be NULL or equal to k_pool; H_kv = 1, D_qk = 576, D_v = 512.
     * Codes 0x7F / 0xFF decode to NaN (and so poison the rows that read
     * them), as in the bf16 and per-tensor formats; the quantiser,
     * decode_attn_append_kv, never writes them: it saturates at +-448. */
    DA_KV_FP8_MLA656 = 2,
    /* k_pool, v_pool: 8-bit codes [num_pages][page_size][H_kv][128], e4m3 or
     * int8; k_scale, v_scale: fp32 [num_pages][H_kv][page_size / 16], one scale
     * per block of 16 tokens, KV head and tensor. Element value = code * scale
     * of its block. page_size 16, 32 or a multiple of 64. Attention takes any
     * scales; those that decode_attn_append_block writes are powers of two. (No
     * counterpart on the source pages, whose e4m3 scales are per tensor.) */
    DA_KV_FP8_BLOCK = 3,
    DA_KV_INT8_BLOCK = 4
} da_kv_dtype;

/* Problem description (host struct, passed by pointer, not retained). */
typedef struct {
    int32_t B;                 /* requests */
    int32_t H_kv;              /* KV heads */
    int32_t G;                 /* query heads per KV head; H_q = H_kv * G */
    int32_t D_qk;              /* q / K head size */
    int32_t D_v;               /* V / out head size */
    int32_t page_size;         /* tokens per page P: 8, 16, 32 or a multiple of 64 (block formats: not 8) */
    int32_t max_pages_per_seq; /* row length of block_table */
    int32_t num_pages;         /* pages in the pool */
    int32_t kv_dtype;          /* da_kv_dtype */
    int32_t splits;            /* 0: balanced over the SMs; S > 0: S splits per request */
    int32_t num_sms;           /* 0: query the current device; the automatic partition then counts
                                  the SMs that can hold the 656-byte kernel's clusters at once, or
                                  two slots per SM for the bf16 D = 64 build with 3-4 query tokens
                                  (it runs two CTAs per SM); > 0: the slot count to partition for */
    float softmax_scale;       /* sigma; 0: 1/sqrt(D_qk) */
    int32_t s_q;               /* query tokens per request (0 means 1); see decode_attn_fwd */
    int32_t window;            /* sliding window W in tokens (0: none); see decode_attn_fwd */
    int32_t topk;              /* sparse decode: positions listed per request (0: dense); see decode_attn_fwd */
} da_desc;

/* Return codes. */
#define DA_OK                  0
#define DA_ERR_NULL           -1   /* a required pointer is NULL */
#define DA_ERR_DIMS           -2   /* a size is out of range */
#define DA_ERR_UNSUPPORTED    -3   /* no kernel for this (dtype, D_qk, D_v, G, page_size, s_q) */
#define DA_ERR_ALIGN          -4   /* a pointer is not 16-byte aligned */
#define DA_ERR_SPLITS         -5   /* splits < 0 or too large */
#define DA_ERR_META_SIZE      -6   /* sched_meta buffer smaller than decode_attn_sched_meta_bytes */
#define DA_ERR_CUDA           -7   /* a CUDA runtime/driver call failed */
#define DA_ERR_SCALE          -8   /* a format of 8 bits without k_scale / v_scale */

/* Device error bits (sched_meta error word). */
#define DA_DEV_BAD_PAGE        1   /* block_table entry outside [0, num_pages): page skipped */
#define DA_DEV_SEQ_TOO_LONG    2   /* cache_seqlens[b] > max_pages_per_seq * page_size: clamped */
#define DA_DEV_NEG_LEN         4   /* cache_seqlens[b] < 0: treated as 0 */
#define DA_DEV_TIMEOUT         8   /* a pipeline wait ran out of time: work unit abandoned */
#define DA_DEV_META_MISMATCH  16   /* sched_meta was built for another desc */
#define DA_DEV_BAD_TOKEN      32   /* a draft token >= vocab: taken as the end of its chain */
#define DA_DEV_BAD_PROBS      64   /* a row without a positive probability: the next token is -1 (verification), all 0 (token_probs) */
#define DA_DEV_BAD_REQUEST   128   /* a request index outside [0, B): the token's K and V are skipped */
#define DA_DEV_NO_PAGES      256   /* fewer free pages than a reservation needs: nothing was changed */

/*
 * Library plumbing from here to decode_attn_num_parts: no page defines these
 * calls; they size and describe the caller-owned sched_meta buffer.
 *
 * Size in bytes of the sched_meta buffer for this desc (host only, no CUDA
 * call except an SM-count query when desc->num_sms is 0). The buffer holds the
 * scheduling metadata, the split-KV partials (fp32 o and lse per split and
 * output row: query token x query head) and the device error word.
 */
int decode_attn_sched_meta_bytes(const da_desc *desc, size_t *bytes);

/*
 * Byte offsets inside sched_meta, for inspection and tests. offs[0..7] =
 * header, parts, chunk_offset, split_offset, num_splits, lse_part, o_part,
 * total size. Header (32 int32): magic, B, H_kv, G, splits, num_parts, cpc,
 * chunk (64), total_chunks, total_splits, per, error word, error detail,
 * kv_dtype, num_sms, s_q, window, topk, then zeros. parts: num_parts records of 8 int32
 * {b0, s0, c0, c1, co0, L0, so0, ns0}: first request, its split index there,
 * global chunk interval [c0, c1), then chunk_offset[b0], min(L_b0,
 * max_pages_per_seq*page_size), split_offset[b0], num_splits[b0] (all 0 when
 * b0 = -1, a part with no work). chunk_offset, split_offset: int32 [B+1]
 * prefix sums; num_splits: int32 [B].
 */
int decode_attn_meta_offsets(const da_desc *desc, size_t offs[8]);

/* Number of parts (grid x of the split-KV kernel) for this desc. */
int decode_attn_num_parts(const da_desc *desc, int32_t *num_parts);

/*
 * Scheduling metadata (FlashMLA page, section "调度": a small kernel hands the
 * (request, KV range) work units to the SMs ahead of time; the main kernel
 * only reads them). Work is counted in chunks of 64 tokens.
 *   splits = S > 0: request b is cut into S ranges of ceil(n_b / S) chunks
 *     (FlashAttention tiling page, section 5.3, block.h split range);
 *   splits = 0: all chunks of all requests are cut into
 *     num_parts = floor(num_sms / (H_kv * cpc)) equal intervals, one per part.
 * With a sliding window (desc->window = W > 0) a request's chunks start at the
 * one holding token max(0, L_b - s_q + 1 - W), the first its first query token
 * sees: the pages before it are never read (XQA page, section
 * "分页 KV:页号怎么变成 TMA 坐标"), and their block_table entries may hold
 * anything. Sparse decode (desc->topk = k > 0) gives every request k slots,
 * ceil(k / 64) chunks, whatever its length.
 * cache_seqlens: device int32 [B]. sched_meta: device, caller-owned, at least
 * decode_attn_sched_meta_bytes. Launches one small kernel on `stream`; the
 * result may be reused by any number of decode_attn_fwd calls while
 * cache_seqlens and desc stay the same. Clears the device error word.
 */
int decode_attn_sched_meta(const da_desc *desc, const int32_t *cache_seqlens,
                           void *sched_meta, size_t sched_meta_bytes, cudaStream_t stream);

/*
 * Decode attention forward. Launches the split-KV kernel and the LSE combine
 * kernel (chained with programmatic dependent launch) on `stream`. With a
 * fixed split count of 2-8 (desc->splits) and all formats but the 656-byte one, the
 * splits of a (request, KV head) run as one thread-block cluster and merge
 * their partials through distributed shared memory: the split-KV kernel then
 * writes out and lse itself and no combine kernel is launched.
 *
 * Several query tokens per request (desc->s_q > 1) verify a chain of draft
 * tokens (XQA page, section "投机解码:XQA 的第二个工作负载", the linear case;
 * FlashMLA's call passes s_q * h_q / h_kv rows per KV head): the request's
 * last s_q tokens are already in the pool (L_b counts them) and draft token
 * j < s_q sees the first L_b - s_q + 1 + j tokens -- the history and the
 * drafts up to itself. A row that sees no token gets out = 0, lse = -inf.
 * Supported: s_q <= 4 for all formats (on the 656-byte format the
 * sliding window and, when s_q > 1, sparse decode are not offered:
 * DA_ERR_UNSUPPORTED). The rows of q, out and lse below are
 * then [B][s_q][H_kv*G]; the scheduling metadata must be built with the same s_q.
 *
 * Sliding window (desc->window = W > 0; XQA page, section
 * "分页 KV:页号怎么变成 TMA 坐标"): a query token at position p sees only the
 * tokens (p - W, p]. Attention sinks (da_launch_opts.sinks; XQA page, section
 * "一个容易漏掉的细节:attention sink"): one fp32 logit per query head, in the
 * units of sigma * q.k, that joins each row's softmax denominator and carries
 * no value: lse = ln(e^sink + sum_t e^{s_t}), out = sum_t e^{s_t - lse} v_t;
 * a row that sees no token gets out = 0 and lse = sink. Both are for the
 * formats but the 656-byte one (DA_ERR_UNSUPPORTED).
 *
 * Sparse top-k decode (desc->topk = k > 0, da_launch_opts.indices; the
 * FlashMLA page's decode call with `indices`, ledger rows "FP8 稀疏解码"): for
 * the 656-byte format only. indices is device int32 [B][k]; request b attends
 * over the token positions indices[b][0..k) instead of [0, L_b): each is a
 * position in the request, mapped through block_table like a dense token;
 * entries outside [0, L_b) (-1 padding, stale positions) are skipped, and a
 * position listed twice counts twice. A request with no valid entry gets
 * out = 0, lse = -inf. Pages that no listed position touches are never read.
 *
 *   q:            bf16 [B][H_kv*G][D_qk], query head h*G+g belongs to KV head h
 *   k_pool/v_pool: see da_kv_dtype
 *   k_scale/v_scale: fp32 [H_kv] for DA_KV_FP8_PER_TENSOR, fp32 [num_pages][H_kv]
 *                 [page_size / 16] for the block formats (only scales of blocks that
 *                 hold a token below L_b are read), else ignored
 *   block_table:  int32 [B][max_pages_per_seq]; entries past ceil(L_b/P) are never read
 *   cache_seqlens: int32 [B] (must match what sched_meta was built from)
 *   sched_meta:   from decode_attn_sched_meta; its partial buffers are overwritten,
 *                 so two calls sharing one sched_meta must not overlap in time
 *   out:          bf16 [B][H_kv*G][D_v]; lse: fp32 [B][H_kv*G]
 * A request with L_b = 0 gets out = 0 and lse = -inf.
 * On all formats of 8 bits q and the softmax weights are multiplied as f16: values of
 * q above 65504 become infinite, those below 2^-14 lose bits.
 */
int decode_attn_fwd(const da_desc *desc, const void *q, const void *k_pool, const void *v_pool,
                    const float *k_scale, const float *v_scale, const int32_t *block_table,
                    const int32_t *cache_seqlens, void *sched_meta, size_t sched_meta_bytes,
                    void *out, float *lse, cudaStream_t stream);

/* Launch options for decode_attn_fwd_ex. */
typedef struct {
    int32_t use_pdl;          /* 1 (default behaviour of decode_attn_fwd): PDL-chain the kernels */
    cudaEvent_t main_begin;   /* if not NULL: recorded on `stream` just before the split-KV kernel */
    cudaEvent_t main_end;     /* if not NULL: recorded just after it (before the combine kernel) */
    const float *sinks;       /* if not NULL: device fp32 [H_kv*G] attention-sink logits (see decode_attn_fwd) */
    const int32_t *indices;   /* sparse decode (desc->topk > 0): device int32 [B][topk] token positions */
} da_launch_opts;

/* decode_attn_fwd with launch options and optional inputs (opts may be NULL). */
int decode_attn_fwd_ex(const da_desc *desc, const void *q, const void *k_pool, const void *v_pool,
                       const float *k_scale, const float *v_scale, const int32_t *block_table,
                       const int32_t *cache_seqlens, void *sched_meta, size_t sched_meta_bytes,
                       void *out, float *lse, const da_launch_opts *opts, cudaStream_t stream);

/*
 * KV append: writes each request's new token into the pool, the step that
 * precedes decode attention (XQA page, section "一次 decode step 的完整时序":
 * the new K/V lands in the paged pool upstream, and the attention kernel then
 * reads it through the page table). Request b's token, at position
 * t = positions[b] (its index in the request: the cache_seqlens[b] of the
 * step before, so the next decode uses t + 1), goes to slot t % page_size of
 * page block_table[b][t / page_size], for every KV head.
 *   desc: B, H_kv, D_qk, D_v, page_size, max_pages_per_seq, num_pages and
 *     kv_dtype are used (the others are ignored). bf16 and e4m3 pools need
 *     D_qk == D_v, a multiple of 8; the 656-byte token H_kv = 1, D_qk = 576,
 *     D_v = 512. The pools are those of decode_attn_fwd.
 *   k_new, v_new: device bf16, request b's row at (k_new + b * new_row_stride):
 *     H_kv x D values (head-major), or for the 656-byte token the 576 values of
 *     the latent vector (512 NoPE, then 64 RoPE) with v_new = NULL (V is the
 *     first 512 of them). new_row_stride counts bf16 elements (0: packed rows;
 *     else at least the row length and a multiple of 8), so rows may sit inside
 *     a larger fused projection output.
 *   positions: device int32 [B]; a negative position skips the request.
 *   block_table: device int32 [B][max_pages_per_seq].
 *   k_pool, v_pool: device, written in place; only the addressed slots change.
 *     v_pool must be NULL or k_pool for the 656-byte token.
 *   k_scale, v_scale: device fp32 [H_kv] for DA_KV_FP8_PER_TENSOR (read only).
 *   device_error: device int32 or NULL; DA_DEV_SEQ_TOO_LONG (t >=
 *     max_pages_per_seq * page_size) and DA_DEV_BAD_PAGE (page id outside
 *     [0, num_pages)) are OR-ed into it, and such a request is skipped.
 * Quantisation (e4m3, OCP FP8: largest finite 448): code = nearest e4m3 to the
 * fp32 quotient x / scale (IEEE division, round to nearest even), ties to the
 * even code, saturating at +-448, NaN -> 0x7F. Per-tensor pools divide by
 * k_scale[h] / v_scale[h] (XQA page, section "Hopper 路径上 V 不做显式反量化");
 * the 656-byte token (FlashMLA page, section "数据加载") takes, per block of 128
 * NoPE values, scale = max|x| / 448 in fp32 (1 for an all-zero block), stores
 * the 512 codes, the 4 fp32 scales and the 64 RoPE values unchanged.
 * Pointers to bf16 rows and pools must be 16-byte aligned, the others 4-byte.
 * Launches one kernel on `stream` (programmatic dependent launch: a following
 * decode_attn_fwd may start early and waits for it before reading the pool).
 * Two requests that address the same slot race. No allocation, no sync.
 */
int decode_attn_append_kv(const da_desc *desc, const void *k_new, const void *v_new, int64_t new_row_stride,
                          const int32_t *positions, const int32_t *block_table, void *k_pool, void *v_pool,
                          const float *k_scale, const float *v_scale, int32_t *device_error, cudaStream_t stream);

/*
 * Append to a cache with scales per block (DA_KV_FP8_BLOCK, DA_KV_INT8_BLOCK), one
 * token per request, a draft chain or ragged prompts. (No counterpart on the source
 * pages.) Request b's new tokens are the rows token_starts[b] .. token_starts[b + 1]
 * of k_new and v_new, and go to positions[b], positions[b] + 1, ... of its cache. Per
 * block of 16 positions, KV head and tensor:
 *   scale = the smallest power of two, at least 2^-126, with max |x| <= 448 scale
 *     (e4m3) or 127 scale (int8) over the block's new tokens (values that are not
 *     finite do not count); where the block holds tokens already (positions below
 *     positions[b]), never below the scale that it has.
 *   code = nearest to x / scale (the fp32 quotient, which is exact for a power of
 *     two), ties to even. e4m3: saturating at +-448, NaN ->
 *     0x7F. int8: saturating at +-127, NaN -> 0.
 * Where a block's scale grows, the codes of its earlier tokens are rounded to the new
 * scale (from their values code * scale, in fp32: exact where the old scale is a power of
 * two; not from what was appended). A value that is appended with
 * its whole block is off by at most half a step; one whose block grew later, by less
 * than a step of the final scale in int8 (halves add up), and in e4m3 by its own
 * rounding only, as long as its code stays normal (|value| >= scale / 64). The
 * positions behind the last new one hold nothing afterwards: their codes are left, the
 * scale may be another.
 *   desc: B, H_kv, D_qk = D_v = 128, page_size, max_pages_per_seq, num_pages, kv_dtype
 *     and, without token_starts, s_q are used.
 *   n_tokens: N in [0, 2^30], rows of k_new and v_new (0: nothing is launched).
 *   k_new, v_new: bf16 [N][H_kv][128], row n at + n * stride (bf16 elements; 0: packed
 *     rows; else at least the row and a multiple of 8).
 *   token_starts: device int32 [B + 1], not descending, within [0, N]; NULL: s_q rows per
 *     request, and N must be B * s_q.
 *   positions: device int32 [B]; negative: the request is skipped.
 *   block_table, device_error: as for decode_attn_append_kv (a token behind the table, or
 *     on a page outside the pool, is skipped).
 *   k_pool, v_pool, k_scale, v_scale: written in place.
 * Two requests that write to one block race: give every request pages of its own (see
 * decode_attn_reserve_pages). Launches one kernel on `stream`. No allocation, no sync.
 */
int decode_attn_append_block(const da_desc *desc, int32_t n_tokens, const void *k_new, int64_t k_stride,
                             const void *v_new, int64_t v_stride, const int32_t *token_starts,
                             const int32_t *positions, const int32_t *block_table, void *k_pool, void *v_pool,
                             float *k_scale, float *v_scale, int32_t *device_error, cudaStream_t stream);

/* Rotary positions with one or several axes (host struct, passed by pointer,
 * not retained). */
typedef struct {
    int32_t rot_dim;      /* rotated values per head: a multiple of 16 in [16, min(D_qk, 512)]; on the 656-byte
                             format at most 64, the first rot_dim of the 64 RoPE values */
    int32_t n_axes;       /* 1..4 (time, height, width, ...) */
    int32_t sections[4];  /* pairs per axis, >= 0; the first n_axes sum to rot_dim / 2, the others are 0 */
    int32_t interleaved;  /* 0: pairs in blocks, the first sections[0] follow axis 0, the next sections[1] axis 1, ...;
                             1: alternating, pair i follows axis a = i mod n_axes while i / n_axes < sections[a],
                             else axis 0 */
    int32_t adjacent;     /* 0: pair i = values (i, i + rot_dim / 2); 1: values (2 i, 2 i + 1) */
} da_rope;

/*
 * Rotary positions and KV append in one pass: rotates the queries and keys of
 * new tokens and writes their K and V into the pool, any number of tokens per
 * request (a draft chain, ragged prompts). With theta = rope_positions[axis(i)][n]
 * * inv_freq[i], pair i of token n goes (x, y) -> (x cos theta - y sin theta,
 * x sin theta + y cos theta) in every query and key head; values past rot_dim
 * pass through. (No counterpart on the source pages, which append finished
 * rows.)
 *   desc: as for decode_attn_append_kv, and G (H_q = H_kv * G).
 *   n_tokens: N in [0, 2^30] (0: nothing is launched). Token n belongs to request
 *     requests[n]; requests = NULL: to request n / s_q, and N must be B * s_q.
 *   q: bf16, token n's [H_q][D_qk] at q + n * q_stride. k_new, v_new: likewise
 *     [H_kv][D]; on the 656-byte format k_new holds the 576 values of the latent
 *     vector and v_new is NULL. Strides count bf16 elements (0: packed rows;
 *     else at least the row and a multiple of 8), so the three may be slices of
 *     one projection output.
 *   inv_freq: fp32 [rot_dim / 2], radians per position. At any int32 position the
 *     angle modulo a turn is held to 24 bits: it is off by at most 2^-26 of a turn
 *     (1e-7 radians), and |position| (|inv_freq| + 1) 2^-64 of a turn besides. An
 *     infinite or NaN frequency gives NaN.
 *   rope_positions: int32 [n_axes][N]. positions: int32 [N], the token's index
 *     in its request's cache (slot t % page_size of page block_table[b][t /
 *     page_size]); negative: the token is skipped, its q_out row left as it was.
 *   q_out: bf16 [N][H_q][D_qk], the q of decode_attn_fwd when the tokens come
 *     request by request. It may be q itself (packed rows); else it must not
 *     overlap q, k_new or v_new (DA_ERR_UNSUPPORTED).
 *   k_pool, v_pool, k_scale, v_scale, device_error: as for decode_attn_append_kv.
 *     Besides its bits, DA_DEV_BAD_REQUEST; such a token's q is still rotated.
 * Products and sums are fp32; each value is rounded once, K to the pool's format
 * from its fp32 value by the rules of decode_attn_append_kv. Two tokens that
 * address the same slot race. Launches one kernel on `stream`. No allocation,
 * no sync.
 */
int decode_attn_rope_append(const da_desc *desc, const da_rope *rope, int32_t n_tokens, const void *q,
                            int64_t q_stride, const void *k_new, int64_t k_stride, const void *v_new,
                            int64_t v_stride, const float *inv_freq, const int32_t *rope_positions,
                            const int32_t *requests, const int32_t *positions, const int32_t *block_table,
                            void *q_out, void *k_pool, void *v_pool, const float *k_scale, const float *v_scale,
                            int32_t *device_error, cudaStream_t stream);

/*
 * Attention weight gathered by cached tokens, the measure by which
 * decode_attn_evict keeps them. After a decode step, for every token t < L_b of
 * request b and KV head h,
 *     w[t] <- (t < weighted_lens[b] ? decay * w[t] : 0)
 *             + sum_j sum_g exp(sigma * q_{b,j,hG+g} . k_t - lse[b,j,hG+g])
 * over the query tokens j <= num_accepted[b] that see t (t <= L_b - s_q + j).
 * (No counterpart on the source pages.) The bf16, e4m3 (a scale per head) and
 * 656-byte formats; no sliding window and no sparse decode (DA_ERR_UNSUPPORTED). On the 656-byte format
 * max_pages_per_seq * page_size may be 2^31 - 257 at most.
 *   desc, q, k_pool, k_scale, block_table, cache_seqlens, sched_meta, lse: those
 *     of the step's decode_attn_fwd call, with the same requirements and the
 *     lengths as they were then (not new_seqlens of a verification); sinks
 *     need no argument (they are in lse). Page errors go to sched_meta's word.
 *   num_accepted: device int32 [B] or NULL (all s_q count): of a draft chain
 *     whose verification accepted a drafts, query tokens 0..a count; negative:
 *     none does.
 *   weighted_lens: device int32 [B] or NULL (all of L_b): the tokens that have
 *     a weight already; the others (this step's, a prompt's at the first call)
 *     start from 0, whatever their slot held.
 *   decay: finite, >= 0.
 *   weights: device fp32 [num_pages][H_kv][page_size], written in place; only
 *     slots of tokens t < L_b change. A page that two requests share, or that
 *     one lists twice, would be updated twice at once: give every request pages of
 *     its own.
 * A query row whose lse is -inf adds nothing. Scores are products of what the
 * attention call multiplies, so that they match its lse: on e4m3 pools q goes to
 * f16 (bf16 values above 65504 become infinite and give NaN, those below 2^-14
 * lose bits), on the 656-byte format K is bf16(e4m3 * scale); exponentials are the
 * hardware's ex2 (2 ulp). Each weight is summed in fp32 in a fixed order. Launches one kernel on `stream`. No allocation, no sync.
 */
int decode_attn_accum_weights(const da_desc *desc, const void *q, const void *k_pool, const float *k_scale,
                              const int32_t *block_table, const int32_t *cache_seqlens, void *sched_meta,
                              size_t sched_meta_bytes, const float *lse, const int32_t *num_accepted,
                              const int32_t *weighted_lens, float decay, float *weights, cudaStream_t stream);

/*
 * Eviction: cuts every request's cache down to `budget` tokens per KV head,
 * copied in their order to the pages of a second block table. (No counterpart
 * on the source pages.) For request b and KV head h: all tokens when L_b <=
 * budget; else the first keep_first, the last keep_last, and of those between
 * them the heaviest by `weights`, budget tokens in all. Equal weights (-0 = +0):
 * the lower position is kept; a NaN weighs more than any number. Heads choose
 * independently, so slot i of a page may hold different tokens of different
 * heads: positions have to be in the keys already (rotated).
 *   desc: B, H_kv, D_qk, D_v, page_size, max_pages_per_seq, num_pages and
 *     kv_dtype are used. bf16 pools need D_qk == D_v, a multiple of 8, e4m3 pools
 *     a multiple of 16; the 656-byte token as for decode_attn_append_kv.
 *   budget >= 1, at most max_pages_per_seq * page_size (itself at most 2^30); keep_first, keep_last >=
 *     0 with keep_first + keep_last <= budget.
 *   block_table, dst_block_table: device int32 [B][max_pages_per_seq]; entries
 *     past ceil(L_b / P) and past ceil(min(L_b, budget) / P) are never read. The
 *     pages of dst_block_table must be distinct and hold no token that this call
 *     reads. Afterwards dst_block_table is the requests' block table.
 *   k_pool, v_pool (NULL or k_pool for the 656-byte token), weights (fp32
 *     [num_pages][H_kv][page_size]): written in the kept tokens' new slots only.
 *   kept: device int32 [B][H_kv][budget], the kept positions in ascending order,
 *     then -1. new_seqlens: device int32 [B], min(L_b, budget); not
 *     cache_seqlens itself (DA_ERR_UNSUPPORTED).
 *   device_error: device int32 or NULL; DA_DEV_NEG_LEN (taken as 0),
 *     DA_DEV_SEQ_TOO_LONG (clamped) and DA_DEV_BAD_PAGE (a token on a page
 *     outside [0, num_pages) weighs less than any other; its row, or one whose
 *     new page is outside, is not copied) are OR-ed into it.
 * Launches two kernels on `stream`. No allocation, no sync.
 */
int decode_attn_evict(const da_desc *desc, int32_t budget, int32_t keep_first, int32_t keep_last,
                      const int32_t *cache_seqlens, const int32_t *block_table, const int32_t *dst_block_table,
                      void *k_pool, void *v_pool, float *weights, int32_t *kept, int32_t *new_seqlens,
                      int32_t *device_error, cudaStream_t stream);

/*
 * The pages of a cache, for callers that keep its tables on the device. (No counterpart
 * on the source pages.) The state is the block table, cache_seqlens, and
 *   held: int32 [B], the table entries [0, held[b]) that request b holds (at least
 *     those of its tokens; more after a reservation),
 *   refs: int32 [num_pages], how many hold each page: table entries, and whoever else
 *     counts (a prefix cache adds its own). 0: the page is free.
 * A fork shares pages; a reservation makes what is written next the request's own:
 *
 *     fork_pages -> reserve_pages -> copy_pages -> append -> sched_meta -> fwd ...
 *
 * One set of tables serves all layers: copies (pairs of pages) are planned once and
 * decode_attn_copy_pages carries them out in each layer's pools. Of desc these calls read
 * B (at most 8192), page_size, max_pages_per_seq, num_pages (at most 2^23) and, where
 * noted, s_q. device_error: device int32 or NULL; DA_DEV_BAD_PAGE (an entry outside
 * [0, num_pages): skipped) is OR-ed into it by all of them. Pointers are device
 * pointers, 4-byte aligned (copies: 8). Results do not depend on the order of anything on
 * the device. Launches on `stream`; no allocation, no sync.
 *
 * fork_pages: new row i continues row parents[i] of the old rows (-1: an empty row), a
 * beam step or parallel samples: the entries of the parent's tokens, ceil(L / P) of them,
 * are shared, entries that it holds beyond are not. Every old row lets go of what it
 * holds, so a row that is no one's parent is freed. new_held, new_seqlens: of the new
 * rows; entries of new_block_table past new_held keep what they were. The new buffers are
 * not the old ones (DA_ERR_UNSUPPORTED). A parent >= B: DA_DEV_BAD_REQUEST, the row is
 * empty. A negative length counts as 0 (DA_DEV_NEG_LEN). One kernel.
 */
int decode_attn_fork_pages(const da_desc *desc, const int32_t *parents, const int32_t *cache_seqlens,
                           const int32_t *block_table, const int32_t *held, int32_t *refs, int32_t *new_block_table,
                           int32_t *new_held, int32_t *new_seqlens, int32_t *device_error, cudaStream_t stream);

/*
 * free_pages: rows with done[b] != 0 let go of all that they hold, in place; held[b] and
 * cache_seqlens[b] become 0. One kernel.
 */
int decode_attn_free_pages(const da_desc *desc, const int32_t *done, int32_t *cache_seqlens,
                           const int32_t *block_table, int32_t *held, int32_t *refs, int32_t *device_error,
                           cudaStream_t stream);

/*
 * reserve_pages: room for new_tokens[b] more tokens of each request (NULL: s_q each;
 * <= 0: none, the row is left alone), which nobody else holds. In place:
 *   - entries are added up to ceil((L_b + n) / P), held[b] follows;
 *   - where the page of the next token has tokens on it (L_b mod P != 0) and others hold
 *     it, the row gets a fresh page in its place and copies[b] = (old, new); if every
 *     holder is a row of this call that asks for room there, the lowest row keeps the page
 *     without a copy. Rows without a copy: (-1, -1);
 *   - entries that the row holds past its tokens, if others hold one that it would write
 *     to, are given back and fresh ones taken.
 * Fresh pages are the lowest that were free before the call, in the order of the rows, and
 * in a row the copy's first. copies: int32 [B][2], the copies argument of
 * decode_attn_copy_pages. missing: int32 [1], 0; or, where the pool has too few free
 * pages, how many are missing: then nothing is changed (all copies are -1,
 * DA_DEV_NO_PAGES). A row that would pass max_pages_per_seq * page_size is left alone
 * (DA_DEV_SEQ_TOO_LONG); a negative length counts as 0 (DA_DEV_NEG_LEN). One kernel.
 */
int decode_attn_reserve_pages(const da_desc *desc, const int32_t *new_tokens, const int32_t *cache_seqlens,
                              int32_t *block_table, int32_t *held, int32_t *refs, int32_t *copies, int32_t *missing,
                              int32_t *device_error, cudaStream_t stream);

/*
 * compact_pages: plans the move of all pages in use (refs > 0), N of them, to [0, N): the
 * i-th page in use at or above N goes to the i-th free one below it. Out of place, so
 * that the old state is good until the copies are done:
 *   new_page: int32 [num_pages], where each page goes (itself if it stays, -1 if it is
 *     free), also for holders outside the table. new_refs: int32 [num_pages].
 *     new_block_table: the held entries, mapped (the others keep what they were).
 *   copies: int32 [num_pages / 2][2], the pairs; counts: int32 [2], N and the number of
 *     pairs (the num_copies of decode_attn_copy_pages is counts + 1).
 * None of the new buffers is an old one (DA_ERR_UNSUPPORTED). Two kernels.
 */
int decode_attn_compact_pages(const da_desc *desc, const int32_t *block_table, const int32_t *held, const int32_t *refs,
                              int32_t *new_block_table, int32_t *new_refs, int32_t *new_page, int32_t *copies,
                              int32_t *counts, int32_t *device_error, cudaStream_t stream);

/*
 * copy_pages: copies whole pages of a cache, all formats: K, V, their scales (block
 * formats) and, if given, the weights of decode_attn_accum_weights.
 *   desc: H_kv, D_qk, D_v, page_size, num_pages, kv_dtype; a page of a pool has to be a
 *     multiple of 16 bytes (DA_ERR_UNSUPPORTED).
 *   copies: device int32 [max_copies][2] (source, destination), a negative source: none;
 *     a page outside the pool: skipped (DA_DEV_BAD_PAGE). num_copies: device int32 [1] or
 *     NULL (all): only the first of them. No destination may be a source, or stand twice.
 *     A pipeline wait that runs out sets DA_DEV_TIMEOUT; pages are then missing.
 *   k_scale, v_scale: the block formats' scales, else ignored. weights: fp32
 *     [num_pages][H_kv][page_size] or NULL. v_pool: NULL or k_pool for the 656-byte token.
 * One kernel.
 */
int decode_attn_copy_pages(const da_desc *desc, int32_t max_copies, const int32_t *copies, const int32_t *num_copies,
                           void *k_pool, void *v_pool, float *k_scale, float *v_scale, float *weights,
                           int32_t *device_error, cudaStream_t stream);

/* Types of the probabilities of decode_attn_verify_drafts, and of the logits and
 * probabilities of decode_attn_token_probs. */
typedef enum {
    DA_PROB_F32 = 0,
    DA_PROB_BF16 = 1,
    DA_PROB_F16 = 2
} da_prob_dtype;

/* What decode_attn_token_probs does to logits (host struct, passed by pointer, not
 * retained; its pointers are device pointers, 4-byte aligned, and may each be NULL). */
typedef struct {
    const float *temperature;     /* [B]; NULL: 1. Not above 0: greedy */
    const float *repetition;      /* [B], > 0; NULL: 1 */
    const float *frequency;       /* [B]; NULL: 0 */
    const float *presence;        /* [B]; NULL: 0 */
    const int32_t *history;       /* [B][history_cols]: the request's tokens, prompt first */
    const int32_t *history_lens;  /* [B]: tokens of each row (needed with history; cut to [0, history_cols]) */
    const int32_t *prompt_lens;   /* [B]: how many of them are the prompt's; NULL: none */
    const int32_t *draft_tokens;  /* [B][n_draft], those of decode_attn_verify_drafts */
    const int32_t *bias_starts;   /* [B + 1]: request b's biases are entries [bias_starts[b], bias_starts[b + 1]) */
    const int32_t *bias_tokens;   /* [n_bias] */
    const float *bias_values;     /* [n_bias] */
    const uint32_t *allowed;      /* row (b, j): ceil(V / 32) words, bit v mod 32 of word v / 32 set: token v is allowed */
    int64_t allowed_stride;       /* words from row to row; 0: ceil(V / 32) */
    int32_t history_cols, n_bias;
} da_token_rules;

/*
 * Probabilities out of the target's logits: what decode_attn_verify_drafts takes. (No
 * counterpart on the source pages.) Row (b, j) follows the first j drafts of request b. With
 * c(v) = how often token v was generated (stands in the history behind the prompt, or
 * among those j drafts, up to the first negative one):
 *   x(v) = the logit; where v was generated or is in the prompt: x / repetition if x > 0, else
 *     x * repetition; then - frequency * c(v), and - presence if c(v) > 0; then + its
 *     biases, in the list's order (a token may stand there several times);
 *   p(v) = e^(x(v) / temperature) / sum over the allowed tokens, 0 for the others, whatever
 *     their logits are; with a temperature that is not above 0, 1 for the largest x (the
 *     lowest token of equals; a NaN is not the largest) and 0 for the others.
 * A pipeline wait that runs out sets DA_DEV_TIMEOUT; the probabilities are then not valid.
 * A row without an allowed token whose x is above -infinity is 0 throughout
 * (DA_DEV_BAD_PROBS). A NaN or +infinity among the allowed x makes a row NaN throughout
 * (not a greedy one).
 *   B >= 1, n_draft in [0, 63], vocab V in [1, 2^19 - 7]. logits_dtype, prob_dtype:
 *     da_prob_dtype, independent of each other.
 *   logits: row j of request b at (b * (n_draft + 1) + j) * logits_stride elements; probs:
 *     likewise with probs_stride (0: V, else >= V; rows aligned to their type only). probs may
 *     be logits itself (same type and stride); else they must not overlap
 *     (DA_ERR_UNSUPPORTED).
 *   rules: NULL for none. Tokens outside [0, V) in any of its lists are ignored. A request
 *     may have any number of biases, one on every token too (n_bias: 2^30 at most).
 *     history_cols may be as wide as the longest text (2^28 at most): the tokens used cost, not the columns.
 * x is fp32 in the order above, each step rounded; exponentials are the hardware's ex2 (2
 * ulp), sums fp32 in a fixed order; p is rounded once to its type. Launches one kernel on
 * `stream`. No allocation, no sync.
 */
int decode_attn_token_probs(int32_t B, int32_t n_draft, int32_t vocab, int32_t logits_dtype, const void *logits,
                            int64_t logits_stride, int32_t prob_dtype, void *probs, int64_t probs_stride,
                            const da_token_rules *rules, int32_t *device_error, cudaStream_t stream);

/*
 * Verification of a chain of drafted tokens against the target's probabilities,
 * from given random numbers: the step after a decode call with s_q = n_draft + 1
 * query tokens (XQA page, section "投机解码:XQA 的第二个工作负载", ends at the
 * attention; the rule is not there). Request b has K = n_draft drafts x_0 ..
 * x_{K-1}, the target's probabilities p_0 .. p_K (p_j after the first j drafts)
 * and the draft model's q_0 .. q_{K-1}. Draft j is accepted when u_j * q_j(x_j)
 * < p_j(x_j), compared exactly, and all before it were. With a drafts accepted,
 * the next token is drawn from max(p_a - q_a, 0) where draft a was refused, from
 * p_a where the chain had ended: the first v for which the sum of the weights up
 * to v exceeds floor(u_K * total), each weight its fp32 value rounded to a whole
 * number of steps of 2^-44. The sums are exact integers.
 *   B >= 1, n_draft in [0, 63] (0: draws one token per request), vocab V in
 *     [1, 2^20), prob_dtype: of both probabilities.
 *   target_probs: device, row j of request b at (b * (n_draft + 1) + j) *
 *     target_stride elements; draft_probs: (b * n_draft + j) * draft_stride, or
 *     NULL for drafts that are certain (q_j(x_j) = 1). Strides: 0 for V, else >= V;
 *     aligned to their type only.
 *   draft_tokens: device int32 [B][n_draft]; a negative one ends its chain (ragged
 *     chains), one >= V too (DA_DEV_BAD_TOKEN).
 *   uniform: device fp32 [B][n_draft + 1] in [0, 1); u_K is clamped into it.
 *   Probabilities that are NaN or negative count as 0 in the draw, above 1 as 1; a
 *     comparison with NaN refuses the draft. Where no weight of p_a - q_a is left,
 *     p_a is drawn from; where none of p_a either, the token is -1 (DA_DEV_BAD_PROBS).
 *   num_accepted: device int32 [B], a. out_tokens: device int32 [B][n_draft + 1]:
 *     the accepted drafts, the next token, then -1.
 *   cache_seqlens, new_seqlens: device int32 [B], both or neither; new = max(L_b
 *     - n_draft + a, 0), the length that keeps the accepted drafts (a row that pads
 *     the batch, of length 0 and without drafts, keeps 0). They may be the same
 *     buffer, if no later call wants the step's own lengths (decode_attn_accum_weights
 *     does).
 *   device_error: device int32 or NULL.
 * Launches one kernel on `stream`. No allocation, no sync.
 */
int decode_attn_verify_drafts(int32_t B, int32_t n_draft, int32_t vocab, int32_t prob_dtype,
                              const void *target_probs, int64_t target_stride, const void *draft_probs,
                              int64_t draft_stride, const int32_t *draft_tokens, const float *uniform,
                              const int32_t *cache_seqlens, int32_t *num_accepted, int32_t *out_tokens,
                              int32_t *new_seqlens, int32_t *device_error, cudaStream_t stream);

/*
 * Reads the device error word of sched_meta into *device_error (host int32).
 * Synchronises `stream`. Library plumbing: no page defines this call.
 */
int decode_attn_get_error(const void *sched_meta, int32_t *device_error, cudaStream_t stream);

/* Size of the library's fixed device scratch buffer (16 MiB). */
#define DA_STATIC_SCRATCH_BYTES (16u << 20)

/*
 * decode_attn_sched_meta + decode_attn_fwd in one call that allocates
 * nothing and needs no caller-provided scratch. (No counterpart on the source
 * pages: it exists for deployment.) It is meant for callers that cannot
 * allocate device memory or hand the library a buffer -- a server that plans
 * all device memory up front and may not call cudaMalloc later, a plug-in that
 * cannot reach its host's allocator, a real-time path that must not risk an
 * allocation.
 *
 * The scheduling metadata and the split-KV partials live in a static device
 * array of DA_STATIC_SCRATCH_BYTES that the library owns; every GPU that loads
 * the library keeps it until the process exits. Problems whose
 * decode_attn_sched_meta_bytes exceeds that size are rejected with
 * DA_ERR_META_SIZE. With the 656-byte format the automatic split count
 * (desc->splits = 0) of a GB300 needs (76 + B) x 256 KB of partials at s_q = 1,
 * over 16 MiB for any B, and is rejected: pass a fixed split count or a
 * smaller desc->num_sms. Sparse decode (desc->topk > 0) needs
 * indices, which this call cannot take: DA_ERR_UNSUPPORTED.
 * The first call on a device looks up the array's device address
 * (cudaGetSymbolAddress, with that device current): make that first call
 * before any stream capture. The address is kept per device and CUDA context;
 * after a device reset the next call looks it up again. Every call reuses the
 * same array and leaves its contents behind; the scheduling kernel rewrites
 * all it reads, so nothing needs clearing, but calls whose work overlaps on
 * the GPU race on the array. Every argument is checked on the host before
 * anything is launched, so a rejected call leaves the array untouched.
 * Arguments, layouts and errors are those of decode_attn_fwd; device errors
 * land in the array's error word and are not readable from outside.
 */
int decode_attn_fwd_static_scratch(const da_desc *desc, const void *q, const void *k_pool, const void *v_pool,
                                   const float *k_scale, const float *v_scale, const int32_t *block_table,
                                   const int32_t *cache_seqlens, void *out, float *lse, cudaStream_t stream);

/* Static description of a return code (never NULL). Library plumbing: no
 * page defines this call. */
const char *decode_attn_strerror(int code);

#ifdef DA_PAGE_TRACE
/* Test build only (the library compiled with -DDA_PAGE_TRACE; the product
 * build does not export it). Makes every later decode_attn_fwd record the
 * pool rows its kernels read into `trace` (device memory, int32, caller-owned,
 * written in place): for the GQA formats, per (part, KV head) unit, per chunk
 * in reading order, per TMA box of min(page_size, 64) tokens, the first pool
 * row of the box (page * page_size + offset within the page), or -2 for a box
 * past the sequence; for the 656-byte format, per part, per chunk, per token,
 * the token's pool row or -2. `cap` chunks are kept per unit (later ones are
 * not recorded); the unit stride is cap * rows_per_chunk. A null `trace`
 * stops recording. Returns DA_ERR_DIMS for cap < 1 with a non-null trace.
 * There is no counterpart on the pages: it checks the page gather (block
 * table -> page -> slot, XQA page section "Hopper:一次 TMA 只搬一个页") bit for
 * bit against a reference built from the partition and the block table. */
int decode_attn_debug_page_trace(int32_t *trace, int32_t cap);

/* Test build only. Limits every bounded wait (mbarrier phase, peer CTA) of
 * later launches to `ns` nanoseconds; 0 restores the product limit of 2 s. A
 * wait that runs out sets DA_DEV_TIMEOUT in the device error word, the
 * kernel's CTAs stop their work units and return, and the CUDA context stays
 * usable; it exists so that tests can make waits run out without a fault.
 * No counterpart on the pages. Always returns DA_OK. */
int decode_attn_debug_wait_limit(uint64_t ns);

/* Test build only. With `on` != 0, the consumer warps of later GQA-format
 * launches first wait (bounded, see above) on an mbarrier that nothing
 * completes: the wait runs out, DA_DEV_TIMEOUT is set and the CTAs return.
 * 0 turns it off. No counterpart on the pages. Always returns DA_OK. */
int decode_attn_debug_stall(int32_t on);

/* Test build only. The page operators and the token probabilities launch
 * clusters of at most `ctas` CTAs (8 or 16; else DA_ERR_DIMS), as they do on a
 * device that has no room for 16. 16 restores the product's choice. No
 * counterpart on the pages. */
int decode_attn_debug_max_cluster(int32_t ctas);
#endif

#ifdef __cplusplus
}
#endif

#endif /* DECODE_ATTN_H */
