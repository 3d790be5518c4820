// Host/device shared definitions: sched_meta layout and kernel parameter blocks.
#pragma once

#include <cstddef>
#include <cstdint>

namespace da {

constexpr int kChunk = 64;                 // tokens per scheduling chunk
constexpr int kScaleBlock = 16;            // tokens that share a scale (block formats)
constexpr int kTmaElemBytes = 8;           // element size the pool tensor maps are described with
constexpr int32_t kMetaMagic = 0x44414d31;  // "DAM1"
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s per pipeline wait
constexpr int kMaxSqD64 = 4;               // query tokens per request: bf16 D = 64 kernel
constexpr int kMaxSqD128 = 4;              // bf16 / e4m3 D = 128 kernels
constexpr int kMaxSqMla = 4;               // 656-byte latent format (one CTA pair per query token)

// sched_meta header words
enum MetaHeader : int {
    kHMagic = 0,
    kHB = 1,
    kHHkv = 2,
    kHG = 3,
    kHSplits = 4,
    kHNumParts = 5,
    kHCpc = 6,
    kHChunk = 7,
    kHTotalChunks = 8,
    kHTotalSplits = 9,
    kHPer = 10,
    kHError = 11,
    kHErrorDetail = 12,
    kHKvDtype = 13,
    kHNumSms = 14,
    kHSq = 15,
    kHWindow = 16,
    kHTopk = 17,
    kHeaderWords = 32,
};

// One part record (32 bytes): the part's first request b0, that request's
// split index s0 there, the global chunk interval [c0, c1), and -- so that the
// split-KV kernel needs no further dependent load for the first segment --
// chunk_offset[b0], min(L_b0, max_len), split_offset[b0], num_splits[b0].
struct PartRec {
    int32_t b0, s0, c0, c1, co0, L0, so0, ns0;
};
constexpr int kPartRecInts = 8;

struct MetaLayout {
    size_t header, parts, chunk_offset, split_offset, num_splits, lse_part, o_part, total;
    int32_t num_parts, max_splits, cpc;
};

// Device-side view of sched_meta.
struct MetaView {
    int32_t *header;
    const int4 *parts;            // PartRec as two int4 per part
    const int32_t *chunk_offset;
    const int32_t *split_offset;
    const int32_t *num_splits;
    float *lse_part;   // [max_splits][s_q * H_q]
    float *o_part;     // [max_splits][s_q * H_q][D_v]
    int32_t max_splits;
};

struct SchedParams {
    const int32_t *seqlens;
    int32_t *meta;           // header base
    int32_t *parts;          // PartRec records
    int32_t *chunk_offset;
    int32_t *split_offset;
    int32_t *num_splits;
    int32_t B, H_kv, G, splits, num_parts, cpc, max_len, kv_dtype, num_sms, s_q;
    int32_t window;          // sliding window in tokens, 0: none
    int32_t topk;            // sparse decode: listed positions per request (0: dense)
};

// First token that any of a request's s_q query tokens sees, with a sliding
// window of `window` tokens (0: none): the chunks before the one holding it
// are never read (XQA page, section "分页 KV:页号怎么变成 TMA 坐标").
__host__ __device__ inline int window_start(int L, int s_q, int window) {
    const int st = L - s_q + 1 - window;
    return (window > 0 && st > 0) ? st : 0;
}

// Chunks of a request of (clamped) length L in the schedule: the listed
// positions for sparse decode, else the chunks from the one holding the
// window's first token to the end.
__host__ __device__ inline int chunks_of(int L, int s_q, int window, int topk) {
    return topk > 0 ? (topk + kChunk - 1) / kChunk : (L + kChunk - 1) / kChunk - window_start(L, s_q, window) / kChunk;
}

struct GqaParams {
    const void *q;                 // bf16 [B][s_q][H_q][D]
    const int32_t *block_table;    // [B][max_pages]
    const int32_t *seqlens;        // [B]
    const float *k_scale;          // [H_kv] (fp8), [num_pages][H_kv][page_size / 16] (block formats) or null
    const float *v_scale;
    MetaView meta;
    void *out;                     // bf16 [B][s_q][H_q][D]
    float *lse;                    // [B][s_q][H_q]
    int32_t B, H_kv, G, H_q, max_pages, num_pages, page_size, box_tokens, boxes_per_chunk;
    int32_t s_q;                   // query tokens per request (draft j sees L - s_q + 1 + j tokens)
    int32_t window;                // sliding window in tokens (0: none)
    const float *sinks;            // [H_q] attention-sink logits (natural-log units) or null
    int32_t cluster_merge;         // 1: fixed split count 2..8, the splits merge inside a cluster (no combine)
    int32_t half_major;            // 1: the tensor maps deliver boxes as [pool][half][token][128 B]
    int32_t log2_box_tokens;       // box_tokens is 8, 16, 32 or 64
    int32_t kv_swap;               // 1: the V pool lies below the K pool (its rows come first in a box)
    int32_t kv_combined;           // 1: one 5-D map covers both pools; 0: one 4-D map per pool
    int32_t splits, num_parts;
    float scale_log2;              // softmax_scale * log2(e)
    uint64_t wait_limit_ns;
    int32_t *page_trace;           // page-trace test build only (null otherwise): rows read, per box
    int32_t page_trace_cap;        // chunks recorded per CTA
    int32_t debug_stall;           // test build only: consumers first wait on a barrier nothing completes
};

struct MlaParams {
    const void *q;                 // bf16 [B][s_q][H_q][576]
    const uint8_t *pool;           // 656-byte tokens
    const int32_t *block_table;
    const int32_t *seqlens;
    MetaView meta;
    void *out;                     // bf16 [B][s_q][H_q][512]
    float *lse;                    // [B][s_q][H_q]
    int32_t B, H_q, max_pages, num_pages, page_size;
    int32_t s_q;                   // query tokens per request (draft j sees L - s_q + 1 + j tokens)
    int32_t log2_page;             // log2(page_size) when it is a power of two, else -1
    int32_t splits, num_parts;
    float scale_log2;
    uint64_t wait_limit_ns;
    int32_t *page_trace;           // page-trace test build only (null otherwise): rows read, per token
    int32_t page_trace_cap;        // chunks recorded per part
    const int32_t *indices;        // sparse decode: [B][topk] token positions, or null
    int32_t topk;                  // 0: dense (tokens [0, L_b))
    int32_t debug_stall;           // test build only: the softmax warps first wait on a barrier nothing completes
};

struct CombineParams {
    MetaView meta;
    void *out;       // bf16 [B][rows][D_v]
    float *lse;      // [B][rows]
    int32_t B, rows, D_v, H_kv, G, splits, num_parts, s_q;   // rows = s_q * H_q per request
    int32_t window, topk;
    const float *sinks;  // [H_q] or null: joins each row's denominator after the merge
};

struct AppendParams {
    const uint16_t *k_new;         // bf16 rows, request b at k_new + b * row_stride
    const uint16_t *v_new;         // same layout (unused for the 656-byte token)
    const int32_t *positions;      // [B]; < 0: request skipped
    const int32_t *block_table;    // [B][max_pages]
    uint8_t *k_pool, *v_pool;
    const float *k_scale, *v_scale;  // [H_kv], e4m3 pools only
    int32_t *error;                // device word, error bits OR-ed in; may be null
    int64_t row_stride;            // bf16 elements between consecutive requests of k_new / v_new
    int32_t B, H_kv, D, page_size, max_pages, num_pages;
};

// Append to a cache with scales per block (append_block.cu).
struct AppendBlockParams {
    const uint16_t *k, *v;         // bf16 rows, token n at + n * stride
    int64_t k_stride, v_stride;
    const int32_t *starts;         // [B + 1] first row of each request, or null: s_q rows each
    const int32_t *positions;      // [B] where the first row goes; < 0: request skipped
    const int32_t *block_table;    // [B][max_pages]
    uint8_t *k_pool, *v_pool;
    float *k_scale, *v_scale;      // [num_pages][H_kv][page_size / 16]
    int32_t *error;                // may be null
    int32_t N, B, H_kv, s_q, page_size, max_pages, num_pages;
    int32_t per_request;           // block slots of a request where starts is null
    int64_t jobs;                  // block slots x 2 H_kv
};

// Rotary positions + append (rope.cu).
struct RopeParams {
    const uint16_t *q, *k, *v;     // bf16 rows, token n at + n * stride
    int64_t q_stride, k_stride, v_stride;
    const float *inv_freq;         // [rot / 2]
    const int32_t *rope_pos;       // [n_axes][N]
    const int32_t *requests;       // [N] or null: n / s_q
    const int32_t *positions;      // [N] slot in the request; < 0: token skipped
    const int32_t *block_table;    // [B][max_pages]
    uint16_t *q_out;               // bf16 [N][H_q][D]
    uint8_t *k_pool, *v_pool;
    const float *k_scale, *v_scale;
    int32_t *error;
    int32_t N, B, H_q, H_kv, D, s_q, page_size, max_pages, num_pages;
    int32_t rot;                   // rotated values per head, a multiple of 16
    int32_t sections[4];           // pairs per axis
    int32_t n_axes, interleaved, adjacent;
    int32_t in_place;              // q_out is q: values that are not rotated stay where they are
    int32_t items;                 // 16-value items per head
    int32_t heads;                 // head slots per token: q heads, then K and V heads (not for the 656-byte token)
    int32_t tokens;                // tokens of a tile
    int32_t parts;                 // blocks that share a tile's rows
    int32_t q_blocks;              // 656-byte token: blocks before this one rotate q, the others write tokens
};

// Attention weight gathered by cached tokens (accum.cu).
struct AccumParams {
    const void *q;                 // bf16 [B][s_q][H_q][D]
    const uint8_t *k_pool;
    const float *k_scale;          // [H_kv], e4m3 pools only
    const int32_t *block_table;
    const int32_t *seqlens;
    MetaView meta;
    const float *lse;              // [B][s_q][H_q]
    const int32_t *accepted;       // [B] or null: query tokens 0..accepted[b] count
    const int32_t *weighted;       // [B] or null: tokens whose weight is valid (the others start from 0)
    float *weights;                // [num_pages][H_kv][page_size]
    float decay, scale_log2;
    int32_t B, H_kv, G, H_q, s_q, page_size, max_pages, num_pages, splits, num_parts;
    int32_t box_tokens, boxes_per_chunk;  // as in GqaParams
    int32_t log2_page;             // log2(page_size) when it is a power of two, else -1
    int32_t parts_per_cta, heads_per_cta;
    uint64_t wait_limit_ns;
    int32_t debug_stall;           // test build only: the warps that sum first wait on a barrier nothing completes
};

// Eviction by weight (evict.cu).
struct EvictParams {
    const int32_t *seqlens;        // [B]
    const int32_t *src_table, *dst_table;  // [B][max_pages]
    uint8_t *k_pool, *v_pool;      // v_pool null: one pool (656-byte token)
    float *weights;                // [num_pages][H_kv][page_size]
    int32_t *kept;                 // [B][H_kv][budget]
    int32_t *new_seqlens;          // [B]
    int32_t *error;                // may be null
    int32_t B, H_kv, page_size, log2_page, max_pages, num_pages;
    int32_t row_bytes;             // of one token and head, a multiple of 16
    int32_t budget, first, last;
};

// The pages of a cache (pages.cu).
constexpr int kMaxPageRows = 8192;         // requests of a page operator
constexpr int kMaxPoolPages = 1 << 23;     // pages of one
// shared memory of the planning kernels: a bit per page of an eighth of the pool, three words a request
constexpr int kPlanSmemMax = kMaxPoolPages / 8 / 8 + 4 * (3 * kMaxPageRows + 1);
struct PagesParams {
    const int32_t *parents;        // [B] (fork)
    const int32_t *done;           // [B] (free)
    const int32_t *new_tokens;     // [B] or null: s_q each (reserve)
    const int32_t *seqlens_in;     // [B]
    const int32_t *table_in;       // [B][max_pages]
    const int32_t *held_in;        // [B]
    const int32_t *refs_in;        // [num_pages]
    int32_t *seqlens, *table, *held, *refs;  // written; `refs` may be refs_in (reserve)
    int32_t *new_page;             // [num_pages] (compact)
    int32_t *copies;               // pairs (source page, destination page)
    int32_t *counts;               // [2]: live pages, pairs (compact)
    int32_t *missing;              // [1] (reserve)
    int32_t *error;                // may be null
    int32_t B, s_q, page_size, max_pages, num_pages;
    int32_t ctas, share_words;     // of a planning kernel's cluster; words of 32 pages to a CTA
    int32_t max_cluster;           // CTAs of a cluster at most: 16 (the test build may lower it to 8)
};
struct CopyPagesParams {
    const int32_t *copies;         // [max_copies] pairs; a negative source: none
    const int32_t *num_copies;     // [1] or null: max_copies
    uint8_t *k_pool, *v_pool;      // v_pool null: one pool
    float *k_scale, *v_scale;      // per page scale_len values, or null
    float *weights;                // per page weight_len values, or null
    int32_t *error;                // may be null
    int64_t k_units, v_units;      // 16-byte units of a page
    uint64_t wait_limit_ns;
    int32_t debug_stall;           // test build only: the first store waits on a barrier nothing completes
    int32_t max_copies, num_pages, k_pieces, pieces, scale_len, weight_len;
};

// Probabilities out of logits (probs.cu). Sixteen CTAs hold 2^19 values in groups of eight; a row's first group may start
// seven values before it.
constexpr int kMaxProbsVocab = (1 << 19) - 7;
struct ProbsParams {
    const void *logits;            // [B][K + 1] rows of V
    void *probs;                   // likewise
    int64_t logits_stride, probs_stride;  // elements between consecutive rows
    const float *temperature, *repetition, *frequency, *presence;  // [B] or null
    const int32_t *history;        // [B][history_cols] or null
    const int32_t *history_lens, *prompt_lens;  // [B]; prompt_lens may be null
    const int32_t *drafts;         // [B][K] or null
    const int32_t *bias_starts;    // [B + 1] or null
    const int32_t *bias_tokens;
    const float *bias_values;
    const uint32_t *allowed;       // [B][K + 1] rows of ceil(V / 32) words, or null
    int64_t allowed_stride;        // words between consecutive rows
    int32_t *error;                // may be null
    int32_t logits_dtype, prob_dtype, history_cols, n_bias, B, K, V;
    int32_t slots;                 // pieces of a streaming share that shared memory holds
    int32_t cap;                   // listed tokens of a share at most
    uint64_t wait_limit_ns;
    int32_t debug_stall;           // test build only: the walkers first wait on a barrier nothing completes
    int32_t ctas, share;           // CTAs of a row; groups of eight values to a CTA
    int32_t max_cluster;           // CTAs of a cluster at most: 16 (the test build may lower it to 8)
};

// Verification of drafted tokens (verify.cu).
struct VerifyParams {
    const void *target;            // [B][K + 1] rows of V probabilities
    const void *draft;             // [B][K] rows, or null: the drafts are certain
    int64_t target_stride, draft_stride;  // elements between consecutive rows
    const int32_t *tokens;         // [B][K]
    const float *uniform;          // [B][K + 1]
    const int32_t *seqlens;        // [B] or null
    int32_t *accepted;             // [B]
    int32_t *out;                  // [B][K + 1]
    int32_t *new_seqlens;          // [B] or null
    int32_t *error;                // may be null
    int32_t B, K, V;
};

}  // namespace da
