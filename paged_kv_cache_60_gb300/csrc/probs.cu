// The probabilities that a verification draws from, out of logits: penalties for
// repeated tokens, biases, grammar masks, temperature, softmax.
//
// Row (b, j), the target's logits after the first j drafts of request b; c(v): how
// often v was generated (behind the prompt in the request's history, and among those
// drafts), seen(v): that, or in the prompt.
//     x(v) = logit(v);  seen: x > 0 ? x / r : x r;  x -= f c(v) + (c(v) > 0 ? a : 0)
//     x += its biases;  p(v) = softmax over the allowed v of x(v) / T
// T = 0: everything on the largest x (the lowest of equals). A token that the mask
// forbids takes no part, whatever its logit.
//
// A row, or a contiguous share of it where a cluster of CTAs works on one, is walked
// twice: once for the largest x and the sum of 2^(x - largest), once to write. Shares of
// at most two groups of eight values a thread stay in registers in between. Longer ones stream
// through a ring of 16 KB pieces in shared memory (bulk copies, issued by one thread as the
// slots come free); what the ring holds at the first walk's end is written first, the rest
// comes again, out of L2 for the most part: two CTAs an SM with shares of at most 256 KB.
// Measured on 1024 rows of 131072 bf16 logits to bf16: 109 us without a history (4.9
// TB/s, 0.73 of the measured copy rate), 190 with histories of 1024 to 8192 tokens (30
// instructions a value, 60 % of the issue slots; the rest are loads waited for, the lists in front of each row, and a
// fourth wave of CTAs that is a third full), 232 with masks too. (Rows held in registers throughout, by clusters of
// eight: 308 and 476 us; 128 warps a row, whose fixed work was more than the values'.)
//
// The tokens that the history, the drafts and the biases touch are few, and go their own
// way: a bit per token of the share, a prefix sum over its words, and so a place for each
// in a list, with its count (and marks: in the prompt, has a bias). They are left out
// of the first walk; a thread per listed token then computes its x, which takes its
// part in maximum and sum, and is written over what the second walk left there. A token's
// biases are added in their order, so that one that stands twice has one result. Where there are
// many, a pass over them adds each to its token's x (looked through by every token that has one, as a
// few are, a bias on each of 131072 tokens took 342 ms for one row, now 0.57); and where the list is too short
// for a share's tokens, they are taken window by window.
//
// Sums: a thread's own in fp32, then warps, then the (largest, sum) pairs of the CTAs, in a
// fixed order.
//
// Rows start anywhere: groups of eight values start where the logits are aligned to
// eight of them, the first and last of a row are taken value by value. Where the
// probabilities' row is aligned like the logits' they are written in vectors, else value
// by value.
#include <cuda_runtime.h>

#include <atomic>
#include <cfloat>
#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "decode_attn.h"
#include "layout.h"
#include "quant.cuh"

namespace da {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kShareBytes = 256 << 10;          // of a CTA at most: 2^17 values
// groups of a thread in a piece of a share that streams: 16 KB a piece
template <typename T>
constexpr int kPerThread = sizeof(T) == 2 ? 2 : 1;
constexpr int kPieceBytes = 16 << 10;
constexpr int kMaxSlots = 12;
constexpr int kAhead = 8, kAbreast = 4;        // tokens of the history, listed tokens that a thread has under way
constexpr int kSmemMax = 224 << 10, kSmemTwo = 112 << 10;  // of a CTA; where two fit an SM
// Tokens that a list has room for at most, beside the marks of a share of 2^17 and two pieces: where two CTAs fit an SM, and else
constexpr int kListRoomTwo = 9344, kListRoom = 27904;
static_assert(2 * kPieceBytes + kShareBytes / 2 / 32 * 6 + kListRoomTwo * 6 + kListRoomTwo / 8 <= kSmemTwo, "two CTAs an SM");
static_assert(2 * kPieceBytes + kShareBytes / 2 / 32 * 6 + kListRoom * 6 + kListRoom / 8 <= kSmemMax, "one");
constexpr int kBiasRoom = 1024;
// biases of a request that every token with one looks through; more are added to the list's x instead (two barriers more and a chain of
// loads: one row of 32000 with up to 4 biases 8.6 instead of 7.3 us, 576 rows of 131072 with up to 300 125 instead of 225)
constexpr int kFewBiases = 32;
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kPrompt = 0x80000000u, kBias = 0x40000000u, kCount = kBias - 1;

template <typename T>
__device__ __forceinline__ float2 pair_to_f32(uint32_t w);
template <>
__device__ __forceinline__ float2 pair_to_f32<__half>(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}
template <>
__device__ __forceinline__ float2 pair_to_f32<__nv_bfloat16>(uint32_t w) {
    return make_float2(bf16_lo(w), bf16_hi(w));
}
// Eight values as they lie in memory: 16 bytes of a two-byte type, 32 of fp32.
template <typename T>
struct Raw {
    static constexpr int kWords = 2 * (int)sizeof(T);
    static constexpr uint32_t kNone = sizeof(T) == 4 ? 0xFF800000u : __is_same(T, __half) ? 0xFC00FC00u : 0xFF80FF80u;  // -infinity
    uint32_t w[kWords];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = kNone;
    }
    __device__ __forceinline__ void load(const T *at) {
#pragma unroll
        for (int i = 0; i < kWords; i += 4) {
            const uint4 v = *reinterpret_cast<const uint4 *>(at + i * 4 / (int)sizeof(T));
            w[i] = v.x, w[i + 1] = v.y, w[i + 2] = v.z, w[i + 3] = v.w;
        }
    }
    // from shared memory that a bulk copy fills again once it is released: volatile, so that the loads stay ahead of the
    // release (plain ones, released before their values had been used, gave some rows the next piece's values)
    __device__ __forceinline__ void load_shared(uint32_t at) {
#pragma unroll
        for (int i = 0; i < kWords; i += 4)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w[i]), "=r"(w[i + 1]), "=r"(w[i + 2]), "=r"(w[i + 3])
                         : "r"(at + i * 4)
                         : "memory");
    }
    // value by value, those of [0, V); t: the first one's token
    __device__ __forceinline__ void load_some(const T *row, int t, int V) {
        clear();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (t + i < 0 || t + i >= V) continue;
            if constexpr (sizeof(T) == 4) {
                w[i] = __float_as_uint(row[t + i]);
            } else {
                const uint32_t h = *reinterpret_cast<const uint16_t *>(row + t + i);
                w[i / 2] = i & 1 ? (w[i / 2] & 0xFFFFu) | h << 16 : (w[i / 2] & 0xFFFF0000u) | h;
            }
        }
    }
    // -infinity where keep's bit is not set. Four bits at a time become the signs of four bytes (the product's terms meet
    // nowhere), and those the masks of the words, by a permute that repeats signs: 11 instructions for eight two-byte values.
    __device__ __forceinline__ void drop(uint32_t keep) {
        constexpr int kHalf = kWords / 2;
        const uint32_t signs[2] = {(keep & 0xFu) * 0x10204080u, (keep >> 4 & 0xFu) * 0x10204080u};
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
            const int k = i % kHalf;
            const uint32_t sel = sizeof(T) == 4 ? 0x8888u + 0x1111u * k : k ? 0xBBAAu : 0x9988u;
            uint32_t m;
            asm("prmt.b32 %0, %1, 0, %2;" : "=r"(m) : "r"(signs[i / kHalf]), "r"(sel));
            w[i] = (w[i] & m) | (kNone & ~m);
        }
    }
    __device__ __forceinline__ void widen(float (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if constexpr (sizeof(T) == 4) {
                x[i] = __uint_as_float(w[i]);
            } else if (i % 2 == 0) {
                const float2 f = pair_to_f32<T>(w[i / 2]);
                x[i] = f.x, x[i + 1] = f.y;
            }
        }
    }
};
// the larger of two pairs, or of two fp32; NaN where one is
template <typename T>
__device__ __forceinline__ uint32_t max_word(uint32_t a, uint32_t b) {
    uint32_t d;
    if constexpr (sizeof(T) == 4)
        return __float_as_uint(fmax_nan(__uint_as_float(a), __uint_as_float(b)));
    else if constexpr (__is_same(T, __half))
        asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    else
        asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
template <typename T, int kN>
__device__ __forceinline__ float largest_of(const Raw<T> (&r)[kN]) {
    uint32_t m[kN];
#pragma unroll
    for (int k = 0; k < kN; ++k) {
        m[k] = r[k].w[0];
#pragma unroll
        for (int i = 1; i < Raw<T>::kWords; ++i) m[k] = max_word<T>(m[k], r[k].w[i]);
    }
#pragma unroll
    for (int k = 1; k < kN; ++k) m[0] = max_word<T>(m[0], m[k]);
    if constexpr (sizeof(T) == 4) {
        return __uint_as_float(m[0]);
    } else {
        const float2 f = pair_to_f32<T>(m[0]);
        return fmax_nan(f.x, f.y);
    }
}
// (32 bytes at once: as two stores of 16, each of which leaves half of every sector out, a row of
// 131072 took 15.4 us to write instead of 6)
__device__ __forceinline__ void store8(float *at, const float (&x)[8]) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "f"(x[0]), "f"(x[1]), "f"(x[2]),
                 "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7])
                 : "memory");
}
__device__ __forceinline__ void store8(__nv_bfloat16 *at, const float (&x)[8]) {
    st_v4(at, make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])));
}
__device__ __forceinline__ void store8(__half *at, const float (&x)[8]) {
    st_v4(at, make_uint4(pack_f16(x[0], x[1]), pack_f16(x[2], x[3]), pack_f16(x[4], x[5]), pack_f16(x[6], x[7])));
}
__device__ __forceinline__ void store1(float *at, float x) { *at = x; }
__device__ __forceinline__ void store1(__nv_bfloat16 *at, float x) { *at = __float2bfloat16_rn(x); }
__device__ __forceinline__ void store1(__half *at, float x) { *at = __float2half_rn(x); }

// A row of probabilities: a group of eight, of which only tokens in [0, V) are there, those in `skip` left as they are (vec: it is
// aligned like the logits' group)
template <typename T>
__device__ __forceinline__ void store_group(T *row, int t, int V, bool vec, uint32_t skip, const float (&x)[8]) {
    if (vec && t >= 0 && t + 8 <= V && skip == 0) {
        store8(row + t, x);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (t + i >= 0 && t + i < V && !(skip >> i & 1)) store1(row + t + i, x[i]);
    }
}

__device__ __forceinline__ float warp_max_nan(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmax_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
}
__device__ __forceinline__ float warp_add(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
// 2^((x - from) scale + off) of eight values. (Packed two to an instruction the differences and products cost more
// moves than they save: 8 instead of 4 instructions a value.)
struct Exps {
    float from, scale, off;
    __device__ __forceinline__ float operator()(float x) const { return ex2(fmaf(x - from, scale, off)); }
    __device__ __forceinline__ void of(float (&x)[8]) const {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (*this)(x[i]);
    }
};
__device__ __forceinline__ float sum8(const float (&x)[8]) {
    return ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
}

// A running maximum with the sum of 2^((x - m) s), or the largest x with its token.
struct Run {
    float m = -INFINITY, sum = 0.f;
    int at = INT32_MAX;
    // raises the maximum to `to` at least; what differences are taken from then (finite where nothing has been seen)
    __device__ __forceinline__ float raise(float to, float s) {
        const float n = fmax_nan(m, to), from = n == -INFINITY ? 0.f : n;
        sum *= ex2((m - from) * s);  // 1 where it stays, 0 where nothing has been seen
        m = n;
        return from;
    }
    __device__ __forceinline__ void take(float x, int token) {
        if (x > m || (x == m && token < at && x > -INFINITY)) m = x, at = token;
    }
};

// Words of a share's marks, a run of eight for each thread that has one: those of a share fit.
static_assert(kShareBytes / 2 / 32 <= 8 * kThreads, "a run of eight words per thread");
__host__ __device__ inline int words_of(int share) { return (share * 8 + 255) / 256 * 8; }
__host__ __device__ inline int many_words(int cap) { return (cap + 127) / 128 * 4; }  // a bit per place of a list

// What x becomes, but for its biases, of a logit with a count and marks (kPrompt, kCount).
__device__ __forceinline__ float penalised(float y, uint32_t c, float rep, float freq, float pres) {
    const uint32_t n = c & kCount;
    if (n > 0 || (c & kPrompt)) y = y > 0.f ? __fdiv_rn(y, rep) : __fmul_rn(y, rep);
    y = __fsub_rn(y, __fmul_rn(freq, (float)n));
    return n > 0 ? __fsub_rn(y, pres) : y;
}

// The list of the touched tokens in shared memory: those of [lowest, lowest + span), of which `before` of the share's stand in
// front. From `mark` on there lie: a bit per token of the share (`words` of them); for each listed token (cap) its count and marks, then
// its x; for each a bit, whether it has several biases; for each word the marks in the words before, without multiples of
// 65536; the listed tokens, from t0 on, without 65536: they ascend, `upper` and up have it.
struct List {
    uint32_t *mark;
    int words, cap;
    int t0, lowest, span, before, upper;
    __device__ __forceinline__ uint32_t *value() const { return mark + words; }
    __device__ __forceinline__ uint32_t *many() const { return mark + words + cap; }
    __device__ __forceinline__ uint16_t *place() const { return reinterpret_cast<uint16_t *>(mark + words + cap + many_words(cap)); }
    __device__ __forceinline__ uint16_t *tokens() const { return place() + words; }
    __device__ __forceinline__ int at(int i) const {  // token t0 + i, which is here
        return (uint16_t)(place()[i / 32] + __popc(mark[i / 32] & ((1u << (i & 31)) - 1)) - before);
    }
    __device__ __forceinline__ int place_of(int token) const {  // -1: not here
        return (unsigned)(token - lowest) < (unsigned)span ? at(token - t0) : -1;
    }
    __device__ __forceinline__ int token_at(int k) const { return t0 + tokens()[k] + (k >= upper ? 65536 : 0); }
    __device__ __forceinline__ uint32_t *enlist(int i) const {  // token t0 + i
        const int k = at(i);
        tokens()[k] = (uint16_t)i;
        return value() + k;
    }
    __device__ __forceinline__ void enlist_bias(int i) const {
        uint32_t *v = enlist(i);
        const int k = (int)(v - value());
        if (atomicOr(v, kBias) & kBias) atomicOr(many() + k / 32, 1u << (k & 31));
    }
    __device__ __forceinline__ bool has_many(int k) const { return many()[k / 32] >> (k & 31) & 1; }
};
// f(token, its index) for the tokens [from, to) of an array, kAhead loads of a thread under way at once.
template <typename F>
__device__ __forceinline__ void each_token(const int32_t *tokens, int from, int to, F f) {
    for (int i0 = from + (int)threadIdx.x; i0 < to; i0 += kAhead * kThreads) {
        int tok[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) tok[k] = i0 + k * kThreads < to ? tokens[i0 + k * kThreads] : -1;
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (tok[k] >= 0) f(tok[k], i0 + k * kThreads);
    }
}
// The biases [lo, hi), added to the x of the list, each token's in their order: a token with one bias takes it from whichever thread
// meets it; those with several, if there are any, from one warp that goes through the biases in order. All threads of the CTA;
// the sums are there when it returns. (Inlined, as what follows: called out of line they made the walks around them spill.)
__device__ __forceinline__ void add_biases(const ProbsParams &p, List l, int lo, int hi) {
    bool later = false;
    __syncthreads();
    for (int i0 = lo + (int)threadIdx.x; i0 < hi; i0 += kAhead * kThreads) {
        int tok[kAhead];
        float v[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int i = i0 + k * kThreads;
            tok[k] = i < hi ? p.bias_tokens[i] : -1;
            v[k] = i < hi ? p.bias_values[i] : 0.f;
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int at = l.place_of(tok[k]);
            if (at < 0) continue;
            if (l.has_many(at))
                later = true;
            else
                l.value()[at] = __float_as_uint(__fadd_rn(__uint_as_float(l.value()[at]), v[k]));
        }
    }
    if (!__syncthreads_or(later)) return;
    if (threadIdx.x < 32) {
        const int lane = (int)threadIdx.x;
        for (int i0 = lo; i0 < hi; i0 += 32) {
            int at = i0 + lane < hi ? l.place_of(p.bias_tokens[i0 + lane]) : -1;
            if (at >= 0 && !l.has_many(at)) at = -1;
            const float v = at >= 0 ? p.bias_values[i0 + lane] : 0.f;
            // lanes with the same token: one behind the other
            const unsigned here = __ballot_sync(0xFFFFFFFFu, at >= 0);
            const int turn = at >= 0 ? __popc(__match_any_sync(here, at) & ((1u << lane) - 1)) : -1;
            const int last = __reduce_max_sync(0xFFFFFFFFu, turn);
            for (int k = 0; k <= last; ++k) {
                if (k == turn) l.value()[at] = __float_as_uint(__fadd_rn(__uint_as_float(l.value()[at]), v));
                __syncwarp();
            }
        }
    }
    __syncthreads();
}
// Draft `tid` of a chain, where it stands before row j and the chain has not ended before it; else -1.
__device__ __forceinline__ int draft_before(const ProbsParams &p, int b, int j, int tid) {
    if (p.drafts == nullptr || tid >= j) return -1;
    const int32_t *drafts = p.drafts + (int64_t)b * p.K;
    int signs = 0;
    for (int i = 0; i < tid; ++i) signs |= drafts[i];
    return signs < 0 ? -1 : drafts[tid];
}

// A row, and a CTA's share of it.
template <typename TI>
struct Place {
    int row, rank, b, j;
    const TI *in;        // the row's logits
    int t0, groups;      // token of the share's first value; group g holds t0 + 8 g ..
    const uint32_t *bits;
    int n_hist, prompt, blo, bhi;
    __device__ __forceinline__ Place(const ProbsParams &p) {
        row = blockIdx.x / p.ctas, rank = blockIdx.x - row * p.ctas;
        b = row / (p.K + 1), j = row - b * (p.K + 1);
        in = static_cast<const TI *>(p.logits) + row * p.logits_stride;
        t0 = rank * p.share * 8 - (int)(reinterpret_cast<uintptr_t>(in) / sizeof(TI) & 7);
        groups = max(min(p.share, (p.V - t0 + 7) / 8), 0);
        bits = p.allowed ? p.allowed + row * p.allowed_stride : nullptr;
        n_hist = p.history ? min(max(p.history_lens[b], 0), p.history_cols) : 0;
        prompt = p.prompt_lens ? p.prompt_lens[b] : 0;
        blo = p.bias_starts ? min(max(p.bias_starts[b], 0), p.n_bias) : 0;
        bhi = p.bias_starts ? min(max(p.bias_starts[b + 1], 0), p.n_bias) : 0;
    }
    __device__ __forceinline__ List list(const ProbsParams &p) const {
        extern __shared__ uint4 smem_v[];
        uint32_t *mark = reinterpret_cast<uint32_t *>(reinterpret_cast<uint8_t *>(smem_v) + (size_t)p.slots * kPieceBytes);
        const int lowest = max(t0, 0);
        return {mark, words_of(p.share), p.cap, t0, lowest, min(p.V - t0, groups * 8) - (lowest - t0), 0, INT32_MAX};
    }
};

// x, biases and all, of the listed tokens, in place of their counts and marks.
template <typename TI>
__device__ __forceinline__ void settle(const ProbsParams &p, const Place<TI> &at, const List &l, int listed) {
    const float rep = p.repetition ? p.repetition[at.b] : 1.f, freq = p.frequency ? p.frequency[at.b] : 0.f;
    const float pres = p.presence ? p.presence[at.b] : 0.f;
    for (int i = threadIdx.x; i < listed; i += kThreads)
        l.value()[i] = __float_as_uint(penalised(static_cast<float>(at.in[l.token_at(i)]), l.value()[i], rep, freq, pres));
    if (at.bhi > at.blo) add_biases(p, l, at.blo, at.bhi);
}
template <typename TI>
__device__ __forceinline__ void settle_list(const ProbsParams &p, int listed) {
    const Place<TI> at(p);
    List l = at.list(p);
    if (l.words > 65536 / 32) l.upper = l.place()[65536 / 32];
    settle(p, at, l, listed);
}

// The touched tokens of a share that has more of them than the list has room for (p.cap), window by window: as many runs of 256 tokens as
// the list holds, enlisted anew from history, drafts and biases. What each thread has met of them, (largest, sum) or (largest, its
// token); or their probabilities are written. All threads of the CTA.
enum class Crowd { kSum, kLargest, kWrite, kWriteZero, kWriteNan };
template <typename TI>
__device__ __forceinline__ float2 crowded_tokens(const ProbsParams &p, Crowd what, float scale, float from, float off) {
    constexpr int kRunTokens = 256;
    __shared__ int sums[kWarps + 1];
    const Place<TI> at(p);
    const List whole = at.list(p);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, runs = whole.words / 8;
    Run run;
    const int32_t *hist = p.history + (int64_t)at.b * p.history_cols;
    const int draft = draft_before(p, at.b, at.j, tid);
    const int out_size = p.prob_dtype == DA_PROB_F32 ? 4 : 2;
    uint8_t *out = static_cast<uint8_t *>(p.probs) + at.row * p.probs_stride * out_size;
    // marks up to the end of this thread's run
    int end = 0;
    for (int k = 0; k < 8 && tid < runs; ++k) end += __popc(whole.mark[tid * 8 + k]);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xFFFFFFFFu, end, o);
        if (lane >= o) end += u;
    }
    if (lane == 31) sums[warp] = end;
    __syncthreads();
    for (int w = 0; w < warp; ++w) end += sums[w];
    for (int r0 = 0, base = 0; r0 < runs;) {
        // (a run fits: a list that may be too short has room for 1024 tokens)
        const int r1 = r0 + __syncthreads_count(tid >= r0 && tid < runs && end - base <= p.cap);
        if (tid == r1 - 1) sums[kWarps] = end;
        List l = whole;
        for (int i = tid; i < p.cap; i += kThreads) l.value()[i] = 0u;
        for (int i = tid; i < many_words(p.cap); i += kThreads) l.many()[i] = 0u;
        __syncthreads();
        const int n = sums[kWarps] - base;
        l.lowest = max(whole.lowest, l.t0 + r0 * kRunTokens);
        l.span = max(min(whole.lowest + whole.span, l.t0 + r1 * kRunTokens) - l.lowest, 0);
        l.before = base;
        l.upper = r0 * kRunTokens >= 65536 ? 0 : r1 * kRunTokens > 65536 ? (uint16_t)(l.place()[65536 / 32] - base) : INT32_MAX;
        const auto here = [&](int token) -> bool { return (unsigned)(token - l.lowest) < (unsigned)l.span; };
        each_token(hist, 0, at.n_hist, [&](int token, int i) {
            if (!here(token)) return;
            uint32_t *v = l.enlist(token - l.t0);
            if (i < at.prompt)
                atomicOr(v, kPrompt);
            else
                atomicAdd(v, 1u);
        });
        if (draft >= 0 && here(draft)) atomicAdd(l.enlist(draft - l.t0), 1u);
        each_token(p.bias_tokens, at.blo, at.bhi, [&](int token, int) {
            if (here(token)) l.enlist_bias(token - l.t0);
        });
        __syncthreads();
        settle(p, at, l, n);
        __syncthreads();
        for (int i = tid; i < n; i += kThreads) {
            const int t = l.token_at(i);
            const float y = __uint_as_float(l.value()[i]);
            const float v = !at.bits || (at.bits[t >> 5] >> (t & 31) & 1) ? y : -INFINITY;
            if (what == Crowd::kSum) {
                const float to = run.raise(v, scale);
                run.sum += ex2((v - to) * scale);
            } else if (what == Crowd::kLargest) {
                run.take(v, t);
            } else {
                const float x = what == Crowd::kWrite ? Exps{from, scale, off}(v) : what == Crowd::kWriteZero ? 0.f : NAN;
                if (p.prob_dtype == DA_PROB_F32)
                    store1(reinterpret_cast<float *>(out) + t, x);
                else if (p.prob_dtype == DA_PROB_BF16)
                    store1(reinterpret_cast<__nv_bfloat16 *>(out) + t, x);
                else
                    store1(reinterpret_cast<__half *>(out) + t, x);
            }
        }
        base += n;
        r0 = r1;
    }
    __syncthreads();
    return make_float2(run.m, what == Crowd::kLargest ? __int_as_float(run.at) : run.sum);
}

// kG: groups of eight values that a thread holds between the walks; 0: the share streams. kMany: built for requests that may have many
// biases or more tokens than the list has room for (which costs the others: 1024 rows of 131072 with histories 200 instead of
// 190 us, one row of 32000 7.5 instead of 7.0).
template <typename TI, int kG, bool kMany>
__global__ void __launch_bounds__(kThreads, 2) probs_kernel(const __grid_constant__ ProbsParams p) {
    extern __shared__ uint4 smem_v[];
    __shared__ float2 warp_pair[kWarps];
    __shared__ float2 cta_pair;          // largest, and sum (or the token, as bits)
    __shared__ int warp_sum[kWarps];
    __shared__ int s_listed;
    __shared__ uint64_t full[kMaxSlots], empty[kMaxSlots];
    __shared__ int given_up;
#ifdef DA_PAGE_TRACE
    __shared__ uint64_t never;  // a barrier that nothing completes
#endif
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Place<TI> here(p);
    const int row = here.row, rank = here.rank, b = here.b, j = here.j;
    const int V = p.V;
    const TI *in = here.in;
    const int out_size = p.prob_dtype == DA_PROB_F32 ? 4 : 2;
    uint8_t *out_at = static_cast<uint8_t *>(p.probs) + row * p.probs_stride * out_size;
    const bool vec = (int)(reinterpret_cast<uintptr_t>(out_at) / out_size & 7) == (int)(reinterpret_cast<uintptr_t>(in) / sizeof(TI) & 7);
    const int t0 = here.t0, groups = here.groups;
    const uint32_t *bits = here.bits;
    const int words = (V + 31) / 32;

    // the logits of a group, -infinity where there is none
    const auto load_group = [&](int g, Raw<TI> &r) {
        const int t = t0 + g * 8;
        if (t >= 0 && t + 8 <= V)
            r.load(in + t);
        else
            r.load_some(in, t, V);
    };
    // bit i: token i of the group is allowed
    const auto allowed_of = [&](int g) -> uint32_t {
        const int t = t0 + g * 8, w = t >> 5;  // w is -1 in front of the row
        const uint32_t lo = w >= 0 ? bits[w] : 0u, hi = w + 1 < words ? bits[w + 1] : 0u;
        return __funnelshift_r(lo, hi, t & 31) & 0xFFu;
    };
    // whole groups of the share: [whole0, whole1)
    const int whole0 = t0 < 0 ? 1 : 0, whole1 = V - t0 >= 8 ? min(groups, (V - t0) / 8) : 0;
    // a share that streams: its whole groups in pieces, through a ring of slots. Load l (piece l on the first walk; on the second,
    // piece l - pieces, those that the first has left in the ring are not loaded again) goes to slot l % slots. Thread 0
    // issues load l + slots once all warps have released what load l's slot held, a piece behind its own reading.
    constexpr int kPer = kPerThread<TI>, kPiece = kPer * kThreads;
    static_assert(kPiece * 8 * (int)sizeof(TI) == kPieceBytes, "pieces of 16 KB");
    const int slots = p.slots, pieces = whole1 > whole0 ? (whole1 - whole0 + kPiece - 1) / kPiece : 0;
    const auto issue = [&](int l, int slot) {
        const int g = whole0 + (l < pieces ? l : l - pieces) * kPiece;
        const uint32_t bytes = (uint32_t)min(kPiece, whole1 - g) * 8u * (uint32_t)sizeof(TI);
        mbar_arrive_expect_tx(&full[slot], bytes);
        bulk_load(reinterpret_cast<uint8_t *>(smem_v) + (size_t)slot * kPieceBytes, in + t0 + g * 8, bytes, &full[slot]);
    };
    // what the lists and the walks wait for, read ahead of the rest
    const int n_hist = here.n_hist, blo = here.blo, bhi = here.bhi, prompt = here.prompt;
    const float T = p.temperature ? p.temperature[b] : 1.f;
    const int draft = draft_before(p, b, j, tid);
    if (kG == 0 && tid == 0) {
        for (int k = 0; k < slots; ++k) {
            mbar_init(&full[k], 1);
            mbar_init(&empty[k], kWarps);
        }
        given_up = 0;
#ifdef DA_PAGE_TRACE
        mbar_init(&never, 1);
#endif
        fence_barrier_init();
        fence_proxy_async_smem();
        for (int l = 0; l < min(slots, pieces); ++l) issue(l, l);
    }
    const auto wait = [&](uint64_t *bar, int phase) -> bool {
        if (mbar_try_wait(bar, phase & 1)) return true;
        const uint64_t begin = global_ns();
        do {  // (asleep, rather than polling: the other warps need the issue slots)
            if (mbar_try_wait_sleep(bar, phase & 1, 20000u)) return true;
        } while (*(volatile int *)&given_up == 0 && global_ns() - begin < p.wait_limit_ns);
        *(volatile int *)&given_up = 1;
        if (p.error) atomicOr(p.error, DA_DEV_TIMEOUT);
        return false;
    };
    // the ring's next slot, and how often it has been round
    struct Turn {
        int slot = 0, round = 0;
        __device__ __forceinline__ void next(int slots) {
            if (++slot == slots) slot = 0, ++round;
        }
    };
    Turn at_load;   // thread 0: of the next load that a release lets go, load slots + this
    int loads = min(slots, pieces);  // issued
    const auto refill = [&] {
        if (*(volatile int *)&given_up != 0 || !wait(&empty[at_load.slot], at_load.round)) return;
        issue(loads, at_load.slot);
        ++loads;
        at_load.next(slots);
    };
    const auto release = [&](int slot) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[slot]);
    };
    // this thread's groups of a piece that starts with group g, in its slot
    const auto read_slot = [&](int slot, int g, auto &r, auto all) {
        const uint32_t at = smem_u32(smem_v) + (uint32_t)(slot * kPieceBytes + tid * 8 * (int)sizeof(TI));
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (all || g + i * kThreads + tid < whole1)
                r[i].load_shared(at + i * kThreads * 8 * (int)sizeof(TI));
            else
                r[i].clear();
        }
    };
    Raw<TI> held[kG > 0 ? kG : 1];
    if constexpr (kG > 0) {
#pragma unroll
        for (int k = 0; k < kG; ++k) {
            held[k].clear();
            if (k * kThreads + tid < groups) load_group(k * kThreads + tid, held[k]);
        }
    }
    const bool warm = T > 0.f;
    // (a temperature next to 0: 0 times its reciprocal stays 0; an infinite one: -infinity stays that)
    const float scale = warm ? fmaxf(fminf(__fdiv_rn(kLog2e, T), FLT_MAX), FLT_MIN) : 1.f;

    // ------------------------------------------------ the tokens that history, drafts and biases touch
    const bool touched = n_hist > 0 || (p.drafts != nullptr && j > 0) || bhi > blo;  // the same for the whole CTA
    const int share_words = words_of(p.share);
    uint32_t *mark = reinterpret_cast<uint32_t *>(reinterpret_cast<uint8_t *>(smem_v) +
                                                  (kG == 0 ? (size_t)slots * kPieceBytes : 0));  // a bit per token of the share
    // of each listed token: count and marks, then x
    uint32_t *value = mark + share_words;
    uint16_t *place = reinterpret_cast<uint16_t *>(value + p.cap + many_words(p.cap));  // marks in the words before
    uint16_t *list = place + share_words;  // the listed tokens, from t0 on, without 65536: they ascend, `upper` and up have it
    int upper = INT32_MAX;
    const auto token_at = [&](int i) -> int { return t0 + list[i] + (i >= upper ? 65536 : 0); };
    int listed = 0;
    bool crowded = false;  // more than the list has room for
    const int32_t *hist = p.history + (int64_t)b * p.history_cols;
    if (touched) {
        const int first_bias = blo + tid < bhi ? p.bias_tokens[blo + tid] : -1;
        const int cap = (min(p.cap, n_hist + j + bhi - blo) + 3) / 4;
        for (int i = tid; i < share_words / 4; i += kThreads) reinterpret_cast<uint4 *>(mark)[i] = make_uint4(0u, 0u, 0u, 0u);
        for (int i = tid; i < cap; i += kThreads) reinterpret_cast<uint4 *>(value)[i] = make_uint4(0u, 0u, 0u, 0u);
        if (kMany && bhi - blo > kFewBiases)
            for (int i = tid; i < many_words(4 * cap); i += kThreads) value[p.cap + i] = 0u;
        __syncthreads();
        const int lowest = max(t0, 0), span = min(V - t0, groups * 8) - (lowest - t0);
        // f(token's place in the share) for every token of the history in [from, to)
        const auto each = [&](int from, int to, auto f) {
            for (int i0 = from + tid; i0 < to; i0 += kAhead * kThreads) {
                int tok[kAhead];
#pragma unroll
                for (int k = 0; k < kAhead; ++k) tok[k] = i0 + k * kThreads < to ? hist[i0 + k * kThreads] : -1;
#pragma unroll
                for (int k = 0; k < kAhead; ++k)
                    if ((unsigned)(tok[k] - lowest) < (unsigned)span) f(tok[k] - t0);
            }
        };
        // and for those of the drafts and biases
        const auto drafted = [&](auto f) {
            if (draft >= 0 && (unsigned)(draft - lowest) < (unsigned)span) f(draft - t0);
        };
        const auto biased = [&](auto f) {
            for (int i = blo + tid; i < bhi; i += kThreads) {
                const int tok = i == blo + tid ? first_bias : p.bias_tokens[i];
                if ((unsigned)(tok - lowest) < (unsigned)span) f(tok - t0);
            }
        };
        const auto touch = [&](int i) { atomicOr(mark + i / 32, 1u << (i & 31)); };
        each(0, n_hist, touch);
        drafted(touch);
        biased(touch);
        __syncthreads();
        // prefix sum over the words, a run of eight per thread
        uint32_t m[8];
        int mine = 0;
        const bool has = tid * 8 < share_words;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const uint4 v = has ? reinterpret_cast<const uint4 *>(mark)[tid * 2 + k] : make_uint4(0u, 0u, 0u, 0u);
            m[4 * k] = v.x, m[4 * k + 1] = v.y, m[4 * k + 2] = v.z, m[4 * k + 3] = v.w;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) mine += __popc(m[k]);
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o) incl += u;
        }
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
        int at = incl - mine;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) at += w < warp ? warp_sum[w] : 0;
        if (tid == kThreads - 1) s_listed = at + mine;
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
            const int second = at + __popc(m[k]);
            const uint32_t both = ((uint32_t)at & 0xFFFFu) | (uint32_t)second << 16;  // (a share may have more than 65535)
            at = second + __popc(m[k + 1]);
            m[k / 2] = both;  // (read by now)
        }
        if (has) reinterpret_cast<uint4 *>(place)[tid] = make_uint4(m[0], m[1], m[2], m[3]);
        __syncthreads();
        listed = s_listed;
        if (share_words > 65536 / 32) upper = place[65536 / 32];
        const auto enlist = [&](int i) -> uint32_t * {  // its place in the list
            const int at = place[i / 32] + __popc(mark[i / 32] & ((1u << (i & 31)) - 1));
            list[at] = (uint16_t)i;
            return value + at;
        };
        crowded = kMany && listed > p.cap;
        if (!crowded) {
            each(0, min(prompt, n_hist), [&](int i) { atomicOr(enlist(i), kPrompt); });
            each(max(prompt, 0), n_hist, [&](int i) { atomicAdd(enlist(i), 1u); });
            drafted([&](int i) { atomicAdd(enlist(i), 1u); });
            biased([&](int i) {
                uint32_t *v = enlist(i);
                if (const uint32_t was = atomicOr(v, kBias); kMany && bhi - blo > kFewBiases && (was & kBias))
                    atomicOr(value + p.cap + (v - value) / 32, 1u << ((v - value) & 31));
            });
        }
        __syncthreads();
    }
    if (kG == 0) __syncthreads();  // the ring's barriers are initialised
    // ------------------------------------------------ the first walk: all tokens but those
    Run run;
    const auto keep_of = [&](int g) -> uint32_t {
        uint32_t keep = bits ? allowed_of(g) : 0xFFu;
        if (listed > 0) keep &= ~(uint32_t) reinterpret_cast<const uint8_t *>(mark)[g];
        return keep;
    };
    // of a thread's whole groups in a piece, read before the piece is waited for
    const auto keeps = [&](int g, bool marked, uint32_t (&keep)[kPer]) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) keep[i] = 0xFFu;
        if (bits) {  // the byte with the group's first bit, and the one with its last
            const uint8_t *bytes = reinterpret_cast<const uint8_t *>(bits);
            uint32_t lo[kPer], hi[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int t = t0 + (g + i * kThreads) * 8;
                const bool there = g + i * kThreads < whole1;
                lo[i] = there ? bytes[t >> 3] : 0u;
                hi[i] = there ? bytes[(t + 7) >> 3] : 0u;
            }
#pragma unroll
            for (int i = 0; i < kPer; ++i) keep[i] = (lo[i] | hi[i] << 8) >> (t0 & 7) & 0xFFu;
        }
        if (marked && listed > 0) {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (g + i * kThreads < whole1) keep[i] &= ~(uint32_t) reinterpret_cast<const uint8_t *>(mark)[g + i * kThreads];
        }
    };
    // groups g, g + kThreads, ..
    const auto walk = [&](int g, const auto &r) {
        constexpr int kN = (int)(sizeof(r) / sizeof(r[0]));
        if (warm) {
            const Exps exps{run.raise(largest_of(r), scale), scale, 0.f};
#pragma unroll
            for (int k = 0; k < kN; ++k) {
                float e[8];
                r[k].widen(e);
                exps.of(e);
                run.sum += sum8(e);
            }
        } else {
            if (largest_of(r) < run.m) return;  // (not where one is NaN)
#pragma unroll
            for (int k = 0; k < kN; ++k) {
                float v[8];
                r[k].widen(v);
#pragma unroll
                for (int i = 0; i < 8; ++i) run.take(v[i], t0 + (g + k * kThreads) * 8 + i);
            }
        }
    };
    const auto drop_untaken = [&](int g, auto &r) {
        constexpr int kN = (int)(sizeof(r) / sizeof(r[0]));
        if (!bits && listed == 0) return;
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            if (g + k * kThreads >= groups) continue;
            const uint32_t keep = keep_of(g + k * kThreads);
            if (keep != 0xFFu) r[k].drop(keep);
        }
    };
    if constexpr (kG > 0) {
        drop_untaken(tid, held);
        walk(tid, held);
    } else {
        const auto edge = [&](int g) {
            Raw<TI> r[1];
            load_group(g, r[0]);
            r[0].drop(keep_of(g));
            walk(g, r);
        };
        if (tid == 0 && whole0 > 0 && groups > 0) edge(0);
        if (tid == 32 && whole1 < groups && (whole1 > 0 || whole0 == 0)) edge(groups - 1);
#ifdef DA_PAGE_TRACE
        if (p.debug_stall) wait(&never, 0);  // test build: a wait that runs out
#endif
        Turn now;
        for (int k = 0; k < pieces; ++k, now.next(slots)) {
            const int g = whole0 + k * kPiece;
            uint32_t keep[kPer];
            if (bits || listed > 0) keeps(g + tid, true, keep);
            if (tid == 0 && k > 0 && k - 1 + slots < pieces) refill();
            wait(&full[now.slot], now.round);
            Raw<TI> r[kPer];
            const auto part = [&](auto all, auto untouched) {  // (all: whole pieces; untouched: no token is left out)
                read_slot(now.slot, g, r, all);
                if (!untouched && (bits || listed > 0)) {
#pragma unroll
                    for (int i = 0; i < kPer; ++i)
                        if (keep[i] != 0xFFu) r[i].drop(keep[i]);
                }
                walk(g + tid, r);
            };
            if (g + kPiece <= whole1 && !bits && listed == 0)
                part(std::true_type(), std::true_type());
            else if (g + kPiece <= whole1)
                part(std::true_type(), std::false_type());
            else
                part(std::false_type(), std::false_type());
            if (k + slots < pieces) {
                asm volatile("" ::"f"(run.m), "f"(run.sum));  // everything read has been used
                release(now.slot);
            }
        }
    }
    // the listed tokens
    if (kMany && crowded) {
        const float2 met = crowded_tokens<TI>(p, warm ? Crowd::kSum : Crowd::kLargest, scale, 0.f, 0.f);
        if (warm) {
            const float from = run.raise(met.x, scale);
            run.sum += met.y * ex2((met.x - from) * scale);  // (none: 0 times 0)
        } else {
            run.take(met.x, __float_as_int(met.y));
        }
    } else if (listed > 0) {
        const float rep = p.repetition ? p.repetition[b] : 1.f, freq = p.frequency ? p.frequency[b] : 0.f;
        const float pres = p.presence ? p.presence[b] : 0.f;
        const bool summed = kMany && bhi - blo > kFewBiases;  // x stands in the list then, biases and all
        if (summed) {
            settle_list<TI>(p, listed);
            __syncthreads();
        }
        for (int i0 = tid; i0 < listed; i0 += kAbreast * kThreads) {
            int t[kAbreast];
            float v[kAbreast];
#pragma unroll
            for (int k = 0; k < kAbreast; ++k) {
                const int i = i0 + k * kThreads;
                t[k] = i < listed ? token_at(i) : 0;
                v[k] = i >= listed ? -INFINITY : summed ? __uint_as_float(value[i]) : static_cast<float>(in[t[k]]);
            }
            float top = -INFINITY;
#pragma unroll
            for (int k = 0; k < kAbreast; ++k) {
                const int i = i0 + k * kThreads;
                if (i >= listed) continue;
                float y = v[k];
                if (!summed) {
                    y = penalised(y, value[i], rep, freq, pres);
                    if (value[i] & kBias)
                        for (int e = blo; e < bhi; ++e)
                            if (p.bias_tokens[e] == t[k]) y = __fadd_rn(y, p.bias_values[e]);
                }
                v[k] = !bits || (bits[t[k] >> 5] >> (t[k] & 31) & 1) ? y : -INFINITY;
                value[i] = __float_as_uint(v[k]);
                if (!warm) run.take(v[k], t[k]);
                top = fmax_nan(top, v[k]);
            }
            if (warm) {
                const float from = run.raise(top, scale);
#pragma unroll
                for (int k = 0; k < kAbreast; ++k)
                    if (i0 + k * kThreads < listed) run.sum += ex2((v[k] - from) * scale);
            }
        }
    }

    // ------------------------------------------------ of the CTA, then of the row
    // (largest, sum) of two runs as one; a run without a token has sum 0
    const auto merged = [&](float m, float sum) {
        const float M = warp_max_nan(m);
        return make_float2(M, warp_add(m == -INFINITY ? 0.f : sum * ex2((m - M) * scale)));
    };
    const auto largest = [&](float2 a) {
        Run r;
        r.m = a.x, r.at = __float_as_int(a.y);
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const float v = __shfl_xor_sync(0xFFFFFFFFu, r.m, o);
            r.take(v, __shfl_xor_sync(0xFFFFFFFFu, r.at, o));
        }
        return make_float2(r.m, __int_as_float(r.at));
    };
    const float2 none = make_float2(-INFINITY, warm ? 0.f : __int_as_float(INT32_MAX));
    float2 best = warm ? merged(run.m, run.sum) : largest(make_float2(run.m, __int_as_float(run.at)));
    if (lane == 0) warp_pair[warp] = best;
    __syncthreads();
    best = lane < kWarps ? warp_pair[lane] : none;
    best = warm ? merged(best.x, best.y) : largest(best);
    if (p.ctas > 1) {
        if (tid == 0) cta_pair = best;
        cluster_sync_all();
        best = none;
        if (lane < p.ctas) {
            const uint32_t at = mapa_shared(smem_u32(&cta_pair), (uint32_t)lane);
            best = make_float2(ld_cluster_f32(at), ld_cluster_f32(at + 4));
        }
        __syncwarp();
        cluster_arrive_all();
        best = warm ? merged(best.x, best.y) : largest(best);
    }
    if (best.x == -INFINITY && rank == 0 && tid == 0 && p.error) atomicOr(p.error, DA_DEV_BAD_PROBS);

    // ------------------------------------------------ the second walk: 2^((x - largest) s - log2(sum))
    // (without a token: everything 0, by an exponent of -infinity; a NaN or +infinity has left no sum: NaN everywhere)
    const bool nothing = best.x == -INFINITY;
    const float from = nothing ? 0.f : best.x, off = nothing ? -INFINITY : -log2f(best.y);
    const bool bad = warm && !nothing && !(best.y < INFINITY);  // (largest NaN or infinite)
    const Exps exps{from, scale, off};
    const bool ordinary = warm && !bad && !nothing && !crowded && vec;
    const auto second = [&](auto *row) {  // of the probabilities, as what they are
        const auto probabilities = [&](int g, const Raw<TI> &r, float (&v)[8]) {
            if (warm) {
                r.widen(v);
                exps.of(v);
                if (bad || nothing) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = bad ? NAN : 0.f;
                }
            } else {
                const int t = t0 + g * 8, at = __float_as_int(best.y);
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = t + i == at ? 1.f : 0.f;
            }
        };
        // of a group, the tokens that have been written before the walk
        const auto written = [&](int g) -> uint32_t {
            return crowded && warm ? (uint32_t) reinterpret_cast<const uint8_t *>(mark)[g] : 0u;
        };
        const auto write = [&](int g, const Raw<TI> &r) {
            float v[8];
            probabilities(g, r, v);
            store_group(row, t0 + g * 8, V, vec, written(g), v);
        };
        if constexpr (kG > 0) {
#pragma unroll
            for (int k = 0; k < kG; ++k)
                if (k * kThreads + tid < groups) write(k * kThreads + tid, held[k]);
        } else {
            const auto edge = [&](int g) {
                Raw<TI> r;
                load_group(g, r);
                if (bits) r.drop(allowed_of(g));
                write(g, r);
            };
            if (tid == 0 && whole0 > 0 && groups > 0) edge(0);
            if (tid == 32 && whole1 < groups && (whole1 > 0 || whole0 == 0)) edge(groups - 1);
            // first the pieces that the ring still has, the last ones; then the others, loaded again behind them
            const int left = min(pieces, slots);
            Turn now;
            if (pieces > slots) now.slot = pieces % slots, now.round = pieces / slots;
            for (int k = 0; k < pieces; ++k, now.next(slots)) {
                const int g = whole0 + (k < left ? pieces - left + k : k - left) * kPiece;
                auto *at = row + t0 + (int64_t)(g + tid) * 8;
                uint32_t keep[kPer];
                if (bits && warm) keeps(g + tid, false, keep);
                const auto part = [&](auto all, auto plain, auto masked) {  // (all: a whole piece; plain: nothing but the formula)
                    Raw<TI> r[kPer];
                    if (plain || warm) {
                        if (tid == 0 && k > 0 && k - 1 < pieces - left) refill();
                        if (k >= left) wait(&full[now.slot], now.round - 1);
                        read_slot(now.slot, g, r, all);
                    }
#pragma unroll
                    for (int i = 0; i < kPer; ++i) {
                        const int gi = g + i * kThreads + tid;
                        if (!all && gi >= whole1) continue;
                        float v[8];
                        if (masked && warm && keep[i] != 0xFFu) r[i].drop(keep[i]);
                        if (plain) {
                            r[i].widen(v);
                            exps.of(v);
                            store8(at + i * kThreads * 8, v);
                            continue;
                        }
                        probabilities(gi, r[i], v);
                        store_group(row, t0 + gi * 8, V, vec, written(gi), v);
                    }
                };
                const bool whole = g + kPiece <= whole1 && ordinary;
                if (whole && !bits)
                    part(std::true_type(), std::true_type(), std::false_type());
                else if (whole)
                    part(std::true_type(), std::true_type(), std::true_type());
                else
                    part(std::false_type(), std::false_type(), bits != nullptr);
                if (warm && k < pieces - left) release(now.slot);
            }
        }
        if (listed > 0 && !crowded && warm) {
            __syncthreads();  // over what the walk has left at the listed tokens
            for (int i0 = tid; i0 < listed; i0 += kAbreast * kThreads) {
#pragma unroll
                for (int k = 0; k < kAbreast; ++k) {
                    const int i = i0 + k * kThreads;
                    if (i >= listed) continue;
                    const float v = exps(__uint_as_float(value[i]));
                    store1(row + token_at(i), bad ? NAN : nothing ? 0.f : v);
                }
            }
        }
    };
    if (kMany && crowded && warm)  // ahead of the walk: it may write over the logits
        crowded_tokens<TI>(p, bad ? Crowd::kWriteNan : nothing ? Crowd::kWriteZero : Crowd::kWrite, scale, from, off);
    if (p.prob_dtype == DA_PROB_F32)
        second(reinterpret_cast<float *>(out_at));
    else if (p.prob_dtype == DA_PROB_BF16)
        second(reinterpret_cast<__nv_bfloat16 *>(out_at));
    else
        second(reinterpret_cast<__half *>(out_at));
    if constexpr (kG == 0) {
        // where a wait has run out, the copies in flight land before the CTA exits (else all have been waited for)
        if (__syncthreads_or(*(volatile int *)&given_up) && tid == 0)
            for (int l = max(loads - slots, 0); l < loads; ++l) mbar_wait_timed(&full[l % slots], (l / slots) & 1, 100000000ull);
    }
    if (p.ctas > 1) cluster_wait_all();  // this CTA's pair stays until all have read it
}

// Whether the current device can hold a cluster of 16 CTAs of this kernel, asked once per device for CTAs of which two fit an SM and
// for larger ones (by the most shared memory that such a one takes). cfg: of the launch, attr[0] its cluster.
template <typename TI, int kG, bool kMany>
bool wide_clusters(cudaLaunchConfig_t cfg, cudaLaunchAttribute *attr) {
    static std::atomic<int> known[64][2];  // 1: no, 2: yes
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    const bool large = cfg.dynamicSmemBytes > (size_t)kSmemTwo;
    int k = known[dev][large].load(std::memory_order_relaxed);
    if (k == 0) {
        cfg.gridDim = dim3(attr[0].val.clusterDim.x);
        cfg.dynamicSmemBytes = large ? kSmemMax : kSmemTwo;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        const bool ok = cudaOccupancyMaxActiveClusters(&n, probs_kernel<TI, kG, kMany>, &cfg) == cudaSuccess && n >= 1;
        if (!ok) cudaGetLastError();
        k = ok ? 2 : 1;
        known[dev][large].store(k, std::memory_order_relaxed);
    }
    return k == 2;
}

// How a row is divided: its CTAs, groups to each, the list's room, slots of the ring, shared memory of a CTA.
struct Split {
    int ctas, share, cap, slots;
    bool many;
    size_t smem;
};

template <typename TI, int kG, bool kMany>
cudaError_t launch_one(ProbsParams p, const Split &how, cudaStream_t stream, bool pdl, bool *no_room) {
    p.ctas = how.ctas;
    p.share = how.share;
    p.cap = how.cap;
    p.slots = how.slots;
    const auto kern = probs_kernel<TI, kG, kMany>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (e == cudaSuccess && p.ctas > 8) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    const int64_t grid = (int64_t)p.B * (p.K + 1) * p.ctas;
    if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = how.smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (p.ctas > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim = {(unsigned)p.ctas, 1, 1};
        ++n;
    }
    if (p.ctas > 8 && !wide_clusters<TI, kG, kMany>(cfg, attr)) {
        *no_room = true;
        return cudaSuccess;
    }
    if (pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

template <typename TI, bool kMany>
cudaError_t launch_held(const ProbsParams &p, const Split &how, cudaStream_t stream, bool pdl, bool *no_room) {
    return how.share <= kThreads       ? launch_one<TI, 1, kMany>(p, how, stream, pdl, no_room)
           : how.share <= 2 * kThreads ? launch_one<TI, 2, kMany>(p, how, stream, pdl, no_room)
                                       : launch_one<TI, 0, kMany>(p, how, stream, pdl, no_room);
}

// rows of [0, V) over clusters of at most `most` CTAs
template <typename TI>
Split split_rows(const ProbsParams &p, int num_sms, int most) {
    // groups of the longest row: the first of them may start before it
    const int head = p.logits_stride % 8 == 0 ? (int)(reinterpret_cast<uintptr_t>(p.logits) / sizeof(TI) & 7) : 7;
    const int groups = (p.V + head + 7) / 8;
    const int64_t rows = (int64_t)p.B * (p.K + 1);
    // tokens that a list may need room for: those of the history and drafts, and of the biases as many as a request has in
    // earnest (n_bias is all requests'). How much of the history's columns is used is known on the device alone: a buffer as wide as
    // the longest text does not decide how rows are divided, the list stays as short as two CTAs an SM allow it where CTAs wait
    // for SMs, and a share with more takes them window by window. (With room for all columns, by clusters of up to 16: 1024 rows of
    // 131072 with up to 64 tokens in 131072 columns 775 us instead of 154, with 8192 to 16384 tokens 1250 instead of 430, with 65536
    // to 131072 4360 instead of 3190.)
    const int64_t touches = (int64_t)p.history_cols + (p.drafts ? p.K : 0) + (p.bias_starts ? min(p.n_bias, kBiasRoom) : 0);
    const int64_t piece = kPieceBytes;
    // As few CTAs as hold a row; where that leaves SMs idle, more, down to eight values a thread: two or four as long as all
    // have a place at once (64 rows of 128259: 18.0 us with four, 28.0 with one), eight or sixteen for half the SMs at most (32
    // rows: 12.9 us with four, 15.2 with eight, as clusters of eight do not fill the chip; one row: 9.1 with sixteen, 12.0
    // with four).
    int c = 1;
    while (c < most && (int64_t)((groups + c - 1) / c) * 8 * (int)sizeof(TI) > kShareBytes) c *= 2;
    while (c < most && rows * c * 2 <= (c < 4 ? 2 * num_sms : num_sms / 2) && groups > c * kThreads) c *= 2;
    Split how = {};
    how.ctas = c;
    how.share = (groups + c - 1) / c;
    const int64_t need = touches < (int64_t)how.share * 8 ? touches : (int64_t)how.share * 8;
    const int64_t most_listed = rows * c <= num_sms ? kListRoom : kListRoomTwo;
    how.cap = (int)(need < most_listed ? need + 3 : most_listed) / 4 * 4;
    how.many = (p.bias_starts && p.n_bias > kFewBiases) || need > most_listed;
    how.smem = touches == 0 ? 0 : ((size_t)words_of(how.share) * 6 + (size_t)how.cap * 6 + (size_t)many_words(how.cap) * 4 + 15) / 16 * 16;
    if (how.share > 2 * kThreads) {
        const int64_t all = ((int64_t)how.share * 8 * sizeof(TI) + piece - 1) / piece;
        const int64_t room = ((how.cap > kListRoomTwo ? kSmemMax : kSmemTwo) - (int64_t)how.smem) / piece;
        how.slots = (int)(room < all ? room : all);
        if (how.slots > kMaxSlots) how.slots = kMaxSlots;
        how.smem += (size_t)how.slots * piece;
    }
    return how;
}
// the longest row over the fewest CTAs that a device may be limited to
static_assert((int64_t)(kMaxProbsVocab + 7) / 8 / 8 * 8 * 4 <= kShareBytes, "eight CTAs hold the longest row");

template <typename TI>
cudaError_t launch_types(const ProbsParams &p, int num_sms, cudaStream_t stream, bool pdl) {
    bool no_room = false;
    for (int most = p.max_cluster;; most = 8) {
        const Split how = split_rows<TI>(p, num_sms, most);
        if ((how.share > 2 * kThreads && how.slots < 2) || how.smem > (size_t)kSmemMax) return cudaErrorInvalidConfiguration;
        no_room = false;
        const cudaError_t e = how.many ? launch_held<TI, true>(p, how, stream, pdl, &no_room) : launch_held<TI, false>(p, how, stream, pdl, &no_room);
        if (!no_room) return e;
    }
}

}  // namespace

cudaError_t launch_probs(const ProbsParams &p, int num_sms, cudaStream_t stream, bool pdl) {
    return p.logits_dtype == DA_PROB_F32    ? launch_types<float>(p, num_sms, stream, pdl)
           : p.logits_dtype == DA_PROB_BF16 ? launch_types<__nv_bfloat16>(p, num_sms, stream, pdl)
                                            : launch_types<__half>(p, num_sms, stream, pdl);
}

}  // namespace da
