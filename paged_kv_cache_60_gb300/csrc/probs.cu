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
// at most two groups of eight values a thread stay in registers in between; longer ones are read
// again, out of L2: a share is at most 256 KB, so that what two CTAs on each SM have
// begun stays within it. (Rows held in registers throughout, by clusters of eight, took
// 308 us for 1024 rows of 131072 bf16 logits without a history: 128 warps with 32 values
// a lane each, whose fixed work was more than the values'.)
//
// The tokens that the history, the drafts and the biases touch are few, and go their own
// way: a bit per token of the share, a prefix sum over its words, and so a place for each
// in a list, with its count (and marks: in the prompt, has a bias). They are left out
// of the first walk; a thread per listed token then computes its x, which takes its
// part in maximum and sum, and is written over what the second walk left there. Biases
// are added in the list's order, so that a token that stands twice has one result.
//
// Sums: a thread's own in fp32, then warps, then the (largest, sum) pairs of the CTAs, in a
// fixed order.
//
// Rows start anywhere: groups of eight values start where the logits are aligned to
// eight of them, the first and last of a row are taken value by value. Where the
// probabilities' row is aligned like the logits' they are written in vectors, else value
// by value.
#include <cuda_runtime.h>

#include <cfloat>
#include <cstdint>

#include "common.cuh"
#include "decode_attn.h"
#include "layout.h"
#include "quant.cuh"

namespace da {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kUnroll = 4;                      // groups of a thread in flight while a share is read
constexpr int kShareBytes = 256 << 10;
constexpr int kSmemMax = 224 << 10, kSmemTwo = 110 << 10;  // of a CTA; where two fit an SM
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
// eight values: 16 bytes of a two-byte type, 32 of fp32
template <typename T>
struct Raw {
    uint4 v[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T *at) {
    Raw<T> r;
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.v[i] = *reinterpret_cast<const uint4 *>(at + 4 * i);
    return r;
}
template <typename T>
__device__ __forceinline__ void widen(const Raw<T> &r, float (&x)[8]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            x[4 * i] = __uint_as_float(r.v[i].x), x[4 * i + 1] = __uint_as_float(r.v[i].y);
            x[4 * i + 2] = __uint_as_float(r.v[i].z), x[4 * i + 3] = __uint_as_float(r.v[i].w);
        }
    } else {
        const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = pair_to_f32<T>(w[i]);
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
    }
}
__device__ __forceinline__ void store8(float *at, const float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
        st_v4(at + 4 * i, make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]),
                                     __float_as_uint(x[4 * i + 2]), __float_as_uint(x[4 * i + 3])));
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

// The row of probabilities; its type is told apart per store.
struct OutRow {
    void *at;
    int dtype;
    bool vec;  // aligned to eight values where the logits are
    template <typename T>
    __device__ __forceinline__ void group_as(int t, int V, const float (&x)[8]) const {
        T *o = static_cast<T *>(at) + t;
        if (vec && t >= 0 && t + 8 <= V) {
            store8(o, x);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (t + i >= 0 && t + i < V) store1(o + i, x[i]);
        }
    }
    __device__ __forceinline__ void group(int t, int V, const float (&x)[8]) const {
        if (dtype == DA_PROB_F32)
            group_as<float>(t, V, x);
        else if (dtype == DA_PROB_BF16)
            group_as<__nv_bfloat16>(t, V, x);
        else
            group_as<__half>(t, V, x);
    }
    __device__ __forceinline__ void one(int t, float x) const {
        if (dtype == DA_PROB_F32)
            store1(static_cast<float *>(at) + t, x);
        else if (dtype == DA_PROB_BF16)
            store1(static_cast<__nv_bfloat16 *>(at) + t, x);
        else
            store1(static_cast<__half *>(at) + t, x);
    }
};

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
// (a, b) <- 2^((a - m) s + c): the differences and products in one packed instruction each
__device__ __forceinline__ void exp_pair(float &a, float &b, float m, float s, float c) {
    asm("{\n.reg .b64 x, y;\nmov.b64 x, {%0, %1};\nmov.b64 y, {%2, %2};\nadd.rn.f32x2 x, x, y;\n"
        "mov.b64 y, {%4, %4};\n.reg .b64 z;\nmov.b64 z, {%3, %3};\nfma.rn.f32x2 x, x, z, y;\nmov.b64 {%0, %1}, x;\n}"
        : "+f"(a), "+f"(b)
        : "f"(-m), "f"(s), "f"(c));
    a = ex2(a);
    b = ex2(b);
}

// A running maximum with the sum of 2^((x - m) s), or the largest x with its token.
struct Run {
    float m = -INFINITY, sum = 0.f;
    int at = INT32_MAX;
    // what differences are taken from: finite where nothing has been seen
    __device__ __forceinline__ float base() const { return m == -INFINITY ? 0.f : m; }
    __device__ __forceinline__ void raise(float to, float s) {
        const float n = fmax_nan(m, to);
        if (n != m) {  // (and where it is NaN)
            sum = m == -INFINITY ? 0.f : sum * ex2((m - n) * s);
            m = n;
        }
    }
    __device__ __forceinline__ void take(float x, int token) {
        if (x > m || (x == m && token < at && x > -INFINITY)) m = x, at = token;
    }
};

// kG: groups of eight values that a thread holds between the walks; 0: the share is read again
template <typename TI, int kG>
__global__ void __launch_bounds__(kThreads, kG == 0 ? 2 : 1) probs_kernel(const __grid_constant__ ProbsParams p) {
    extern __shared__ uint4 smem_v[];
    __shared__ float2 warp_pair[kWarps];
    __shared__ float2 cta_pair;          // largest, and sum (or the token, as bits)
    __shared__ int warp_sum[kWarps];
    __shared__ int s_listed;
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = blockIdx.x / p.ctas, rank = blockIdx.x - row * p.ctas;
    const int b = row / (p.K + 1), j = row - b * (p.K + 1);
    const int V = p.V;
    const TI *in = static_cast<const TI *>(p.logits) + row * p.logits_stride;
    const int out_size = p.prob_dtype == DA_PROB_F32 ? 4 : 2;
    uint8_t *out_at = static_cast<uint8_t *>(p.probs) + row * p.probs_stride * out_size;
    const int head = (int)(reinterpret_cast<uintptr_t>(in) / sizeof(TI) & 7);
    const OutRow out{out_at, p.prob_dtype, (int)(reinterpret_cast<uintptr_t>(out_at) / out_size & 7) == head};
    const int t0 = rank * p.share * 8 - head;  // token of the share's first value; group g holds t0 + 8 g ..
    const int groups = max(min(p.share, (V - t0 + 7) / 8), 0);
    const uint32_t *bits = p.allowed ? p.allowed + row * p.allowed_stride : nullptr;
    const int words = (V + 31) / 32;

    // the logits of a group, -infinity where there is none
    const auto load_group = [&](int g, float (&x)[8]) {
        const int t = t0 + g * 8;
        if (t >= 0 && t + 8 <= V) {
            widen(load_raw(in + t), x);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = t + i >= 0 && t + i < V ? static_cast<float>(in[t + i]) : -INFINITY;
        }
    };
    // bit i: token i of the group is allowed
    const auto allowed_of = [&](int g) -> uint32_t {
        const int t = t0 + g * 8, w = t >> 5;  // w is -1 in front of the row
        const uint32_t lo = w >= 0 ? bits[w] : 0u, hi = w + 1 < words ? bits[w + 1] : 0u;
        return __funnelshift_r(lo, hi, t & 31) & 0xFFu;
    };
    const auto drop = [&](uint32_t keep, float (&x)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!(keep >> i & 1)) x[i] = -INFINITY;
    };

    float x[kG > 0 ? kG : 1][8];
    if constexpr (kG > 0) {
#pragma unroll
        for (int k = 0; k < kG; ++k) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[k][i] = -INFINITY;
            if (k * kThreads + tid < groups) load_group(k * kThreads + tid, x[k]);
        }
    }
    const float T = p.temperature ? p.temperature[b] : 1.f;
    const bool warm = T > 0.f;
    // (a temperature next to 0: 0 times its reciprocal stays 0; an infinite one: -infinity stays that)
    const float scale = warm ? fmaxf(fminf(__fdiv_rn(kLog2e, T), FLT_MAX), FLT_MIN) : 1.f;

    // ------------------------------------------------ the tokens that history, drafts and biases touch
    const int n_hist = p.history ? min(max(p.history_lens[b], 0), p.history_cols) : 0;
    const int blo = p.bias_starts ? min(max(p.bias_starts[b], 0), p.n_bias) : 0;
    const int bhi = p.bias_starts ? min(max(p.bias_starts[b + 1], 0), p.n_bias) : 0;
    const bool touched = n_hist > 0 || (p.drafts != nullptr && j > 0) || bhi > blo;  // the same for the whole CTA
    const int share_words = (p.share * 8 + 31) / 32;
    uint32_t *mark = reinterpret_cast<uint32_t *>(smem_v);   // a bit per token of the share
    int *place = reinterpret_cast<int *>(mark + share_words);  // marks in the words before
    uint32_t *value = reinterpret_cast<uint32_t *>(place + share_words);  // of each listed token: count and marks, then x
    uint32_t *list = value + p.cap;                          // their tokens, from t0 on (16 bits each where that will do)
    const auto token_at = [&](int i) -> int {
        return t0 + (int)(p.short_list ? reinterpret_cast<const uint16_t *>(list)[i] : list[i]);
    };
    int listed = 0;
    if (touched) {
        for (int i = tid; i < share_words; i += kThreads) mark[i] = 0u;
        __syncthreads();
        const int prompt = p.prompt_lens ? p.prompt_lens[b] : 0;
        const int32_t *hist = p.history + (int64_t)b * p.history_cols;
        // f(place in the share, what it adds) for every touch
        const auto each = [&](auto f) {
            const auto touch = [&](int token, uint32_t what, bool atomic_add) {
                const unsigned i = (unsigned)(token - t0);
                if (token >= 0 && token < V && i < (unsigned)groups * 8u) f((int)i, what, atomic_add);
            };
            for (int i0 = tid; i0 < n_hist; i0 += 4 * kThreads) {
                int tok[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) tok[k] = i0 + k * kThreads < n_hist ? hist[i0 + k * kThreads] : -1;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const bool asked = i0 + k * kThreads < prompt;
                    touch(tok[k], asked ? kPrompt : 1u, !asked);
                }
            }
            if (p.drafts != nullptr && tid < j) {  // draft tid, unless the chain has ended before it
                const int32_t *d = p.drafts + (int64_t)b * p.K;
                bool there = true;
                for (int i = 0; i <= tid; ++i) there = there && d[i] >= 0;
                if (there) touch(d[tid], 1u, true);
            }
            for (int i = blo + tid; i < bhi; i += kThreads) touch(p.bias_tokens[i], kBias, false);
        };
        each([&](int i, uint32_t, bool) {
            const uint32_t bit = 1u << (i & 31);
            if (!(*(volatile uint32_t *)(mark + i / 32) & bit)) atomicOr(mark + i / 32, bit);
        });
        __syncthreads();
        // prefix sum over the words: a run of them per thread
        const int per = (share_words + kThreads - 1) / kThreads;
        int mine = 0;
        for (int k = 0; k < per; ++k)
            if (tid * per + k < share_words) mine += __popc(mark[tid * per + k]);
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o) incl += u;
        }
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
        int at = incl - mine;
        for (int w = 0; w < warp; ++w) at += warp_sum[w];
        if (tid == kThreads - 1) s_listed = at + mine;
        for (int k = 0; k < per; ++k)
            if (tid * per + k < share_words) {
                place[tid * per + k] = at;
                at += __popc(mark[tid * per + k]);
            }
        __syncthreads();
        listed = s_listed;
        for (int i = tid; i < listed; i += kThreads) value[i] = 0u;
        __syncthreads();
        each([&](int i, uint32_t what, bool atomic_add) {
            const int at = place[i / 32] + __popc(mark[i / 32] & ((1u << (i & 31)) - 1));
            if (atomic_add)
                atomicAdd(value + at, what);
            else
                atomicOr(value + at, what);
            if (p.short_list)
                reinterpret_cast<uint16_t *>(list)[at] = (uint16_t)i;
            else
                list[at] = (uint32_t)i;
        });
        __syncthreads();
    }

    // ------------------------------------------------ the first walk: all tokens but those
    Run run;
    const auto keep_of = [&](int g) -> uint32_t {
        uint32_t keep = bits ? allowed_of(g) : 0xFFu;
        if (listed > 0) keep &= ~(uint32_t) reinterpret_cast<const uint8_t *>(mark)[g];
        return keep;
    };
    const auto walk = [&](int g, const float (&v)[8]) {
        if (warm) {
            float m = v[0];
#pragma unroll
            for (int i = 1; i < 8; ++i) m = fmax_nan(m, v[i]);
            run.raise(m, scale);
            const float from = run.base();
            float e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = v[i];
#pragma unroll
            for (int i = 0; i < 8; i += 2) exp_pair(e[i], e[i + 1], from, scale, 0.f);
            run.sum += ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) run.take(v[i], t0 + g * 8 + i);
        }
    };
    if constexpr (kG > 0) {
#pragma unroll
        for (int k = 0; k < kG; ++k) {
            const int g = k * kThreads + tid;
            if (g >= groups) continue;
            const uint32_t keep = keep_of(g);
            if (keep != 0xFFu) drop(keep, x[k]);
            walk(g, x[k]);
        }
    } else {
        for (int g0 = tid; g0 < groups; g0 += kUnroll * kThreads) {
            Raw<TI> r[kUnroll];
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) {
                const int g = g0 + k * kThreads, t = t0 + g * 8;
                if (g < groups && t >= 0 && t + 8 <= V) r[k] = load_raw(in + t);
            }
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) {
                const int g = g0 + k * kThreads, t = t0 + g * 8;
                if (g >= groups) continue;
                float v[8];
                if (t >= 0 && t + 8 <= V)
                    widen(r[k], v);
                else
                    load_group(g, v);
                const uint32_t keep = keep_of(g);
                if (keep != 0xFFu) drop(keep, v);
                walk(g, v);
            }
        }
    }
    // the listed tokens
    if (listed > 0) {
        const float rep = p.repetition ? p.repetition[b] : 1.f, freq = p.frequency ? p.frequency[b] : 0.f;
        const float pres = p.presence ? p.presence[b] : 0.f;
        for (int i = tid; i < listed; i += kThreads) {
            const int t = token_at(i);
            const uint32_t c = value[i], n = c & kCount;
            float v = static_cast<float>(in[t]);
            if (n > 0 || (c & kPrompt)) v = v > 0.f ? __fdiv_rn(v, rep) : __fmul_rn(v, rep);
            v = __fsub_rn(v, __fmul_rn(freq, (float)n));
            if (n > 0) v = __fsub_rn(v, pres);
            if (c & kBias)
                for (int e = blo; e < bhi; ++e)
                    if (p.bias_tokens[e] == t) v = __fadd_rn(v, p.bias_values[e]);
            if (bits && !(bits[t >> 5] >> (t & 31) & 1)) v = -INFINITY;
            value[i] = __float_as_uint(v);
            if (warm) {
                run.raise(v, scale);
                run.sum += ex2((v - run.base()) * scale);
            } else {
                run.take(v, t);
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
    const bool empty = best.x == -INFINITY;
    const float from = empty ? 0.f : best.x, off = empty ? -INFINITY : -log2f(best.y);
    const bool bad = warm && !empty && !(best.y < INFINITY);  // (largest NaN or infinite)
    const auto probability = [&](int g, float (&v)[8]) {
        if (warm) {
#pragma unroll
            for (int i = 0; i < 8; i += 2) exp_pair(v[i], v[i + 1], from, scale, off);
            if (bad || empty) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = bad ? NAN : 0.f;
            }
        } else {
            const int t = t0 + g * 8, at = __float_as_int(best.y);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = t + i == at ? 1.f : 0.f;
        }
        out.group(t0 + g * 8, V, v);
    };
    if constexpr (kG > 0) {
#pragma unroll
        for (int k = 0; k < kG; ++k)
            if (k * kThreads + tid < groups) probability(k * kThreads + tid, x[k]);
    } else {
        for (int g0 = tid; g0 < groups; g0 += kUnroll * kThreads) {
            Raw<TI> r[kUnroll];
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) {
                const int g = g0 + k * kThreads, t = t0 + g * 8;
                if (warm && g < groups && t >= 0 && t + 8 <= V) r[k] = load_raw(in + t);
            }
#pragma unroll
            for (int k = 0; k < kUnroll; ++k) {
                const int g = g0 + k * kThreads, t = t0 + g * 8;
                if (g >= groups) continue;
                float v[8];
                if (!warm) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = 0.f;
                } else {
                    if (t >= 0 && t + 8 <= V)
                        widen(r[k], v);
                    else
                        load_group(g, v);
                    if (bits) {
                        const uint32_t keep = allowed_of(g);
                        if (keep != 0xFFu) drop(keep, v);
                    }
                }
                probability(g, v);
            }
        }
    }
    if (listed > 0 && warm) {
        __syncthreads();  // over what the walk has left at the listed tokens
        for (int i = tid; i < listed; i += kThreads) {
            float v = __uint_as_float(value[i]), w = 0.f;
            exp_pair(v, w, from, scale, off);
            out.one(token_at(i), bad ? NAN : empty ? 0.f : v);
        }
    }
    if (p.ctas > 1) cluster_wait_all();  // this CTA's pair stays until all have read it
}

template <typename TI, int kG>
cudaError_t launch_one(const ProbsParams &p, size_t smem, cudaStream_t stream, bool pdl) {
    const auto kern = probs_kernel<TI, kG>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
    if (e == cudaSuccess && p.ctas > 8) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    const int64_t grid = (int64_t)p.B * (p.K + 1) * p.ctas;
    if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (p.ctas > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim = {(unsigned)p.ctas, 1, 1};
        ++n;
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

template <typename TI>
cudaError_t launch_types(ProbsParams p, int num_sms, cudaStream_t stream, bool pdl) {
    // groups of the longest row: the first of them may start before it
    const int head = p.logits_stride % 8 == 0 ? (int)(reinterpret_cast<uintptr_t>(p.logits) / sizeof(TI) & 7) : 7;
    const int groups = (p.V + head + 7) / 8;
    const int64_t rows = (int64_t)p.B * (p.K + 1);
    const int64_t touches = (int64_t)p.history_cols + (p.drafts ? p.K : 0) + (p.bias_starts ? p.n_bias : 0);
    const auto split = [&](int c) -> size_t {  // a row over c CTAs: the shared memory of one
        p.ctas = c;
        p.share = (groups + c - 1) / c;
        const int64_t tokens = (int64_t)p.share * 8;
        p.short_list = tokens <= 65536;
        p.cap = (int)((touches < tokens ? touches : tokens) + 3) / 4 * 4;
        if (touches == 0) return 0;
        return 8 * ((size_t)p.share * 8 / 32 + 1) + (size_t)p.cap * (p.short_list ? 6 : 8);
    };
    // as few CTAs as hold a row; where that leaves SMs idle, more, down to eight values a thread
    int c = 1;
    while (c < kMaxCluster && ((int64_t)((groups + c - 1) / c) * 8 * (int)sizeof(TI) > kShareBytes || split(c) > kSmemTwo)) c *= 2;
    while (c < kMaxCluster && rows * c * 2 <= num_sms && groups > c * kThreads) c *= 2;
    const size_t smem = split(c);
    if (smem > (size_t)kSmemMax) return cudaErrorInvalidConfiguration;
    const int need = (p.share + kThreads - 1) / kThreads;
    return need <= 1   ? launch_one<TI, 1>(p, smem, stream, pdl)
           : need <= 2 ? launch_one<TI, 2>(p, smem, stream, pdl)
                       : launch_one<TI, 0>(p, smem, stream, pdl);
}

}  // namespace

cudaError_t launch_probs(const ProbsParams &p, int num_sms, cudaStream_t stream, bool pdl) {
    return p.logits_dtype == DA_PROB_F32    ? launch_types<float>(p, num_sms, stream, pdl)
           : p.logits_dtype == DA_PROB_BF16 ? launch_types<__nv_bfloat16>(p, num_sms, stream, pdl)
                                            : launch_types<__half>(p, num_sms, stream, pdl);
}

}  // namespace da
