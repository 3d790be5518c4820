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
// One cluster of CTAs per row, a contiguous share of the vocabulary each: a thread
// loads its logits once, 16 bytes at a time, and keeps them in registers until the
// probabilities are written, so a row is read once and written once. Which tokens the
// history, the drafts and the biases touch is a count per token of the share in
// shared memory: 14 bits of count and two marks (seen in the prompt, has a bias), or 30
// bits where the history is longer than 14 bits count. Only tokens with a count that is
// not 0 do any of the arithmetic; their biases are added in the list's order, so that
// a token that stands twice has one result.
//
// Every warp takes the largest of its own values and the sum of 2^(x - largest);
// one exchange through distributed shared memory brings the (largest, sum) pairs of all
// warps of the row together, and each lane scales what it has: one barrier a row.
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
constexpr float kLog2e = 1.4426950408889634f;

// The types are told apart at run time, once per thread and direction: a build for each
// pair of them, size and width of the counts took four minutes to compile.
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
// eight values from 16 bytes (two-byte types) or 32
template <typename T>
__device__ __forceinline__ void load8(const T *at, float (&x)[8]) {
    if constexpr (sizeof(T) == 4) {
        const uint4 a = ld_stream_v4(at), b = ld_stream_v4(at + 4);
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
    } else {
        const uint4 a = ld_stream_v4(at);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
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

// A thread's groups of a row: group k * kThreads + tid of the share holds the tokens t0 + 8 group ..
template <typename T, int kG>
__device__ __forceinline__ void load_row(const ProbsParams &p, const T *in, int t0, float (&x)[kG][8]) {
#pragma unroll
    for (int k = 0; k < kG; ++k) {
        const int g = k * kThreads + threadIdx.x, t = t0 + g * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[k][i] = -INFINITY;
        if (g >= p.share || t >= p.V) continue;
        if (t >= 0 && t + 8 <= p.V) {
            load8(in + t, x[k]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (t + i >= 0 && t + i < p.V) x[k][i] = static_cast<float>(in[t + i]);
        }
    }
}
template <typename T, int kG>
__device__ __forceinline__ void store_row(const ProbsParams &p, T *out, int t0, int head, const float (&x)[kG][8]) {
    const bool vec = (int)(reinterpret_cast<uintptr_t>(out) / sizeof(T) & 7) == head;
#pragma unroll
    for (int k = 0; k < kG; ++k) {
        const int g = k * kThreads + threadIdx.x, t = t0 + g * 8;
        if (g >= p.share || t >= p.V) continue;
        if (vec && t >= 0 && t + 8 <= p.V) {
            store8(out + t, x[k]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (t + i >= 0 && t + i < p.V) store1(out + t + i, x[k][i]);
        }
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

// Counts of a share's tokens, 16 bits each or (wide) 32: two marks above the count.
struct Counts {
    uint32_t *words;
    bool wide;
    static constexpr uint32_t kPrompt = 0x80000000u, kBias = 0x40000000u, kCount = kBias - 1;  // as group() gives them
    __device__ __forceinline__ void add(int i) {
        if (wide)
            atomicAdd(words + i, 1u);
        else
            atomicAdd(words + i / 2, i & 1 ? 0x10000u : 1u);
    }
    __device__ __forceinline__ void mark(int i, uint32_t m) {
        if (wide)
            atomicOr(words + i, m);
        else
            atomicOr(words + i / 2, i & 1 ? m : m >> 16);
    }
    // whether any of group g's eight tokens has one
    __device__ __forceinline__ bool any(int g) const {
        const uint4 *v = reinterpret_cast<const uint4 *>(words);
        const uint4 a = v[wide ? 2 * g : g];
        uint32_t w = a.x | a.y | a.z | a.w;
        if (wide) {
            const uint4 b = v[2 * g + 1];
            w |= b.x | b.y | b.z | b.w;
        }
        return w != 0;
    }
    __device__ __forceinline__ uint32_t of(int i) const {
        if (wide) return words[i];
        const uint32_t c = words[i / 2] >> (i & 1) * 16;
        return (c & 0xC000u) << 16 | (c & 0x3FFFu);
    }
};

// kG: groups of eight values that a thread holds
template <int kG>
__global__ void __launch_bounds__(kThreads) probs_kernel(const __grid_constant__ ProbsParams p) {
    extern __shared__ uint4 smem_v[];
    __shared__ float2 pairs[kWarps];   // of each warp: largest, and sum (or the index, as bits)
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = blockIdx.x / p.ctas, rank = blockIdx.x - row * p.ctas;
    const int b = row / (p.K + 1), j = row - b * (p.K + 1);
    const int V = p.V;
    const int in_size = p.logits_dtype == DA_PROB_F32 ? 4 : 2, out_size = p.prob_dtype == DA_PROB_F32 ? 4 : 2;
    const uint8_t *in = static_cast<const uint8_t *>(p.logits) + row * p.logits_stride * in_size;
    uint8_t *out = static_cast<uint8_t *>(p.probs) + row * p.probs_stride * out_size;
    const int head = (int)(reinterpret_cast<uintptr_t>(in) / in_size & 7);
    const int g0 = rank * p.share;        // first group of this CTA; group g holds tokens 8 g - head ..
    const int t0 = g0 * 8 - head;         // token of the share's first value

    float x[kG][8];
    if (p.logits_dtype == DA_PROB_F32)
        load_row(p, reinterpret_cast<const float *>(in), t0, x);
    else if (p.logits_dtype == DA_PROB_BF16)
        load_row(p, reinterpret_cast<const __nv_bfloat16 *>(in), t0, x);
    else
        load_row(p, reinterpret_cast<const __half *>(in), t0, x);
    const float T = p.temperature ? p.temperature[b] : 1.f;

    // ------------------------------------------------ what the history, drafts and biases touch
    const int n_hist = p.history ? min(max(p.history_lens[b], 0), p.history_cols) : 0;
    const int blo = p.bias_starts ? min(max(p.bias_starts[b], 0), p.n_bias) : 0;
    const int bhi = p.bias_starts ? min(max(p.bias_starts[b + 1], 0), p.n_bias) : 0;
    const bool counted = n_hist > 0 || (p.drafts != nullptr && j > 0) || bhi > blo;  // the same for the whole CTA
    Counts counts{reinterpret_cast<uint32_t *>(smem_v), p.wide != 0};
    if (counted) {
        const int vecs = p.share * (p.wide ? 2 : 1);
        for (int i = tid; i < vecs; i += kThreads) smem_v[i] = make_uint4(0u, 0u, 0u, 0u);
        __syncthreads();
        const auto local = [&](int token) {  // its place in the share, or -1
            const unsigned i = (unsigned)(token - t0);
            return token >= 0 && token < V && i < (unsigned)p.share * 8u ? (int)i : -1;
        };
        const int prompt = p.prompt_lens ? p.prompt_lens[b] : 0;
        const int32_t *hist = p.history + (int64_t)b * p.history_cols;
        for (int i0 = tid; i0 < n_hist; i0 += 4 * kThreads) {
            int tok[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) tok[k] = i0 + k * kThreads < n_hist ? hist[i0 + k * kThreads] : -1;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int at = local(tok[k]);
                if (at < 0) continue;
                if (i0 + k * kThreads < prompt)
                    counts.mark(at, Counts::kPrompt);
                else
                    counts.add(at);
            }
        }
        if (p.drafts != nullptr && tid < j) {  // draft tid, unless the chain has ended before it
            const int32_t *d = p.drafts + (int64_t)b * p.K;
            bool there = true;
            for (int i = 0; i <= tid; ++i) there = there && d[i] >= 0;
            const int at = there ? local(d[tid]) : -1;
            if (at >= 0) counts.add(at);
        }
        for (int i = blo + tid; i < bhi; i += kThreads) {
            const int at = local(p.bias_tokens[i]);
            if (at >= 0) counts.mark(at, Counts::kBias);
        }
        __syncthreads();
        const float rep = p.repetition ? p.repetition[b] : 1.f, freq = p.frequency ? p.frequency[b] : 0.f;
        const float pres = p.presence ? p.presence[b] : 0.f;
#pragma unroll
        for (int k = 0; k < kG; ++k) {
            const int g = k * kThreads + tid;
            if (g >= p.share || !counts.any(g)) continue;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t c = counts.of(8 * g + i), n = c & Counts::kCount;
                if (c == 0) continue;
                float v = x[k][i];
                if (n > 0 || (c & Counts::kPrompt)) v = v > 0.f ? __fdiv_rn(v, rep) : __fmul_rn(v, rep);
                v = __fsub_rn(v, __fmul_rn(freq, (float)n));
                if (n > 0) v = __fsub_rn(v, pres);
                if (c & Counts::kBias)
                    for (int e = blo; e < bhi; ++e)
                        if (p.bias_tokens[e] == t0 + g * 8 + i) v = __fadd_rn(v, p.bias_values[e]);
                x[k][i] = v;
            }
        }
    }
    if (p.allowed != nullptr) {
        const uint32_t *bits = p.allowed + row * p.allowed_stride;
        const int words = (V + 31) / 32;
#pragma unroll
        for (int k = 0; k < kG; ++k) {
            const int g = k * kThreads + tid, t = t0 + g * 8;
            if (g >= p.share || t >= V) continue;
            const int w = t >> 5;  // -1 in front of the row
            const uint32_t lo = w >= 0 ? bits[w] : 0u, hi = w + 1 < words ? bits[w + 1] : 0u;
            const uint32_t m = __funnelshift_r(lo, hi, t & 31);
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (!(m >> i & 1)) x[k][i] = -INFINITY;
        }
    }

    const auto pair_of = [&](int i) {  // of warp i of the row
        const uint32_t at = mapa_shared(smem_u32(pairs + i % kWarps), (uint32_t)(i / kWarps));
        return make_float2(ld_cluster_f32(at), ld_cluster_f32(at + 4));
    };

    if (T > 0.f) {
        // (a temperature next to 0: 0 times its reciprocal stays 0)
        const float scale = fminf(__fdiv_rn(kLog2e, T), FLT_MAX);
        float m = -INFINITY, sum = 0.f;
#pragma unroll
        for (int k = 0; k < kG; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) m = fmax_nan(m, x[k][i]);
        m = warp_max_nan(m);
#pragma unroll
        for (int k = 0; k < kG; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[k][i] = x[k][i] == -INFINITY ? 0.f : ex2((x[k][i] - m) * scale);
                sum += x[k][i];
            }
        sum = warp_add(sum);
        if (lane == 0) pairs[warp] = make_float2(m, sum);
        cluster_sync_all();
        float2 q[kMaxCluster * kWarps / 32];
        float M = -INFINITY, total = 0.f;
#pragma unroll
        for (int k = 0; k < kMaxCluster * kWarps / 32; ++k) {
            const int i = k * 32 + lane;
            q[k] = i < p.ctas * kWarps ? pair_of(i) : make_float2(-INFINITY, 0.f);
            M = fmax_nan(M, q[k].x);
        }
        cluster_arrive_all();
        M = warp_max_nan(M);
#pragma unroll
        for (int k = 0; k < kMaxCluster * kWarps / 32; ++k)
            total += q[k].x == -INFINITY ? 0.f : q[k].y * ex2((q[k].x - M) * scale);
        total = warp_add(total);
        // (a NaN or +infinity anywhere leaves no total: NaN everywhere)
        const float fac = M == -INFINITY ? 0.f : (m == -INFINITY ? 0.f : ex2((m - M) * scale)) / total;
#pragma unroll
        for (int k = 0; k < kG; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) x[k][i] *= fac;
        if (M == -INFINITY && rank == 0 && tid == 0 && p.error) atomicOr(p.error, DA_DEV_BAD_PROBS);
    } else {
        float best = -INFINITY;
        int at = INT32_MAX;
        const auto take = [&](float v, int i) {
            if (v > best || (v == best && i < at)) best = v, at = i;
        };
#pragma unroll
        for (int k = 0; k < kG; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (x[k][i] > -INFINITY) take(x[k][i], t0 + (k * kThreads + tid) * 8 + i);
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const float v = __shfl_xor_sync(0xFFFFFFFFu, best, o);
            take(v, __shfl_xor_sync(0xFFFFFFFFu, at, o));
        }
        if (lane == 0) pairs[warp] = make_float2(best, __int_as_float(at));
        cluster_sync_all();
#pragma unroll
        for (int k = 0; k < kMaxCluster * kWarps / 32; ++k) {
            const int i = k * 32 + lane;
            if (i >= p.ctas * kWarps) continue;
            const float2 q = pair_of(i);
            take(q.x, __float_as_int(q.y));
        }
        cluster_arrive_all();
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            const float v = __shfl_xor_sync(0xFFFFFFFFu, best, o);
            take(v, __shfl_xor_sync(0xFFFFFFFFu, at, o));
        }
#pragma unroll
        for (int k = 0; k < kG; ++k) {
            const int t = t0 + (k * kThreads + tid) * 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) x[k][i] = t + i == at ? 1.f : 0.f;
        }
        if (best == -INFINITY && rank == 0 && tid == 0 && p.error) atomicOr(p.error, DA_DEV_BAD_PROBS);
    }
    if (p.prob_dtype == DA_PROB_F32)
        store_row(p, reinterpret_cast<float *>(out), t0, head, x);
    else if (p.prob_dtype == DA_PROB_BF16)
        store_row(p, reinterpret_cast<__nv_bfloat16 *>(out), t0, head, x);
    else
        store_row(p, reinterpret_cast<__half *>(out), t0, head, x);
    cluster_wait_all();  // this CTA's pairs stay until all have read them
}

template <int kG>
cudaError_t launch_one(const ProbsParams &p, cudaStream_t stream, bool pdl) {
    const auto kern = probs_kernel<kG>;
    const bool counts = p.history || p.bias_starts || p.drafts;
    const size_t smem = counts ? (size_t)p.share * 8 * (p.wide ? 4 : 2) : 0;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kThreads * kG * 8 * 4);
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
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {(unsigned)p.ctas, 1, 1};
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_probs(ProbsParams p, int num_sms, cudaStream_t stream, bool pdl) {
    // groups of the longest row: the first of them may start before it
    const int es = p.logits_dtype == DA_PROB_F32 ? 4 : 2;
    const int head = p.logits_stride % 8 == 0 ? (int)(reinterpret_cast<uintptr_t>(p.logits) / es & 7) : 7;
    const int groups = (p.V + head + 7) / 8;
    const int64_t rows = (int64_t)p.B * (p.K + 1);
    // as few CTAs as hold a row with 32 values a thread; where that leaves SMs idle, more, down to 8 values
    int c = 1;
    while (c < kMaxCluster && c * kThreads * 4 < groups) c *= 2;
    while (c < kMaxCluster && rows * c * 2 <= num_sms && groups > c * kThreads) c *= 2;
    p.ctas = c;
    p.share = (groups + c - 1) / c;
    p.wide = (int64_t)p.history_cols + p.K > 0x3FFF;  // counts of more than 14 bits
    const int need = (p.share + kThreads - 1) / kThreads;
    return need <= 1   ? launch_one<1>(p, stream, pdl)
           : need <= 2 ? launch_one<2>(p, stream, pdl)
           : need <= 4 ? launch_one<4>(p, stream, pdl)
           : need <= 8 ? launch_one<8>(p, stream, pdl)
                       : cudaErrorInvalidConfiguration;
}

}  // namespace da
