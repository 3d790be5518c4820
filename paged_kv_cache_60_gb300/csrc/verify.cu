// Verification of drafted tokens against the target model's probabilities,
// from given random numbers.
//
// Request b has a chain of K drafts x_0 .. x_{K-1} (a negative one ends it), the
// target's distributions p_0 .. p_K (p_j: after the first j drafts) and the
// draft model's q_0 .. q_{K-1}. Draft j is accepted when u_j q_j(x_j) <
// p_j(x_j) and every draft before it was; a drafts are accepted. One more
// token follows, drawn with u_K from the weights
//     w(v) = max(p_a(v) - q_a(v), 0)   where draft a was refused,
//     w(v) = p_a(v)                    where the chain had ended,
// so that the tokens are distributed as the target's own.
//
// The weights are counted in whole steps of 2^-44 (their fp32 values rounded to
// nearest even, at most 2^44 each), so their sums are 64-bit integers: exact,
// the same in any order and on any split, and below 2^64 for fewer than 2^20
// entries. The token is the first v whose running sum exceeds floor(u_K *
// total). A step is 2^-44: next to an fp32 probability of 1e-6 it is below the
// rounding of the probability itself.
//
// Bound by reading one row of p, and one of q where a draft was refused. One
// cluster of CTAs per request, a contiguous share of the row each; pass 1
// leaves a sum per tile, and only the tile with the token is read again.
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "decode_attn.h"
#include "layout.h"

namespace da {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 1024;                        // entries per tile, one warp each
constexpr int kMaxVocab = 1 << 20;                // exclusive
constexpr int kMaxTiles = kMaxVocab / kTile;

template <typename T>
__device__ __forceinline__ float to_f32(T x) {
    return static_cast<float>(x);
}

// Running sum of round(w 2^44), w in [0, 1], kept as two 32-bit sums: the part
// in steps of 2^-22 and a signed remainder in steps of 2^-44. Adding 2 rounds
// w to a multiple of 2^-22 (an fp32 in [2, 4) has that ulp), the difference is
// exact, and adding 1.5 * 2^-21 rounds it to a multiple of 2^-44; both land in
// the mantissa bits, so the sums are integer adds. Up to 512 values.
struct Fixed {
    uint32_t hi = 0;
    int32_t lo = 0;
    __device__ __forceinline__ void add(float w) {
        const float t = __fadd_rn(w, 2.f);
        const float r = __fsub_rn(w, __fsub_rn(t, 2.f));
        const float s = __fadd_rn(r, 0x1.8p-21f);
        hi += __float_as_uint(t) - __float_as_uint(2.f);
        lo += __float_as_int(s) - __float_as_int(0x1.8p-21f);
    }
    __device__ __forceinline__ uint64_t sum() const { return ((uint64_t)hi << 22) + (int64_t)lo; }
};

// w(v) as the sums take it: NaN and negative count as 0, above 1 as 1
__device__ __forceinline__ float weight(float p, float q) {
    return fminf(fmaxf(__fsub_rn(p, q), 0.f), 1.f);
}

__device__ __forceinline__ uint64_t shfl_u64(uint64_t v, int src) {
    return __shfl_sync(0xffffffffu, (unsigned long long)v, src);
}
__device__ __forceinline__ uint64_t warp_sum_u64(uint64_t v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, (unsigned long long)v, o);
    return v;
}
__device__ __forceinline__ uint64_t ld_cluster_u64(uint32_t caddr) {
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(caddr) : "memory");
    return v;
}

// Which weights a row takes: p - q, p, or p without the refused (certain) draft.
template <typename T>
struct Row {
    const T *p, *q;   // q null: nothing is subtracted
    int without;      // >= 0: this entry has weight 0 (the draft was certain)
    __device__ __forceinline__ float at(int v) const {
        const float w = weight(to_f32(p[v]), q ? to_f32(q[v]) : 0.f);
        return v == without ? 0.f : w;
    }
};

// Sum of one tile's weights, by one warp.
template <typename T>
__device__ __forceinline__ uint64_t tile_sum(const Row<T> &r, int v0, int v1, int lane) {
    Fixed f;
    if (v0 + kTile <= v1) {
#pragma unroll
        for (int g = 0; g < kTile / 32; g += 16) {
            float p[16], q[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                p[i] = to_f32(r.p[v0 + (g + i) * 32 + lane]);
                q[i] = r.q ? to_f32(r.q[v0 + (g + i) * 32 + lane]) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) f.add(v0 + (g + i) * 32 + lane == r.without ? 0.f : weight(p[i], q[i]));
        }
    } else {
        for (int v = v0 + lane; v < v1; v += 32) f.add(r.at(v));
    }
    return warp_sum_u64(f.sum());
}

template <typename T, int kC>
__global__ void __launch_bounds__(kThreads) verify_kernel(const __grid_constant__ VerifyParams p) {
    __shared__ uint64_t s_tile[kMaxTiles];
    __shared__ uint64_t s_total, s_warp[kWarps];
    __shared__ int s_a, s_ended, s_bad;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = kC > 1 ? (int)cluster_ctarank() : 0;
    const int b = blockIdx.x / kC, K = p.K, V = p.V;
    pdl_wait();
    pdl_launch_dependents();
    const T *target = static_cast<const T *>(p.target) + (int64_t)b * (K + 1) * p.target_stride;
    const T *draft = p.draft ? static_cast<const T *>(p.draft) + (int64_t)b * K * p.draft_stride : nullptr;
    const int32_t *tokens = p.tokens + (int64_t)b * K;
    const float *u = p.uniform + (int64_t)b * (K + 1);

    // how many drafts are accepted (two lanes' worth of drafts: K <= 63)
    if (warp == 0) {
        bool go0 = false, go1 = false, end0 = false, end1 = false, bad = false;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int j = lane + 32 * k;
            bool go = false, end = j >= K;
            if (j < K) {
                const int x = tokens[j];
                end = x < 0 || x >= V;
                bad |= x >= V;
                if (!end) {
                    const double px = to_f32(target[(int64_t)j * p.target_stride + x]);
                    const double qx = draft ? to_f32(draft[(int64_t)j * p.draft_stride + x]) : 1.f;
                    go = (double)u[j] * qx < px;  // the product of two fp32 is exact in fp64
                }
            }
            if (k == 0) {
                go0 = go;
                end0 = end;
            } else {
                go1 = go;
                end1 = end;
            }
        }
        const uint64_t go = (uint64_t)__ballot_sync(0xffffffffu, go0) | (uint64_t)__ballot_sync(0xffffffffu, go1) << 32;
        const uint64_t end = (uint64_t)__ballot_sync(0xffffffffu, end0) | (uint64_t)__ballot_sync(0xffffffffu, end1) << 32;
        const int a = __ffsll((long long)~go) - 1;  // bit 63 is never set: K <= 63
        const bool any_bad = __any_sync(0xffffffffu, bad);
        if (lane == 0) {
            s_a = a;
            s_ended = (int)((end >> a) & 1);
            s_bad = any_bad;
        }
    }
    __syncthreads();
    const int a = s_a;
    const bool ended = s_ended != 0;
    Row<T> row;
    row.p = target + (int64_t)a * p.target_stride;
    row.q = !ended && draft ? draft + (int64_t)a * p.draft_stride : nullptr;
    row.without = !ended && !draft ? tokens[a] : -1;

    const int tiles = (V + kTile - 1) / kTile;
    const int t0 = (int)((int64_t)tiles * rank / kC), t1 = (int)((int64_t)tiles * (rank + 1) / kC);
    uint64_t before = 0, total = 0;
    for (int attempt = 0;; ++attempt) {
        uint64_t mine = 0;
        for (int t = t0 + warp; t < t1; t += kWarps) {
            const uint64_t s = tile_sum(row, t * kTile, min(V, (t + 1) * kTile), lane);
            if (lane == 0) s_tile[t - t0] = s;
            mine += s;
        }
        if (lane == 0) s_warp[warp] = mine;
        __syncthreads();
        if (warp == 0) {
            const uint64_t s = warp_sum_u64(lane < kWarps ? s_warp[lane] : 0ull);
            if (lane == 0) s_total = s;
        }
        if (kC > 1) {
            __syncwarp();
            cluster_sync_all();
        } else {
            __syncthreads();
        }
        before = 0;
        total = 0;
#pragma unroll
        for (int r = 0; r < kC; ++r) {
            const uint64_t s = kC > 1 ? ld_cluster_u64(mapa_shared(smem_u32(&s_total), r)) : s_total;
            if (r < rank) before += s;
            total += s;
        }
        if (total != 0 || attempt == 1 || (!row.q && row.without < 0)) break;
        // nothing is left of p - q (it may be when the rows do not sum to one): draw from p itself
        row.q = nullptr;
        row.without = -1;
        if (kC > 1) {
            __syncwarp();
            cluster_sync_all();  // every CTA has read the totals
        } else {
            __syncthreads();
        }
    }

    // first entry whose running sum exceeds floor(u total); u clamped into [0, 1)
    const float uk = fminf(fmaxf(u[K], 0.f), 0x1.fffffep-1f);  // NaN: 0
    uint64_t until;
    {
        const uint32_t bits = __float_as_uint(uk);
        const int e = (int)(bits >> 23) - 150 + 64;  // uk 2^64 = m 2^e
        const uint64_t m = (bits & 0x7FFFFFu) | ((bits >> 23) ? 0x800000u : 0u);
        const uint64_t U = e >= 0 ? m << e : e > -24 ? m >> -e : 0ull;
        until = __umul64hi(U, total);
    }
    auto finish = [&](int token) {
        for (int i = 0; i <= K; ++i)
            p.out[(int64_t)b * (K + 1) + i] = i < a ? tokens[i] : i == a ? token : -1;
        p.accepted[b] = a;
        if (p.new_seqlens) p.new_seqlens[b] = p.seqlens[b] - K + a;
        if (p.error) {
            if (s_bad) atomicOr(p.error, DA_DEV_BAD_TOKEN);
            if (token < 0) atomicOr(p.error, DA_DEV_BAD_PROBS);
        }
    };
    if (total == 0) {
        if (rank == 0 && tid == 0) finish(-1);
    } else if (warp == 0) {
        if (before <= until && until < before + s_total) {
            // the tile with it: lane l looks at tiles l, l + 32, ... 32 at a time
            uint64_t run = before;
            int t = t0;
            for (; t < t1; t += 32) {
                const uint64_t s = t + lane < t1 ? s_tile[t + lane - t0] : 0ull;
                uint64_t inc = s;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint64_t x = __shfl_up_sync(0xffffffffu, (unsigned long long)inc, o);
                    if (lane >= o) inc += x;
                }
                const uint32_t over = __ballot_sync(0xffffffffu, run + inc > until);
                if (over) {
                    const int k = __ffs(over) - 1;
                    run += shfl_u64(inc - s, k);
                    t += k;
                    break;
                }
                run += shfl_u64(inc, 31);
            }
            const int v1 = min(V, (t + 1) * kTile);
            for (int v0 = t * kTile; v0 < v1; v0 += 32) {
                Fixed f;
                if (v0 + lane < v1) f.add(row.at(v0 + lane));
                const uint64_t s = f.sum();
                uint64_t inc = s;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const uint64_t x = __shfl_up_sync(0xffffffffu, (unsigned long long)inc, o);
                    if (lane >= o) inc += x;
                }
                const uint32_t over = __ballot_sync(0xffffffffu, run + inc > until);
                if (over) {
                    if (lane == 0) finish(v0 + __ffs(over) - 1);
                    break;
                }
                run += shfl_u64(inc, 31);
            }
        }
    }
    if (kC > 1) {
        __syncwarp();
        cluster_sync_all();  // every CTA stays until the others have read its total
    }
}

template <typename T, int kC>
cudaError_t launch(const VerifyParams &p, cudaStream_t stream, bool pdl) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.B * kC));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (kC > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim = {kC, 1, 1};
        ++n;
    }
    if (pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, verify_kernel<T, kC>, p);
}

template <typename T>
cudaError_t launch_for(const VerifyParams &p, int num_sms, cudaStream_t stream, bool pdl) {
    // CTAs per request: as many as there are SMs for, two resident on each, while each has a tile per warp
    int c = 1;
    while (c < 8 && (int64_t)p.B * c * 2 <= 2 * num_sms && p.V / c > kTile * kWarps / 2) c *= 2;
    switch (c) {
        case 8: return launch<T, 8>(p, stream, pdl);
        case 4: return launch<T, 4>(p, stream, pdl);
        case 2: return launch<T, 2>(p, stream, pdl);
        default: return launch<T, 1>(p, stream, pdl);
    }
}

}  // namespace

cudaError_t launch_verify(int prob_dtype, const VerifyParams &p, int num_sms, cudaStream_t stream, bool pdl) {
    switch (prob_dtype) {
        case DA_PROB_BF16: return launch_for<__nv_bfloat16>(p, num_sms, stream, pdl);
        case DA_PROB_F16: return launch_for<__half>(p, num_sms, stream, pdl);
        default: return launch_for<float>(p, num_sms, stream, pdl);
    }
}

}  // namespace da
