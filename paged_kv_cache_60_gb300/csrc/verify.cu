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
// leaves a sum per tile, and only the tile with the token is read again. Rows
// start anywhere (a vocabulary need not be a multiple of anything), so tiles
// start where p is 16-byte aligned, and q, whose rows are aligned otherwise, is
// read in aligned vectors too, with the start of the next one, and shifted in
// registers.
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "decode_attn.h"
#include "layout.h"

namespace da {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTile = 1024;                        // entries per tile, one warp each
constexpr int kMaxVocab = 1 << 20;                // exclusive
constexpr int kMaxTiles = kMaxVocab / kTile + 1;  // the first may start before the row

template <typename T>
__device__ __forceinline__ float to_f32(T x) {
    return static_cast<float>(x);
}
// the i-th value of a 16-byte vector held as four words
template <typename T>
__device__ __forceinline__ float value_of(const uint32_t *w, int i);
template <>
__device__ __forceinline__ float value_of<float>(const uint32_t *w, int i) {
    return __uint_as_float(w[i]);
}
template <>
__device__ __forceinline__ float value_of<__nv_bfloat16>(const uint32_t *w, int i) {
    return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
}
template <>
__device__ __forceinline__ float value_of<__half>(const uint32_t *w, int i) {
    const __half2 h = *reinterpret_cast<const __half2 *>(w + i / 2);
    return i & 1 ? __high2float(h) : __low2float(h);
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
// inclusive sums over the lanes
__device__ __forceinline__ uint64_t warp_scan_u64(uint64_t v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t x = __shfl_up_sync(0xffffffffu, (unsigned long long)v, o);
        if (lane >= o) v += x;
    }
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

// Sum of the weights of entries [v0, v0 + kTile) that lie in the row, by one
// warp; p is 16-byte aligned at v0 (which may be below 0). kShift: whole words
// by which q is off a 16-byte boundary there, -1 without q; 16-bit rows may be
// off by half a word more.
template <typename T, int kShift>
__device__ __forceinline__ uint64_t tile_sum(const Row<T> &r, int v0, int V, int lane) {
    constexpr bool kHasQ = kShift >= 0, kHalf = sizeof(T) == 2;
    constexpr int VE = 16 / (int)sizeof(T);       // values per vector
    constexpr int NV = kTile / 32 / VE;           // vectors per lane
    constexpr int U = kHasQ || NV < 8 ? 4 : 8;    // of them in flight (and as many or twice as many of q)
    Fixed f;
    // whole vectors of p, and of q around them, inside the row
    if (v0 >= VE && v0 + kTile + VE <= V && !(r.without >= v0 && r.without < v0 + kTile)) {
        const uint4 *p = reinterpret_cast<const uint4 *>(r.p + v0) + lane;
        const uintptr_t qa = reinterpret_cast<uintptr_t>(r.q + v0);
        const uint4 *q = reinterpret_cast<const uint4 *>(qa & ~(uintptr_t)15) + lane;
        const bool half = kHalf && (qa & 2);      // uniform over the warp
        const int bits = half ? 16 : 0;
#pragma unroll
        for (int g = 0; g < NV; g += U) {
            uint4 x[U];
            uint32_t y[U][8];                     // the vector of q at p's, and what is needed of the next one
#pragma unroll
            for (int i = 0; i < U; ++i) {
                x[i] = ld_unwritten(p + (g + i) * 32);
                if constexpr (kHasQ) {
                    const uint4 *qi = q + (g + i) * 32;
                    const uint4 u = ld_unwritten(qi);
                    y[i][0] = u.x, y[i][1] = u.y, y[i][2] = u.z, y[i][3] = u.w;
                    y[i][4] = y[i][5] = y[i][6] = y[i][7] = 0u;
                    if constexpr (kShift == 0 && kHalf) {
                        if (half) y[i][4] = ld_unwritten(reinterpret_cast<const uint32_t *>(qi + 1));
                    } else if constexpr (kShift == 1 && !kHalf) {
                        y[i][4] = ld_unwritten(reinterpret_cast<const uint32_t *>(qi + 1));
                    } else if constexpr (kShift == 1 || (kShift == 2 && !kHalf)) {
                        const uint2 z = ld_unwritten(reinterpret_cast<const uint2 *>(qi + 1));
                        y[i][4] = z.x, y[i][5] = z.y;
                    } else if constexpr (kShift > 0) {
                        const uint4 z = ld_unwritten(qi + 1);
                        y[i][4] = z.x, y[i][5] = z.y, y[i][6] = z.z, y[i][7] = z.w;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < U; ++i) {
                const uint32_t a[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                uint32_t c[4] = {0u, 0u, 0u, 0u};
                if constexpr (kHasQ) {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        c[k] = kHalf ? __funnelshift_r(y[i][kShift + k], y[i][kShift + k + 1], bits) : y[i][kShift + k];
                }
#pragma unroll
                for (int k = 0; k < VE; ++k) f.add(weight(value_of<T>(a, k), kHasQ ? value_of<T>(c, k) : 0.f));
            }
        }
    } else {
#pragma unroll
        for (int g = 0; g < kTile / 32; g += 16) {
            float x[16], y[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {  // (loads of a clamped index: no branch keeps them apart)
                const int v = min(max(v0 + (g + i) * 32 + lane, 0), V - 1);
                x[i] = to_f32(r.p[v]);
                y[i] = kHasQ ? to_f32(r.q[v]) : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int v = v0 + (g + i) * 32 + lane;
                f.add(v >= 0 && v < V && v != r.without ? weight(x[i], y[i]) : 0.f);
            }
        }
    }
    return warp_sum_u64(f.sum());
}

template <typename T, int kC>
__global__ void __launch_bounds__(kThreads, 2) verify_kernel(const __grid_constant__ VerifyParams p) {
    __shared__ uint64_t s_tile[kMaxTiles];
    __shared__ uint64_t s_total, s_warp[kWarps];
    __shared__ int s_a, s_ended, s_bad, s_token[64];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = kC > 1 ? (int)cluster_ctarank() : 0;
    const int b = blockIdx.x / kC, K = p.K, V = p.V;
    pdl_wait();
    pdl_launch_dependents();
    const T *target = static_cast<const T *>(p.target) + (int64_t)b * (K + 1) * p.target_stride;
    const T *draft = p.draft ? static_cast<const T *>(p.draft) + (int64_t)b * K * p.draft_stride : nullptr;
    const int32_t *tokens = p.tokens + (int64_t)b * K;
    const float *u = p.uniform + (int64_t)b * (K + 1);

    // read ahead of their use at the end
    const float u_last = u[K];
    const int len = p.seqlens ? p.seqlens[b] : 0;
    // how many drafts are accepted (two lanes' worth of drafts: K <= 63)
    if (warp == 0) {
        bool go0 = false, go1 = false, end0 = false, end1 = false, bad = false;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int j = lane + 32 * k;
            bool go = false, end = j >= K;
            if (j < K) {
                const int x = tokens[j];
                s_token[j] = x;
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
        const auto both = [](bool lo, bool hi) {
            return (uint64_t)__ballot_sync(0xffffffffu, lo) | (uint64_t)__ballot_sync(0xffffffffu, hi) << 32;
        };
        const uint64_t go = both(go0, go1), end = both(end0, end1);
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
    row.without = !ended && !draft ? s_token[a] : -1;

    // tile t: entries [t kTile - lead, (t + 1) kTile - lead)
    const int lead = (int)(reinterpret_cast<uintptr_t>(row.p) & 15u) / (int)sizeof(T);
    const int tiles = (V + lead + kTile - 1) / kTile;
    const int t0 = (int)((int64_t)tiles * rank / kC), t1 = (int)((int64_t)tiles * (rank + 1) / kC);
    uint64_t before = 0, total = 0;
    for (int attempt = 0;; ++attempt) {
        uint64_t mine = 0;
        // q's distance from a 16-byte boundary where p is on one, in words
        const int shift = row.q ? (int)((reinterpret_cast<uintptr_t>(row.q - lead) & 15u) >> 2) : -1;
        for (int t = t0 + warp; t < t1; t += kWarps) {
            const int v0 = t * kTile - lead;
            uint64_t s;
            switch (shift) {
                case 0: s = tile_sum<T, 0>(row, v0, V, lane); break;
                case 1: s = tile_sum<T, 1>(row, v0, V, lane); break;
                case 2: s = tile_sum<T, 2>(row, v0, V, lane); break;
                case 3: s = tile_sum<T, 3>(row, v0, V, lane); break;
                default: s = tile_sum<T, -1>(row, v0, V, lane); break;
            }
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

    if (kC > 1) {
        __syncwarp();
        cluster_arrive_all();  // done with the other CTAs' totals; waited for before the exit
    }
    // first entry whose running sum exceeds floor(u total); u clamped into [0, 1)
    const float uk = fminf(fmaxf(u_last, 0.f), 0x1.fffffep-1f);  // NaN: 0
    uint64_t until;
    {
        const uint32_t bits = __float_as_uint(uk);
        const int e = (int)(bits >> 23) - 150 + 64;  // uk 2^64 = m 2^e
        const uint64_t m = (bits & 0x7FFFFFu) | ((bits >> 23) ? 0x800000u : 0u);
        const uint64_t U = e >= 0 ? m << e : e > -24 ? m >> -e : 0ull;
        until = __umul64hi(U, total);
    }
    auto finish = [&](int token) {  // by one warp
        for (int i = lane; i <= K; i += 32) p.out[(int64_t)b * (K + 1) + i] = i < a ? s_token[i] : i == a ? token : -1;
        if (lane == 0) {
            p.accepted[b] = a;
            if (p.new_seqlens) p.new_seqlens[b] = max(max(len, 0) - K + a, 0);  // (a padded row of length 0 stays one)
            if (p.error && (s_bad || token < 0))
                atomicOr(p.error, (s_bad ? DA_DEV_BAD_TOKEN : 0) | (token < 0 ? DA_DEV_BAD_PROBS : 0));
        }
    };
    if (total == 0) {
        if (rank == 0 && warp == 0) finish(-1);
    } else if (warp == 0) {
        if (before <= until && until < before + s_total) {
            // the tile with it: lane l looks at tiles l, l + 32, ... 32 at a time
            uint64_t run = before;
            int t = t0;
            for (; t < t1; t += 32) {
                const uint64_t s = t + lane < t1 ? s_tile[t + lane - t0] : 0ull;
                const uint64_t inc = warp_scan_u64(s, lane);
                const uint32_t over = __ballot_sync(0xffffffffu, run + inc > until);
                if (over) {
                    const int k = __ffs(over) - 1;
                    run += shfl_u64(inc - s, k);
                    t += k;
                    break;
                }
                run += shfl_u64(inc, 31);
            }
            // within the tile: 32 groups of 32 entries, all loaded at once, lane l holding entry l of each
            const int v0 = t * kTile - lead + lane;
            uint32_t hi[32];
            int32_t lo[32];
            {
                float x[32], y[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const int v = min(max(v0 + 32 * i, 0), V - 1);
                    x[i] = to_f32(row.p[v]);
                    y[i] = 0.f;
                }
                if (row.q) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) y[i] = to_f32(row.q[min(max(v0 + 32 * i, 0), V - 1)]);
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const int v = v0 + 32 * i;
                    Fixed f;
                    f.add(v >= 0 && v < V && v != row.without ? weight(x[i], y[i]) : 0.f);
                    hi[i] = f.hi;
                    lo[i] = f.lo;
                }
            }
            // sums of the groups, group l's in lane l: each step adds the half that the lane keeps to its partner's
#pragma unroll
            for (int o = 16; o; o >>= 1)
#pragma unroll
                for (int i = 0; i < o; ++i) {
                    const bool up = (lane & o) != 0;
                    const uint32_t gh = up ? hi[i] : hi[i + o];
                    const int32_t gl = up ? lo[i] : lo[i + o];
                    hi[i] = (up ? hi[i + o] : hi[i]) + __shfl_xor_sync(0xffffffffu, gh, o);
                    lo[i] = (up ? lo[i + o] : lo[i]) + __shfl_xor_sync(0xffffffffu, gl, o);
                }
            Fixed group;
            group.hi = hi[0];
            group.lo = lo[0];
            const uint64_t in_group = group.sum(), groups = warp_scan_u64(in_group, lane);
            const int g = __ffs(__ballot_sync(0xffffffffu, run + groups > until)) - 1;
            run += shfl_u64(groups - in_group, g);
            Fixed f;
            const int v = v0 + 32 * g;
            if (v >= 0 && v < V) f.add(row.at(v));
            const uint64_t entries = warp_scan_u64(f.sum(), lane);
            finish(v - lane + __ffs(__ballot_sync(0xffffffffu, run + entries > until)) - 1);
        }
    }
    if (kC > 1) {
        __syncwarp();
        cluster_wait_all();  // every CTA stays until the others have read its total
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
    // CTAs per request: as many as are resident at once, while each warp has a tile. Two CTAs of 256 threads on an SM
    // and up to 128 registers a thread, for the vectors in flight: three (80 registers, spilled) took 30.3 us where two
    // take 22.6 for 128 requests of 131072 entries with q, and 5.7 us against 4.6 for one request of 32000.
    int c = 1;
    while (c < 8 && (int64_t)p.B * c * 2 <= 2 * num_sms && p.V / c > kTile * kWarps) c *= 2;
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
