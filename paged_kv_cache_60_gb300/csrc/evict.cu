// Eviction of cached tokens by the attention weight that they have gathered.
//
// For request b of length L and KV head h, with a budget of N tokens: all
// tokens when L <= N; else the first F, the last R, and of those between them
// the N - F - R heaviest, equal weights going to the lower index. The kept
// tokens' rows (K, V, weight) are copied in their order to slots 0, 1, ... of
// the pages that a second block table names; the old pages are only read.
//
// Two kernels, chained with programmatic dependent launch.
//
// evict_select_kernel: one thread-block cluster per (request, KV head), each
// CTA holding a contiguous share of the middle tokens' keys in shared memory.
// A key orders the weights as unsigned integers; the key of the last token
// kept is found digit by digit (11, 11 and 10 bits) from histograms that the
// CTAs of the cluster add up through distributed shared memory. The counts of
// heavier and of equal tokens in the lower shares then give every CTA its
// place in the list, and ballots keep the order within it. No atomic changes
// an order: the histograms are integer sums.
//
// evict_copy_kernel: one CTA per (request, tile of kept tokens); the source and
// destination slots of the tile are looked up once into shared memory, then
// the rows are copied 16 bytes a thread. Bound by HBM: each kept byte is read
// and written once.
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "decode_attn.h"
#include "layout.h"

namespace da {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kBins = 2048;
constexpr int kKeyCap = 40960;  // keys a CTA keeps in shared memory (160 KB); later ones are read again from the pool

__device__ __forceinline__ int page_index(int t, int page_size, int log2_page) {
    return log2_page >= 0 ? t >> log2_page : t / page_size;
}

// Unsigned key in the order of the weights: -inf lowest, -0 = +0, NaN (any)
// above +inf.
__device__ __forceinline__ uint32_t key_of(float w) {
    if (w != w) return 0xFFFFFFFFu;
    const uint32_t u = __float_as_uint(w + 0.f);
    return (u >> 31) ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t caddr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(caddr) : "memory");
    return v;
}

struct SelSmem {
    uint32_t hist[3][kBins];   // this CTA's counts, one histogram a digit
    uint32_t warp_sum[32];
    uint32_t wgt[33], weq[33];
    uint32_t digit, above;     // the digit found, tokens above it
    uint32_t gt, eq;           // this CTA's tokens above / at the last kept key
};

// kC: CTAs per cluster
template <int kC>
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const __grid_constant__ EvictParams p) {
    extern __shared__ uint32_t keys[];
    __shared__ SelSmem s;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = kC > 1 ? (int)cluster_ctarank() : 0;
    const int row = blockIdx.x / kC, b = row / p.H_kv, h = row - b * p.H_kv;
    pdl_wait();
    pdl_launch_dependents();

    const int64_t max_len = (int64_t)p.max_pages * p.page_size;
    int L = __ldg(p.seqlens + b);
    if (h == 0 && rank == 0 && tid == 0 && p.error) {
        if (L < 0) atomicOr(p.error, DA_DEV_NEG_LEN);
        if (L > max_len) atomicOr(p.error, DA_DEV_SEQ_TOO_LONG);
    }
    L = (int)min((int64_t)max(L, 0), max_len);
    const int N = p.budget;
    int32_t *kept = p.kept + (int64_t)row * N;
    if (h == 0 && rank == 0 && tid == 0) p.new_seqlens[b] = min(L, N);
    if (L <= N) {
        for (int i = rank * kSelThreads + tid; i < N; i += kC * kSelThreads) kept[i] = i < L ? i : -1;
        return;
    }
    const int F = p.first, R = p.last;
    for (int i = rank * kSelThreads + tid; i < F; i += kC * kSelThreads) kept[i] = i;
    for (int i = rank * kSelThreads + tid; i < R; i += kC * kSelThreads) kept[N - R + i] = L - R + i;
    const int M = L - F - R;      // tokens to choose from
    uint32_t want = N - F - R;    // tokens to choose, < M
    if (want == 0) return;        // uniform over the cluster, as every exit above

    // this CTA's share [m0, m1) of the middle, a multiple of 32 tokens
    const int share = ((M + kC - 1) / kC + 31) / 32 * 32;
    const int m0 = min(M, rank * share), m1 = min(M, m0 + share), n = m1 - m0;
    const int32_t *table = p.src_table + (int64_t)b * p.max_pages;
    auto weight_key = [&](int i) -> uint32_t {
        const int t = F + m0 + i, pi = page_index(t, p.page_size, p.log2_page);
        const int page = __ldg(table + pi);
        if (page < 0 || page >= p.num_pages) {
            if (p.error) atomicOr(p.error, DA_DEV_BAD_PAGE);
            return 0u;  // below every weight
        }
        return key_of(__ldg(p.weights + ((int64_t)page * p.H_kv + h) * p.page_size + (t - pi * p.page_size)));
    };
    for (int i = tid; i < kBins; i += kSelThreads) s.hist[0][i] = s.hist[1][i] = s.hist[2][i] = 0;
    const int nc = min(n, kKeyCap);
    for (int i = tid; i < nc; i += kSelThreads) keys[i] = weight_key(i);
    __syncthreads();
    auto key = [&](int i) -> uint32_t { return i < kKeyCap ? keys[i] : weight_key(i); };

    // digits, highest first
    uint32_t prefix = 0, mask = 0, local_above = 0;
#pragma unroll
    for (int d = 0; d < 3; ++d) {
        const int shift = d == 0 ? 21 : d == 1 ? 10 : 0;
        const int bins = d == 2 ? 1024 : kBins;
        uint32_t *hist = s.hist[d];
        for (int i0 = 0; i0 < n; i0 += kSelThreads) {
            const int i = i0 + tid;
            const uint32_t k = i < n ? key(i) : 0u;
            const bool in = i < n && (k & mask) == prefix;
            const uint32_t bin = (k >> shift) & (bins - 1);
            // one add per warp where all its keys share a bin (equal weights)
            const uint32_t act = __ballot_sync(0xffffffffu, in);
            if (act) {
                const uint32_t b0 = __shfl_sync(0xffffffffu, bin, __ffs(act) - 1);
                if (__all_sync(0xffffffffu, !in || bin == b0)) {
                    if (lane == 0) atomicAdd(hist + b0, (uint32_t)__popc(act));
                } else if (in) {
                    atomicAdd(hist + bin, 1u);
                }
            }
        }
        if (kC > 1)
            cluster_sync_all();
        else
            __syncthreads();
        // the whole row's counts, two bins a thread from the top, and their suffix sums
        const int top = bins - 1 - 2 * tid;  // bins top and top - 1
        uint32_t c0 = 0, c1 = 0;
        if (top > 0) {
            const uint32_t a = smem_u32(hist + top - 1);
#pragma unroll
            for (int r = 0; r < kC; ++r) {
                if (kC > 1) {
                    c1 += ld_cluster_u32(mapa_shared(a, r));
                    c0 += ld_cluster_u32(mapa_shared(a + 4, r));
                } else {
                    c1 += hist[top - 1];
                    c0 += hist[top];
                }
            }
        }
        uint32_t v = c0 + c1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += x;
        }
        if (lane == 31) s.warp_sum[warp] = v;
        __syncthreads();
        uint32_t before = 0;
        {
            uint32_t w = lane < warp ? s.warp_sum[lane] : 0u;
            before = __reduce_add_sync(0xffffffffu, w);
        }
        const uint32_t incl = before + v, excl = incl - c0 - c1;  // counts above these bins
        if (top > 0) {
            if (excl < want && want <= excl + c0) {
                s.digit = top;
                s.above = excl;
            } else if (excl + c0 < want && want <= incl) {
                s.digit = top - 1;
                s.above = excl + c0;
            }
        }
        __syncthreads();
        const uint32_t digit = s.digit;
        want -= s.above;
        // this CTA's tokens above the digit
        uint32_t mine = 0;
        for (int i = digit + 1 + tid; i < bins; i += kSelThreads) mine += hist[i];
        mine = __reduce_add_sync(0xffffffffu, mine);
        if (lane == 0) s.wgt[warp] = mine;
        __syncthreads();
        local_above += __reduce_add_sync(0xffffffffu, s.wgt[lane]);
        if (d == 2 && tid == 0) {
            s.gt = local_above;
            s.eq = hist[digit];
        }
        prefix |= digit << shift;
        mask |= (uint32_t)(bins - 1) << shift;
        __syncthreads();  // s.digit and s.wgt are written again
    }
    if (kC > 1)
        cluster_sync_all();  // every CTA's gt and eq
    else
        __syncthreads();
    const uint32_t T = prefix;  // tokens above T are kept, and the first `want` of those at T
    uint32_t gt_before = 0, eq_before = 0;
    if (kC > 1) {
        if (lane < rank) {
            gt_before = ld_cluster_u32(mapa_shared(smem_u32(&s.gt), lane));
            eq_before = ld_cluster_u32(mapa_shared(smem_u32(&s.eq), lane));
        }
        gt_before = __reduce_add_sync(0xffffffffu, gt_before);
        eq_before = __reduce_add_sync(0xffffffffu, eq_before);
        cluster_arrive_all();  // done with the other CTAs' memory; waited for before the exit
    }
    // each warp counts, then lists, a contiguous run of this CTA's share
    const int per = ((n + 31) / 32 + 31) / 32 * 32;
    const int w0 = min(n, warp * per), w1 = min(n, w0 + per);
    uint32_t gt = 0, eq = 0;
    for (int i = w0 + lane; i < w1; i += 32) {
        const uint32_t k = key(i);
        gt += k > T;
        eq += k == T;
    }
    gt = __reduce_add_sync(0xffffffffu, gt);
    eq = __reduce_add_sync(0xffffffffu, eq);
    if (lane == 0) {
        s.wgt[warp] = gt;
        s.weq[warp] = eq;
    }
    __syncthreads();
    gt_before += __reduce_add_sync(0xffffffffu, lane < warp ? s.wgt[lane] : 0u);
    eq_before += __reduce_add_sync(0xffffffffu, lane < warp ? s.weq[lane] : 0u);
    const uint32_t below = (1u << lane) - 1u;
    for (int i0 = w0; i0 < w1; i0 += 32) {
        const int i = i0 + lane;
        const uint32_t k = i < w1 ? key(i) : 0u;
        const bool g = i < w1 && k > T, e = i < w1 && k == T;
        const uint32_t bg = __ballot_sync(0xffffffffu, g), be = __ballot_sync(0xffffffffu, e);
        const uint32_t eb = eq_before + __popc(be & below);   // equal tokens before this one
        if (g || (e && eb < want)) {
            const uint32_t at = gt_before + __popc(bg & below) + min(eb, want);
            kept[F + at] = F + m0 + i;
        }
        gt_before += __popc(bg);
        eq_before += __popc(be);
    }
    if (kC > 1) cluster_wait_all();
}

constexpr int kCopyThreads = 256;

// Copies one tile of kept tokens of one request. A thread keeps its place in a
// row and walks over the rows, kUnroll at a time, K and V of each.
template <int kUnroll>
__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(const __grid_constant__ EvictParams p, int tile,
                                                                  int tiles) {
    extern __shared__ int64_t rows[];  // [tile * H_kv] source rows (-1: none), then as many destination rows
    const int tid = threadIdx.x, H = p.H_kv;
    const int b = blockIdx.x / tiles, i0 = (blockIdx.x - b * tiles) * tile;
    pdl_wait();
    pdl_launch_dependents();
    const int n = min(tile, p.new_seqlens[b] - i0);
    if (n <= 0) return;
    int64_t *src = rows, *dst = rows + (int64_t)tile * H;
    const int32_t *st = p.src_table + (int64_t)b * p.max_pages, *dt = p.dst_table + (int64_t)b * p.max_pages;
    for (int k = tid; k < n * H; k += kCopyThreads) {
        const int h = k / n, i = k - h * n;
        const int t = p.kept[((int64_t)b * H + h) * p.budget + i0 + i];
        const int si = page_index(t, p.page_size, p.log2_page), di = page_index(i0 + i, p.page_size, p.log2_page);
        const int sp = __ldg(st + si), dp = __ldg(dt + di);
        const bool ok = sp >= 0 && sp < p.num_pages && dp >= 0 && dp < p.num_pages;
        if (!ok && p.error) atomicOr(p.error, DA_DEV_BAD_PAGE);
        const int ss = t - si * p.page_size, ds = i0 + i - di * p.page_size;
        src[i * H + h] = ok ? ((int64_t)sp * p.page_size + ss) * H + h : -1;
        dst[i * H + h] = ((int64_t)dp * p.page_size + ds) * H + h;
        if (ok)
            p.weights[((int64_t)dp * H + h) * p.page_size + ds] = p.weights[((int64_t)sp * H + h) * p.page_size + ss];
    }
    __syncthreads();
    const int vecs = p.row_bytes / 16, across = min(vecs, kCopyThreads), down = kCopyThreads / across;
    const int r0 = tid / across, v0 = tid - r0 * across;
    if (r0 >= down) return;
    for (int v = v0; v < vecs; v += across) {
        for (int r = r0; r < n * H; r += down * kUnroll) {
            uint4 xk[kUnroll], xv[kUnroll];
            int64_t from[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int k = r + u * down;
                from[u] = k < n * H ? src[k] : -1;
                if (from[u] >= 0) {
                    xk[u] = ldg_stream16(p.k_pool + from[u] * p.row_bytes + v * 16);
                    if (p.v_pool) xv[u] = ldg_stream16(p.v_pool + from[u] * p.row_bytes + v * 16);
                }
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (from[u] >= 0) {
                    const int64_t to = dst[r + u * down] * p.row_bytes + v * 16;
                    *reinterpret_cast<uint4 *>(p.k_pool + to) = xk[u];
                    if (p.v_pool) *reinterpret_cast<uint4 *>(p.v_pool + to) = xv[u];
                }
            }
        }
    }
}

template <int kC>
cudaError_t launch_select(const EvictParams &p, int key_bytes, cudaStream_t stream, bool pdl) {
    const auto kern = evict_select_kernel<kC>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeyCap * 4);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.B * p.H_kv * kC));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = key_bytes;
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
    return cudaLaunchKernelEx(&cfg, kern, p);
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, int num_sms, cudaStream_t stream, bool pdl) {
    // CTAs per row: as many as there are SMs for, while each still has a few thousand tokens of the longest
    // length the block table allows
    const int64_t rows = (int64_t)p.B * p.H_kv, longest = (int64_t)p.max_pages * p.page_size;
    int c = 1;
    while (c < 8 && rows * c * 2 <= num_sms && longest / c > 4096) c *= 2;
    const int64_t share = (longest + c - 1) / c + 32;
    const int key_bytes = (int)(share < kKeyCap ? share : kKeyCap) * 4;
    cudaError_t e = c == 8   ? launch_select<8>(p, key_bytes, stream, pdl)
                    : c == 4 ? launch_select<4>(p, key_bytes, stream, pdl)
                    : c == 2 ? launch_select<2>(p, key_bytes, stream, pdl)
                             : launch_select<1>(p, key_bytes, stream, pdl);
    if (e != cudaSuccess) return e;
    // tile: about 64 KB of rows per CTA
    const int64_t token_bytes = (int64_t)p.H_kv * p.row_bytes * (p.v_pool ? 2 : 1);
    int64_t tile = (64 << 10) / token_bytes;
    tile = tile < 1 ? 1 : tile > 64 ? 64 : tile;
    cudaLaunchConfig_t cfg = {};
    const int64_t tiles = (p.budget + tile - 1) / tile;
    if (tiles * p.B > INT32_MAX) return cudaErrorInvalidConfiguration;
    cfg.gridDim = dim3((unsigned)(tiles * p.B));
    cfg.blockDim = dim3(kCopyThreads);
    cfg.dynamicSmemBytes = (size_t)tile * p.H_kv * 16;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, evict_copy_kernel<4>, p, (int)tile, (int)tiles);
}

}  // namespace da
