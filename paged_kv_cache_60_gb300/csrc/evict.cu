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
// kept is found digit by digit (8, 12 and 12 bits) from histograms that the
// CTAs of the cluster add up through distributed shared memory. Weights crowd
// into few exponents, so the first digit is short enough for every lane to
// count into a copy of its own (256 bins x 32 lanes, one bank each): its shared
// atomics never meet in a warp. The later digits are mantissa bits and spread
// over 4096 bins; where most keys share the first digit's bin they are counted
// with one add per warp when they are equal (weights that are all zero). With
// 2048 bins in four copies the first digit alone took half of the selection.
// After two digits a few tokens are usually left in the row: where they are at
// most 256, their keys are brought together and compared with each other, one
// exchange in a cluster instead of the third digit's three (two latent caches of
// 115 thousand tokens, sixteen CTAs each: 29.5 us for both kernels on one state,
// out of a warm L2, against 32.9, with the first digit's 256 bins read by every
// CTA instead of shared out; 37.3 over six states).
// The counts of heavier and of equal tokens in the lower shares then give every
// CTA its place in the list, and ballots keep the order within it. No atomic
// changes a result: the histograms are integer sums, and of the few keys only
// counts are taken.
//
// evict_copy_kernel: one CTA per (request, tile of kept tokens); the source and
// destination slots of the tile are looked up once into shared memory, then
// the rows are copied 16 bytes a thread. Bound by HBM: each kept byte is read
// and written once.
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "common.cuh"
#include "decode_attn.h"
#include "layout.h"

namespace da {
namespace {

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins0 = 256, kBins = 4096;   // bins of the first digit, and of the two others
constexpr int kFew = 256;       // tokens left after two digits that are compared with each other instead of a third
static_assert(3 * kFew + 2 <= kBins && kFew <= kSelThreads, "their keys lie where the third digit's counts would");
constexpr int kKeyCap = 36864;  // keys a CTA keeps in shared memory (144 KB); later ones are read again from the pool

__device__ __forceinline__ int page_index(int t, int page_size, int log2_page) {
    return log2_page >= 0 ? t >> log2_page : t / page_size;
}

// Unsigned key in the order of the weights: -inf lowest, -0 = +0, NaN (any)
// above +inf. 0 is below every weight's.
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
__device__ __forceinline__ uint4 ld_cluster_v4(uint32_t caddr) {
    uint4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(caddr)
                 : "memory");
    return v;
}
// One token's key; 0 for a token on a page outside the pool.
__device__ __noinline__ uint32_t weight_key(const EvictParams &p, const int32_t *table, int h, int t) {
    const int pi = page_index(t, p.page_size, p.log2_page), page = ld_unwritten(table + pi);
    if (page < 0 || page >= p.num_pages) {
        if (p.error) atomicOr(p.error, DA_DEV_BAD_PAGE);
        return 0u;
    }
    return key_of(ld_unwritten(p.weights + ((int64_t)page * p.H_kv + h) * p.page_size + (t - pi * p.page_size)));
}

struct SelSmem {
    // this CTA's counts: the first digit's, a copy per lane; then the other two digits', in the same place
    union {
        uint32_t lanes[kBins0][32];
        uint32_t hist[2][kBins];
    };
    uint32_t hist0[kBins0];        // the first digit's, summed over the lanes
    uint32_t row0[kBins0];         // and, in a cluster, over its CTAs
    uint32_t warp_sum[kSelWarps], wgt[kSelWarps], weq[kSelWarps];
    uint32_t digit, above, at;     // the digit found, tokens above it and at it, in the row
    uint32_t slice;                // this CTA's slice of the row's histogram: all of its tokens
    uint32_t gt, eq;               // this CTA's tokens above / at the last kept key
};
static_assert(sizeof(uint32_t) * kBins0 * 32 == sizeof(uint32_t) * 2 * kBins, "one region");
constexpr int kSelBase = (sizeof(SelSmem) + 15) / 16 * 16;
// in a cluster, behind it: this CTA's slice of the row's histogram; then the keys
constexpr int sel_keys_at(int cluster) { return kSelBase + (cluster > 1 ? kBins / cluster * 4 : 0); }

// sum of one value per warp over the warps below `upto`
__device__ __forceinline__ uint32_t sum_below(const uint32_t *per_warp, int upto, int lane) {
    return __reduce_add_sync(0xffffffffu, lane < upto ? per_warp[lane] : 0u);
}

// Counts one key per lane that is `in`: one add for the whole warp where its keys share a bin.
__device__ __forceinline__ void count_crowded(uint32_t *hist, uint32_t bin, bool in, int lane) {
    const uint32_t act = __ballot_sync(0xffffffffu, in);
    if (!act) return;
    const uint32_t b0 = __shfl_sync(0xffffffffu, bin, __ffs(act) - 1);
    if (__all_sync(0xffffffffu, !in || bin == b0)) {
        if (lane == 0) atomicAdd(hist + b0, (uint32_t)__popc(act));
    } else if (in) {
        atomicAdd(hist + bin, 1u);
    }
}

// kC: CTAs per cluster
template <int kC>
__global__ void __launch_bounds__(kSelThreads, 2) evict_select_kernel(const __grid_constant__ EvictParams p) {
    extern __shared__ __align__(16) uint8_t sel_smem[];
    SelSmem &s = *reinterpret_cast<SelSmem *>(sel_smem);
    uint32_t *row_slice = reinterpret_cast<uint32_t *>(sel_smem + kSelBase);
    uint32_t *keys = reinterpret_cast<uint32_t *>(sel_smem + sel_keys_at(kC));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = kC > 1 ? (int)cluster_ctarank() : 0;
    const int row = blockIdx.x / kC, b = row / p.H_kv, h = row - b * p.H_kv;
    for (int i = tid; i < kBins0 * 32 / 4; i += kSelThreads)
        reinterpret_cast<uint4 *>(&s.lanes[0][0])[i] = make_uint4(0u, 0u, 0u, 0u);
    if (kC > 1 && tid < kBins0) s.row0[tid] = 0u;
    pdl_wait();
    pdl_launch_dependents();

    const int64_t max_len = (int64_t)p.max_pages * p.page_size;
    int L = p.seqlens[b];
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

    // this CTA's share [m0, m1) of the middle, a multiple of 128 tokens
    const int share = (int)((((int64_t)M + kC - 1) / kC + 127) / 128 * 128);
    const int m0 = (int)min((int64_t)M, (int64_t)rank * share), n = min(share, M - m0);
    const int t0 = F + m0;
    const int32_t *table = known_from_here(p.src_table + (int64_t)b * p.max_pages);
    __syncthreads();  // the histograms are clear
    // kBatch pages, then their weights: two latencies for kBatch * kSelThreads keys
    constexpr int kBatch = 8;
    const int nc = min(n, kKeyCap);
    const int64_t page_stride = (int64_t)p.H_kv * p.page_size;
    const float *head = p.weights + (int64_t)h * p.page_size;
    for (int i0 = 0; i0 < nc; i0 += kBatch * kSelThreads) {
        int page[kBatch], slot[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int t = t0 + min(i0 + u * kSelThreads + tid, nc - 1);
            const int pi = page_index(t, p.page_size, p.log2_page);
            slot[u] = t - pi * p.page_size;
            page[u] = ld_unwritten(table + pi);
        }
        float w[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const bool ok = (uint32_t)page[u] < (uint32_t)p.num_pages;
            w[u] = ld_unwritten(head + (ok ? page[u] : 0) * page_stride + slot[u]);
            if (!ok) slot[u] = -1;
        }
#pragma unroll
        for (int u = 0; u < kBatch; ++u) {
            const int i = i0 + u * kSelThreads + tid;
            if (i < nc) {
                uint32_t k = key_of(w[u]);
                if (slot[u] < 0) {
                    k = 0u;
                    if (p.error) atomicOr(p.error, DA_DEV_BAD_PAGE);
                }
                keys[i] = k;
                atomicAdd(&s.lanes[k >> 24][lane], 1u);
            }
        }
    }
    for (int i = nc + tid; i < n; i += kSelThreads)  // keys beyond shared memory
        atomicAdd(&s.lanes[weight_key(p, table, h, t0 + i) >> 24][lane], 1u);
    __syncthreads();
    {   // two threads a bin, each half of the lanes, starting at different ones
        const int bin = tid >> 1, half = (tid & 1) * 16;
        uint32_t c = 0;
#pragma unroll
        for (int k = 0; k < 16; ++k) c += s.lanes[bin][half + ((k + bin) & 15)];
        c += __shfl_xor_sync(0xffffffffu, c, 1);
        if (!(tid & 1)) s.hist0[bin] = c;
        static_assert(kSelThreads == 2 * kBins0, "two threads a bin");
    }
    __syncthreads();
    for (int i = tid; i < 2 * kBins / 4; i += kSelThreads)
        reinterpret_cast<uint4 *>(&s.hist[0][0])[i] = make_uint4(0u, 0u, 0u, 0u);
    __syncthreads();
    // keys i .. i + 3 (i a multiple of 4); what lies past n is not a key
    auto keys4 = [&](int i, uint32_t(&k)[4]) {
        if (i < kKeyCap) {
            const uint4 v = *reinterpret_cast<const uint4 *>(keys + i);
            k[0] = v.x, k[1] = v.y, k[2] = v.z, k[3] = v.w;
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u) k[u] = i + u < n ? weight_key(p, table, h, t0 + i + u) : 0u;
        }
    };

    // each warp has a contiguous run of this CTA's share, 128 keys at a time
    const int per = (n + kSelWarps * 128 - 1) / (kSelWarps * 128) * 128;
    const int w0 = (int)min((int64_t)n, (int64_t)warp * per), w1 = min(n, w0 + per);

    // digits of 8, 12 and 12 bits, highest first
    uint32_t prefix = 0, mask = 0, local_above = 0, at = (uint32_t)M;
    uint32_t gt_before = 0, eq_before = 0;   // tokens above / at the last kept key in the lower shares (and runs)
    bool few = false;
#pragma unroll
    for (int d = 0; d < 3; ++d) {
        const int shift = d == 0 ? 24 : d == 1 ? 12 : 0;
        const int bins = d == 0 ? kBins0 : kBins;
        uint32_t *hist = d == 0 ? s.hist0 : s.hist[d - 1];
        if (d == 2 && at <= (uint32_t)kFew) {
            // few tokens are left in the row: their keys are brought together (in any order, only counts are taken
            // from them), and each is compared with all; what is above them is counted run by run on the way
            uint32_t *own = s.hist[1], *all = kC > 1 ? own + kFew : own, *run = own + 2 * kFew;
            uint32_t *head = own + 3 * kFew;   // this CTA's count of them, and of the tokens above them
            uint32_t gt = 0;
            for (int i = w0 + 4 * lane; i < w1; i += 128) {
                uint32_t k[4];
                keys4(i, k);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const bool in = i + u < w1;
                    gt += in && (k[u] & mask) > prefix;
                    if (in && (k[u] & mask) == prefix) {
                        const uint32_t slot = atomicAdd(head, 1u);
                        own[slot] = k[u];
                        run[slot] = warp;
                    }
                }
            }
            gt = __reduce_add_sync(0xffffffffu, gt);
            if (lane == 0) s.wgt[warp] = gt;
            __syncthreads();
            uint32_t lower = 0;                          // of them, those of lower shares
            if constexpr (kC > 1) {
                if (warp == 0) {
                    gt = sum_below(s.wgt, kSelWarps, lane);
                    if (lane == 0) head[1] = gt;
                    __syncwarp();
                }
                cluster_sync_all();  // every CTA's keys and counts
                static_assert(kC <= kSelWarps, "a warp copies the keys of one rank");
                uint32_t first = 0;                      // (as if there were 32: one latency instead of two)
                if (warp < kC) first = ld_cluster_u32(mapa_shared(smem_u32(own + lane), warp));
                uint32_t count = 0, above = 0;           // lane r: rank r's
                if (lane < kC) {
                    count = ld_cluster_u32(mapa_shared(smem_u32(head), lane));
                    above = ld_cluster_u32(mapa_shared(smem_u32(head + 1), lane));
                }
                gt_before = __reduce_add_sync(0xffffffffu, lane < rank ? above : 0u);
                lower = __reduce_add_sync(0xffffffffu, lane < rank ? count : 0u);
                const uint32_t to = __reduce_add_sync(0xffffffffu, lane < warp ? count : 0u);
                const int from = __shfl_sync(0xffffffffu, count, warp);
                if (warp < kC) {
                    if (lane < from) all[to + lane] = first;
                    for (int i = lane + 32; i < from; i += 32)
                        all[to + i] = ld_cluster_u32(mapa_shared(smem_u32(own + i), warp));
                }
                __syncwarp();
                cluster_arrive_all();  // done with the other CTAs' memory; waited for before the exit
                __syncthreads();
            }
            if (tid < (int)at) {
                const uint32_t k = all[tid];
                uint32_t over = 0, same = 0;
                for (int i = 0; i < (int)at; ++i) {
                    over += all[i] > k;
                    same += all[i] == k;
                }
                if (over < want && want <= over + same) {  // (equal keys write the same)
                    s.digit = k;
                    s.above = over;
                }
            }
            __syncthreads();
            prefix = s.digit;
            want -= s.above;
            uint32_t over = 0, same = 0;
            if (kC > 1) {
                for (int i = lane; i < (int)lower; i += 32) {
                    over += all[i] > prefix;
                    same += all[i] == prefix;
                }
            }
            for (int i = lane; i < (int)head[0]; i += 32) {
                over += run[i] < warp && own[i] > prefix;
                same += run[i] < warp && own[i] == prefix;
            }
            gt_before += __reduce_add_sync(0xffffffffu, over) + sum_below(s.wgt, warp, lane);
            eq_before = __reduce_add_sync(0xffffffffu, same);
            few = true;
            break;
        }
        if (d > 0) {
            const bool crowded = at > (uint32_t)M / 2;  // most keys are in the bins found so far
            for (int i0 = 4 * (tid - lane); i0 < n; i0 += 4 * kSelThreads) {
                const int i = i0 + 4 * lane;
                uint32_t k[4] = {0u, 0u, 0u, 0u};
                if (i < n) keys4(i, k);
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const bool in = i + u < n && (k[u] & mask) == prefix;
                    const uint32_t bin = (k[u] >> shift) & (bins - 1);
                    if (crowded)
                        count_crowded(hist, bin, in, lane);
                    else if (in)
                        atomicAdd(hist + bin, 1u);
                }
            }
            __syncthreads();
        }
        // the row's counts: kPer bins a thread, from the top of the bins, or in a cluster of the slice of them that
        // holds the digit
        constexpr int kPer = kC == 1 ? 8 : 4;
        const int slice = d == 0 ? bins : bins / kC;     // (the first digit's bins are few enough for every CTA)
        const int base = slice - kPer * (tid + 1);
        uint32_t c[kPer], first_bin = 0, over = 0;       // over: tokens above the slice
#pragma unroll
        for (int i = 0; i < kPer; ++i) c[i] = 0u;
        auto put = [&](int i, uint4 q) { c[i] = q.x, c[i + 1] = q.y, c[i + 2] = q.z, c[i + 3] = q.w; };
        if constexpr (kC == 1) {
            if (base >= 0) {
                put(0, *reinterpret_cast<const uint4 *>(hist + base));
                put(kPer - 4, *reinterpret_cast<const uint4 *>(hist + base + kPer - 4));
            }
        } else if (d == 0) {
            __syncwarp();
            cluster_sync_all();  // every CTA's counts
            const int at4 = 4 * (tid & (kBins0 / 4 - 1));
            for (int r = tid / (kBins0 / 4); r < kC; r += kSelThreads / (kBins0 / 4)) {
                const uint4 x = ld_cluster_v4(mapa_shared(smem_u32(hist + at4), r));
                if (x.x) atomicAdd(s.row0 + at4, x.x);
                if (x.y) atomicAdd(s.row0 + at4 + 1, x.y);
                if (x.z) atomicAdd(s.row0 + at4 + 2, x.z);
                if (x.w) atomicAdd(s.row0 + at4 + 3, x.w);
            }
            __syncthreads();
            if (base >= 0) put(0, *reinterpret_cast<const uint4 *>(s.row0 + base));
        } else {
            __syncwarp();
            cluster_sync_all();  // every CTA's counts
            // this CTA adds up its slice of all CTAs' bins
            uint32_t sum = 0;
            if (4 * tid < slice) {
                const uint32_t a = smem_u32(hist + rank * slice + 4 * tid);
                uint4 q = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int r = 0; r < kC; ++r) {
                    const uint4 x = ld_cluster_v4(mapa_shared(a, r));
                    q.x += x.x, q.y += x.y, q.z += x.z, q.w += x.w;
                }
                *reinterpret_cast<uint4 *>(row_slice + 4 * tid) = q;
                sum = q.x + q.y + q.z + q.w;
            }
            sum = __reduce_add_sync(0xffffffffu, sum);
            if (lane == 0) s.wgt[warp] = sum;
            __syncthreads();
            if (warp == 0) {
                sum = sum_below(s.wgt, kSelWarps, lane);
                if (lane == 0) s.slice = sum;
                __syncwarp();
            }
            cluster_sync_all();  // every CTA's slice
            uint32_t all = 0, mine = 0;                  // lane r: tokens of rank r's slice, and of those above it
            if (lane < kC) mine = ld_cluster_u32(mapa_shared(smem_u32(&s.slice), lane));
#pragma unroll
            for (int r = 0; r < kC; ++r) {
                const uint32_t x = __shfl_sync(0xffffffffu, mine, r);
                all += r > lane ? x : 0u;
            }
            const int owner = __ffs(__ballot_sync(0xffffffffu, lane < kC && all < want && want <= all + mine)) - 1;
            over = __shfl_sync(0xffffffffu, all, owner);
            first_bin = owner * slice;
            if (base >= 0) put(0, ld_cluster_v4(mapa_shared(smem_u32(row_slice + base), owner)));
        }
        uint32_t mine8 = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) mine8 += c[i];
        uint32_t v = mine8;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t x = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += x;
        }
        if (lane == 31) s.warp_sum[warp] = v;
        __syncthreads();
        uint32_t above = over + sum_below(s.warp_sum, warp, lane) + v - mine8;   // tokens above this thread's bins
        if (base >= 0) {
#pragma unroll
            for (int i = kPer - 1; i >= 0; --i) {
                if (above < want && want <= above + c[i]) {
                    s.digit = first_bin + base + i;
                    s.above = above;
                    s.at = c[i];
                }
                above += c[i];
            }
        }
        __syncthreads();
        const uint32_t digit = s.digit;
        want -= s.above;
        at = s.at;
        if (kC > 1 && (d != 1 || at > (uint32_t)kFew)) {  // this CTA's tokens above the digit
            uint32_t mine = 0;
            for (int i = digit + 1 + tid; i < bins; i += kSelThreads) mine += hist[i];
            mine = __reduce_add_sync(0xffffffffu, mine);
            if (lane == 0) s.wgt[warp] = mine;
            __syncthreads();
            local_above += sum_below(s.wgt, kSelWarps, lane);
            if (d == 2 && tid == 0) {
                s.gt = local_above;
                s.eq = hist[digit];
            }
        }
        __syncthreads();  // s.digit and s.wgt are written again
        prefix |= digit << shift;
        mask |= (uint32_t)(bins - 1) << shift;
    }
    const uint32_t T = prefix;  // tokens above T are kept, and the first `want` of those at T
    if (kC > 1 && !few) {
        cluster_sync_all();  // every CTA's gt and eq
        if (lane < rank) {
            gt_before = ld_cluster_u32(mapa_shared(smem_u32(&s.gt), lane));
            eq_before = ld_cluster_u32(mapa_shared(smem_u32(&s.eq), lane));
        }
        gt_before = __reduce_add_sync(0xffffffffu, gt_before);
        eq_before = __reduce_add_sync(0xffffffffu, eq_before);
        cluster_arrive_all();  // done with the other CTAs' memory; waited for before the exit
    }
    if (!few) {
        uint32_t gt = 0, eq = 0;
        for (int i = w0 + 4 * lane; i < w1; i += 128) {
            uint32_t k[4];
            keys4(i, k);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                gt += i + u < w1 && k[u] > T;
                eq += i + u < w1 && k[u] == T;
            }
        }
        gt = __reduce_add_sync(0xffffffffu, gt);
        eq = __reduce_add_sync(0xffffffffu, eq);
        if (lane == 0) {
            s.wgt[warp] = gt;
            s.weq[warp] = eq;
        }
        __syncthreads();
        gt_before += sum_below(s.wgt, warp, lane);
        eq_before += sum_below(s.weq, warp, lane);
    }
    // the runs' kept tokens, in order
    const uint32_t below = (1u << lane) - 1u;
    for (int i0 = w0; i0 < w1; i0 += 128) {
        const int i = i0 + 4 * lane;
        uint32_t k[4] = {0u, 0u, 0u, 0u};
        if (i < w1) keys4(i, k);
        bool g[4], e[4];
        uint32_t at = gt_before, eb = eq_before;   // tokens above / at T before this lane's
        bool any_e = false;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            g[u] = i + u < w1 && k[u] > T;
            e[u] = i + u < w1 && k[u] == T;
            any_e |= e[u];
            const uint32_t m = __ballot_sync(0xffffffffu, g[u]);
            at += __popc(m & below);
            gt_before += __popc(m);
        }
        if (__any_sync(0xffffffffu, any_e)) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint32_t m = __ballot_sync(0xffffffffu, e[u]);
                eb += __popc(m & below);
                eq_before += __popc(m);
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (g[u] || (e[u] && eb < want)) kept[F + at + min(eb, want)] = F + m0 + i + u;
            at += g[u];
            eb += e[u];
        }
    }
    if (kC > 1) {
        __syncwarp();
        cluster_wait_all();
    }
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
        const int sp = st[si], dp = dt[di];
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

// Whether the current device can hold a cluster of 16 selecting CTAs (asked once per device, with the most shared
// memory that one takes).
bool wide_clusters() {
    static std::atomic<int> known[64];   // 1: no, 2: yes
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    int k = known[dev].load(std::memory_order_relaxed);
    if (!k) {
        const auto kern = evict_select_kernel<16>;
        const int smem = sel_keys_at(16) + kKeyCap * 4;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(16);
        cfg.blockDim = dim3(kSelThreads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim = {16, 1, 1};
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int n = 0;
        const bool ok = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) == cudaSuccess &&
                        cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess && n >= 1;
        if (!ok) cudaGetLastError();
        k = ok ? 2 : 1;
        known[dev].store(k, std::memory_order_relaxed);
    }
    return k == 2;
}

template <int kC>
cudaError_t launch_select(const EvictParams &p, int64_t keys, cudaStream_t stream, bool pdl) {
    const auto kern = evict_select_kernel<kC>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         sel_keys_at(kC) + kKeyCap * 4);
    if (e != cudaSuccess) return e;
    if (kC > 8 && (e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess)
        return e;
    const int smem = sel_keys_at(kC) + (int)(keys < kKeyCap ? keys : kKeyCap) * 4;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.B * p.H_kv * kC));
    cfg.blockDim = dim3(kSelThreads);
    cfg.dynamicSmemBytes = smem;
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
    // CTAs per row: as many as there are SMs for, while each still has a few thousand tokens of the longest length
    // that the block table allows
    const int64_t rows = (int64_t)p.B * p.H_kv, longest = (int64_t)p.max_pages * p.page_size;
    int c = 1;
    while (c < 16 && rows * c * 2 <= num_sms && longest / c > 4096) c *= 2;
    if (c == 16 && !wide_clusters()) c = 8;
    const int64_t share = (longest + c - 1) / c + 128;
    cudaError_t e = c == 16  ? launch_select<16>(p, share, stream, pdl)
                    : c == 8 ? launch_select<8>(p, share, stream, pdl)
                    : c == 4 ? launch_select<4>(p, share, stream, pdl)
                    : c == 2 ? launch_select<2>(p, share, stream, pdl)
                             : launch_select<1>(p, share, stream, pdl);
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
    cfg.dynamicSmemBytes = (size_t)tile * p.H_kv * 16;  // 64 KB at most (one token of 4096 heads)
    e = cudaFuncSetAttribute(evict_copy_kernel<4>, cudaFuncAttributeMaxDynamicSharedMemorySize, 64 << 10);
    if (e != cudaSuccess) return e;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, evict_copy_kernel<4>, p, (int)tile, (int)tiles);
}

}  // namespace da
