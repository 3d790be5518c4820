// The pages of a cache: forking rows, reserving room, freeing, compacting, copying.
//
// The state is a count per page (`refs`: how many table entries hold it, others
// such as a prefix cache counted too; 0: free) and, per request, the entries of the block
// table that it holds (`held`). There is no free list: a page is free because nothing
// counts it, and the lowest free pages are taken first, so that the same calls give
// the same pages. All counting is in integers; atomics change no result.
//
// fork and free touch table entries and counts only, one thread per entry.
//
// reserve and compact need all counts: one cluster of up to sixteen CTAs, each
// with a contiguous share of them, reads the counts once, keeps one bit a page in shared
// memory and learns its place among the others' pages from their totals through
// distributed shared memory. A share is cut into one run of words per warp, so that a
// page's rank is the sum over lower CTAs, lower warps, lower words and lower lanes. A single
// CTA reads 8192 counts (eight loads a lane) in one round trip; that many pages a CTA
// decides the cluster's size.
//
// copy moves whole pages as bulk copies: bound by HBM.
#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <cstdint>

#include "common.cuh"
#include "decode_attn.h"
#include "layout.h"
#include "quant.cuh"

namespace da {
namespace {

constexpr int kPlanThreads = 1024, kPlanWarps = kPlanThreads / 32;
constexpr int kBatch = 8;              // words that a warp reads at once
constexpr int kPagesPerCta = kPlanWarps * kBatch * 32;
constexpr int kFewRows = kPlanThreads, kSlots = 2 * kFewRows;  // requests with a hash table, and its places
constexpr int kForkThreads = 256, kForkColumns = 1024;
constexpr int kCopyThreads = 64, kCopyPiece = 8 << 10, kCopyStages = 8;

__device__ __forceinline__ void report(int32_t *error, int bits) {
    if (error) atomicOr(error, bits);
}
__device__ __forceinline__ bool page_ok(int page, int num_pages) { return page >= 0 && page < num_pages; }
__device__ __forceinline__ uint32_t cluster_u32(const void *local, uint32_t rank) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(local), rank)) : "memory");
    return v;
}
// all threads of the planning CTAs, and what they have written
__device__ __forceinline__ void sync_ctas(uint32_t ctas) {
    if (ctas > 1)
        cluster_sync_all();
    else
        __syncthreads();
}
__device__ __forceinline__ int warp_sum(int v) { return __reduce_add_sync(0xFFFFFFFFu, v); }

// ------------------------------------------------------------------ fork, free
// One CTA per (row, 1024 table entries). As an old row it lets its pages go, less
// those that its children take over: what n children hold of a page is counted in one
// atomic. As a new row it copies its parent's entries.
__global__ void __launch_bounds__(kForkThreads) fork_kernel(const __grid_constant__ PagesParams p, int tiles) {
    pdl_wait();
    pdl_launch_dependents();
    const int b = blockIdx.x / tiles, col0 = blockIdx.x % tiles * kForkColumns, tid = threadIdx.x;
    const auto held_of = [&](int row) { return min(max(p.held_in[row], 0), p.max_pages); };
    const auto used_of = [&](int row, int held) {
        return (int)min(((int64_t)max(p.seqlens_in[row], 0) + p.page_size - 1) / p.page_size, (int64_t)held);
    };
    // both rows are looked up before anything is written: two chains of loads under way at once
    const int parent = p.parents[b];
    const bool has = parent >= 0 && parent < p.B;
    const int held = held_of(b), used = used_of(b, held);
    const int n = has ? used_of(parent, held_of(parent)) : 0;
    const int32_t *old = p.table_in + (int64_t)b * p.max_pages;
    const int32_t *from = p.table_in + (int64_t)(has ? parent : 0) * p.max_pages;
    int32_t *to = p.table + (int64_t)b * p.max_pages;
    int mine[kForkColumns / kForkThreads], taken[kForkColumns / kForkThreads];
#pragma unroll
    for (int k = 0; k < kForkColumns / kForkThreads; ++k) {
        const int j = col0 + k * kForkThreads + tid;
        mine[k] = j < held ? old[j] : -1;
        taken[k] = j < n ? from[j] : -1;
    }
    int children = 0;
    for (int i = 0; i < p.B; i += kForkThreads)
        children += __syncthreads_count(i + tid < p.B && p.parents[i + tid] == b);
#pragma unroll
    for (int k = 0; k < kForkColumns / kForkThreads; ++k) {
        const int j = col0 + k * kForkThreads + tid;
        const int delta = (j < used ? children : 0) - 1;
        if (j < held && delta != 0) {
            if (page_ok(mine[k], p.num_pages))
                atomicAdd(p.refs + mine[k], delta);
            else
                report(p.error, DA_DEV_BAD_PAGE);
        }
        if (j < n) {
            if (!page_ok(taken[k], p.num_pages)) report(p.error, DA_DEV_BAD_PAGE);
            to[j] = taken[k];
        }
    }
    if (col0 == 0 && tid == 0) {
        const int L = has ? p.seqlens_in[parent] : 0;
        if (parent >= p.B) report(p.error, DA_DEV_BAD_REQUEST);
        if (L < 0) report(p.error, DA_DEV_NEG_LEN);
        p.held[b] = n;
        p.seqlens[b] = max(L, 0);
    }
}

// One CTA per row.
__global__ void __launch_bounds__(kForkThreads) free_kernel(const __grid_constant__ PagesParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const int b = blockIdx.x;
    if (p.done[b] == 0) return;
    const int held = min(max(p.held[b], 0), p.max_pages);
    const int32_t *row = p.table_in + (int64_t)b * p.max_pages;
    for (int j = threadIdx.x; j < held; j += kForkThreads) {
        if (page_ok(row[j], p.num_pages))
            atomicSub(p.refs + row[j], 1);
        else
            report(p.error, DA_DEV_BAD_PAGE);
    }
    __syncthreads();  // every thread has read held
    if (threadIdx.x == 0) {
        p.held[b] = 0;
        p.seqlens[b] = 0;
    }
}

// ------------------------------------------------------------------ what reserve and compact share
// A CTA's share of the pages: [first, end), as `words` bit words in shared memory.
struct Share {
    uint32_t rank, ctas;
    int first, end, words, per_warp;  // per_warp: words of a warp's run
};
__device__ __forceinline__ Share share_of(const PagesParams &p) {
    Share s;
    s.rank = cluster_ctarank();
    s.ctas = (uint32_t)p.ctas;
    const int words = p.share_words;
    s.first = (int)min((int64_t)s.rank * words * 32, (int64_t)p.num_pages);
    s.end = (int)min((int64_t)s.first + (int64_t)words * 32, (int64_t)p.num_pages);
    s.words = (s.end - s.first + 31) / 32;
    s.per_warp = (words + kPlanWarps - 1) / kPlanWarps;
    return s;
}
// bit of a page set where refs > 0 (live) or refs == 0; returns this warp's bits
template <bool kLive>
__device__ __forceinline__ int read_bits(const PagesParams &p, const Share &s, uint32_t *bits, int warp, int lane) {
    int count = 0;
    const int w1 = min((warp + 1) * s.per_warp, s.words);
    for (int w = warp * s.per_warp; w < w1; w += kBatch) {
        int v[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int page = s.first + (w + k) * 32 + lane;
            v[k] = w + k < w1 && page < s.end ? p.refs_in[page] : (kLive ? 0 : 1);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const uint32_t m = __ballot_sync(0xFFFFFFFFu, kLive ? v[k] > 0 : v[k] == 0);
            if (w + k < w1 && lane == k) bits[w + k] = m;
            count += __popc(m);
        }
    }
    __syncwarp();
    return count;
}

// ------------------------------------------------------------------ reserve
// Row by row: what is written next may not be held by anybody else. A shared last page
// with tokens on it is copied (its new page is the first of the row's fresh ones), but
// where all its holders are rows of this call that write to it, the lowest of them
// keeps it. Then room up to ceil((L + n) / P) pages.
//
// Who keeps a page: for up to 1024 requests a hash table in shared memory counts the
// writers of each page and finds the lowest. More of them settle it in `refs` itself: every
// writer takes its hold back; where nothing is left the writers put their row (as a
// negative number) with an atomic minimum, and who finds its own has the page. (Four round
// trips to L2: 6.8 us instead of 4.8 for a small pool.) The counts of free pages were taken
// before, so nothing that this does is seen as free.
//
// Fresh pages are given out 32 words at a time, a thread per page: they crowd where the pool
// is free from its front (a warp per run of words had all of them: 13 us of 512 requests'
// 24).
__global__ void __launch_bounds__(kPlanThreads, 1) reserve_kernel(const __grid_constant__ PagesParams p) {
    extern __shared__ uint32_t smem[];
    __shared__ int warp_free[kPlanWarps], warp_tmp[kPlanWarps];
    __shared__ int s_free, s_need, s_ok;
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Share s = share_of(p);
    uint32_t *bits = smem;
    int *offs = reinterpret_cast<int *>(bits + p.share_words);  // [B + 1]: fresh pages of the rows before
    int *from = offs + p.B + 1;   // [B]: first fresh entry of the row's growth; -1 - it: held entries are given back
    int *tail = from + p.B;       // [B]: the shared page that is copied, or -1
    int *slot_page = tail + p.B, *slot_writers = slot_page + kSlots, *slot_lowest = slot_writers + kSlots;  // few requests

    const int mine = read_bits<false>(p, s, bits, warp, lane);
    if (lane == 0) warp_free[warp] = mine;
    bool any_tail = false;
    const auto rows_of = [&](int b, int &L, int &need, int &held) {  // false: the row asks for nothing
        const int n = p.new_tokens ? p.new_tokens[b] : p.s_q;
        L = max(p.seqlens_in[b], 0);
        held = min(max(p.held[b], 0), p.max_pages);
        if (n <= 0 || (int64_t)L + n > (int64_t)p.max_pages * p.page_size) return false;
        need = (L + n - 1) / p.page_size + 1;
        return true;
    };
    if (s.rank == 0) {
        for (int b = tid; b < p.B; b += kPlanThreads) {
            int L, need = 0, held;
            const bool asks = rows_of(b, L, need, held);
            if (p.seqlens_in[b] < 0) report(p.error, DA_DEV_NEG_LEN);
            if (!asks && (p.new_tokens ? p.new_tokens[b] : p.s_q) > 0) report(p.error, DA_DEV_SEQ_TOO_LONG);
            int page = -1, start = held, fresh = 0;
            if (asks) {
                const int32_t *row = p.table + (int64_t)b * p.max_pages;
                const int last = L / p.page_size, first = last + (L % p.page_size != 0);
                if (first > last && last < held) {
                    page = row[last];
                    if (!page_ok(page, p.num_pages)) {
                        report(p.error, DA_DEV_BAD_PAGE);
                        page = -1;
                    } else if (p.refs[page] <= 1) {
                        page = -1;
                    }
                }
                for (int j = first; j < min(held, need); ++j)
                    if (page_ok(row[j], p.num_pages) && p.refs[row[j]] > 1) start = first;
                fresh = max(need - start, 0) + (page >= 0);
                any_tail |= page >= 0;
                if (start < held) start = -1 - start;
            }
            from[b] = start;
            tail[b] = page;
            offs[b + 1] = fresh;
        }
    }
    __syncthreads();
    if (tid == 0) {
        int n = 0;
        for (int w = 0; w < kPlanWarps; ++w) n += warp_free[w];
        s_free = n;
    }
    sync_ctas(s.ctas);  // all counts are read; every CTA's total is there
    if (s.rank == 0) {
        const bool few = p.B <= kFewRows;
        if (__syncthreads_or(any_tail)) {
            if (few) {
                for (int i = tid; i < kSlots; i += kPlanThreads) slot_page[i] = -1, slot_writers[i] = 0, slot_lowest[i] = INT_MAX;
                __syncthreads();
                const int b = tid, page = b < p.B ? tail[b] : -1;
                unsigned at = ((unsigned)page * 0x9E3779B1u) % kSlots;
                if (page >= 0) {
                    for (;; at = (at + 1) % kSlots) {  // (there are twice as many places as requests)
                        const int was = atomicCAS(slot_page + at, -1, page);
                        if (was == -1 || was == page) break;
                    }
                    atomicAdd(slot_writers + at, 1);
                    atomicMin(slot_lowest + at, b);
                }
                __syncthreads();
                if (page >= 0 && slot_lowest[at] == b && slot_writers[at] == p.refs[page]) {
                    tail[b] = -1;
                    --offs[b + 1];
                }
            } else {
                for (int b = tid; b < p.B; b += kPlanThreads)
                    if (tail[b] >= 0) atomicSub(p.refs + tail[b], 1);
                __syncthreads();
                for (int b = tid; b < p.B; b += kPlanThreads)
                    if (tail[b] >= 0 && __ldcg(p.refs + tail[b]) <= 0) atomicMin(p.refs + tail[b], INT_MIN + b);
                __syncthreads();
                for (int b = tid; b < p.B; b += kPlanThreads)
                    if (tail[b] >= 0 && __ldcg(p.refs + tail[b]) == INT_MIN + b) {
                        tail[b] = -2 - tail[b];
                        --offs[b + 1];
                    }
                __syncthreads();
                for (int b = tid; b < p.B; b += kPlanThreads)
                    if (tail[b] < -1) {
                        p.refs[-2 - tail[b]] = 1;
                        tail[b] = -1;
                    }
            }
            __syncthreads();
        }
        // prefix sum of the fresh pages
        int carry = 0;
        for (int b0 = 0; b0 < p.B; b0 += kPlanThreads) {
            const int b = b0 + tid;
            int v = b < p.B ? offs[b + 1] : 0;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int u = __shfl_up_sync(0xFFFFFFFFu, v, d);
                if (lane >= d) v += u;
            }
            if (lane == 31) warp_tmp[warp] = v;
            __syncthreads();
            const int below = warp_sum(lane < warp ? warp_tmp[lane] : 0), all = warp_sum(warp_tmp[lane]);
            if (b < p.B) offs[b + 1] = carry + below + v;
            carry += all;
            __syncthreads();
        }
        if (tid == 0) {
            int free_pages = 0;
            for (uint32_t c = 0; c < s.ctas; ++c) free_pages += (int)cluster_u32(&s_free, c);
            offs[0] = 0;
            s_need = carry;
            s_ok = carry <= free_pages;
            *p.missing = s_ok ? 0 : carry - free_pages;
            if (!s_ok) report(p.error, DA_DEV_NO_PAGES);
        }
        __syncthreads();
        const bool ok = s_ok != 0;
        for (int b = tid; b < p.B; b += kPlanThreads) {
            const int page = tail[b], f = from[b];
            reinterpret_cast<int2 *>(p.copies)[b] = make_int2(ok ? page : -1, -1);
            if (!ok) {
                if (page >= 0 && !few) atomicAdd(p.refs + page, 1);  // as it was
                continue;
            }
            if (page >= 0 && few) atomicSub(p.refs + page, 1);
            int L, need, held;
            if (!rows_of(b, L, need, held)) continue;
            const int32_t *row = p.table + (int64_t)b * p.max_pages;
            if (f < 0)  // entries behind the tokens that others hold: given back, fresh ones in their place
                for (int j = -1 - f; j < held; ++j)
                    if (page_ok(row[j], p.num_pages)) atomicSub(p.refs + row[j], 1);
            p.held[b] = f < 0 ? need : max(held, need);
        }
    }
    sync_ctas(s.ctas);  // offs, from, tail of rank 0 are final; copies are initialised
    const int want = cluster_u32(&s_ok, 0) ? (int)cluster_u32(&s_need, 0) : 0;
    int base = 0;
    for (uint32_t c = 0; c < s.rank; ++c) base += (int)cluster_u32(&s_free, c);
    if (s.rank != 0 && base < want)  // the prefix sums, for the searches below
        for (int b = tid; b <= p.B; b += kPlanThreads) offs[b] = (int)cluster_u32(offs + b, 0);
    __syncthreads();
    for (int w0 = 0; w0 < s.words && base < want; w0 += kPlanWarps) {
        const uint32_t word = w0 + lane < s.words ? bits[w0 + lane] : 0u;  // the tile's words, one a lane; this warp's is `warp`
        const int n = __popc(word);
        int incl = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int u = __shfl_up_sync(0xFFFFFFFFu, incl, d);
            if (lane >= d) incl += u;
        }
        const uint32_t m = __shfl_sync(0xFFFFFFFFu, word, warp);
        const int r = base + __shfl_sync(0xFFFFFFFFu, incl - n, warp) + __popc(m & ((1u << lane) - 1));
        base += __shfl_sync(0xFFFFFFFFu, incl, 31);
        if (!(m >> lane & 1) || r >= want) continue;
        int lo = 0, hi = p.B;  // the last row whose first fresh page is not behind r, among those that get some
        while (hi - lo > 1) {
            const int mid = (lo + hi) / 2;
            if (offs[mid] <= r)
                lo = mid;
            else
                hi = mid;
        }
        const int page = s.first + (w0 + warp) * 32 + lane;
        const int copied = (int)cluster_u32(tail + lo, 0) >= 0, f = (int)cluster_u32(from + lo, 0);
        const int k = r - offs[lo] - copied;
        int j = (f < 0 ? -1 - f : f) + k;
        if (k < 0) {
            j = max(p.seqlens_in[lo], 0) / p.page_size;
            p.copies[2 * lo + 1] = page;
        }
        p.table[(int64_t)lo * p.max_pages + j] = page;
        p.refs[page] = 1;
    }
    sync_ctas(s.ctas);  // rank 0's shared memory stays until all have read it
}

// ------------------------------------------------------------------ compact
// With N live pages, the i-th live page at or above N goes to the i-th free one below it.
__global__ void __launch_bounds__(kPlanThreads, 1) compact_kernel(const __grid_constant__ PagesParams p) {
    extern __shared__ uint32_t smem[];
    __shared__ int warp_live[kPlanWarps], warp_far[kPlanWarps], warp_gap[kPlanWarps];
    __shared__ int s_live, s_far, s_gap;
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const Share s = share_of(p);
    uint32_t *bits = smem;
    const int mine = read_bits<true>(p, s, bits, warp, lane);
    if (lane == 0) warp_live[warp] = mine;
    __syncthreads();
    if (warp == 0) {
        const int n = warp_sum(warp_live[lane]);
        if (lane == 0) s_live = n;
    }
    sync_ctas(s.ctas);
    int N = 0;
    for (uint32_t c = 0; c < s.ctas; ++c) N += (int)cluster_u32(&s_live, c);
    // live pages at or above N, and free ones below it, of this warp
    const int w0 = warp * s.per_warp, w1 = min(w0 + s.per_warp, s.words);
    const auto below_n = [&](int w) -> uint32_t {  // bits of the word's pages below N
        const int n = N - (s.first + w * 32);
        return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1;
    };
    int far = 0, gap = 0;
    for (int w = w0 + lane; w < w1; w += 32) {
        const uint32_t m = bits[w], low = below_n(w);
        far += __popc(m & ~low);
        gap += __popc(~m & low);
    }
    far = warp_sum(far);
    gap = warp_sum(gap);
    if (lane == 0) warp_far[warp] = far, warp_gap[warp] = gap;
    __syncthreads();
    if (warp == 0) {
        const int f = warp_sum(warp_far[lane]), g = warp_sum(warp_gap[lane]);
        if (lane == 0) s_far = f, s_gap = g;
    }
    sync_ctas(s.ctas);
    int moves = 0, far_at = 0, gap_at = 0;
    for (uint32_t c = 0; c < s.ctas; ++c) {
        const int f = (int)cluster_u32(&s_far, c), g = (int)cluster_u32(&s_gap, c);
        if (c < s.rank) far_at += f, gap_at += g;
        moves += f;
    }
    far_at += warp_sum(lane < warp ? warp_far[lane] : 0);
    gap_at += warp_sum(lane < warp ? warp_gap[lane] : 0);
    const uint32_t under = (1u << lane) - 1;
    for (int wb = w0; wb < w1; wb += kBatch) {
        int refs[kBatch];  // of the pages that stay
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int w = wb + k;
            refs[k] = w < w1 && (bits[w] & below_n(w)) >> lane & 1 ? p.refs_in[s.first + w * 32 + lane] : 0;
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int w = wb + k, page = s.first + w * 32 + lane;
            if (w >= w1) break;
            const uint32_t m = bits[w], low = below_n(w), f = m & ~low, g = ~m & low;
            if (page < s.end) {
                const bool live = m >> lane & 1, is_low = low >> lane & 1;
                if (!live || is_low) p.new_page[page] = live ? page : -1;  // (where a page goes that moves, and
                if (live || !is_low) p.refs[page] = is_low ? refs[k] : 0;  // the count of a gap, are written below)
                if (f >> lane & 1) p.copies[2 * (far_at + __popc(f & under))] = page;
                if (g >> lane & 1) p.copies[2 * (gap_at + __popc(g & under)) + 1] = page;
            }
            far_at += __popc(f);
            gap_at += __popc(g);
        }
    }
    if (s.rank == 0 && tid == 0) {
        p.counts[0] = N;
        p.counts[1] = moves;
    }
    sync_ctas(s.ctas);  // the pairs are complete; and no CTA's shared memory is read any more
    for (int i = (int)s.rank * kPlanThreads + tid; i < moves; i += (int)s.ctas * kPlanThreads) {
        const int2 c = __ldcg(reinterpret_cast<const int2 *>(p.copies) + i);
        p.new_page[c.x] = c.y;
        p.refs[c.y] = p.refs_in[c.x];
    }
}

// the tables, through the map that compact_kernel has left
__global__ void __launch_bounds__(kForkThreads) remap_kernel(const __grid_constant__ PagesParams p, int tiles) {
    pdl_wait();
    pdl_launch_dependents();
    const int b = blockIdx.x / tiles, col0 = blockIdx.x % tiles * kForkColumns;
    const int held = min(max(p.held_in[b], 0), p.max_pages);
    const int64_t row = (int64_t)b * p.max_pages;
#pragma unroll
    for (int k = 0; k < kForkColumns / kForkThreads; ++k) {
        const int j = col0 + k * kForkThreads + threadIdx.x;
        if (j >= held) continue;
        const int page = p.table_in[row + j];
        const bool ok = page_ok(page, p.num_pages);
        if (!ok) report(p.error, DA_DEV_BAD_PAGE);
        p.table[row + j] = ok ? p.new_page[page] : -1;
    }
}

// ------------------------------------------------------------------ copy
// Pieces of at most 8 KB, each within one page of one pool, go through shared memory as bulk
// copies, both ways asynchronous: one warp looks 32 pieces up at a time, its first lane issues their
// loads and, as they arrive, their stores, through a ring of stages. Another warp copies the pages'
// scales and weights (4-byte values). Three CTAs an SM with eight stages each: 25239 pages of 32 KB
// in 247 to 257 us, 6.4 to 6.7 TB/s or 0.95 to 0.99 of the measured copy rate (pieces of 16 KB, six stages, two CTAs: 274; 16
// bytes a thread and load, four in flight, 2048 threads an SM: 288).
__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const __grid_constant__ CopyPagesParams p) {
    extern __shared__ uint4 ring_v[];
    __shared__ uint64_t full[kCopyStages], never;  // (never: a barrier that nothing completes, in the test build)
    __shared__ uint8_t *dst_of[kCopyStages];  // where the stages' pieces go, and their sizes
    __shared__ uint32_t size_of[kCopyStages];
    pdl_wait();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int n = p.num_copies ? min(max(*p.num_copies, 0), p.max_copies) : p.max_copies;
    if (warp == 0) {
        uint8_t *ring = reinterpret_cast<uint8_t *>(ring_v);
        if (lane < kCopyStages) mbar_init(&full[lane], 1);
        if (lane == kCopyStages) mbar_init(&never, 1);
        fence_barrier_init();
        fence_proxy_async_smem();
        __syncwarp();
        const int64_t items = (int64_t)n * p.pieces, mine = items > blockIdx.x ? (items - blockIdx.x + gridDim.x - 1) / gridDim.x : 0;
        int loads = 0, stores = 0;          // of this CTA, so far (lane 0)
        bool lost = false;                  // a wait has run out: nothing more is loaded or stored
        const auto store_next = [&] {
            const int st = stores % kCopyStages;
            uint64_t *bar = &full[st];
            uint32_t phase = (stores / kCopyStages) & 1;
#ifdef DA_PAGE_TRACE
            if (p.debug_stall) bar = &never, phase = 0;
#endif
            if (lost) {
                mbar_wait_timed(&full[st], (stores / kCopyStages) & 1, 100000000ull);  // lands before the CTA exits
            } else if (mbar_wait_timed(bar, phase, p.wait_limit_ns)) {
                bulk_store(dst_of[st], ring + st * kCopyPiece, size_of[st]);
            } else {
                report(p.error, DA_DEV_TIMEOUT);
                lost = true;
                return;  // (and is waited for again, as the others)
            }
            ++stores;
        };
        for (int64_t b = 0; b < mine; b += 32) {
            const int64_t it = blockIdx.x + (b + lane) * gridDim.x;
            const uint8_t *from = nullptr;
            uint8_t *into = nullptr;
            uint32_t bytes = 0;
            if (b + lane < mine) {
                const int64_t i = it / p.pieces;
                const int piece = (int)(it - i * p.pieces);
                const int src = p.copies[2 * i], dst = p.copies[2 * i + 1];
                if (src >= 0) {
                    if (src >= p.num_pages || !page_ok(dst, p.num_pages)) {
                        if (piece == 0) report(p.error, DA_DEV_BAD_PAGE);
                    } else {
                        const bool is_v = piece >= p.k_pieces;
                        const int64_t at = (int64_t)(is_v ? piece - p.k_pieces : piece) * kCopyPiece;
                        const int64_t page_bytes = 16 * (is_v ? p.v_units : p.k_units);
                        uint8_t *pool = is_v ? p.v_pool : p.k_pool;
                        bytes = (uint32_t)min((int64_t)kCopyPiece, page_bytes - at);
                        from = pool + src * page_bytes + at;
                        into = pool + dst * page_bytes + at;
                    }
                }
            }
            unsigned todo = __ballot_sync(0xFFFFFFFFu, bytes > 0);
            while (todo) {
                const int l = __ffs(todo) - 1;
                todo &= todo - 1;
                const uint8_t *f = reinterpret_cast<const uint8_t *>(__shfl_sync(0xFFFFFFFFu, (unsigned long long)from, l));
                uint8_t *t = reinterpret_cast<uint8_t *>(__shfl_sync(0xFFFFFFFFu, (unsigned long long)into, l));
                const uint32_t z = __shfl_sync(0xFFFFFFFFu, bytes, l);
                if (lane == 0 && !lost) {
                    const int st = loads % kCopyStages;
                    // half of the ring loads, half stores
                    if (loads - stores >= kCopyStages / 2) store_next();
                    if (!lost) {
                        if (loads >= kCopyStages) bulk_wait_read<kCopyStages / 2 - 1>();
                        dst_of[st] = t;
                        size_of[st] = z;
                        mbar_arrive_expect_tx(&full[st], z);
                        bulk_load(ring + st * kCopyPiece, f, z, &full[st]);
                        ++loads;
                    }
                }
                __syncwarp();
            }
        }
        if (lane == 0) {
            while (stores < loads) store_next();
            bulk_wait_all();
        }
        return;
    }
    if (p.k_scale == nullptr && p.weights == nullptr) return;
    for (int64_t i = blockIdx.x; i < n; i += gridDim.x) {
        const int src = p.copies[2 * i], dst = p.copies[2 * i + 1];
        if (src < 0 || src >= p.num_pages || !page_ok(dst, p.num_pages)) continue;
#pragma unroll
        for (int a = 0; a < 3; ++a) {
            float *t = a == 0 ? p.k_scale : a == 1 ? p.v_scale : p.weights;
            const int len = a == 2 ? p.weight_len : p.scale_len;
            if (t == nullptr) continue;
            for (int e = threadIdx.x - 32; e < len; e += kCopyThreads - 32) t[(int64_t)dst * len + e] = t[(int64_t)src * len + e];
        }
    }
}

// Clusters of 16 CTAs: not every device has room for one (asked once per device).
bool wide_clusters() {
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    int k = known[dev].load(std::memory_order_relaxed);
    if (k == 0) {
        bool ok = true;
        for (const void *kern : {(const void *)reserve_kernel, (const void *)compact_kernel}) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(16);
            cfg.blockDim = dim3(kPlanThreads);
            cfg.dynamicSmemBytes = kPlanSmemMax;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim = {16, 1, 1};
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int n = 0;
            ok = ok && cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                 cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kPlanSmemMax) == cudaSuccess &&
                 cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess && n >= 1;
        }
        if (!ok) cudaGetLastError();
        k = ok ? 2 : 1;
        known[dev].store(k, std::memory_order_relaxed);
    }
    return k == 2;
}

template <typename... Args>
cudaError_t launch(void (*kern)(Args...), int64_t grid, int threads, size_t smem, int cluster, cudaStream_t stream,
                   bool pdl, Args... args) {
    if (grid < 1 || grid > INT32_MAX) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (cluster > 0) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim = {(unsigned)cluster, 1, 1};
        ++n;
    }
    if (pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

// the cluster's size and shares of a planning kernel
cudaError_t plan(const void *kern, PagesParams &p) {
    int c = 1;
    while (c < 16 && (int64_t)c * kPagesPerCta < p.num_pages) c *= 2;
    if (c == 16 && (p.max_cluster < 16 || !wide_clusters())) c = 8;
    p.ctas = c;
    const int64_t words = ((int64_t)p.num_pages + 31) / 32;
    p.share_words = (int)((words + c - 1) / c);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kPlanSmemMax);
    if (e == cudaSuccess && c > 8) e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    return e;
}

int tiles_of(const PagesParams &p) { return (p.max_pages + kForkColumns - 1) / kForkColumns; }

}  // namespace

cudaError_t launch_fork(const PagesParams &p, cudaStream_t stream, bool pdl) {
    const int tiles = tiles_of(p);
    return launch(fork_kernel, (int64_t)p.B * tiles, kForkThreads, 0, 0, stream, pdl, p, tiles);
}

cudaError_t launch_free(const PagesParams &p, cudaStream_t stream, bool pdl) {
    return launch(free_kernel, p.B, kForkThreads, 0, 0, stream, pdl, p);
}

cudaError_t launch_reserve(PagesParams p, cudaStream_t stream, bool pdl) {
    const cudaError_t e = plan((const void *)reserve_kernel, p);
    if (e != cudaSuccess) return e;
    const size_t smem = 4 * ((size_t)p.share_words + 3 * (size_t)p.B + 1 + (p.B <= kFewRows ? 3 * kSlots : 0));
    return launch(reserve_kernel, p.ctas, kPlanThreads, smem, p.ctas, stream, pdl, p);
}

cudaError_t launch_compact(PagesParams p, cudaStream_t stream, bool pdl) {
    cudaError_t e = plan((const void *)compact_kernel, p);
    if (e != cudaSuccess) return e;
    e = launch(compact_kernel, p.ctas, kPlanThreads, 4 * (size_t)p.share_words, p.ctas, stream, pdl, p);
    if (e != cudaSuccess) return e;
    const int tiles = tiles_of(p);
    return launch(remap_kernel, (int64_t)p.B * tiles, kForkThreads, 0, 0, stream, pdl, p, tiles);
}

cudaError_t launch_copy_pages(CopyPagesParams p, int num_sms, cudaStream_t stream, bool pdl) {
    const int64_t kp = (p.k_units * 16 + kCopyPiece - 1) / kCopyPiece, vp = (p.v_units * 16 + kCopyPiece - 1) / kCopyPiece;
    if (kp + vp > INT32_MAX) return cudaErrorInvalidConfiguration;
    p.k_pieces = (int)kp;
    p.pieces = (int)(kp + vp);
    const int64_t items = (int64_t)p.max_copies * p.pieces, most = (int64_t)num_sms * 3;
    const cudaError_t e = cudaFuncSetAttribute(copy_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kCopyStages * kCopyPiece);
    if (e != cudaSuccess) return e;
    return launch(copy_kernel, items < most ? items : most, kCopyThreads, kCopyStages * kCopyPiece, 0, stream, pdl, p);
}

}  // namespace da
