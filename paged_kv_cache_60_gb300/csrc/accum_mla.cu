// Attention weight gathered by cached tokens, on the 656-byte latent format.
//
// The sum of accum.cu with one KV head, G = 128 query heads and 576 dims, of
// which 512 are e4m3 with a scale per 128 (dequantised as the attention kernel
// does: bf16(fp32(e4m3) * scale)) and 64 bf16.
//
// 147 thousand floating-point operations a token and query token against 656
// bytes: HBM and the bf16 tensor peak would take about the same time, so the
// products run on the 5th-generation tensor cores, as
//     S = K Q^T      M = 128 tokens, N = 128 heads, K = 576 dims: 36 MMAs,
// with the tokens as rows: a token's scores then lie in one lane of tensor
// memory, and the sum over its heads is one thread's. K is read once and needed
// once, so it never becomes a shared-memory operand: raw rows come in by bulk
// copies (whole runs of a page), are dequantised by the thread that has the
// token's lane and stored to tensor memory as the A operand, in pieces of 64
// dims. The 128 query rows of one query token stay in shared memory as B (147 KB)
// for a whole pass; several query tokens take one pass over the tokens each.
//
// Roles (512 threads): warp 0 issues MMAs and owns the tensor memory; warp 1
// copies rows, 32 tokens (a quarter of a unit of 128) at a time into the
// quarter's buffer; warps 4-7 sum the exponentials of a finished S and update the
// weights; warps 8-15 dequantise, two to a quarter, each one half of the dims:
// a warp takes its part of the rows into registers, hands the buffer back, and
// converts while the next rows arrive. Operand slots are a ring of four, each
// with a piece of either half, and S has two buffers.
//
// Measured on 32 caches of 4 to 128 thousand tokens (997 thousand in all, 97 us
// from HBM at 6.8 TB/s): 148 us, 1003 TFLOP/s, where warp-level products on
// dequantised tiles in shared memory took 454 us. The three roles run different
// code at the same time and each SM has few warps to hide a fetch of
// instructions behind, so their loops are kept short: unrolled fully they took
// 280 us, rolled as they are below 171. The warp that issues is the next bound:
// with a barrier and a commit to every piece of a half instead of every pair of
// pieces it took 171 us.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "decode_attn.h"
#include "layout.h"
#include "segwalk.cuh"

namespace da {
namespace {

constexpr int kThreads = 512;
constexpr int kHeads = 128, kDim = 576;
constexpr int kRow = 656, kScaleAt = 512, kRopeAt = 528;
constexpr int kUnit = 128, kQuarter = 32;            // tokens
constexpr int kQSlice = kHeads * 128;                // 64 dims of the query rows, 128-byte swizzle: 16 KB
constexpr int kItems = 5;                            // operand pieces of a half per unit: four of 64 dims, one of 32
constexpr int kSlots = 4;                            // operand slots, each with a piece of either half
constexpr int kOffRaw = 9 * kQSlice;
constexpr int kOffLse = kOffRaw + 4 * kQuarter * kRow;
constexpr int kOffBars = kOffLse + kHeads * 4;
constexpr int kBars = 4 + 4 + 2 * kSlots + 2 + 2 + 1;
constexpr int kOffTmem = kOffBars + kBars * 8;
constexpr int kSmem = kOffTmem + 16;                 // no slack: the base has to be 1024-byte aligned, see below
static_assert(kSmem <= 232448, "shared memory budget");
static_assert(kOffRaw % 1024 == 0 && kOffBars % 8 == 0, "alignment");
// tensor memory (512 columns x 128 lanes; lane = token of the unit): S twice, then the operand slots (32 columns each)
constexpr uint32_t kTmemCols = 512, kACol = 256;

struct Bars {
    uint64_t *rfull, *rempty;    // [quarter] raw rows
    uint64_t *afull, *aempty;    // [slot] operand pieces, both halves'
    uint64_t *sfull, *sempty;    // [2] scores
    uint64_t *drain;
};
__device__ __forceinline__ Bars bars_at(uint8_t *smem) {
    uint64_t *b = reinterpret_cast<uint64_t *>(smem + kOffBars);
    return Bars{b, b + 4, b + 8, b + 8 + kSlots, b + 8 + 2 * kSlots, b + 10 + 2 * kSlots, b + 12 + 2 * kSlots};
}

// Untiled bulk copy of `bytes` (a multiple of 16) into shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
            smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

// 16 e4m3 values times the scale, as 16 bf16 in eight words.
__device__ __forceinline__ void dequant16(uint4 v, float scale, uint32_t *o) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t lo = e4m3x2_to_f16x2((uint16_t)(w[k] & 0xFFFFu)), hi = e4m3x2_to_f16x2((uint16_t)(w[k] >> 16));
        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
        const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
        o[2 * k] = pack_bf16(__fmul_rn(a.x, scale), __fmul_rn(a.y, scale));
        o[2 * k + 1] = pack_bf16(__fmul_rn(b.x, scale), __fmul_rn(b.y, scale));
    }
}

template <bool B>
struct Bool {
    static constexpr bool value = B;
};

// One pass: query token j of a segment over its tokens. Units are dealt out to the CTAs of a part.
struct Pass {
    int b, L, j, nj;
    int base, end;      // tokens [base, end)
    int units;          // units of 128 of them that are this CTA's: u = z + Z k
};

__global__ void __launch_bounds__(kThreads, 1) accum_mla_kernel(const __grid_constant__ AccumParams p) {
    extern __shared__ __align__(1024) uint8_t smem[];
    const Bars bar = bars_at(smem);
    float *lse2 = reinterpret_cast<float *>(smem + kOffLse);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + kOffTmem);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + kOffTmem + 4);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, quad = warp & 3;
    const int Z = gridDim.z, z = blockIdx.z;
    const int part0 = blockIdx.x * p.parts_per_cta, part1 = min(part0 + p.parts_per_cta, p.num_parts);

    const int P = p.page_size, bt = min(P, kQuarter), nb = kQuarter / bt;   // tokens of a copy, copies of a quarter
    if (tid == 0) {
        for (int i = 0; i < 4; ++i) {
            mbar_init(&bar.rfull[i], nb);
            mbar_init(&bar.rempty[i], 2);
        }
        for (int i = 0; i < kSlots; ++i) {
            mbar_init(&bar.afull[i], 8);
            mbar_init(&bar.aempty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bar.sfull[i], 1);
            mbar_init(&bar.sempty[i], 4);
        }
        mbar_init(bar.drain, 1);
        *abort_flag = 0;
#ifdef DA_PAGE_TRACE
        mbar_init(reinterpret_cast<uint64_t *>(smem + kOffTmem + 8), 1);  // never arrived at
#endif
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if (warp == 0) tmem_alloc(tmem_slot, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    pdl_launch_dependents();

    const bool meta_ok =
        meta_header_ok(load_meta_header(p.meta.header), p.B, p.H_kv, p.G, p.splits, p.num_parts, p.s_q, 0, 0);
    // the query tiles' swizzle needs a 1024-byte aligned base (the declaration asks for it, and dynamic shared memory
    // without static starts there; were it not so, the call would do nothing and report a wait that ran out)
    const bool aligned = (smem_u32(smem) & 1023u) == 0;
    if (tid == 0 && !meta_ok) atomicOr(&p.meta.header[kHError], DA_DEV_META_MISMATCH);
    if (tid == 0 && !aligned) atomicOr(&p.meta.header[kHError], DA_DEV_TIMEOUT);
    const int max_len = p.max_pages * P;
    // every thread walks the same passes
    int part = part0 - 1;
    bool open = false;   // wk holds a part
    SegWalker wk;
    Seg sg;
    Pass ps;
    ps.j = ps.nj = 0;
    const auto next_pass = [&]() -> bool {
        if (ps.j + 1 < ps.nj) {
            ++ps.j;
            return true;
        }
        for (;;) {
            while (!open || !wk.next(sg)) {
                if (++part >= part1) return false;
                wk = make_walker(p.meta, p.meta.parts[2 * part], p.meta.parts[2 * part + 1], p.B, p.seqlens, max_len,
                                 p.s_q, 0, 0);
                open = true;
            }
            ps.base = sg.lc0 * kChunk;
            ps.end = min(sg.lc1 * kChunk, sg.L);
            const int all = (ps.end - ps.base + kUnit - 1) / kUnit;
            ps.units = all > z ? (all - z + Z - 1) / Z : 0;
            if (ps.units > 0) break;
        }
        ps.b = sg.b;
        ps.L = sg.L;
        ps.j = 0;
        // query tokens that count; where none does, one pass all the same, for the decay
        ps.nj = p.accepted ? min(p.accepted[ps.b], p.s_q - 1) + 1 : p.s_q;
        return true;
    };
    const auto unit_base = [&](int k) { return ps.base + (z + k * Z) * kUnit; };

    bool ok = true;
    int done = 0, pass = 0;         // units and passes so far
    const auto give_up = [&]() {
        if (lane == 0) {
            atomicOr(&p.meta.header[kHError], DA_DEV_TIMEOUT);
            *abort_flag = 1;
        }
        ok = false;
    };
    const auto wait = [&](uint64_t *b, uint32_t parity) -> bool {
        if (ok && !mbar_wait_warp_ool(b, parity, abort_flag, p.wait_limit_ns)) give_up();
        return ok;
    };
    int issued = 0;                 // producer: quarters whose copies this lane has issued
    const uint64_t pol = policy_evict_first();
    const uint64_t dq = umma_desc(smem_u32(smem), 16, 1024);
    constexpr uint32_t kIdesc = umma_idesc_bf16(128, 128, 0, 0);
    const uint32_t trow = tmem + ((uint32_t)(32 * quad) << 16);

    while (meta_ok && aligned && next_pass()) {
        // all roles are done with the last pass (the MMA warp has seen its products complete)
        if (__syncthreads_or(*abort_flag != 0)) break;
        {
            const size_t row0 = ((size_t)ps.b * p.s_q + ps.j) * kHeads;
            const uint4 *q = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.q) + row0 * kDim);
            for (int i = tid; i < kHeads * (kDim / 8); i += kThreads) {
                const int head = i / (kDim / 8), c = i - head * (kDim / 8);
                *reinterpret_cast<uint4 *>(smem + (c >> 3) * kQSlice + head * 128 + (((c & 7) ^ (head & 7)) << 4)) = q[i];
            }
            if (tid < kHeads) {
                const float l = p.lse[row0 + tid];
                lse2[tid] = l == -INFINITY || ps.j >= ps.nj ? INFINITY : l * 1.4426950408889634f;
            }
        }
        fence_proxy_async_smem();
        __syncthreads();
        const int32_t *table = p.block_table + (size_t)ps.b * p.max_pages;
        const auto page_at = [&](int t) -> int {
            return t < ps.end ? ld_unwritten(table + (p.log2_page >= 0 ? t >> p.log2_page : t / P)) : -2;
        };
        const auto slot_at = [&](int t) { return p.log2_page >= 0 ? t & (P - 1) : t % P; };
        if (warp == 0) {
            // -------------------------------------------------------- MMA issuer
            int m = done * kItems;
            for (int k = 0; k < ps.units && ok; ++k) {
                const int n = done + k, d = n & 1;
                if (!wait(&bar.sempty[d], ((n >> 1) & 1) ^ 1)) break;
                tc_fence_after();
                const uint32_t acc = tmem + 128 * d;
#pragma unroll 1
                for (int o = 0; o < kItems; ++o, ++m) {
                    const int slot = m & (kSlots - 1);
                    if (!wait(&bar.afull[slot], (uint32_t)(m / kSlots) & 1u)) break;
                    tc_fence_after();
                    const uint32_t a0 = tmem + kACol + 32 * slot, a1 = a0 + 32 * kSlots;
                    const uint64_t b0 = dq + (uint64_t)((o < 4 ? o : 8) * (kQSlice >> 4));
                    const uint64_t b1 = b0 + (uint64_t)(o < 4 ? 4 * (kQSlice >> 4) : 4);
                    umma_bf16_tmem_a_w(acc, a0, b0, kIdesc, o > 0);
                    umma_bf16_tmem_a_w(acc, a0 + 8, b0 + 2, kIdesc, true);
                    umma_bf16_tmem_a_w(acc, a1, b1, kIdesc, true);
                    umma_bf16_tmem_a_w(acc, a1 + 8, b1 + 2, kIdesc, true);
                    if (o < 4) {
                        umma_bf16_tmem_a_w(acc, a0 + 16, b0 + 4, kIdesc, true);
                        umma_bf16_tmem_a_w(acc, a0 + 24, b0 + 6, kIdesc, true);
                        umma_bf16_tmem_a_w(acc, a1 + 16, b1 + 4, kIdesc, true);
                        umma_bf16_tmem_a_w(acc, a1 + 24, b1 + 6, kIdesc, true);
                    }
                    umma_commit_w(&bar.aempty[slot]);
                }
                if (ok) umma_commit_w(&bar.sfull[d]);
            }
            // every product has read its operands before the query rows are replaced or the tensor memory goes away
            umma_commit_w(bar.drain);
            // (the limit of every other wait, and where a test shortens that, time enough for the products all the same)
            if (!mbar_wait_timed(bar.drain, (uint32_t)pass & 1u, max(p.wait_limit_ns, (uint64_t)100000000))) give_up();
        } else if (warp == 1) {
            // -------------------------------------------------------- rows into the quarters' buffers
            if (lane < nb) {
                int id[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) id[c] = page_at(unit_base(0) + c * kQuarter + lane * bt);
                for (int k = 0; k < ps.units && ok; ++k) {
                    const int n = done + k;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        int pg = id[c];
                        const int t = unit_base(k) + c * kQuarter + lane * bt;
                        if (k + 1 < ps.units) id[c] = page_at(unit_base(k + 1) + c * kQuarter + lane * bt);
                        if (!mbar_wait_bounded(&bar.rempty[c], ((uint32_t)n & 1u) ^ 1u, abort_flag, p.wait_limit_ns)) {
                            atomicOr(&p.meta.header[kHError], DA_DEV_TIMEOUT);
                            *abort_flag = 1;
                            ok = false;
                            break;
                        }
                        if (pg != -2 && (uint32_t)pg >= (uint32_t)p.num_pages) {
                            atomicOr(&p.meta.header[kHError], DA_DEV_BAD_PAGE);
                            p.meta.header[kHErrorDetail] = pg;
                            pg = -2;  // skipped: its rows keep stale bytes, its weights stay
                        }
                        mbar_arrive_expect_tx(&bar.rfull[c], pg < 0 ? 0u : (uint32_t)(bt * kRow));
                        if (pg >= 0)
                            bulk_load(smem + kOffRaw + (c * kQuarter + lane * bt) * kRow,
                                      p.k_pool + ((size_t)pg * P + slot_at(t)) * kRow, (uint32_t)(bt * kRow),
                                      &bar.rfull[c], pol);
                        ++issued;
                    }
                }
            }
            __syncwarp();
        } else if (warp >= 4 && warp < 8) {
            // -------------------------------------------------------- sums and weights: one token a thread
            const int own = quad * 32 + lane;
            const int last = ps.L - p.s_q + ps.j;    // last token that query token j sees
            const int wl = p.weighted ? p.weighted[ps.b] : ps.L;
            const auto weight_at = [&](int t, int pg) -> float * {
                return (uint32_t)pg < (uint32_t)p.num_pages ? p.weights + (size_t)pg * P + slot_at(t) : nullptr;
            };
            const auto old_at = [&](int t, const float *w) -> float {
                return !w ? 0.f : ps.j > 0 ? *w : t < wl ? *w * p.decay : 0.f;   // later passes add to the first
            };
            bool off = false;                        // some head adds nothing
            for (int h = lane; h < kHeads; h += 32) off |= lse2[h] == INFINITY;
            off = __any_sync(0xffffffffu, off);
            int pg = page_at(unit_base(0) + own);
            for (int k = 0; k < ps.units && ok; ++k) {
                const int n = done + k, d = n & 1, t = unit_base(k) + own;
                float *w = weight_at(t, pg);
                const float old = old_at(t, w);
                if (k + 1 < ps.units) pg = page_at(unit_base(k + 1) + own);
#ifdef DA_PAGE_TRACE
                // test build: a wait on a barrier that nothing completes runs out
                if (p.debug_stall && !wait(reinterpret_cast<uint64_t *>(smem + kOffTmem + 8), 0)) break;
#endif
                if (!wait(&bar.sfull[d], (uint32_t)(n >> 1) & 1u)) break;
                tc_fence_after();
                float sum[4] = {0.f, 0.f, 0.f, 0.f};
                const auto part_sum = [&](auto guard, const uint32_t (&s)[16], int c) {
#pragma unroll
                    for (int h = 0; h < 16; h += 4) {
                        const float4 l = *reinterpret_cast<const float4 *>(lse2 + c + h);
                        const float ls[4] = {l.x, l.y, l.z, l.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float e = ex2(fmaf(__uint_as_float(s[h + i]), p.scale_log2, -ls[i]));
                            sum[i] += guard.value && ls[i] == INFINITY ? 0.f : e;   // whatever the score
                        }
                    }
                };
                const auto all_heads = [&](auto guard) {
#pragma unroll 1
                    for (int c = 0; c < kHeads; c += 32) {
                        uint32_t s0[16], s1[16];
                        tmem_ld16_sync(trow + 128 * d + c, s0);
                        tmem_ld16_sync(trow + 128 * d + c + 16, s1);
                        part_sum(guard, s0, c);
                        part_sum(guard, s1, c + 16);
                    }
                };
                if (off)
                    all_heads(Bool<true>{});
                else
                    all_heads(Bool<false>{});
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.sempty[d]);
                const float add = t <= last ? (sum[0] + sum[1]) + (sum[2] + sum[3]) : 0.f;
                if (w) *w = old + add;
            }
        } else if (warp >= 8) {
            // -------------------------------------------------------- dequantise: one token a thread, half of its dims
            const int half = (warp - 8) >> 2;
            const uint8_t *row = smem + kOffRaw + (quad * kQuarter + lane) * kRow;
            for (int k = 0; k < ps.units && ok; ++k) {
                const int n = done + k;
                if (!wait(&bar.rfull[quad], (uint32_t)n & 1u)) break;
                uint4 v[16], r[4];
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = *reinterpret_cast<const uint4 *>(row + half * 256 + 16 * i);
#pragma unroll
                for (int i = 0; i < 4; ++i) r[i] = *reinterpret_cast<const uint4 *>(row + kRopeAt + half * 64 + 16 * i);
                const float2 sc = *reinterpret_cast<const float2 *>(row + kScaleAt + 8 * half);
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.rempty[quad]);
                int m = n * kItems;
                const auto at = [&]() -> uint32_t {   // operand columns of piece m, once they are free
                    const int slot = m & (kSlots - 1);
                    wait(&bar.aempty[slot], ((uint32_t)(m / kSlots) & 1u) ^ 1u);
                    tc_fence_after();
                    return trow + kACol + 32 * (half * kSlots + slot);
                };
                const auto full = [&]() {
                    tmem_wait_st();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.afull[m & (kSlots - 1)]);
                    ++m;
                };
#pragma unroll 1   // two pieces' code, see above; a roll of one moves registers too often (171 -> 189 us)
                for (int o = 0; o < 4 && ok; o += 2) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t to = at();
                        if (!ok) break;
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t x[16];
                            dequant16(v[4 * e + 2 * i], o < 2 ? sc.x : sc.y, x);
                            dequant16(v[4 * e + 2 * i + 1], o < 2 ? sc.x : sc.y, x + 8);
                            tmem_st16(to + 16 * i, x);
                        }
                        full();
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) v[i] = v[i + 8];
                }
                const uint32_t to = at();
                if (!ok) break;
                uint32_t x[16];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[4 * i] = r[i].x, x[4 * i + 1] = r[i].y, x[4 * i + 2] = r[i].z, x[4 * i + 3] = r[i].w;
                tmem_st16(to, x);
                full();
            }
        }
        done += ps.units;
        ++pass;
    }
    __syncthreads();
    if (*abort_flag && warp == 1 && lane < nb) {
        // copies that were issued land before the CTA exits: at most one a quarter is in flight
        for (int c = 0; c < 4; ++c) {
            const int mine = (issued + 3 - c) / 4;   // copies of quarter c
            if (mine) mbar_wait_timed(&bar.rfull[c], (uint32_t)(mine - 1) & 1u, 100000000ull);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, kTmemCols);
}

}  // namespace

cudaError_t launch_accum_mla(AccumParams p, int num_sms, cudaStream_t stream, bool pdl) {
    cudaError_t e = cudaFuncSetAttribute(accum_mla_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    // one CTA per SM: several to a part where there are fewer parts, several parts to one where there are more
    int64_t z = (int64_t)num_sms / p.num_parts;
    z = z < 1 ? 1 : z > 8 ? 8 : z;
    p.parts_per_cta = (p.num_parts + num_sms - 1) / num_sms;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)((p.num_parts + p.parts_per_cta - 1) / p.parts_per_cta), 1, (unsigned)z);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, accum_mla_kernel, p);
}

}  // namespace da
