// Attention weight gathered by cached tokens.
//
// After a decode step, for every cached token t of request b and KV head h,
//     w[t] <- (decay w[t], or 0 for a token that has none yet)
//             + sum_j sum_g exp(sigma q_{j,g} . k_t - lse_{j,g})
// over the query tokens j of the step that count and see t, and the G query
// heads of h: the softmax weights of the step's attention call, from its lse.
//
// Bound by HBM: K is read once (V is not needed), w read and written once.
// The kernel has the attention kernel's shape without its V half: it walks the
// parts of the scheduling metadata in 64-token chunks, a producer warp brings
// K pages into a ring of shared-memory stages with one TMA copy per page, and
// every consumer warp takes whole chunks, round robin, as four 16-token tiles
// on the M side of a warp MMA with the 8 query heads as N. The lse is final, so
// a tile's exponentials are the weights themselves: there is no running
// maximum, no state between chunks and nothing to merge, and the warps of all
// CTAs write disjoint tokens. Where the metadata has fewer (part, head) pairs
// than the GPU has room for (a short fixed split), several CTAs share a pair's
// chunks.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "decode_attn.h"
#include "layout.h"
#include "segwalk.cuh"

namespace da {
namespace {

// NQ: query tokens held in registers. HP: KV heads of a CTA (neighbours, whose rows lie side by side).
template <int D, bool FP8, int NQ, int HP>
struct AccumCfg {
    static constexpr int ROW = D * (FP8 ? 1 : 2);      // bytes of one token's head
    static constexpr int SROW = ROW * HP;              // bytes of one token in a stage
    static constexpr int NX = SROW / 128;
    static constexpr int KS = D / 16;                  // MMA steps
    static constexpr int STAGE = kChunk * SROW;
    // Consumer warps, and stages (a multiple, so that a stage always belongs to one warp): 192 KB in flight on an SM. A
    // producer warp issues a chunk in about 0.35 us, which 16 KB chunks hide behind HBM; the builds with 8 KB chunks
    // take two CTAs, and so two producers, per SM, with five consumer warps each for four query tokens: twelve warps on
    // an SM leave a thread 168 registers. Rows of 128 bytes are best taken two heads at a time: the CTAs of
    // the heads drift apart, and DRAM then sees 128-byte reads 128 H_kv bytes apart (64 x 32768 e4m3 tokens of 4 heads,
    // three pools in turn: 181 us against 212 with one head to a CTA).
    static constexpr int NCW = HP == 2 ? 12 : NQ < 4 ? 6 : SROW == 128 ? 5 : 7;
    static constexpr int NS = HP == 2 ? NCW : 2 * NCW;
    static constexpr int MIN_BLOCKS = SROW == 128 ? 2 : 1;
    static constexpr int THREADS = (NCW + 1) * 32;
    static constexpr int OFF_BAR = NS * STAGE;
    static constexpr int OFF_FLAG = OFF_BAR + 2 * NS * 8;
    static constexpr int SMEM = OFF_FLAG + 16 + 1024;  // + alignment slack
};

template <int D, bool FP8, int NQ, int HP>
__global__ void __launch_bounds__(AccumCfg<D, FP8, NQ, HP>::THREADS, AccumCfg<D, FP8, NQ, HP>::MIN_BLOCKS)
    accum_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ AccumParams p) {
    using C = AccumCfg<D, FP8, NQ, HP>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *empty = full + C::NS;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_FLAG);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = blockIdx.y * HP, Z = gridDim.z;   // (first of) this CTA's KV head(s)
    // this CTA's parts, one after the other through the same ring
    const int part0 = blockIdx.x * p.parts_per_cta, part1 = min(part0 + p.parts_per_cta, p.num_parts);

    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NS; ++i) {
            mbar_init(&full[i], p.boxes_per_chunk);  // one arrival per producer lane
            mbar_init(&empty[i], 1);
        }
        *abort_flag = 0;
#ifdef DA_PAGE_TRACE
        mbar_init(reinterpret_cast<uint64_t *>(smem + C::OFF_FLAG + 8), 1);  // never arrived at
#endif
        fence_barrier_init();
        fence_proxy_async_smem();
    }
    if (warp == C::NCW && lane == 0) prefetch_tmap(&tm_k);
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();

    // the next part's record is loaded while this one is worked on
    int4 rec0 = p.meta.parts[2 * part0];
    int4 rec1 = p.meta.parts[2 * part0 + 1];
    {
        if (!meta_header_ok(load_meta_header(p.meta.header), p.B, p.H_kv, p.G, p.splits, p.num_parts, p.s_q, 0, 0)) {
            if (threadIdx.x == 0) atomicOr(&p.meta.header[kHError], DA_DEV_META_MISMATCH);
            return;
        }
    }
    const int max_len = p.max_pages * p.page_size;
    // this CTA's chunks of a segment: lc0 + (z - lc0) mod Z, then every Z-th
    const auto first_chunk = [&](int lc0) { return lc0 + (int)(((int)blockIdx.z + Z - lc0 % Z) % Z); };
    SegWalker wk;
    int part = part0 - 1;
    const auto enter = [&]() {
        ++part;
        wk = make_walker(p.meta, rec0, rec1, p.B, p.seqlens, max_len, p.s_q, 0, 0);
        if (part + 1 < part1) {
            rec0 = p.meta.parts[2 * part + 2];
            rec1 = p.meta.parts[2 * part + 3];
        }
    };
    Seg sg;
    const auto next_segment = [&]() -> bool {
        for (;;) {
            if (wk.next(sg)) return true;
            if (part + 1 >= part1) return false;
            enter();
        }
    };
    enter();
    int i = 0;  // this CTA's chunks so far

    if (warp == C::NCW) {
        // ------------------------------------------------------------ producer
        // Lane j < boxes_per_chunk owns box j of every chunk and keeps the page ids of its next four chunks in
        // registers, loaded four chunks ahead.
        const int nb = p.boxes_per_chunk, bt = p.box_tokens, P = p.page_size;
        if (lane >= nb) return;
        const uint64_t pol = policy_evict_first();
        const uint32_t box_bytes = (uint32_t)bt * C::SROW;
        bool aborted = false;
        while (!aborted && next_segment()) {
            const int32_t *table = p.block_table + (size_t)sg.b * p.max_pages;
            auto id_of = [&](int lc) -> int {
                const int tok = lc * kChunk + lane * bt;
                return (lc < sg.lc1 && tok < sg.L) ? table[tok / P] : -2;
            };
            const int lcf = first_chunk(sg.lc0);
            int ring[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) ring[k] = id_of(lcf + k * Z);
            for (int lc = lcf; lc < sg.lc1 && !aborted; lc += 4 * Z) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int c = lc + k * Z;
                    if (c >= sg.lc1) break;
                    int pg = ring[k];
                    ring[k] = id_of(c + 4 * Z);
                    const int stage = i % C::NS;
                    if (!mbar_wait_bounded(&empty[stage], ((i / C::NS) & 1) ^ 1, abort_flag, p.wait_limit_ns)) {
                        atomicOr(&p.meta.header[kHError], DA_DEV_TIMEOUT);
                        *abort_flag = 1;
                        aborted = true;
                        break;
                    }
                    if (pg != -2 && (pg < 0 || pg >= p.num_pages)) {
                        atomicOr(&p.meta.header[kHError], DA_DEV_BAD_PAGE);
                        p.meta.header[kHErrorDetail] = pg;
                        pg = -2;  // skipped: its rows keep stale bytes, its weights stay
                    }
                    mbar_arrive_expect_tx(&full[stage], pg < 0 ? 0u : box_bytes);
                    if (pg >= 0) {
                        const int tok = c * kChunk + lane * bt;
                        const int in_page = (P > kChunk) ? (tok % P) : 0;
                        tma_load_4d(smem + (size_t)stage * C::STAGE + lane * box_bytes, &tm_k, &full[stage], 0, 0, h,
                                    pg * P + in_page, pol);
                    }
                    ++i;
                }
            }
        }
        // Copies in flight land before the CTA exits, whoever gives up (ignoring the abort flag): a consumer may after
        // this warp has issued its last copy. Where nobody does, the consumers wait for the same copies.
        for (int k = max(0, i - C::NS); k < i; ++k)
            mbar_wait_timed(&full[k % C::NS], (k / C::NS) & 1, 100000000ull);
        return;
    }

    // ---------------------------------------------------------------- consumers
    const int r8 = lane >> 2, c4 = lane & 3, lrow = lane & 7, lmat = lane >> 3;
    float sl2[HP];
#pragma unroll
    for (int e = 0; e < HP; ++e) sl2[e] = p.scale_log2 * (FP8 ? p.k_scale[h + e] : 1.f);
    // tokens whose weights this lane updates: 16 c4 + r8 of a chunk, and the eighth one after it
    const int own = 16 * c4 + r8;
    while (next_segment()) {
        const int b = sg.b, L = sg.L;
        const int lcf = first_chunk(sg.lc0);
        const int n = lcf < sg.lc1 ? (sg.lc1 - lcf + Z - 1) / Z : 0;   // this CTA's chunks of the segment
        // the first of them that is this warp's
        const int skip = (warp + C::NCW - i % C::NCW) % C::NCW;
        if (skip >= n) {
            i += n;
            continue;
        }
        // q: B fragments, n = query head r8; lse of the two heads whose scores this lane gets
        uint32_t qf[HP][C::KS][NQ][2];
        float lse2[HP][NQ][2];
        int last[HP][NQ][2];  // last token that query token j sees, -1 for a head that adds nothing
        const int nj = p.accepted ? min(p.accepted[b], p.s_q - 1) + 1 : p.s_q;  // query tokens that count
        const int wl = p.weighted ? p.weighted[b] : L;
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            const bool on = j < nj;
#pragma unroll
            for (int e = 0; e < HP; ++e) {
                lse2[e][j][0] = lse2[e][j][1] = 0.f;
                last[e][j][0] = last[e][j][1] = -1;
#pragma unroll
                for (int ks = 0; ks < C::KS; ++ks) qf[e][ks][j][0] = qf[e][ks][j][1] = 0u;
                if (!on) continue;
                const size_t head0 = ((size_t)b * p.s_q + j) * p.H_q + (size_t)(h + e) * 8;
                const float2 ls = *reinterpret_cast<const float2 *>(p.lse + head0 + 2 * c4);
                constexpr float kLog2e = 1.4426950408889634f;
                lse2[e][j][0] = ls.x * kLog2e;
                lse2[e][j][1] = ls.y * kLog2e;
                last[e][j][0] = ls.x == -INFINITY ? -1 : L - p.s_q + j;
                last[e][j][1] = ls.y == -INFINITY ? -1 : L - p.s_q + j;
                const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) + (head0 + r8) * D;
                if constexpr (!FP8) {
                    const uint32_t *q32 = reinterpret_cast<const uint32_t *>(q);
#pragma unroll
                    for (int ks = 0; ks < C::KS; ++ks) {
                        qf[e][ks][j][0] = q32[ks * 8 + c4];
                        qf[e][ks][j][1] = q32[ks * 8 + 4 + c4];
                    }
                } else {
#pragma unroll
                    for (int ks = 0; ks < C::KS; ++ks) {
                        const uint2 v = *reinterpret_cast<const uint2 *>(q + ks * 16 + c4 * 4);
                        qf[e][ks][j][0] = pack_f16(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u));
                        qf[e][ks][j][1] = pack_f16(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u));
                    }
                }
            }
        }
        const int i1 = i + n;
        int c = lcf + skip * Z;
        // the weights that this lane updates, loaded a chunk ahead of their use, their pages two: they come from DRAM
        // (217 -> 212 us on the largest e4m3 workload, one head to a CTA)
        const int32_t *table = p.block_table + (size_t)b * p.max_pages;
        const auto page_of = [&](int chunk, int k) -> int {
            const int t = chunk * kChunk + own + 8 * k;
            if (chunk >= sg.lc1 || t >= L) return -1;
            return ld_unwritten(table + (p.log2_page >= 0 ? t >> p.log2_page : t / p.page_size));
        };
        const auto weight_at = [&](int chunk, int k, int pg) -> float * {
            const int t = chunk * kChunk + own + 8 * k;
            return (uint32_t)pg < (uint32_t)p.num_pages
                       ? p.weights + ((size_t)pg * p.H_kv + h) * p.page_size +
                             (p.log2_page >= 0 ? t & (p.page_size - 1) : t % p.page_size)
                       : nullptr;
        };
        const int step = C::NCW * Z;
        float *wp[2];           // the first head's; the next head's is a page of floats behind it
        float old[HP][2];
        int pg[2];
        const auto old_of = [&](int chunk, int k, const float *w, float(&to)[HP][2]) {
#pragma unroll
            for (int e = 0; e < HP; ++e)
                to[e][k] = w && chunk * kChunk + own + 8 * k < wl ? w[(size_t)e * p.page_size] : 0.f;
        };
#pragma unroll
        for (int k = 0; k < 2; ++k) pg[k] = page_of(c, k);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            wp[k] = weight_at(c, k, pg[k]);
            old_of(c, k, wp[k], old);
            pg[k] = page_of(c + step, k);
        }
        for (i += skip; i < i1; i += C::NCW, c += C::NCW * Z) {
            const int stage = i % C::NS;
#ifdef DA_PAGE_TRACE
            // test build: a wait on a barrier that nothing completes runs out
            if (p.debug_stall &&
                !mbar_wait_warp(reinterpret_cast<uint64_t *>(smem + C::OFF_FLAG + 8), 0, abort_flag, p.wait_limit_ns)) {
                if (lane == 0) {
                    atomicOr(&p.meta.header[kHError], DA_DEV_TIMEOUT);
                    *abort_flag = 1;
                }
                return;
            }
#endif
            if (!mbar_wait_warp(&full[stage], (i / C::NS) & 1, abort_flag, p.wait_limit_ns)) {
                if (lane == 0) {
                    atomicOr(&p.meta.header[kHError], DA_DEV_TIMEOUT);
                    *abort_flag = 1;
                }
                return;
            }
            const int t0 = c * kChunk;
            float *wp_next[2];
            float old_next[HP][2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                wp_next[k] = weight_at(c + step, k, pg[k]);
                old_of(c + step, k, wp_next[k], old_next);
                pg[k] = page_of(c + 2 * step, k);
            }
            const uint32_t s_base = smem_u32(smem + (size_t)stage * C::STAGE);
            float add[HP][2];
#pragma unroll
            for (int e = 0; e < HP; ++e) add[e][0] = add[e][1] = 0.f;
            // the chunk's products with the first NJ query tokens: one build for each count
            const auto products = [&](auto count) {
                // TT: tiles in registers at a time. The e4m3 build for three and four query tokens, whose code with the
                // conversions is the longest, takes one tile in a loop: unrolled it waits for instructions (32 x 8192
                // tokens of 8 heads: 89 us against 71 for four query tokens, 74 against 55 for three; two tiles in a
                // loop 75 and 63)
                constexpr bool kLoop = FP8 && NQ > 2;
                constexpr int NJ = decltype(count)::value, TT = NJ == 1 && !kLoop ? 4 : kLoop && NJ > 2 ? 1 : 2;
#pragma unroll
                for (int e = 0; e < HP; ++e) {
#pragma unroll(kLoop ? 1 : 4 / TT)
                    for (int tt = 0; tt < 4; tt += TT) {
                        float s[TT][NJ][4];
#pragma unroll
                        for (int t = 0; t < TT; ++t)
#pragma unroll
                            for (int j = 0; j < NJ; ++j) s[t][j][0] = s[t][j][1] = s[t][j][2] = s[t][j][3] = 0.f;
                        if constexpr (!FP8) {
#pragma unroll
                            for (int ks = 0; ks < C::KS; ++ks)
#pragma unroll
                                for (int t = 0; t < TT; ++t) {
                                    const int tok = 16 * (tt + t) + lrow + (lmat & 1) * 8;
                                    // (with two heads a row is one 128-byte box)
                                    const int d = ks * 16 + (lmat >> 1) * 8, x = (d >> 6) + e;
                                    const uint32_t addr = s_base + tok * C::SROW + x * 128 +
                                                          ((((d & 63) >> 3) ^ ((tok * C::NX + x) & 7)) << 4);
                                    uint32_t a[4];
                                    ldsm_x4(addr, a[0], a[1], a[2], a[3]);
#pragma unroll
                                    for (int j = 0; j < NJ; ++j)
                                        mma_bf16(s[t][j], a, qf[e][ks][j][0], qf[e][ks][j][1]);
                                }
                        } else {
#pragma unroll
                            for (int kk = 0; kk < D / 32; ++kk)
#pragma unroll
                                for (int t = 0; t < TT; ++t) {
                                    const int tok = 16 * (tt + t) + lrow + (lmat & 1) * 8;
                                    const uint32_t addr = s_base + tok * C::SROW + e * 128 +
                                                          (((kk * 2 + (lmat >> 1)) ^ ((tok * C::NX + e) & 7)) << 4);
                                    uint32_t R[4];
                                    ldsm_x4(addr, R[0], R[1], R[2], R[3]);
#pragma unroll
                                    for (int hf = 0; hf < 2; ++hf) {
                                        const uint32_t ra = R[hf * 2], rb = R[hf * 2 + 1];
                                        const uint32_t a[4] = {e4m3x2_to_f16x2((uint16_t)(ra & 0xffff)),
                                                               e4m3x2_to_f16x2((uint16_t)(rb & 0xffff)),
                                                               e4m3x2_to_f16x2((uint16_t)(ra >> 16)),
                                                               e4m3x2_to_f16x2((uint16_t)(rb >> 16))};
#pragma unroll
                                        for (int j = 0; j < NJ; ++j)
                                            mma_f16(s[t][j], a, qf[e][kk * 2 + hf][j][0], qf[e][kk * 2 + hf][j][1]);
                                    }
                                }
                        }
                        // a row that does not see the token adds nothing, whatever its score
#pragma unroll
                        for (int t = 0; t < TT; ++t) {
                            float e0 = 0.f, e1 = 0.f;
                            const int ta = t0 + 16 * (tt + t) + r8;
#pragma unroll
                            for (int j = 0; j < NJ; ++j)
#pragma unroll
                                for (int g = 0; g < 2; ++g) {
                                    const float x = ex2(fmaf(s[t][j][g], sl2[e], -lse2[e][j][g]));
                                    const float y = ex2(fmaf(s[t][j][2 + g], sl2[e], -lse2[e][j][g]));
                                    e0 += ta <= last[e][j][g] ? x : 0.f;
                                    e1 += ta + 8 <= last[e][j][g] ? y : 0.f;
                                }
                            e0 += __shfl_xor_sync(0xffffffffu, e0, 1);
                            e1 += __shfl_xor_sync(0xffffffffu, e1, 1);
                            e0 += __shfl_xor_sync(0xffffffffu, e0, 2);
                            e1 += __shfl_xor_sync(0xffffffffu, e1, 2);
                            if (c4 == tt + t) {
                                add[e][0] = e0;
                                add[e][1] = e1;
                            }
                        }
                    }
                }
            };
            if constexpr (NQ == 4) {
                if (nj >= 4) products(std::integral_constant<int, 4>{});
                if (nj == 3) products(std::integral_constant<int, 3>{});
            }
            if constexpr (NQ >= 2) {
                if (nj == 2) products(std::integral_constant<int, 2>{});
            }
            if (nj == 1) products(std::integral_constant<int, 1>{});
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[stage]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int e = 0; e < HP; ++e) {
                    const float kept = t0 + own + 8 * k < wl ? old[e][k] * p.decay : 0.f;
                    if (wp[k]) wp[k][(size_t)e * p.page_size] = kept + add[e][k];
                    old[e][k] = old_next[e][k];
                }
                wp[k] = wp_next[k];
            }
        }
        i = i1;
    }
}

template <int D, bool FP8, int NQ, int HP>
cudaError_t launch(const CUtensorMap &tk, AccumParams p, int num_sms, cudaStream_t stream, bool pdl) {
    using C = AccumCfg<D, FP8, NQ, HP>;
    const auto kern = accum_kernel<D, FP8, NQ, HP>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return e;
    // As many CTAs as fit the GPU at once: several to a (part, head) pair where there are fewer pairs, several parts to
    // a CTA where there are more (a fixed split of many requests: a CTA for every short part spends most of its time
    // starting, 70 us against 47 for 32 requests of 2048 to 4096 tokens of 8 bf16 heads in 8 splits).
    const int64_t room = (int64_t)num_sms * C::MIN_BLOCKS, pairs = (int64_t)p.num_parts * (p.H_kv / HP);
    int64_t z = room / pairs;
    z = z < 1 ? 1 : z > 8 ? 8 : z;
    p.parts_per_cta = (int32_t)((pairs + room - 1) / room);
    const int gx = (p.num_parts + p.parts_per_cta - 1) / p.parts_per_cta;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)gx, (unsigned)(p.H_kv / HP), (unsigned)z);
    cfg.blockDim = dim3(C::THREADS);
    cfg.dynamicSmemBytes = C::SMEM;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, tk, p);
}

template <int D, bool FP8>
cudaError_t launch_for(const CUtensorMap &tk, const AccumParams &p, int num_sms, cudaStream_t stream, bool pdl) {
    if constexpr (D * (FP8 ? 1 : 2) == 128)
        if (p.heads_per_cta == 2) return launch<D, FP8, 1, 2>(tk, p, num_sms, stream, pdl);
    if (p.s_q == 1) return launch<D, FP8, 1, 1>(tk, p, num_sms, stream, pdl);
    if (p.s_q == 2) return launch<D, FP8, 2, 1>(tk, p, num_sms, stream, pdl);
    return launch<D, FP8, 4, 1>(tk, p, num_sms, stream, pdl);
}

}  // namespace

// KV heads that a CTA takes (the tensor map's box has as many): two where their rows are 128 bytes, for one query
// token (more tokens' queries of two heads do not fit the registers).
int accum_heads(int row_bytes, int H_kv, int s_q) { return row_bytes == 128 && H_kv % 2 == 0 && s_q == 1 ? 2 : 1; }

cudaError_t launch_accum(int D, bool fp8, const CUtensorMap &tk, const AccumParams &p, int num_sms,
                         cudaStream_t stream, bool pdl) {
    if (fp8) return launch_for<128, true>(tk, p, num_sms, stream, pdl);
    return D == 64 ? launch_for<64, false>(tk, p, num_sms, stream, pdl)
                   : launch_for<128, false>(tk, p, num_sms, stream, pdl);
}

}  // namespace da
