// Attention weight gathered by cached tokens.
//
// After a decode step, for every cached token t of request b and KV head h,
//     w[t] <- (decay w[t], or 0 for a token that has none yet)
//             + sum_j sum_g exp(sigma q_{j,g} . k_t - lse_{j,g})
// over the query tokens j of the step that count and see t, and the G query
// heads of h: the softmax weights of the step's attention call, from its lse.
//
// Bound by HBM: K is read once (V is not needed), w read and written once.
// Like the attention kernel it walks the parts of the scheduling metadata; the
// warps of a part share its tiles round robin and never wait for each other.
// The K rows go from global memory straight into the A fragments of the warp
// MMA (K tile as M, the 8 query heads as N): a dot product does not care in
// which order its terms are added, so the k index of the MMA stands for
// whichever dims make each lane's share of a row contiguous, in q as in K.
// Lane (r, c) of a warp reads 16 contiguous bytes of row r at a time, the four
// lanes of a row 64.
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "decode_attn.h"
#include "layout.h"
#include "segwalk.cuh"

namespace da {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// D, e4m3, query tokens held in registers
template <int D, bool FP8, int NQ>
struct Cfg {
    static constexpr int ROW = D * (FP8 ? 1 : 2);      // bytes
    static constexpr int NV = ROW / 64;                // 16-byte vectors per lane and row
    static constexpr int KS = D / 16;                  // MMA steps
    static constexpr int MT = ROW == 256 ? 1 : 2;      // 16-token m tiles per warp tile: 4 KB
    static constexpr int TOK = 16 * MT;
    static constexpr int TPC = kChunk / TOK;           // tiles per chunk
    static constexpr int NG = 2 * MT;                  // 8-token groups per tile
};

template <int D, bool FP8, int NQ>
__global__ void __launch_bounds__(kThreads) accum_kernel(const __grid_constant__ AccumParams p) {
    using C = Cfg<D, FP8, NQ>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r8 = lane >> 2, c4 = lane & 3;
    const int part = blockIdx.x, h = blockIdx.y;
    pdl_wait();
    pdl_launch_dependents();

    const int4 rec0 = p.meta.parts[2 * part];
    const int4 rec1 = p.meta.parts[2 * part + 1];
    {
        const bool ok = meta_header_ok(load_meta_header(p.meta.header), p.B, p.H_kv, p.G, p.splits, p.num_parts,
                                       p.s_q, 0, 0) &
                        ((int)gridDim.x == p.num_parts);
        if (!ok) {
            if (threadIdx.x == 0) atomicOr(&p.meta.header[kHError], DA_DEV_META_MISMATCH);
            return;
        }
    }
    const int max_len = p.max_pages * p.page_size;
    const float sl2 = p.scale_log2 * (FP8 ? __ldg(p.k_scale + h) : 1.f);
    const int W = kWarps * gridDim.z, w = blockIdx.z * kWarps + warp;  // warps of this part

    SegWalker wk = make_walker(p.meta, rec0, rec1, p.B, p.seqlens, max_len, p.s_q, 0, 0);
    Seg sg;
    int done = 0;  // tiles of the part's earlier segments
    while (wk.next(sg)) {
        const int b = sg.b, L = sg.L;
        const int tiles = min((sg.lc1 - sg.lc0) * C::TPC, (L - sg.lc0 * kChunk + C::TOK - 1) / C::TOK);
        if (tiles <= 0) continue;
        const int first = (w + W - done % W) % W;
        done += tiles;
        if (first >= tiles) continue;
        // q: B fragments, n = query head r8; lse of the two heads whose scores this lane gets
        uint32_t qf[NQ][C::KS][2];
        float lse2[NQ][2];
        int last[NQ];  // last token that query token j sees, -1 where it does not count
        const int acc = p.accepted ? p.accepted[b] : p.s_q - 1;
        const int wl = p.weighted ? p.weighted[b] : L;
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            const bool on = j < p.s_q && j <= acc;
            last[j] = on ? L - p.s_q + j : -1;
            lse2[j][0] = lse2[j][1] = 0.f;
            if (!on) {
#pragma unroll
                for (int k = 0; k < C::KS; ++k) qf[j][k][0] = qf[j][k][1] = 0u;
                continue;
            }
            const size_t head0 = ((size_t)b * p.s_q + j) * p.H_q + (size_t)h * 8;
            const float2 ls = *reinterpret_cast<const float2 *>(p.lse + head0 + 2 * c4);
            constexpr float kLog2e = 1.4426950408889634f;
            lse2[j][0] = ls.x * kLog2e;
            lse2[j][1] = ls.y * kLog2e;
            const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) + (head0 + r8) * D;
            if constexpr (!FP8) {
                // vector x: dims x 32 + c4 8 .. + 7 feed two MMA steps, four dims each
#pragma unroll
                for (int x = 0; x < C::NV; ++x) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(q + x * 32 + c4 * 8);
                    qf[j][2 * x][0] = v.x;
                    qf[j][2 * x][1] = v.y;
                    qf[j][2 * x + 1][0] = v.z;
                    qf[j][2 * x + 1][1] = v.w;
                }
            } else {
                // vector x: dims x 64 + c4 16 .. + 15 feed four steps
#pragma unroll
                for (int x = 0; x < C::NV; ++x)
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(q + x * 64 + c4 * 16 + y * 8);
                        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            qf[j][4 * x + 2 * y + i / 2][i & 1] =
                                pack_f16(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xFFFF0000u));
                    }
            }
        }
        const int32_t *table = p.block_table + (size_t)b * p.max_pages;
        // page and slot of the 8-token group g of a tile (groups start on multiples of 8, pages are multiples of 8)
        auto page_of = [&](int t) -> int {
            if (t >= L) return -2;
            return table[p.log2_page >= 0 ? t >> p.log2_page : t / p.page_size];
        };
        auto slot_of = [&](int t) -> int {
            return p.log2_page >= 0 ? t & (p.page_size - 1) : t % p.page_size;
        };
        const int base0 = sg.lc0 * kChunk;
        int page[C::NG];
#pragma unroll
        for (int g = 0; g < C::NG; ++g) page[g] = page_of(base0 + first * C::TOK + 8 * g);
        for (int ti = first; ti < tiles; ti += W) {
            const int t0 = base0 + ti * C::TOK;
            uint4 kv[C::NG][C::NV];
            float *wp = nullptr;   // the weight that this lane updates: row r8 of group c4
            float old = 0.f;
#pragma unroll
            for (int g = 0; g < C::NG; ++g) {
                const int t = t0 + 8 * g;
                int pg = page[g];
                if (pg != -2 && (pg < 0 || pg >= p.num_pages)) {
                    if (lane == 0) {
                        atomicOr(&p.meta.header[kHError], DA_DEV_BAD_PAGE);
                        p.meta.header[kHErrorDetail] = pg;
                    }
                    pg = -2;
                }
                const int slot = slot_of(t);
                const bool in = pg >= 0 && t + r8 < L;
                const uint8_t *k = p.k_pool + (((size_t)max(pg, 0) * p.page_size + slot + r8) * p.H_kv + h) * C::ROW;
#pragma unroll
                for (int x = 0; x < C::NV; ++x)
                    kv[g][x] = in ? ldg_stream16(k + x * 64 + c4 * 16) : make_uint4(0u, 0u, 0u, 0u);
                if (g == c4 && in) {
                    wp = p.weights + ((size_t)pg * p.H_kv + h) * p.page_size + slot + r8;
                    old = t + r8 < wl ? *wp * p.decay : 0.f;
                }
            }
            // the next tile's pages, a tile ahead of their use
            if (ti + W < tiles) {
#pragma unroll
                for (int g = 0; g < C::NG; ++g) page[g] = page_of(t0 + W * C::TOK + 8 * g);
            }
            float sum[C::NG];
#pragma unroll
            for (int m = 0; m < C::MT; ++m) {
                float s[NQ][4];
#pragma unroll
                for (int j = 0; j < NQ; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
#pragma unroll
                for (int x = 0; x < C::NV; ++x) {
                    const uint4 lo = kv[2 * m][x], hi = kv[2 * m + 1][x];
                    if constexpr (!FP8) {
                        const uint32_t a0[4] = {lo.x, hi.x, lo.y, hi.y}, a1[4] = {lo.z, hi.z, lo.w, hi.w};
#pragma unroll
                        for (int j = 0; j < NQ; ++j) {
                            mma_bf16(s[j], a0, qf[j][2 * x][0], qf[j][2 * x][1]);
                            mma_bf16(s[j], a1, qf[j][2 * x + 1][0], qf[j][2 * x + 1][1]);
                        }
                    } else {
                        const uint32_t l[4] = {lo.x, lo.y, lo.z, lo.w}, u[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t a[4] = {
                                e4m3x2_to_f16x2((uint16_t)(l[i] & 0xffff)), e4m3x2_to_f16x2((uint16_t)(u[i] & 0xffff)),
                                e4m3x2_to_f16x2((uint16_t)(l[i] >> 16)), e4m3x2_to_f16x2((uint16_t)(u[i] >> 16))};
#pragma unroll
                            for (int j = 0; j < NQ; ++j) mma_f16(s[j], a, qf[j][4 * x + i][0], qf[j][4 * x + i][1]);
                        }
                    }
                }
                // a row that does not count or see the token adds nothing, whatever its score
                float e0 = 0.f, e1 = 0.f;
                const int ta = t0 + 16 * m + r8;
#pragma unroll
                for (int j = 0; j < NQ; ++j) {
                    const bool on0 = lse2[j][0] != -INFINITY, on1 = lse2[j][1] != -INFINITY;
                    if (ta <= last[j]) {
                        e0 += on0 ? ex2(fmaf(s[j][0], sl2, -lse2[j][0])) : 0.f;
                        e0 += on1 ? ex2(fmaf(s[j][1], sl2, -lse2[j][1])) : 0.f;
                    }
                    if (ta + 8 <= last[j]) {
                        e1 += on0 ? ex2(fmaf(s[j][2], sl2, -lse2[j][0])) : 0.f;
                        e1 += on1 ? ex2(fmaf(s[j][3], sl2, -lse2[j][1])) : 0.f;
                    }
                }
                e0 += __shfl_xor_sync(0xffffffffu, e0, 1);
                e1 += __shfl_xor_sync(0xffffffffu, e1, 1);
                e0 += __shfl_xor_sync(0xffffffffu, e0, 2);
                e1 += __shfl_xor_sync(0xffffffffu, e1, 2);
                sum[2 * m] = e0;
                sum[2 * m + 1] = e1;
            }
            if (wp) {
                float v = sum[0];
#pragma unroll
                for (int g = 1; g < C::NG; ++g) v = c4 == g ? sum[g] : v;
                *wp = old + v;
            }
        }
    }
}

template <int D, bool FP8, int NQ>
cudaError_t launch(const AccumParams &p, int num_sms, cudaStream_t stream, bool pdl) {
    // blocks per (part, head): enough to fill the SMs, two blocks on each
    const int64_t pairs = (int64_t)p.num_parts * p.H_kv;
    int64_t z = (2 * (int64_t)num_sms + pairs - 1) / pairs;
    z = z < 1 ? 1 : z > 8 ? 8 : z;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.num_parts, (unsigned)p.H_kv, (unsigned)z);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, accum_kernel<D, FP8, NQ>, p);
}

template <int D, bool FP8>
cudaError_t launch_for(const AccumParams &p, int num_sms, cudaStream_t stream, bool pdl) {
    if (p.s_q == 1) return launch<D, FP8, 1>(p, num_sms, stream, pdl);
    if (p.s_q == 2) return launch<D, FP8, 2>(p, num_sms, stream, pdl);
    return launch<D, FP8, 4>(p, num_sms, stream, pdl);
}

}  // namespace

cudaError_t launch_accum(int D, bool fp8, const AccumParams &p, int num_sms, cudaStream_t stream, bool pdl) {
    if (fp8) return launch_for<128, true>(p, num_sms, stream, pdl);
    return D == 64 ? launch_for<64, false>(p, num_sms, stream, pdl) : launch_for<128, false>(p, num_sms, stream, pdl);
}

}  // namespace da
