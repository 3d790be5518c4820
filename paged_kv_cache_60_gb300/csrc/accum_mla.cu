// Attention weight gathered by cached tokens, on the 656-byte latent format.
//
// The sum of accum.cu with one KV head, G = 128 query heads and 576 dims, of
// which 512 are e4m3 with a scale per 128 (dequantised as the attention kernel
// does: bf16(fp32(e4m3) * scale)) and 64 bf16.
//
// 147 thousand floating-point operations a token and query token against 656
// bytes: the products bound it, not HBM. One CTA per SM holds the 128 x 576
// query rows of one query token in shared memory, in the order in which the
// warp MMA's B fragments want them (147 KB, one 8-byte read per lane and
// fragment, no conflicts). A warp takes 32 tokens at a time: the rows go from
// global memory straight into A fragments, every lane reading and dequantising
// 16 contiguous values of a row (a dot product does not care which dims the k
// index of an MMA stands for, as long as q and K agree), each B fragment feeds
// the two 16-token tiles, and the 32 x 128 scores stay in registers until their
// exponentials are summed. Several query tokens take one pass over the tokens
// each, later ones adding to what the same lane stored before.
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
constexpr int kHeads = 128;
constexpr int kDim = 576, kNope = 512;
constexpr int kRow = 656, kScales = 512, kRope = 528;
constexpr int kSteps = kDim / 16;     // MMA steps
constexpr int kNT = kHeads / 8;       // n tiles
constexpr int kTok = 32;              // tokens of a warp's unit
constexpr int kSmem = kSteps * kNT * 32 * 8 + kHeads * 4;

// Two e4m3 values (a 16-bit piece of w) times the scale, as two bf16.
__device__ __forceinline__ uint32_t dequant2(uint32_t w, bool high, float scale) {
    const uint32_t f = e4m3x2_to_f16x2((uint16_t)(high ? w >> 16 : w & 0xFFFFu));
    const __half2 v = *reinterpret_cast<const __half2 *>(&f);
    return pack_bf16(__low2float(v) * scale, __high2float(v) * scale);
}

// s += A B for one step of both tiles and all heads
__device__ __forceinline__ void step(float (&s)[2][kNT][4], const uint32_t (&a)[2][4], const uint2 *qs, int lane) {
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
        const uint2 b = qs[nt * 32 + lane];
        mma_bf16(s[0][nt], a[0], b.x, b.y);
        mma_bf16(s[1][nt], a[1], b.x, b.y);
    }
}

__global__ void __launch_bounds__(kThreads, 1) accum_mla_kernel(const __grid_constant__ AccumParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    uint2 *qs = reinterpret_cast<uint2 *>(smem);                                   // [step][n tile][lane]
    float *lse2 = reinterpret_cast<float *>(smem + kSteps * kNT * 32 * 8);         // [head], +inf: adds nothing
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r8 = lane >> 2, c4 = lane & 3, Z = gridDim.z;
    const int part0 = blockIdx.x * p.parts_per_cta, part1 = min(part0 + p.parts_per_cta, p.num_parts);
    pdl_wait();
    pdl_launch_dependents();
    if (!meta_header_ok(load_meta_header(p.meta.header), p.B, p.H_kv, p.G, p.splits, p.num_parts, p.s_q, 0, 0)) {
        if (tid == 0) atomicOr(&p.meta.header[kHError], DA_DEV_META_MISMATCH);
        return;
    }
    const int max_len = p.max_pages * p.page_size;
    for (int part = part0; part < part1; ++part) {
        SegWalker wk = make_walker(p.meta, p.meta.parts[2 * part], p.meta.parts[2 * part + 1], p.B, p.seqlens, max_len,
                                   p.s_q, 0, 0);
        Seg sg;
        while (wk.next(sg)) {
            // tokens [lc0, lc1) * 64 of the request, 32 to a unit; the warps of the pair's CTAs share them
            const int b = sg.b, L = sg.L, u0 = sg.lc0 * 2;
            const int units = min((sg.lc1 - sg.lc0) * 2, (L - sg.lc0 * kChunk + kTok - 1) / kTok);
            if (units <= 0) continue;
            const int nj = p.accepted ? min(p.accepted[b], p.s_q - 1) + 1 : p.s_q;   // query tokens that count
            const int wl = p.weighted ? p.weighted[b] : L;
            const int32_t *table = p.block_table + (size_t)b * p.max_pages;
            // (no query token counts: one pass all the same, for the decay)
            for (int j = 0; j < max(nj, 1); ++j) {
                const size_t row0 = ((size_t)b * p.s_q + j) * kHeads;
                __syncthreads();  // the previous pass is done with q
                const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(p.q) + row0 * kDim;
                for (int i = tid; i < kHeads * 40; i += kThreads) {
                    // head i / 40: 32 groups of 16 NoPE dims, then 8 groups of 8 RoPE dims
                    const int head = i / 40, g = i - head * 40, nt = head >> 3, ln = (head & 7) * 4;
                    if (g < 32) {
                        const uint4 *src = reinterpret_cast<const uint4 *>(q + (size_t)head * kDim + g * 16);
                        const uint4 x = src[0], y = src[1];
                        uint2 *dst = qs + ((g >> 2) * 4 * kNT + nt) * 32 + ln + (g & 3);
                        dst[0] = make_uint2(x.x, x.y);
                        dst[kNT * 32] = make_uint2(x.z, x.w);
                        dst[2 * kNT * 32] = make_uint2(y.x, y.y);
                        dst[3 * kNT * 32] = make_uint2(y.z, y.w);
                    } else {
                        const int r = g - 32;
                        const uint4 x = *reinterpret_cast<const uint4 *>(q + (size_t)head * kDim + kNope + r * 8);
                        uint2 *dst = qs + ((32 + (r >> 2) * 2) * kNT + nt) * 32 + ln + (r & 3);
                        dst[0] = make_uint2(x.x, x.y);
                        dst[kNT * 32] = make_uint2(x.z, x.w);
                    }
                }
                for (int i = tid; i < kHeads; i += kThreads) {
                    const float l = p.lse[row0 + i];
                    lse2[i] = l == -INFINITY || j >= nj ? INFINITY : l * 1.4426950408889634f;
                }
                __syncthreads();
                const int last = L - p.s_q + j;   // last token that query token j sees
                for (int u = blockIdx.z * kWarps + warp; u < units; u += kWarps * Z) {
                    const int t0 = (u0 + u) * kTok;
                    // the four rows of this lane: tokens t0 + 8 k + r8 (a group of eight lies in one page)
                    const uint8_t *row[4];
                    float *wp = nullptr;
                    float old = 0.f;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int tg = t0 + 8 * k, t = tg + r8;
                        const int pi = p.log2_page >= 0 ? tg >> p.log2_page : tg / p.page_size;
                        int pg = tg < L ? table[pi] : -2;
                        if (pg != -2 && (uint32_t)pg >= (uint32_t)p.num_pages) {
                            if (lane == 0) {
                                atomicOr(&p.meta.header[kHError], DA_DEV_BAD_PAGE);
                                p.meta.header[kHErrorDetail] = pg;
                            }
                            pg = -2;
                        }
                        const size_t slot = (size_t)max(pg, 0) * p.page_size + (tg - pi * p.page_size) + r8;
                        row[k] = pg >= 0 && t < L ? p.k_pool + slot * kRow : nullptr;
                        if (k == c4 && row[k]) {
                            wp = p.weights + slot;     // one KV head: [page][slot]
                            old = j > 0 ? *wp : t < wl ? *wp * p.decay : 0.f;
                        }
                    }
                    float s[2][kNT][4];
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int nt = 0; nt < kNT; ++nt) s[m][nt][0] = s[m][nt][1] = s[m][nt][2] = s[m][nt][3] = 0.f;
                    // vector v of a row: bytes [64 v, 64 v + 64) of it, this lane 16 of them; the RoPE part 128 bytes
                    const auto get = [&](int k, int at) -> uint4 {
                        return row[k] ? ldg_stream16(row[k] + at) : make_uint4(0u, 0u, 0u, 0u);
                    };
                    uint4 next[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) next[k] = get(k, c4 * 16);
#pragma unroll 1
                    for (int x = 0; x < 8; ++x) {
                        uint4 v[4];
                        float sc[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            v[k] = next[k];
                            sc[k] = row[k] ? __ldg(reinterpret_cast<const float *>(row[k] + kScales) + (x >> 1)) : 0.f;
                            next[k] = get(k, x < 7 ? (x + 1) * 64 + c4 * 16 : kRope + c4 * 16);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t a[2][4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint32_t w = i == 0 ? v[k].x : i == 1 ? v[k].y : i == 2 ? v[k].z : v[k].w;
                                a[k >> 1][k & 1] = dequant2(w, false, sc[k]);
                                a[k >> 1][2 + (k & 1)] = dequant2(w, true, sc[k]);
                            }
                            step(s, a, qs + (x * 4 + i) * kNT * 32, lane);
                        }
                    }
#pragma unroll
                    for (int y = 0; y < 2; ++y) {
                        uint4 v[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            v[k] = next[k];
                            if (y == 0) next[k] = get(k, kRope + 64 + c4 * 16);
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            uint32_t a[2][4];
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                a[k >> 1][k & 1] = i ? v[k].z : v[k].x;
                                a[k >> 1][2 + (k & 1)] = i ? v[k].w : v[k].y;
                            }
                            step(s, a, qs + (32 + y * 2 + i) * kNT * 32, lane);
                        }
                    }
                    // a row that does not see the token adds nothing, whatever its score
                    float e[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int nt = 0; nt < kNT; ++nt) {
                        const float2 l = *reinterpret_cast<const float2 *>(lse2 + nt * 8 + 2 * c4);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float x = ex2(fmaf(s[k >> 1][nt][2 * (k & 1)], p.scale_log2, -l.x));
                            const float y = ex2(fmaf(s[k >> 1][nt][2 * (k & 1) + 1], p.scale_log2, -l.y));
                            e[k] += (l.x == INFINITY ? 0.f : x) + (l.y == INFINITY ? 0.f : y);
                        }
                    }
                    float mine = 0.f;
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        if (t0 + 8 * k + r8 > last) e[k] = 0.f;
                        e[k] += __shfl_xor_sync(0xffffffffu, e[k], 1);
                        e[k] += __shfl_xor_sync(0xffffffffu, e[k], 2);
                        if (k == c4) mine = e[k];
                    }
                    if (wp) *wp = old + mine;
                }
            }
        }
    }
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
