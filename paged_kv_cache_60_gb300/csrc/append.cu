// KV append: writes each request's new token into the page slot that its
// block table gives for its position, quantising on the way.
//
// The decode kernels read a pool that already holds the step's new K/V; the
// write itself happens upstream of attention (XQA page, section
// "一次 decode step 的完整时序": the KV append is not part of XQA, the new
// token lands in the pool first and the attention kernel only reads through
// the page table). The formats are those the decode kernels read:
//   * bf16 pools: a copy of the token's H_kv * D values;
//   * e4m3 pools: code = e4m3(x / scale[h]) with one fp32 scale per KV head and
//     tensor (XQA page, section "Hopper 路径上 V 不做显式反量化", largest finite 448);
//   * the 656-byte latent token (FlashMLA page, section "数据加载"): per block
//     of 128 NoPE values, scale = max|x| / 448 (1 for an all-zero block),
//     512 codes, the four fp32 scales, then the 64 RoPE values as bf16.
// Rounding is the IEEE one everywhere: the quotient x / scale is the fp32
// division rounded to nearest (not a plain multiply by a reciprocal), the e4m3
// code the nearest finite value with ties to even, saturating at +-448; NaN
// maps to 0x7F. The quotient is computed by Markstein's correction of the
// reciprocal product where that gives the rounded quotient exactly, and by the
// division elsewhere (see quot_rn). The pool layout is [num_pages][page_size][H_kv][D] (bf16 / e4m3)
// or [num_pages][page_size][1][656].
//
// The work is a scatter of a few hundred bytes per request, HBM / latency
// bound: per thread the same 16-byte vector of K and of V (two loads, two
// 16- or 8-byte stores), coalesced along the token's contiguous H_kv * D
// values; the latent format takes one warp per token (lanes 8k..8k+7 own
// block k and reduce its max with shuffles). Every request's new row is read,
// even when its position skips it.
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "decode_attn.h"
#include "layout.h"
#include "quant.cuh"

namespace da {
namespace {

constexpr int kThreads = 256;
// Shared prologue of both kernels: where request b's token goes, or -1 when
// it is skipped (negative position) or invalid (error bit set by `reporter`).
__device__ __forceinline__ int64_t slot_of(const AppendParams &p, int b, bool reporter) {
    const int t = p.positions[b];
    if (t < 0) return -1;
    if ((int64_t)t >= (int64_t)p.max_pages * p.page_size) {
        if (reporter && p.error) atomicOr(p.error, DA_DEV_SEQ_TOO_LONG);
        return -1;
    }
    const int page = p.block_table[(int64_t)b * p.max_pages + t / p.page_size];
    if (page < 0 || page >= p.num_pages) {
        if (reporter && p.error) atomicOr(p.error, DA_DEV_BAD_PAGE);
        return -1;
    }
    return (int64_t)page * p.page_size + t % p.page_size;
}

// bf16 / e4m3 pools. Work item = kV values (one or two 16-byte vectors of 8)
// at the same place in K and in V of one request (items of a request are
// consecutive). The row loads are issued before the position and page
// lookups, so their latencies overlap. The e4m3 build takes 16 values per item
// (D a multiple of 16): each thread then moves as many bytes per lookup chain
// as a bf16 thread, and stores its 16 codes as one 16-byte vector.
// Six blocks per SM (at most 40 registers a thread): the latency of a work
// item's chain (row loads, position and page lookups, quotients, stores)
// is hidden by more resident threads; measured faster than the four blocks
// that 52 registers allow, despite a few spilled words.
template <bool kFp8, int kV>
__global__ void __launch_bounds__(kThreads, 6) append_gqa_kernel(const AppendParams p) {
    pdl_wait();               // positions, block table and new rows may come from the previous kernel
    pdl_launch_dependents();  // the next kernel waits for this grid before it reads the pool
    constexpr int NV = kV / 8;  // 16-byte input vectors per item
    const int vpr = p.D / kV;
    const int per_req = p.H_kv * vpr;
    const int64_t total = (int64_t)p.B * per_req;
    for (int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x; i < total; i += (int64_t)gridDim.x * kThreads) {
        const int b = (int)(i / per_req);
        const int e = (int)(i - (int64_t)b * per_req);
        const int64_t src = (int64_t)b * p.row_stride + (int64_t)e * kV;
        uint4 xk[NV], xv[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            xk[j] = ld_stream_v4(p.k_new + src + 8 * j);
            xv[j] = ld_stream_v4(p.v_new + src + 8 * j);
        }
        const int64_t slot = slot_of(p, b, e == 0);
        if (slot < 0) continue;
        const int64_t vec = slot * per_req + e;
        if constexpr (!kFp8) {
#pragma unroll
            for (int j = 0; j < NV; ++j) {
                st_v4(p.k_pool + vec * kV * 2 + 16 * j, xk[j]);
                st_v4(p.v_pool + vec * kV * 2 + 16 * j, xv[j]);
            }
        } else {
            const int h = e / vpr;
            const Recip dk = recip_of(p.k_scale[h]), dv = recip_of(p.v_scale[h]);
            if constexpr (NV == 2) {
                const uint2 k0 = quant8(xk[0], dk), k1 = quant8(xk[1], dk);
                const uint2 v0 = quant8(xv[0], dv), v1 = quant8(xv[1], dv);
                st_v4(p.k_pool + vec * kV, make_uint4(k0.x, k0.y, k1.x, k1.y));
                st_v4(p.v_pool + vec * kV, make_uint4(v0.x, v0.y, v1.x, v1.y));
            } else {
                st_v2(p.k_pool + vec * kV, quant8(xk[0], dk));
                st_v2(p.v_pool + vec * kV, quant8(xv[0], dv));
            }
        }
    }
}

__global__ void __launch_bounds__(kThreads, 6) append_mla_kernel(const AppendParams p) {
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    constexpr int kWarps = kThreads / 32;
    for (int b = blockIdx.x * kWarps + (threadIdx.x >> 5); b < p.B; b += gridDim.x * kWarps) {
        // the row loads first, then the position and page lookups
        const LatentIn x = latent_load(p.k_new + (int64_t)b * p.row_stride, lane);
        const int64_t slot = slot_of(p, b, lane == 0);  // uniform over the warp
        if (slot >= 0) latent_store(p.k_pool + slot * kLatentRow, lane, x);
    }
}

}  // namespace

cudaError_t launch_append(int kv_dtype, const AppendParams &p, cudaStream_t stream, bool pdl) {
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    constexpr int64_t kMaxBlocks = 1 << 20;    // grid-stride beyond that
    if (kv_dtype == DA_KV_FP8_MLA656) {
        const int64_t blocks = (p.B + kThreads / 32 - 1) / (kThreads / 32);
        cfg.gridDim = dim3((unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks));
        return cudaLaunchKernelEx(&cfg, append_mla_kernel, p);
    }
    const bool wide = kv_dtype == DA_KV_FP8_PER_TENSOR && p.D % 16 == 0;
    const int64_t items = (int64_t)p.B * p.H_kv * (p.D / (wide ? 16 : 8));
    const int64_t blocks = (items + kThreads - 1) / kThreads;
    cfg.gridDim = dim3((unsigned)(blocks < kMaxBlocks ? blocks : kMaxBlocks));
    if (kv_dtype == DA_KV_FP8_PER_TENSOR)
        return wide ? cudaLaunchKernelEx(&cfg, append_gqa_kernel<true, 16>, p)
                    : cudaLaunchKernelEx(&cfg, append_gqa_kernel<true, 8>, p);
    return cudaLaunchKernelEx(&cfg, append_gqa_kernel<false, 8>, p);
}

}  // namespace da
