// Append to a cache in 8 bits with a scale for each block of 16 tokens and KV
// head (e4m3 or int8 codes): one token per request, draft chains, ragged prompts.
//
// For a block, head and tensor, with Q = 448 (e4m3) or 127 (int8):
//     scale = the smallest power of two with max |x| <= Q scale, never below the
//             scale of tokens that the block holds already
//     code  = round(x / scale), ties to even
// A scale that is a power of two makes x / scale exact, so a value is rounded
// once; and when a later token makes the scale grow, the earlier codes go down by
// whole powers of two: exact in e4m3 but for subnormals, and in int8 the halves of
// a step add up to less than one (a scale that followed the maximum itself would
// be rounded to again at every new maximum, up to fifteen halves). What it costs: an
// int8 step is up to twice the one that the maximum would need; e4m3 loses nothing.
//
// One warp per (block, head, tensor): it holds the block's new rows in registers (16
// rows of 256 bytes, 16 bytes a lane and row, two rows per load), takes their largest
// magnitude by a warp reduction and writes the codes. The rows are read once, and
// nothing is handed on between warps. Block slots are dealt out without a scan: request
// b's start at floor(starts[b] / 16) + 2 b, which leaves room for the blocks that n
// tokens from any position touch (floor((n + 14) / 16) + 1 at most); a warp finds its
// request by a search over that sum, 32 requests at a time.
//
// Bound by HBM: 32771 tokens of 8 heads in 34.3 us, 201 MB, 0.87 of the measured copy
// rate (the saturating conversions for every value: 62.6 us, 63 % of the issue slots).
// Four CTAs an SM, 64 registers a thread: 36.7 us with three, 43.3 with five, which spill.
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "decode_attn.h"
#include "layout.h"
#include "quant.cuh"

namespace da {
namespace {

constexpr int kThreads = 256;
constexpr int kRow = 128;            // values of a head
constexpr int kPasses = kScaleBlock / 2;  // loads of two rows

__device__ __forceinline__ int clamp_start(const AppendBlockParams &p, int b) {
    return min(max(p.starts[b], 0), p.N);
}
// first block slot of request b
__device__ __forceinline__ int64_t slot_base(const AppendBlockParams &p, int b) {
    return (int64_t)(clamp_start(p, b) / kScaleBlock) + 2 * (int64_t)b;
}

// The biased exponent of the scale for a largest magnitude m, the 15 magnitude bits of a bf16.
template <bool I8>
__device__ __forceinline__ int scale_exponent(uint32_t m) {
    // 448 = 1.75 * 2^8, 127 = 1.984375 * 2^6: bf16 significands above those need one more
    constexpr int kExp = I8 ? 6 : 8;
    constexpr uint32_t kSig = I8 ? 126 : 96;
    const int e = (int)(m >> 7) - kExp + ((m & 127u) > kSig ? 1 : 0);
    return max(e, 1);
}

__device__ __forceinline__ uint32_t int8_of(float q) {
    return (uint32_t)min(max(__float2int_rn(q), -127), 127) & 0xFFu;  // NaN -> 0
}

// eight codes of eight values (already divided by the scale)
template <bool I8>
__device__ __forceinline__ uint2 codes8(const float (&q)[8]) {
    uint32_t c[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float *x = q + 4 * i;
        if constexpr (I8)
            c[i] = int8_of(x[0]) | int8_of(x[1]) << 8 | int8_of(x[2]) << 16 | int8_of(x[3]) << 24;
        else
            c[i] = e4m3x2(x[0], x[1]) | e4m3x2(x[2], x[3]) << 16;
    }
    return make_uint2(c[0], c[1]);
}

// Eight codes of eight bf16 values whose scale is the power of two 1 / inv and large enough for all of them: nothing
// saturates and nothing is NaN. int8: adding 1.5 * 2^23 rounds x inv to a whole number (to nearest even, in the same
// instruction as the exact product), which is then the sum's lowest byte.
template <bool I8>
__device__ __forceinline__ uint2 codes8_fitting(uint4 x, float inv) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t c[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        if constexpr (I8) {
            uint32_t r[4];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                r[2 * k] = __float_as_uint(fmaf(bf16_lo(w[2 * i + k]), inv, 12582912.f));
                r[2 * k + 1] = __float_as_uint(fmaf(bf16_hi(w[2 * i + k]), inv, 12582912.f));
            }
            c[i] = prmt(prmt(r[0], r[1], 0x0040u), prmt(r[2], r[3], 0x0040u), 0x5410u);
        } else {
            uint16_t h[2];
#pragma unroll
            for (int k = 0; k < 2; ++k)
                asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
                    : "=h"(h[k])
                    : "f"(bf16_hi(w[2 * i + k]) * inv), "f"(bf16_lo(w[2 * i + k]) * inv));
            c[i] = (uint32_t)h[0] | (uint32_t)h[1] << 16;
        }
    }
    return make_uint2(c[0], c[1]);
}

// the values of eight codes, without their scale
template <bool I8>
__device__ __forceinline__ void values8(uint2 c, float (&x)[8]) {
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        uint32_t h[2];
        if constexpr (I8) {
            h[0] = int8x2_to_f16x2<0, 1>(w[i]);
            h[1] = int8x2_to_f16x2<2, 3>(w[i]);
        } else {
            h[0] = e4m3x2_to_f16x2((uint16_t)(w[i] & 0xFFFFu));
            h[1] = e4m3x2_to_f16x2((uint16_t)(w[i] >> 16));
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[k]));
            x[4 * i + 2 * k] = f.x;
            x[4 * i + 2 * k + 1] = f.y;
        }
    }
}

template <bool I8>
__global__ void __launch_bounds__(kThreads, 4) append_block_kernel(const __grid_constant__ AppendBlockParams p) {
    pdl_wait();               // rows, positions, table and scales may come from the kernel before
    pdl_launch_dependents();  // the next kernel waits for this grid before it reads the pool
    const int lane = threadIdx.x & 31;
    const int64_t job = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    if (job >= p.jobs) return;
    // neighbouring warps: neighbouring heads of K, then of V, of one block
    const int H = p.H_kv;
    const int64_t u = job / (2 * H);
    const int r = (int)(job - u * (2 * H));
    const bool is_v = r >= H;
    const int h = is_v ? r - H : r;

    // the request, its rows [lo, lo + n) and the how-manieth of its blocks
    int b, lo, n;
    int64_t nth;
    if (p.starts == nullptr) {
        b = (int)(u / p.per_request);
        nth = u - (int64_t)b * p.per_request;
        lo = b * p.s_q;
        n = p.s_q;
    } else {
        // the last request whose first slot is not above u: 32 probes a round
        int first = 0, count = p.B;  // it is in [first, first + count)
        while (count > 1) {
            const int step = (count + 31) / 32;
            const int probe = first + lane * step;
            const bool below = lane * step < count && slot_base(p, probe) <= u;
            const unsigned hits = __ballot_sync(0xFFFFFFFFu, below);
            const int at = hits ? 31 - __clz(hits) : 0;
            first += at * step;
            count = min(step, count - at * step);
        }
        b = first;
        nth = u - slot_base(p, b);
        lo = clamp_start(p, b);
        n = clamp_start(p, b + 1) - lo;
    }
    const int pos = p.positions[b];
    if (pos < 0 || n <= 0 || nth < 0) return;
    const int64_t blk = pos / kScaleBlock + nth;  // of the request
    int64_t t0 = max((int64_t)pos, blk * kScaleBlock), t1 = min((int64_t)pos + n, (blk + 1) * kScaleBlock);
    if (t0 >= t1) return;
    const bool reporter = r == 0 && lane == 0;
    if (t1 > (int64_t)p.max_pages * p.page_size) {  // whole blocks: a table ends with one
        if (reporter && p.error) atomicOr(p.error, DA_DEV_SEQ_TOO_LONG);
        return;
    }
    const int s0 = (int)(t0 - blk * kScaleBlock), s1 = (int)(t1 - blk * kScaleBlock);

    // the new rows: lane covers values 8 (lane & 15) .. + 8 of slots 2 i + (lane >> 4)
    const uint16_t *src = (is_v ? p.v : p.k) + (int64_t)h * kRow + (lane & 15) * 8;
    const int64_t stride = is_v ? p.v_stride : p.k_stride;
    const int64_t row0 = lo + (t0 - pos);
    uint4 x[kPasses];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int slot = 2 * i + (lane >> 4);
        x[i] = slot >= s0 && slot < s1 ? ld_stream_v4(src + (row0 + slot - s0) * stride) : make_uint4(0u, 0u, 0u, 0u);
    }
    const int page = p.block_table[(int64_t)b * p.max_pages + blk * kScaleBlock / p.page_size];
    if (page < 0 || page >= p.num_pages) {
        if (reporter && p.error) atomicOr(p.error, DA_DEV_BAD_PAGE);
        return;
    }
    const int in_page = (int)(blk * kScaleBlock % p.page_size);
    float *scale_at = (is_v ? p.v_scale : p.k_scale) +
                      ((int64_t)page * H + h) * (p.page_size / kScaleBlock) + in_page / kScaleBlock;
    const float had = s0 > 0 ? *scale_at : 0.f;

    // largest finite magnitude, by its bits
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) m = __vmaxu2(m, w[k] & 0x7FFF7FFFu);
    }
    m = max(m & 0xFFFFu, m >> 16);
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    const bool finite = m < 0x7F80u;
    if (!finite) {  // the values that are not finite do not count
        m = 0;
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t a = w[k] & 0x7FFFu, c = w[k] >> 16 & 0x7FFFu;
                if (a < 0x7F80u) m = max(m, a);
                if (c < 0x7F80u) m = max(m, c);
            }
        }
        m = __reduce_max_sync(0xFFFFFFFFu, m);
    }
    const float need = __uint_as_float((uint32_t)scale_exponent<I8>(m) << 23);
    const float scale = had >= need ? had : need;
    const uint32_t bits = __float_as_uint(scale), e = bits >> 23;
    const bool power = (bits & 0x7FFFFFu) == 0 && e >= 1 && e <= 253;  // its reciprocal is a normal power of two
    const float inv = __uint_as_float((254u - e) << 23);

    uint8_t *rows = (is_v ? p.v_pool : p.k_pool) +
                    (((int64_t)page * p.page_size + in_page) * H + h) * kRow + (lane & 15) * 8;
    const int64_t pitch = (int64_t)H * kRow;  // from one slot to the next
    if (finite && power) {
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
            const int slot = 2 * i + (lane >> 4);
            if (slot >= s0 && slot < s1) st_v2(rows + slot * pitch, codes8_fitting<I8>(x[i], inv));
        }
    } else {
#pragma unroll 1
        for (int i = 0; i < kPasses; ++i) {
            const int slot = 2 * i + (lane >> 4);
            if (slot < s0 || slot >= s1) continue;
            const uint4 y = ld_stream_v4(src + (row0 + slot - s0) * stride);
            const uint32_t w[4] = {y.x, y.y, y.z, y.w};
            float q[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                q[2 * k] = __fdiv_rn(bf16_lo(w[k]), scale);
                q[2 * k + 1] = __fdiv_rn(bf16_hi(w[k]), scale);
            }
            st_v2(rows + slot * pitch, codes8<I8>(q));
        }
    }
    if (s0 == 0 || scale != had) {
        if (lane == 0) *scale_at = scale;
        // earlier tokens go to the larger scale (`need` then: a power of two)
        for (int slot = lane >> 4; slot < s0; slot += 2) {
            const uint2 c = *reinterpret_cast<const uint2 *>(rows + slot * pitch);
            float q[8];
            values8<I8>(c, q);
#pragma unroll
            for (int k = 0; k < 8; ++k) q[k] = q[k] * had * inv;
            st_v2(rows + slot * pitch, codes8<I8>(q));
        }
    }
}

}  // namespace

cudaError_t launch_append_block(bool int8, const AppendBlockParams &params, cudaStream_t stream, bool pdl) {
    AppendBlockParams p = params;
    p.per_request = (p.s_q + kScaleBlock - 2) / kScaleBlock + 1;
    const int64_t slots =
        p.starts == nullptr ? (int64_t)p.B * p.per_request : (int64_t)p.N / kScaleBlock + 2 * (int64_t)p.B;
    p.jobs = slots * 2 * p.H_kv;
    const int64_t blocks = (p.jobs + kThreads / 32 - 1) / (kThreads / 32);
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    return int8 ? cudaLaunchKernelEx(&cfg, append_block_kernel<true>, p)
                : cudaLaunchKernelEx(&cfg, append_block_kernel<false>, p);
}

}  // namespace da
