// Rotary positions with several axes, fused with the KV append.
//
// Pair i of the rotated values of a head turns by the angle
//     theta = pos[axis(i)][n] * inv_freq[i],
//     (x, y) -> (x cos theta - y sin theta, x sin theta + y cos theta),
// where a token has one position per axis (time, height, width) and axis(i)
// comes from the sections: in blocks (the first sections[0] pairs follow axis
// 0, the next sections[1] axis 1, ...) or alternating. q goes rotated to
// q_out, K rotated and V as it is into the page slot of the token, in the
// pool's format (bf16, e4m3 with one scale per head, the 656-byte token, whose
// last 64 values are the rotated ones). Products and sums are fp32, each value
// is rounded once.
//
// The angle: positions reach far beyond what an fp32 product keeps of an angle
// (position 10^6 has an ulp of 0.06 rad), so the phase is kept in turns as a
// 64-bit fraction, F = inv_freq / (2 pi) mod 1 in units of 2^-64 from the fp32
// bits of inv_freq, and pos * F wraps modulo one turn in integer arithmetic: F
// is short of inv_freq / (2 pi) by less than |inv_freq| + 1 of its units (the
// constant's last unit, then the shift's), the phase by |pos| (|inv_freq| + 1)
// 2^-64 turns. The top 32 bits, as a signed fraction of half a turn, go to
// sincospif; as an fp32 number they keep 24, an error of at most 2^-26 turns
// (1e-7 radians), next to the 2 ulp of sincospif.
//
// Bound by HBM: every value is read and written once. A block works on a tile
// of tokens: it computes each token's angles once, into shared memory, and then
// walks over the tile's rows (a row is one head of q, K or V of one token). Work
// item = 16 values of a row (two 16-byte vectors, the two halves of eight
// pairs); a thread keeps its place in the rows and takes a few rows at a time,
// their loads in flight together. The next tile's angles are computed before
// this tile's rows, so one barrier a tile is all there is.
#include <cuda_runtime.h>

#include <cstdint>

#include "common.cuh"
#include "decode_attn.h"
#include "layout.h"
#include "quant.cuh"

namespace da {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 32;    // tokens of a tile
constexpr int kMaxAngles = 1024;  // angles of a tile (at least one token's)
// rows a thread has in flight (the e4m3 build's quotients leave registers for two)
constexpr int unroll_of(int kv) { return kv == DA_KV_FP8_PER_TENSOR ? 2 : 4; }

// inv_freq / (2 pi) mod 1, in units of 2^-64, from the fp32 bits: mantissa
// (24 bits) times floor(2^64 / (2 pi)), shifted by the exponent. Finite input.
__device__ __forceinline__ uint64_t turns_of(float f) {
    constexpr uint64_t kInv2Pi = 0x28BE60DB9391054Aull;  // floor(2^64 / (2 pi))
    const uint32_t u = __float_as_uint(f);
    const int ex = (int)((u >> 23) & 255u);
    const uint64_t m = (u & 0x7FFFFFu) | (ex ? 0x800000u : 0u);
    const int e = (ex ? ex : 1) - 150;  // f = m 2^e
    const uint64_t lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
    uint64_t r = 0;
    if (e >= 0) {
        if (e < 64) r = lo << e;
    } else if (e > -64) {
        r = (lo >> -e) | (hi << (64 + e));
    } else if (e > -128) {
        r = hi >> (-e - 64);
    }
    return (u >> 31) ? 0ull - r : r;
}

// cos and sin of pos * F turns, each within 2^-22 where F is exact: 2 pi 2^-26 from the conversion to float, and 2 ulp
__device__ __forceinline__ float2 cos_sin(int32_t pos, uint64_t F, bool finite) {
    const uint64_t phase = (uint64_t)(int64_t)pos * F;
    const float half_turns = (float)(int32_t)(phase >> 32) * 0x1p-31f;
    float s, c;
    sincospif(half_turns, &s, &c);
    return finite ? make_float2(c, s) : make_float2(NAN, NAN);
}

__device__ __forceinline__ int axis_of(const RopeParams &p, int i) {
    if (p.interleaved) {
        const int a = i % p.n_axes;
        return i / p.n_axes < p.sections[a] ? a : 0;
    }
    int a = 0, end = p.sections[0];
    while (a + 1 < p.n_axes && i >= end) end += p.sections[++a];
    return a;
}

constexpr int64_t kSkip = -2;    // negative position: the token is skipped
constexpr int64_t kNowhere = -1;  // invalid request, position or page: no K / V row is written

// Pool slot of token n (page * page_size + slot), or one of the above.
__device__ __forceinline__ int64_t slot_of(const RopeParams &p, int n, bool reporter) {
    const int t = p.positions[n];
    if (t < 0) return kSkip;
    const int b = p.requests ? p.requests[n] : n / p.s_q;
    if (b < 0 || b >= p.B) {
        if (reporter && p.error) atomicOr(p.error, DA_DEV_BAD_REQUEST);
        return kNowhere;
    }
    if ((int64_t)t >= (int64_t)p.max_pages * p.page_size) {
        if (reporter && p.error) atomicOr(p.error, DA_DEV_SEQ_TOO_LONG);
        return kNowhere;
    }
    const int page = p.block_table[(int64_t)b * p.max_pages + t / p.page_size];
    if (page < 0 || page >= p.num_pages) {
        if (reporter && p.error) atomicOr(p.error, DA_DEV_BAD_PAGE);
        return kNowhere;
    }
    return (int64_t)page * p.page_size + t % p.page_size;
}

// 16-byte load of q, K or V rows: plain (q may be rotated in place)
__device__ __forceinline__ uint4 ld_row(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p)
                 : "memory");
    return v;
}

__device__ __forceinline__ void unpack8(uint4 x, float *v) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
    }
}
__device__ __forceinline__ uint4 pack8(const float *v) {
    return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

// Rotates the eight pairs of item j; cs: a token's (cos, sin), two pairs to a
// vector, vector k of item j at [k][j] (so that the items' lanes read side by side).
template <bool kAdjacent>
__device__ __forceinline__ void rotate16(float (&x)[16], const float4 *cs, int j, int turned) {
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
        const float4 c2 = cs[(k / 2) * turned + j];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const float c = u ? c2.z : c2.x, s = u ? c2.w : c2.y;
            const int i = kAdjacent ? 2 * (k + u) : k + u, j = kAdjacent ? i + 1 : i + 8;
            const float a = x[i], b = x[j];
            x[i] = a * c - b * s;
            x[j] = a * s + b * c;
        }
    }
}

// One token's latent row, by one warp: NoPE quantised as the append does, the
// RoPE part rotated, lane l its pair l (or the two values that pass through).
template <bool kAdjacent>
__device__ __forceinline__ void latent_token(const RopeParams &p, int n, int lane, uint64_t F, bool finite, int axis) {
    const uint16_t *src = p.k + (int64_t)n * p.k_stride;
    LatentIn x;
    x.a0 = ld_stream_v4(src + lane * 16);
    x.a1 = ld_stream_v4(src + lane * 16 + 8);
    const int half = p.rot / 2;
    const bool turn = lane < half;
    const int i = kAdjacent || !turn ? 2 * lane : lane, j = kAdjacent || !turn ? i + 1 : lane + half;
    const float a = __uint_as_float((uint32_t)src[kLatentNope + i] << 16);
    const float b = __uint_as_float((uint32_t)src[kLatentNope + j] << 16);
    const float2 cs = turn ? cos_sin(p.rope_pos[(int64_t)axis * p.N + n], F, finite) : make_float2(1.f, 0.f);
    const int64_t slot = slot_of(p, n, lane == 0);  // uniform over the warp
    if (slot < 0) return;
    uint8_t *row = p.k_pool + slot * kLatentRow;
    latent_store_nope(row, lane, x);
    uint16_t *out = reinterpret_cast<uint16_t *>(row + kLatentRope);
    const uint32_t ab = turn ? pack_bf16(a * cs.x - b * cs.y, a * cs.y + b * cs.x)
                             : (__float_as_uint(a) >> 16) | (__float_as_uint(b) & 0xFFFF0000u);
    if (kAdjacent || !turn) {
        *reinterpret_cast<uint32_t *>(out + i) = ab;
    } else {
        out[i] = (uint16_t)(ab & 0xFFFFu);
        out[j] = (uint16_t)(ab >> 16);
    }
}

template <int kKv, bool kAdjacent>
__global__ void __launch_bounds__(kThreads, 3) rope_kernel(const __grid_constant__ RopeParams p) {
    extern __shared__ float4 smem[];  // [2][tokens][4][turned] angles
    __shared__ int64_t s_slot[2][kMaxTokens];
    constexpr bool kLatent = kKv == DA_KV_FP8_MLA656;
    constexpr int kUnroll = unroll_of(kKv);
    const int tid = threadIdx.x, pairs = p.rot / 2, turned = p.rot / 16;  // items j < turned are rotated (q and K)
    pdl_wait();
    pdl_launch_dependents();

    if (kLatent && (int)blockIdx.x >= p.q_blocks) {
        const int lane = tid & 31;
        const bool turn = lane < pairs;
        const float f = turn ? p.inv_freq[lane] : 0.f;
        const bool finite = fabsf(f) < INFINITY;
        const uint64_t F = finite ? turns_of(f) : 0;
        const int axis = turn ? axis_of(p, lane) : 0;
        const int64_t step = (int64_t)(gridDim.x - p.q_blocks) * (kThreads / 32);
        for (int64_t n = (int64_t)(blockIdx.x - p.q_blocks) * (kThreads / 32) + (tid >> 5); n < p.N; n += step)
            latent_token<kAdjacent>(p, (int)n, lane, F, finite, axis);
        return;
    }

    // angles: thread (ta, ia) computes pair ia of tokens ta, ta + at, ...
    const int at = kThreads / pairs, ta = tid / pairs, ia = tid - ta * pairs;
    uint64_t F = 0;
    bool finite = true;
    const int32_t *apos = p.rope_pos;
    if (ta < at) {
        const float f = p.inv_freq[ia];
        finite = fabsf(f) < INFINITY;
        F = finite ? turns_of(f) : 0;
        apos += (int64_t)axis_of(p, ia) * p.N;
    }
    const int cs_at = (((ia & 7) >> 1) * turned + (ia >> 3)) * 2 + (ia & 1);  // of its (cos, sin) in a token's angles
    const int tiles = (p.N + p.tokens - 1) / p.tokens;
    // block -> tile (the grid strides over them) and part of the tile's rows
    const int first = blockIdx.x / p.parts, part = blockIdx.x - first * p.parts;
    const int stride = (kLatent ? p.q_blocks : (int)gridDim.x) / p.parts;
    auto prepare = [&](int tile, int buf) {
        const int n0 = tile * p.tokens, nt = min(p.tokens, p.N - n0);
        if (ta < at) {
            float2 *cs = reinterpret_cast<float2 *>(smem) + (size_t)buf * p.tokens * pairs + cs_at;
            for (int t = ta; t < nt; t += at) cs[t * pairs] = cos_sin(apos[n0 + t], F, finite);
        }
        const int t = tid - (kThreads - 32);
        if (t >= 0 && t < nt)
            s_slot[buf][t] = !kLatent                           ? slot_of(p, n0 + t, part == 0)
                             : p.positions[n0 + t] < 0 ? kSkip
                                                               : kNowhere;
    };

    // this thread's place in the rows: item j, of every per_pass-th row
    const int per_pass = kThreads / p.items, hs = tid / p.items, j = tid - hs * p.items;
    const bool in_rot = j < turned;
    // the item's two vectors in q and K rows; on the 656-byte format the rotated values start at 512, and the
    // copied items are those before them, then what is left behind them
    int r0, r1;
    if (in_rot) {
        r0 = (kLatent ? kLatentNope : 0) + (kAdjacent ? 16 * j : 8 * j);
        r1 = r0 + (kAdjacent ? 8 : pairs);
    } else {
        const int c = 16 * (j - turned);
        r0 = !kLatent || c >= kLatentNope ? c + p.rot : c;
        r1 = r0 + 8;
    }
    const int v0 = 16 * j, v1 = 16 * j + 8;              // in V rows
    const bool has1 = in_rot || r1 < p.D, v_has1 = v1 < p.D;  // D = 8 mod 16: the last item has one vector
    const int hq = p.H_q, hk = kLatent ? 0 : p.H_kv;
    const int step_t = per_pass / p.heads, step_h = per_pass - step_t * p.heads;

    if (first >= tiles) return;
    // rows [r, end) of the tile at n0 are left, the first of them head h of token t
    int n0, r, end, t, h;
    auto enter = [&](int tile) {
        n0 = tile * p.tokens;
        const int rows = min(p.tokens, p.N - n0) * p.heads;
        end = (int)((int64_t)rows * (part + 1) / p.parts);
        r = (int)((int64_t)rows * part / p.parts) + hs;
        t = r / p.heads;
        h = r - t * p.heads;
        if (hs >= per_pass) r = end;                     // threads behind the last whole row of a pass
    };
    // a batch of rows: loaded before the tile's slots are known (rows of skipped tokens are read in vain)
    uint4 x0[kUnroll], x1[kUnroll];
    int tt[kUnroll], hh[kUnroll], nb;
    auto load = [&]() {
        nb = n0;
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            tt[u] = t;
            hh[u] = r < end && !(h < hq && p.in_place && !in_rot) ? h : -1;
            x0[u] = x1[u] = make_uint4(0u, 0u, 0u, 0u);
            if (hh[u] >= 0) {
                const int64_t n = n0 + t;
                const bool is_v = !kLatent && h >= hq + hk;
                const uint16_t *src = h < hq        ? p.q + n * p.q_stride + (int64_t)h * p.D
                                      : h < hq + hk ? p.k + n * p.k_stride + (int64_t)(h - hq) * p.D
                                                    : p.v + n * p.v_stride + (int64_t)(h - hq - hk) * p.D;
                x0[u] = ld_row(src + (is_v ? v0 : r0));
                if (is_v ? v_has1 : has1) x1[u] = ld_row(src + (is_v ? v1 : r1));
            }
            r += per_pass;
            t += step_t;
            h += step_h;
            if (h >= p.heads) {
                h -= p.heads;
                ++t;
            }
        }
    };
    int buf = 0;
    auto finish = [&]() {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u) {
            const int hd = hh[u];
            if (hd < 0) continue;
            const int64_t slot = s_slot[buf][tt[u]];
            if (slot == kSkip || (hd >= hq && slot < 0)) continue;
            const float4 *cs = smem + ((size_t)buf * p.tokens + tt[u]) * (pairs / 2);
            const bool is_q = hd < hq, is_k = !is_q && hd < hq + hk, is_v = !is_q && !is_k;
            const bool turn = in_rot && !is_v;
            if (kKv != DA_KV_FP8_PER_TENSOR || is_q) {
                if (turn) {
                    float x[16];
                    unpack8(x0[u], x);
                    unpack8(x1[u], x + 8);
                    rotate16<kAdjacent>(x, cs, j, turned);
                    x0[u] = pack8(x);
                    x1[u] = pack8(x + 8);
                }
                uint16_t *o;
                if (is_q)
                    o = p.q_out + ((int64_t)(nb + tt[u]) * hq + hd) * p.D;
                else
                    o = reinterpret_cast<uint16_t *>(is_k ? p.k_pool : p.v_pool) +
                        (slot * p.H_kv + (is_k ? hd - hq : hd - hq - hk)) * p.D;
                st_v4(o + (is_v ? v0 : r0), x0[u]);
                if (is_v ? v_has1 : has1) st_v4(o + (is_v ? v1 : r1), x1[u]);
            } else {
                const int kh = is_k ? hd - hq : hd - hq - hk;
                float x[16], q[16];
                unpack8(x0[u], x);
                unpack8(x1[u], x + 8);
                if (turn) rotate16<kAdjacent>(x, cs, j, turned);
                quot_rn(x, recip_of((is_k ? p.k_scale : p.v_scale)[kh]), q);
                uint32_t c[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) c[i] = e4m3x2(q[2 * i], q[2 * i + 1]);
                uint8_t *o = (is_k ? p.k_pool : p.v_pool) + (slot * p.H_kv + kh) * p.D;
                st_v2(o + (is_v ? v0 : r0), make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16)));
                if (is_v ? v_has1 : has1)
                    st_v2(o + (is_v ? v1 : r1), make_uint2(c[4] | (c[5] << 16), c[6] | (c[7] << 16)));
            }
        }
    };
    enter(first);
    load();
    prepare(first, 0);
    __syncthreads();
    for (int tile = first; tile < tiles; tile += stride, buf ^= 1) {
        const bool more = tile + stride < tiles;
        if (more) prepare(tile + stride, buf ^ 1);
        for (;;) {
            finish();
            if (r >= end) break;
            load();
        }
        if (more) {
            enter(tile + stride);
            load();
        }
        __syncthreads();  // the next tile's angles and slots are there, this one's have been used
    }
}

template <int kKv>
cudaError_t launch(const cudaLaunchConfig_t &cfg, const RopeParams &p) {
    return p.adjacent ? cudaLaunchKernelEx(&cfg, rope_kernel<kKv, true>, p)
                      : cudaLaunchKernelEx(&cfg, rope_kernel<kKv, false>, p);
}

}  // namespace

// Fills in p.items, heads, tokens, parts and q_blocks and launches.
cudaError_t launch_rope(int kv_dtype, RopeParams p, int num_sms, cudaStream_t stream, bool pdl) {
    const bool latent = kv_dtype == DA_KV_FP8_MLA656;
    p.items = latent && p.in_place ? p.rot / 16 : (p.D + 15) / 16;
    p.heads = p.H_q + (latent ? 0 : 2 * p.H_kv);
    const int64_t per_pass = kThreads / p.items, resident = (int64_t)num_sms * 3;
    // tokens of a tile: what leaves every resident block the same number of tiles, at least what one pass of a block
    // covers, at most what fits
    const int64_t fits = kMaxAngles / (p.rot / 2) < kMaxTokens ? kMaxAngles / (p.rot / 2) : kMaxTokens;
    const int64_t rounds = (p.N + resident * fits - 1) / (resident * fits);
    int64_t t = (p.N + resident * rounds - 1) / (resident * rounds);
    if (t < per_pass / p.heads) t = per_pass / p.heads;
    if (t > fits) t = fits;
    // few rows: whole batches of them, so that no thread waits at the barrier with nothing in flight
    const int64_t batch = per_pass * unroll_of(kv_dtype);
    if (t * p.heads > batch && t * p.heads < 4 * batch) t = t * p.heads / batch * batch / p.heads;
    p.tokens = (int32_t)(t < 1 ? 1 : t);
    const int64_t tiles = ((int64_t)p.N + p.tokens - 1) / p.tokens;
    // few tiles: several blocks share a tile's rows, each still with rows for all its threads
    int64_t parts = resident / tiles;
    const int64_t most = ((int64_t)p.tokens * p.heads + per_pass - 1) / per_pass;
    if (parts > most) parts = most;
    p.parts = (int32_t)(parts < 1 ? 1 : parts);
    int64_t blocks = (tiles < resident / p.parts ? tiles : resident / p.parts) * p.parts;
    if (blocks < p.parts) blocks = p.parts;
    p.q_blocks = (int32_t)blocks;
    if (latent) {
        const int64_t lt = ((int64_t)p.N + kThreads / 32 - 1) / (kThreads / 32);
        blocks += lt < resident ? lt : resident;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)2 * p.tokens * (p.rot / 2) * sizeof(float2);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 1 : 0;
    if (latent) return launch<DA_KV_FP8_MLA656>(cfg, p);
    return kv_dtype == DA_KV_FP8_PER_TENSOR ? launch<DA_KV_FP8_PER_TENSOR>(cfg, p) : launch<DA_KV_BF16>(cfg, p);
}

}  // namespace da
