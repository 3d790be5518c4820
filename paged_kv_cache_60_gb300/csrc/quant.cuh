// Writing KV rows in the pool formats: 16-byte loads and stores, the e4m3
// quantiser (per-head scales, or per block of the 656-byte latent token) and
// the latent token's row, shared by the kernels that write new tokens.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace da {

constexpr int kLatentRow = 656;
constexpr int kLatentNope = 512;
constexpr int kLatentScales = 512;   // byte offset of the 4 fp32 scales
constexpr int kLatentRope = 528;     // byte offset of the 64 bf16 RoPE values
constexpr float kE4m3Max = 448.f;

__device__ __forceinline__ uint4 ld_stream_v4(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

__device__ __forceinline__ void st_v4(void *p, uint4 v) {
    asm volatile("st.global.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

__device__ __forceinline__ void st_v2(void *p, uint2 v) {
    asm volatile("st.global.v2.u32 [%0], {%1, %2};" ::"l"(p), "r"(v.x), "r"(v.y) : "memory");
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two fp32 values -> two e4m3 codes (lo in bits 0..7, hi in bits 8..15):
// round to nearest even, finite results saturate at +-448, NaN -> 0x7F (one
// test per pair on the common path: the sum of two values is NaN when either
// is).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    uint32_t c = r;
    const float t = lo + hi;
    if (t != t) {
        if (lo != lo) c = (c & 0xFF00u) | 0x7Fu;
        if (hi != hi) c = (c & 0x00FFu) | 0x7F00u;
    }
    return c;
}

// The reciprocal of a scale and whether Markstein's correction applies to it:
// y = RN(1 / s) (correctly rounded), for scales in [2^-80, 2^100]: the
// reciprocal stays normal, and an input small enough for the residual below to
// underflow (|x| < 2^-100) gives |x / s| < 2^-20, which codes to a signed zero
// whatever its last bit.
struct Recip {
    float s, y;
    bool ok;
};
__device__ __forceinline__ Recip recip_of(float s) {
    const float a = fabsf(s);
    return Recip{s, __frcp_rn(s), a >= 0x1p-80f && a <= 0x1p100f};
}

// RN(x / s), the quotient rounded to nearest, by Markstein's correction
// (P. Markstein, "Computation of elementary functions on the IBM RISC
// System/6000 processor", IBM J. Res. Develop. 34 (1990)): with y = RN(1/s),
// q0 = RN(x y) is within an ulp of x / s, the residual r = x - q0 s is exact
// in one fused multiply-add, and RN(q0 + r y) is the rounded quotient, as long
// as nothing overflows or underflows on the way. That equality was checked
// exhaustively over every finite bf16 x with |x| >= 2^-100 and |x / s| in
// [2^-12, 2^10] for 5090 scales (powers of two and their neighbours,
// log-uniform 1e-4 .. 1e2, amax / 448): the range in which the e4m3 code
// depends on the quotient's value. For fp32 x (rotated keys) it is the boundaries
// between codes that matter, numbers of five significant bits: within 8 ulps of
// boundary * s the quotient was compared for all 2^23 significands of s and all
// 16 of the boundary (2.28 * 10^9 quotients, no difference); further away an
// ulp or two changes no code. Below that range the code is a signed zero (the
// sign is taken from q0, so -0 stays -0), above it the code saturates, and a
// NaN input gives a NaN quotient, so those need no test. What does: a scale
// outside the range recip_of accepts, an infinite input, and a quotient large
// enough to overflow the residual (|x| y >= 2^100): one running max of |x| per
// group of values tells, and the IEEE division runs only where some active
// lane of the warp has such a value (the vote is over the lanes that reach it:
// requests that are skipped leave the loop first).
// Pairs of values go through the packed fp32 pipe (mul.rn / fma.rn on .f32x2:
// each lane rounds exactly as the scalar instruction does).
__device__ __forceinline__ uint64_t f2pack(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void f2unpack(uint64_t r, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
template <int N>
__device__ __forceinline__ void quot_rn(const float (&x)[N], const Recip &d, float (&q)[N]) {
    static_assert(N % 2 == 0, "pairs of values");
    float mx = 0.f;
    const uint64_t y2 = f2pack(d.y, d.y), ns2 = f2pack(-d.s, -d.s);
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const uint64_t x2 = f2pack(x[i], x[i + 1]);
        uint64_t q02, r2, qq2;
        asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q02) : "l"(x2), "l"(y2));
        asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r2) : "l"(q02), "l"(ns2), "l"(x2));
        asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(qq2) : "l"(r2), "l"(y2), "l"(q02));
        float q0a, q0b, qa, qb;
        f2unpack(q02, q0a, q0b);
        f2unpack(qq2, qa, qb);
        q[i] = copysignf(qa, q0a);
        q[i + 1] = copysignf(qb, q0b);
        mx = fmaxf(mx, fmaxf(fabsf(x[i]), fabsf(x[i + 1])));
    }
    const bool fast = d.ok && mx < INFINITY && mx * fabsf(d.y) < 0x1p100f;
    if (!__all_sync(__activemask(), fast)) {
        if (!fast) {
#pragma unroll
            for (int i = 0; i < N; ++i) q[i] = __fdiv_rn(x[i], d.s);
        }
    }
}

// RN(a / 448), the block scale of the 656-byte token, by the same correction
// with the constant y = RN(1/448); checked exhaustively against the IEEE
// division for every bf16 magnitude >= 2^-100 (the block maxima are bf16
// values). Smaller, infinite or NaN maxima take the division.
__device__ __forceinline__ float div448(float a) {
    constexpr float y = 0x1.24924ap-9f;  // RN(1 / 448)
    if (!(a >= 0x1p-100f && a < INFINITY)) return __fdiv_rn(a, kE4m3Max);
    const float q0 = a * y;
    const float r = fmaf(-q0, kE4m3Max, a);
    return fmaf(r, y, q0);
}

// Eight bf16 values (one 16-byte vector) / s -> eight e4m3 codes.
__device__ __forceinline__ uint2 quant8(uint4 x, const Recip &d) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float v[8], q[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
    }
    quot_rn(v, d, q);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = e4m3x2(q[2 * i], q[2 * i + 1]);
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// 656-byte latent tokens, one warp per token. Lane l holds NoPE values
// [16l, 16l+16); lanes 8k..8k+7 form block k; lanes 0..7 hold the RoPE values.
struct LatentIn {
    uint4 a0, a1, rope;
};
// src: the token's 576 bf16 values (512 NoPE, then 64 RoPE)
__device__ __forceinline__ LatentIn latent_load(const uint16_t *src, int lane) {
    LatentIn x;
    x.a0 = ld_stream_v4(src + lane * 16);
    x.a1 = ld_stream_v4(src + lane * 16 + 8);
    x.rope = lane < 8 ? ld_stream_v4(src + kLatentNope + lane * 8) : make_uint4(0u, 0u, 0u, 0u);
    return x;
}
// The NoPE codes and scales of a token; every lane of the warp calls this for
// the same token. row: its 656 bytes in the pool.
__device__ __forceinline__ void latent_store_nope(uint8_t *row, int lane, const LatentIn &x) {
    const uint32_t w[8] = {x.a0.x, x.a0.y, x.a0.z, x.a0.w, x.a1.x, x.a1.y, x.a1.z, x.a1.w};
    // max |x| by the magnitude bits: exact, and a NaN wins (scale 1 then)
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        m = max(m, (w[i] << 16) & 0x7FFFFFFFu);
        m = max(m, w[i] & 0x7FFF0000u);
    }
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
    const float amax = __uint_as_float(m);
    const float scale = amax > 0.f ? div448(amax) : 1.f;
    const Recip d = recip_of(scale);
    float v[16], q[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
    }
    quot_rn(v, d, q);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = e4m3x2(q[4 * i], q[4 * i + 1]) | (e4m3x2(q[4 * i + 2], q[4 * i + 3]) << 16);
    st_v4(row + lane * 16, make_uint4(c[0], c[1], c[2], c[3]));
    const float s1 = __shfl_sync(0xFFFFFFFFu, scale, 8);
    const float s2 = __shfl_sync(0xFFFFFFFFu, scale, 16);
    const float s3 = __shfl_sync(0xFFFFFFFFu, scale, 24);
    if (lane == 0)
        st_v4(row + kLatentScales,
              make_uint4(__float_as_uint(scale), __float_as_uint(s1), __float_as_uint(s2), __float_as_uint(s3)));
}
__device__ __forceinline__ void latent_store(uint8_t *row, int lane, const LatentIn &x) {
    latent_store_nope(row, lane, x);
    if (lane < 8) st_v4(row + kLatentRope + lane * 16, x.rope);
}

}  // namespace da
