// rope_row.cuh -- a row's rotation and its quantisation, as the cache writes
// share them: thread c of a row's D/16 holds the 8-value chunks that start at
// 8c and at D/2 + 8c.
#pragma once
#include <cuda_fp8.h>

#include "pkv_internal.h"
#include "pkv_ptx.cuh"

namespace pkv {

struct Chunk8 {
    float v[8];
};

__device__ __forceinline__ Chunk8 unpack_bf16x8(uint4 w) {
    Chunk8 c;
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        c.v[2 * i] = bf16_lo(u[i]);
        c.v[2 * i + 1] = bf16_hi(u[i]);
    }
    return c;
}

__device__ __forceinline__ uint4 pack_bf16x8(const Chunk8& c) {
    uint4 w;
    w.x = pack_bf16(c.v[0], c.v[1]);
    w.y = pack_bf16(c.v[2], c.v[3]);
    w.z = pack_bf16(c.v[4], c.v[5]);
    w.w = pack_bf16(c.v[6], c.v[7]);
    return w;
}

// Packed float32 product (sm_100+ f32x2 arithmetic): each lane is rounded
// exactly as the scalar product would be, in one issue slot for two values.
// Where a sum follows (the rotation), the sum is a scalar operation with
// explicit rounding, which is never contracted with the product.
__device__ __forceinline__ void mul_rn_x2(float a0, float a1, float b0, float b1, float& d0, float& d1) {
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d0), "=f"(d1) : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}
// Four E4M3 bytes (a -> byte 0 .. d -> byte 3), saturating round-to-nearest-even.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
        "mov.b32 %0, {l, h};\n\t}"
        : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
    return r;
}

// Per-scale constants of the FP8 quantiser: the reciprocal of the scale
// nudged down and up by 2^-20 (relative), each rounded to float32.
struct E4m3Rcp {
    float lo, hi;
    bool exact_only;  // a scale whose reciprocal could leave float32's normal range
};
__device__ __forceinline__ E4m3Rcp e4m3_rcp(float scale) {
    E4m3Rcp r;
    r.exact_only = !(scale >= 0x1p-100f && scale <= 0x1p100f);
    const float rcp = __frcp_rn(scale);
    r.lo = __fmul_rn(rcp, 1.0f - 0x1p-20f);
    r.hi = __fmul_rn(rcp, 1.0f + 0x1p-20f);
    return r;
}

// E4M3 bytes (low byte first) of the correctly rounded float32 quotients
// Q = RN(y / scale), saturating, for the 8 values of a chunk, without a
// division in the common case. With r = RN(1/scale), r_lo = RN(r (1 - 2^-20))
// and r_hi = RN(r (1 + 2^-20)), the products z_lo = RN(y r_lo) and
// z_hi = RN(y r_hi) differ from y / scale by factors within
// (1 - 2^-20)(1 +- 2^-24)^3 and (1 + 2^-20)(1 +- 2^-24)^3, while Q differs from
// it by a factor within 1 +- 2^-24; so Q lies between z_lo and z_hi (values
// so small that float32 rounds them absolutely are far below E4M3's smallest
// step, where every one of the three gives the zero byte of the right
// sign). E4M3 rounding is monotone, so when z_lo and z_hi give the same byte,
// Q gives it too. When they differ -- Q is within about 2^-19 (relative) of
// an E4M3 rounding boundary, about one value in 2^15 -- the chunk is
// quantised from the IEEE divisions.
__device__ __forceinline__ uint2 pack_e4m3x8(const Chunk8& c, float scale, const E4m3Rcp& r) {
    float zl[8], zh[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        mul_rn_x2(c.v[j], c.v[j + 1], r.lo, r.lo, zl[j], zl[j + 1]);
        mul_rn_x2(c.v[j], c.v[j + 1], r.hi, r.hi, zh[j], zh[j + 1]);
    }
    uint32_t w0 = e4m3x4(zl[0], zl[1], zl[2], zl[3]);
    uint32_t w1 = e4m3x4(zl[4], zl[5], zl[6], zl[7]);
    const uint32_t h0 = e4m3x4(zh[0], zh[1], zh[2], zh[3]);
    const uint32_t h1 = e4m3x4(zh[4], zh[5], zh[6], zh[7]);
    if ((w0 != h0) | (w1 != h1) | r.exact_only) {
        float z[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) z[j] = __fdiv_rn(c.v[j], scale);
        w0 = e4m3x4(z[0], z[1], z[2], z[3]);
        w1 = e4m3x4(z[4], z[5], z[6], z[7]);
    }
    return make_uint2(w0, w1);
}

__device__ __forceinline__ float amax8(const Chunk8& c) {
    float m = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(c.v[j]));
    return m;
}

// Bracketing reciprocals of a divisor d: RN(RN(1/d) (1 -+ 2^-20)). For any y,
// RN(y * lo) and RN(y * hi) enclose the correctly rounded quotient RN(y / d)
// (the argument of pack_e4m3x8), so a monotone rounding that gives both the
// same code gives the quotient that code too. Divisors whose reciprocal could
// leave float32's normal range are marked for the division path.
__device__ __forceinline__ E4m3Rcp bracket_rcp(float d) { return e4m3_rcp(d); }

// The same brackets from the hardware's approximate reciprocal r ~ 1/d
// (rcp.approx.f32, documented within one unit in the last place; measured on
// GB300 over every float32 in [2^-30, 2^30): relative error at most
// 2^-23.27). With
// |r d - 1| < 2^-22 the products RN(y RN(r (1 -+ 2^-20))) still differ from
// y / d by factors within (1 -+ 2^-20)(1 +- 2^-22)(1 +- 2^-24)^2, i.e.
// strictly beyond the 1 +- 2^-24 of RN(y / d) on each side, so they still
// enclose it. Used for the per-block divisors of the NVFP4 quantiser.
__device__ __forceinline__ E4m3Rcp bracket_rcp_approx(float d) {
    E4m3Rcp r;
    r.exact_only = !(d >= 0x1p-100f && d <= 0x1p100f);
    float rcp;
    asm("rcp.approx.f32 %0, %1;" : "=f"(rcp) : "f"(d));
    r.lo = __fmul_rn(rcp, 1.0f - 0x1p-20f);
    r.hi = __fmul_rn(rcp, 1.0f + 0x1p-20f);
    return r;
}

// One 8-value half of an NVFP4 block whose largest magnitude is `amax`,
// under the static scale g (six_g = RN(6 g), r6 = bracket_rcp(six_g)):
// returns the four bytes of E2M1 pairs and the block's E4M3 scale byte,
// which are those of the correctly rounded quotients amax / six_g and
// y / RN(g s). Each is taken from the bracketing products when both
// products give the same code, else (rarely) from the IEEE divisions.
__device__ __forceinline__ uint32_t nvfp4_half(const Chunk8& c, float amax, float g, float six_g,
                                               const E4m3Rcp& r6, uint32_t& sbyte) {
    uint32_t sb;
    {
        uint16_t bl, bh;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(bl) : "f"(__fmul_rn(amax, r6.hi)), "f"(__fmul_rn(amax, r6.lo)));
        bh = static_cast<uint16_t>(bl >> 8);
        bl = static_cast<uint16_t>(bl & 0xFF);
        sb = bl;
        if (bl != bh || r6.exact_only)
            sb = __nv_cvt_float_to_fp8(__fdiv_rn(amax, six_g), __NV_SATFINITE, __NV_E4M3);
    }
    sbyte = sb;
    const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(sb), __NV_E4M3)));
    if (s == 0.f) return 0u;
    const float denom = __fmul_rn(g, s);
    const E4m3Rcp r = bracket_rcp_approx(denom);
    float zl[8], zh[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        mul_rn_x2(c.v[j], c.v[j + 1], r.lo, r.lo, zl[j], zl[j + 1]);
        mul_rn_x2(c.v[j], c.v[j + 1], r.hi, r.hi, zh[j], zh[j + 1]);
    }
    const uint32_t wl = pack_e2m1x8(zl);
    if (wl == pack_e2m1x8(zh) && !r.exact_only) return wl;
    float z[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) z[j] = __fdiv_rn(c.v[j], denom);
    return pack_e2m1x8(z);
}

__device__ __forceinline__ uint32_t lane_id() {
    uint32_t l;
    asm("mov.u32 %0, %%laneid;" : "=r"(l));
    return l;
}

// The cos and sin a thread needs for its two chunks, loaded as four 16-byte
// vectors. NeoX: chunk 8c pairs with chunk D/2 + 8c at frequencies 8c..8c+7.
// Interleaved: chunk 8c holds the pairs of frequencies 4c..4c+3, chunk
// D/2 + 8c those of D/4 + 4c .. D/4 + 4c + 3.
template <int D, bool INTER>
__device__ __forceinline__ void load_cos_sin(const float* cs, int c, float (&cv)[8], float (&sv)[8]) {
    float4 a0, a1, b0, b1;
    if constexpr (!INTER) {
        a0 = *reinterpret_cast<const float4*>(cs + 8 * c);
        a1 = *reinterpret_cast<const float4*>(cs + 8 * c + 4);
        b0 = *reinterpret_cast<const float4*>(cs + D / 2 + 8 * c);
        b1 = *reinterpret_cast<const float4*>(cs + D / 2 + 8 * c + 4);
    } else {
        a0 = *reinterpret_cast<const float4*>(cs + 4 * c);
        a1 = *reinterpret_cast<const float4*>(cs + D / 4 + 4 * c);
        b0 = *reinterpret_cast<const float4*>(cs + D / 2 + 4 * c);
        b1 = *reinterpret_cast<const float4*>(cs + D / 2 + D / 4 + 4 * c);
    }
    cv[0] = a0.x; cv[1] = a0.y; cv[2] = a0.z; cv[3] = a0.w;
    cv[4] = a1.x; cv[5] = a1.y; cv[6] = a1.z; cv[7] = a1.w;
    sv[0] = b0.x; sv[1] = b0.y; sv[2] = b0.z; sv[3] = b0.w;
    sv[4] = b1.x; sv[5] = b1.y; sv[6] = b1.z; sv[7] = b1.w;
}

// y1 = x1 c - x2 s, y2 = x2 c + x1 s for every pair of the row's two chunks,
// each product and the sum / difference rounded on its own, never fused:
// the products are packed f32x2 multiplies (two per instruction, explicit
// round-to-nearest), the sums and differences scalar operations with
// explicit rounding. (A packed sum reading a packed product may be
// contracted into a fused multiply-add by the compiler, which changes the
// rounding; the scalar forms are not.)
template <bool INTER>
__device__ __forceinline__ void rotate_row(Chunk8& lo, Chunk8& hi, const float (&cv)[8], const float (&sv)[8]) {
    if constexpr (!INTER) {
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            float lc0, lc1, hs0, hs1, hc0, hc1, ls0, ls1;
            mul_rn_x2(lo.v[j], lo.v[j + 1], cv[j], cv[j + 1], lc0, lc1);
            mul_rn_x2(hi.v[j], hi.v[j + 1], sv[j], sv[j + 1], hs0, hs1);
            mul_rn_x2(hi.v[j], hi.v[j + 1], cv[j], cv[j + 1], hc0, hc1);
            mul_rn_x2(lo.v[j], lo.v[j + 1], sv[j], sv[j + 1], ls0, ls1);
            lo.v[j] = __fsub_rn(lc0, hs0);
            lo.v[j + 1] = __fsub_rn(lc1, hs1);
            hi.v[j] = __fadd_rn(hc0, ls0);
            hi.v[j + 1] = __fadd_rn(hc1, ls1);
        }
    } else {
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            float p0, p1, q0, q1;
            // lo pair (2m, 2m + 1) at frequency m
            mul_rn_x2(lo.v[2 * m], lo.v[2 * m + 1], cv[m], cv[m], p0, p1);
            mul_rn_x2(lo.v[2 * m + 1], lo.v[2 * m], sv[m], sv[m], q0, q1);
            lo.v[2 * m] = __fsub_rn(p0, q0);
            lo.v[2 * m + 1] = __fadd_rn(p1, q1);
            // hi pair at frequency 4 + m
            mul_rn_x2(hi.v[2 * m], hi.v[2 * m + 1], cv[4 + m], cv[4 + m], p0, p1);
            mul_rn_x2(hi.v[2 * m + 1], hi.v[2 * m], sv[4 + m], sv[4 + m], q0, q1);
            hi.v[2 * m] = __fsub_rn(p0, q0);
            hi.v[2 * m + 1] = __fadd_rn(p1, q1);
        }
    }
}

}  // namespace pkv
