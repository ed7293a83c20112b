// mx_common.cuh -- microscaled blocks: 32 channels that share one power-of-two
// scale, with elements in 8 bits (int8 or e4m3) or 4 bits (e2m1).
//
// A block with largest magnitude a is stored as codes q and a scale byte S,
// value = q * 2^(S - 127).  S is the smallest exponent at which a / 2^(S-127)
// does not pass the format's largest value, so nothing saturates (one case
// aside, below) and, the scale being a power of two, the division is exact and
// the only rounding is that of the element itself, to nearest, ties to even:
// half a step, i.e. 2^-7 of the scale for int8; for e4m3 2^-4 of the value, or
// 2^-10 of the scale below its normal range (2^-6 of the scale); for e2m1 2^-2 of
// the value, or 2^-2 of the scale below 1 times the scale, where a small value
// may round to zero.
// The codes therefore depend on the input alone, not on the order or
// precision of the arithmetic.
//
//   format  largest value       emax (its exponent)  mantissa of the largest
//   int8    127/64 (m / 64)     0                    127/64
//   e4m3    448                 8                    1.75
//   e2m1    6                   2                    1.5
//
// S = 255 marks a block that holds an infinity or NaN; it restores as NaN and
// its codes are zero.  S is clamped to 0..254: at S = 0 the 8-bit formats still
// hold every multiple of 2^-133 (the smallest bf16) that rounds to them, so the
// clamp loses nothing of a bf16 input; at S = 254 an int8 block that needed
// S = 255 saturates at 127.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "mhc_birkhoff.h"

namespace mhc {

constexpr int kMxBlock = 32;    // channels that share a scale
constexpr int kMxScaleNaN = 255;

// Bytes of one row of scales: one per block, padded with zeros to four, so
// that a kernel can fetch scales four bytes at a time.
__host__ __device__ constexpr int64_t mx_scale_pitch(int64_t C) { return 4 * ((C + 127) / 128); }

// Bytes of one row of codes.
__host__ __device__ constexpr int64_t mx_code_pitch(int format, int64_t C)
{
    return format == MHC_MX_E2M1 ? C / 2 : C;
}

template <int kFmt>
struct MxFormat;
template <>
struct MxFormat<MHC_MX_INT8> {
    static constexpr int kEmax = 0;
    static constexpr uint32_t kTopMantissa = 0x7e0000u;  // 127/64 - 1
};
template <>
struct MxFormat<MHC_MX_E4M3> {
    static constexpr int kEmax = 8;
    static constexpr uint32_t kTopMantissa = 0x600000u;  // 0.75
};
template <>
struct MxFormat<MHC_MX_E2M1> {
    static constexpr int kEmax = 2;
    static constexpr uint32_t kTopMantissa = 0x400000u;  // 0.5
};

// Scale byte of a block from the fp32 bits of its largest magnitude.  Adding
// the complement of the top mantissa carries into the exponent exactly when
// the magnitude's mantissa passes it.
template <int kFmt>
__device__ __forceinline__ int mx_scale_byte(uint32_t amax_bits)
{
    if (amax_bits >= 0x7f800000u) return kMxScaleNaN;
    // subnormal: below 2 * 2^-127, which e4m3 and e2m1 hold; int8 holds 127/64 *
    // 2^-127, the largest subnormal bf16, and is given bf16 only
    if (amax_bits < 0x00800000u) return 0;
    const int e = (int)((amax_bits + (0x7fffffu - MxFormat<kFmt>::kTopMantissa)) >> 23) - MxFormat<kFmt>::kEmax;
    return min(max(e, 0), 254);
}

// 2^(S - 127), and 2^(127 - S) for the quantiser.  S = 255 gives NaN; an
// exponent field of zero is the subnormal 2^-127.
__device__ __forceinline__ float mx_scale_value(int S)
{
    const uint32_t b = S == 0 ? 0x00400000u : S == kMxScaleNaN ? 0x7fffffffu : (uint32_t)S << 23;
    return __uint_as_float(b);
}
__device__ __forceinline__ float mx_inverse_scale(int S)
{
    return __uint_as_float(S >= 254 ? 0x00400000u : (uint32_t)(254 - S) << 23);
}

// Eight consecutive elements: two words of 8-bit codes (the second is unused
// for 4-bit codes, which fit in one; the even element is in the low half).
template <int kFmt>
__device__ __forceinline__ uint2 mx_encode8(const float (&f)[8], int S)
{
    if constexpr (kFmt == MHC_MX_INT8) {
        // fma with 1.5 * 2^23 rounds 64 q to an integer, ties to even, into the
        // low bits.  64 / scale is a float for S >= 6, and |64 q| passes 127 at
        // S = 254 only; the other scales take the long way
        uint32_t b[8];
        if (S >= 6 && S < 254) {
            const float inv64 = __uint_as_float((uint32_t)(260 - S) << 23);
#pragma unroll
            for (int e = 0; e < 8; ++e) b[e] = __float_as_uint(fmaf(f[e], inv64, 12582912.0f));
        } else {
            if (S == kMxScaleNaN) return make_uint2(0u, 0u);
            const float inv = mx_inverse_scale(S);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                b[e] = __float_as_uint(fmaf(fminf(fmaxf(f[e] * inv, -1.984375f), 1.984375f), 64.0f, 12582912.0f));
        }
        return make_uint2(__byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410),
                          __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410));
    }
    if (S == kMxScaleNaN) return make_uint2(0u, 0u);
    const float inv = mx_inverse_scale(S);
    float q[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = f[e] * inv;
    if constexpr (kFmt == MHC_MX_E4M3) {
        uint16_t p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(p[e]) : "f"(q[2 * e + 1]), "f"(q[2 * e]));
        return make_uint2((uint32_t)p[0] | (uint32_t)p[1] << 16, (uint32_t)p[2] | (uint32_t)p[3] << 16);
    } else {
        uint32_t w;
        asm("{\n\t.reg .b8 a, b, c, d;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
            "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
            "mov.b32 %0, {a, b, c, d};\n\t}"
            : "=r"(w)
            : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
        return make_uint2(w, 0u);
    }
}

__device__ __forceinline__ void mx_half2_to_float(uint32_t h, float& lo, float& hi)
{
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
        : "=f"(lo), "=f"(hi)
        : "r"(h));
}

// Eight consecutive values from their codes and scale (exact in bf16).
template <int kFmt>
__device__ __forceinline__ void mx_decode8(const uint2 w, float scale, float (&f)[8])
{
    if (kFmt == MHC_MX_INT8) {
        // byte b = m + 128 in the low mantissa bits of 2^23: m = that - (2^23 + 128)
        const float s = scale * 0.015625f;
        const uint32_t u[2] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u};
#pragma unroll
        for (int e = 0; e < 8; ++e)
            f[e] = (__uint_as_float(__byte_perm(u[e >> 2], 0x4b000000u, 0x7440 + (e & 3))) - 8388736.0f) * s;
    } else if (kFmt == MHC_MX_E4M3) {
        const uint32_t u[2] = {w.x, w.y};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint32_t h;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(u[e >> 1] >> (16 * (e & 1)))));
            mx_half2_to_float(h, f[2 * e], f[2 * e + 1]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= scale;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint32_t h;
            asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}"
                : "=r"(h)
                : "r"(w.x >> (8 * e)));
            mx_half2_to_float(h, f[2 * e], f[2 * e + 1]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= scale;
    }
}

// Largest of the four lanes that hold one block (lanes 4k .. 4k + 3 of a full
// warp: a lane holds eight channels).
__device__ __forceinline__ uint32_t mx_block_max(uint32_t v)
{
    v = max(v, __shfl_xor_sync(0xffffffffu, v, 1));
    return max(v, __shfl_xor_sync(0xffffffffu, v, 2));
}

// fp32 bits of the largest magnitude among eight bf16 (an infinity or NaN is
// above every finite magnitude).
__device__ __forceinline__ uint32_t mx_amax8(const uint4 v)
{
    const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
    return max(m & 0xffff0000u, m << 16);
}
__device__ __forceinline__ uint32_t mx_amax8(const float (&f)[8])
{
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(f[e]) & 0x7fffffffu);
    return m;
}

// Writes the scale byte of block k of NB, at its place, and the row's padding
// with its last block.
__device__ __forceinline__ void mx_store_scale(uint8_t* at, int k, int NB, int S)
{
    at[0] = (uint8_t)S;
    if (k == NB - 1)
        for (int p = 1; (k + p) & 3; ++p) at[p] = 0;
}

}  // namespace mhc
