// Block scaling and rounding of 1x32 blocks: the rules of mxfp4_quantize and
// mxfp8_quantize (quantize.cu).  The expert-layer and dense-layer kernels round whole
// blocks with quantize_block and quantize_block_pairs; there, beyond those rules, a block
// that holds an infinity or a NaN gets the scale code 0xFF (NaN), so that the rows
// computed from it show it.
#pragma once

#include <cstdint>

#include "pairs.cuh"

namespace mxfp4 {

// Largest s with 6 * 2^s <= a for a finite a > 0 (float bits): a = f * 2^e
// with f in [1, 2) (or a subnormal), and 6 * 2^s = 1.5 * 2^(s + 2), so
// s = e - 2 when f >= 1.5, else e - 3.
__device__ __forceinline__ int block_exponent(float amax)
{
    if (amax == 0.0f)
        return 0;
    const uint32_t bits = __float_as_uint(amax);
    const int biased = static_cast<int>((bits >> 23) & 0xFFu);
    int s;
    if (biased == 0) {
        s = -127;                                   // below 2^-126: clamps
    } else {
        const int e = biased - 127;
        s = (bits & 0x400000u) ? e - 2 : e - 3;     // f >= 1.5 iff the top significand bit is set
    }
    return s < -127 ? -127 : (s > 127 ? 127 : s);
}

// Two floats -> one byte of two E2M1 codes: `lo` in bits 0-3, `hi` in 4-7.
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi)
{
    uint32_t r;
    asm("{\n\t.reg .b8 t;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n\t"
        "cvt.u32.u8 %0, t;\n\t}"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// floor(log2 amax) - emax from amax's float exponent (a subnormal amax is
// below 2^-126 and clamps).
__device__ __forceinline__ int block_exponent8(float amax, int emax)
{
    if (amax == 0.0f)
        return 0;
    const int biased = static_cast<int>((__float_as_uint(amax) >> 23) & 0xFFu);
    const int s = biased == 0 ? -127 : biased - 127 - emax;
    return s < -127 ? -127 : (s > 127 ? 127 : s);
}

// Output formats of the quantising kernels: packed E2M1, or one E4M3 / E5M2
// code per byte (the ABI's MXFP8_E4M3 and MXFP8_E5M2).
enum class QuantFmt { kE2M1, kE4M3, kE5M2 };

// The scale code of a block for a byte format (its E8M0 byte; 0xFF for an infinity or a NaN among
// its values) and the factor 2^-s, from the largest magnitude.  The code is the float's own biased
// exponent less emax: at most 254 - emax, so 2^-s is a normal number.
template <QuantFmt Q>
__device__ __forceinline__ uint32_t block_scale8(float amax, float &inv)
{
    constexpr int kEmax = Q == QuantFmt::kE4M3 ? 8 : 15;
    const uint32_t bits = __float_as_uint(amax);
    int code = static_cast<int>(bits >> 23) - kEmax;
    code = code < 0 ? 0 : code;
    const bool finite = bits < 0x7F800000u;
    if (bits == 0u || !finite)
        code = 127;
    inv = __uint_as_float(static_cast<uint32_t>(254 - code) << 23);
    return finite ? static_cast<uint32_t>(code) : 0xFFu;
}

// Two floats -> two 8-bit codes: `lo` in bits 0-7, `hi` in bits 8-15.
template <int FMT>
__device__ __forceinline__ uint32_t f8x2(float lo, float hi)
{
    uint32_t r;
    if constexpr (FMT == 0)
        asm("{\n\t.reg .b16 t;\n\t"
            "cvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\n\t"
            "cvt.u32.u16 %0, t;\n\t}"
            : "=r"(r)
            : "f"(hi), "f"(lo));
    else
        asm("{\n\t.reg .b16 t;\n\t"
            "cvt.rn.satfinite.e5m2x2.f32 t, %1, %2;\n\t"
            "cvt.u32.u16 %0, t;\n\t}"
            : "=r"(r)
            : "f"(hi), "f"(lo));
    return r;
}

// 2^-s for s in [-127, 127] (2^127 is normal, 2^-127 subnormal).
__device__ __forceinline__ float exp2_neg(int s)
{
    return s == 127 ? __uint_as_float(0x00400000u) : __uint_as_float(static_cast<uint32_t>(127 - s) << 23);
}

template <QuantFmt Q>
struct QuantTraits {
    static constexpr int kWords = Q == QuantFmt::kE2M1 ? 4 : 8;   // 32-bit words of codes per block
};

// Largest magnitude of three; NaN if any is.
__device__ __forceinline__ float max_abs3(float a, float b, float c)
{
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// One block: 32 values -> codes (element order) and the E8M0 scale code.
template <QuantFmt Q>
__device__ __forceinline__ uint32_t quantize_block(const float (&x)[32], uint32_t (&out)[QuantTraits<Q>::kWords])
{
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; i += 2)
        amax = max_abs3(amax, x[i], x[i + 1]);
    const bool finite = amax <= 3.402823466e38f;     // not for infinities and NaN
    if (!finite)
        amax = 0.0f;
    const int s = Q == QuantFmt::kE2M1 ? block_exponent(amax) : block_exponent8(amax, Q == QuantFmt::kE4M3 ? 8 : 15);
    const float inv = exp2_neg(s);
#pragma unroll
    for (int w = 0; w < QuantTraits<Q>::kWords; ++w) {
        if constexpr (Q == QuantFmt::kE2M1) {
            uint32_t v = 0u;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v |= e2m1x2(x[8 * w + 2 * j] * inv, x[8 * w + 2 * j + 1] * inv) << (8 * j);
            out[w] = v;
        } else {
            constexpr int kF = Q == QuantFmt::kE4M3 ? 0 : 1;
            out[w] = f8x2<kF>(x[4 * w] * inv, x[4 * w + 1] * inv) |
                     (f8x2<kF>(x[4 * w + 2] * inv, x[4 * w + 3] * inv) << 16);
        }
    }
    return finite ? static_cast<uint32_t>(s + 127) : 0xFFu;
}

// quantize_block for a byte format, scaled two values at a time (the same codes).
template <QuantFmt Q>
__device__ __forceinline__ uint32_t quantize_block_pairs(const float (&x)[32], uint32_t (&out)[8])
{
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; i += 2)
        amax = max_abs3(amax, x[i], x[i + 1]);
    float factor;
    const uint32_t code = block_scale8<Q>(amax, factor);
    const F2 inv = f2(factor);
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        constexpr int kF = Q == QuantFmt::kE4M3 ? 0 : 1;
        const float2 lo = parts(f2(x[4 * w], x[4 * w + 1]) * inv), hi = parts(f2(x[4 * w + 2], x[4 * w + 3]) * inv);
        out[w] = f8x2<kF>(lo.x, lo.y) | (f8x2<kF>(hi.x, hi.y) << 16);
    }
    return code;
}

}  // namespace mxfp4
