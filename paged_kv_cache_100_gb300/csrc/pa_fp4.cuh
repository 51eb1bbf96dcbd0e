// Pools held in 4 bits, shared by the kernels that write, read back
// (pa_fp4_cache.cu) and attend to them (pa_fp4_decode.cu).
//
// A tile is a block's 16 rows of one KV head: 9 head_dim bytes, first the rows'
// E2M1 codes, head_dim / 2 bytes each (the even element in a byte's low half), then
// their scales, head_dim / 16 bytes each, one per 16 elements.
//   value = code * scale,  code in +-{0, 0.5, 1, 1.5, 2, 3, 4, 6}
// E2M1 reaches from 0.5 to 6, so its range is the scale's business, and a scale per
// 16 elements follows a row's own outliers where one per block would not.  The
// scale's 8 bits are a positive number of 5 exponent and 3 mantissa bits: bits 14 to
// 7 of an f16, so that it is widened by a shift, needs no second scale (E4M3's
// smallest normal number, 2^-6, would for small values) and has no sign to waste.
// A value has at most 6 significant bits and is a multiple of 2^-18, below 2^16:
// exact in f16, bf16 and f32.
#pragma once

#include <cuda_runtime.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

constexpr uint32_t kFp4TopScale = 0xe2;          // 10240: 6 * 10240 is an f16, the next one's is not
constexpr uint32_t kFp4NanScale = 0xff;          // of 16 elements with a NaN among them
constexpr float kFp4Top = 61440.f;               // 6 * 10240

// Bytes of a tile of rows of `head_dim` elements, and where its scales begin.
__host__ __device__ constexpr int fp4_tile_bytes(int head_dim) { return 9 * head_dim; }
__host__ __device__ constexpr int fp4_scales_at(int head_dim) { return 8 * head_dim; }

// Eight codes (the lowest four bits first) as f16 pairs; exact.
__device__ __forceinline__ void e2m1x8_to_f16x2x4(uint32_t codes, uint32_t (&x)[4]) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
        : "r"(codes));
}

// Codes of eight floats, to nearest, ties to even, 6 at most (the first in the lowest bits).
__device__ __forceinline__ uint32_t f32x8_to_e2m1x8(const float (&x)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// Byte kByte of `w`, a scale, as an f16 pair of it.
template <int kByte>
__device__ __forceinline__ uint32_t fp4_scale_pair(uint32_t w) {
    return __byte_perm(w, 0u, 0x0404u | (kByte << 4) | (kByte << 12)) >> 1;
}

__device__ __forceinline__ float fp4_scale_value(uint32_t byte) {
    return __half2float(__ushort_as_half((unsigned short)(byte << 7)));
}

// The scale of 16 elements of which the largest magnitude is amax: amax / 6 to
// nearest, ties to even, at least the smallest scale and at most kFp4TopScale; 0 for
// 0.  `near` is amax to 2^-20 (not a value that may be further off: of an exact amax, that rounded); the
// decision compares amax itself with *border, six times the number midway between the two scales in
// question, which is exact.
template <typename F>
__device__ __forceinline__ uint32_t fp4_scale_of(float near, F amax, float *border) {
    const float low = fminf(near, 2.f * kFp4Top) * ((1.f - 0x1p-18f) / 6.f);
    const uint32_t at = (uint32_t)__half_as_ushort(__float2half_rz(low)) >> 7;   // amax / 6 lies above it, below the second one above
    *border = 6.f * __half2float(__ushort_as_half((unsigned short)((at << 7) + 64)));
    const bool up = amax > (F)*border || (amax == (F)*border && (at & 1u) != 0);
    const uint32_t s = min(at + (up ? 1u : 0u), kFp4TopScale);
    return amax > (F)0 ? max(s, 1u) : 0u;
}

}  // namespace pa
