// Shared by the attention kernels over E4M3 pools with one scale per block and
// KV head (pa_block8_decode.cu, pa_block8_prefill.cu).
//
// The value of a code in block j is code * sk_j (keys) or code * sv_j (values).
// The key scale is a factor of the block's scores.  The value scale enters the
// exponent instead of the product: with lv_j = log2 sv_j,
//   o = sum_t 2^(s_t - m) sv_j(t) v_t / sum_t 2^(s_t - m)
//     = sum_t w_t v_t / sum_t w_t / sv_j(t),   w_t = 2^(s_t + lv_j(t) - m'),
// with m' the largest s_t + lv_j(t).  So w_t, which is rounded to 16 bits for
// the second product, measures a token by what it can add to the output: a block
// with a large scale neither leaves the 16-bit range nor pushes the others out
// of it.  The denominator's terms w_t / sv_j(t) stay in 32 bits.  Scales lie in
// [2^-32, 2^31] (others are clamped and flagged), so a term of the denominator
// that 2^x flushes to zero is below 2^-63 of the largest one.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {

constexpr float kMinScale = 0x1p-32f, kMaxScale = 0x1p31f;

// The value scale as read, brought into range.
__device__ __forceinline__ float value_scale(float sv, int32_t *status) {
    if (!(sv >= kMinScale && sv <= kMaxScale)) {
        report(status, PA_DEV_RANGE);
        sv = sv > kMaxScale ? kMaxScale : kMinScale;      // NaN and negative ones too
    }
    return sv;
}

// log2 of a positive normal number, exact for powers of two.
__device__ __forceinline__ float log2_scale(float x) {
    const uint32_t u = __float_as_uint(x);
    return (float)((int)(u >> 23) - 127) + log2f(__uint_as_float((u & 0x7fffffu) | 0x3f800000u));
}

// 2-D view of an E4M3 pool as [num_blocks * num_kv_heads * 16 rows][128 codes],
// loaded as boxes of 16 rows, with 128-byte swizzle or as they are.  Defined in
// pa_block8_decode.cu.
bool encode_block8_map(CUtensorMap *map, const void *pool, int64_t rows, bool swizzled);

}  // namespace pa
