// Device helpers of the microscaled formats (OCP MX: blocks of 32 with an E8M0 scale).
#pragma once

#include "device.h"
#include "kernels.h"

namespace moe {

// E8M0 byte of a block: from the exponent of its largest magnitude, one more where
// the mantissa is past the format's (448 = 1.75 * 2^8, 6 = 1.5 * 2^2), so the smallest
// power of two that no value over it exceeds the format's range.  At least 1 (2^-126),
// so the scale and its reciprocal are normal numbers; 127 (scale 1) for an all-zero
// block; 255 where a value is not finite.
template <int FMT>
__device__ __forceinline__ uint32_t mx_block_byte(uint32_t amax_bits) {
    constexpr uint32_t kMant = FMT == kMxE4M3 ? 0x600000u : 0x400000u;
    constexpr int kShift = FMT == kMxE4M3 ? 8 : 2;
    if (amax_bits == 0) return 127u;
    if (amax_bits >= 0x7f800000u) return 255u;
    const int e = (int)(amax_bits >> 23) - kShift + ((amax_bits & 0x7fffffu) > kMant ? 1 : 0);
    return (uint32_t)max(e, 1);
}

__device__ __forceinline__ float e8m0_value(uint32_t b) {
    return b == 255u ? __uint_as_float(0x7fc00000u) : b == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(b << 23);
}
// 2^-x of a scale byte 1 .. 253 (a finite block's is 253 at most).
__device__ __forceinline__ float e8m0_inverse(uint32_t b) { return __uint_as_float((254u - b) << 23); }

// Values of at most 6 as e2m1 codes, rounded to nearest even: codes of a and b in byte
// SEL of w (which keeps its other bytes), a's in the low half.
template <int SEL>
__device__ __forceinline__ uint32_t e2m1x2(uint32_t w, float a, float b) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, a, b, 1.0f, SEL);
}

}  // namespace moe
