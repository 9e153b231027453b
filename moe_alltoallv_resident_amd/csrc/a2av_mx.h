// Device helpers of the 8- and 4-bit formats: e4m3 / E2M1 elements with one power-of-two
// scale byte (E8M0) for every 32 of them.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace a2av {

constexpr int kMxGroup = 32;       // elements that share a scale

// Bytes of an 8-bit row of n elements: elements, scales, zeros up to a multiple of 16.
__host__ __device__ inline int64_t mx8_row_bytes(int64_t n) { return (n + n / kMxGroup + 15) / 16 * 16; }

typedef uint16_t u16;
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

#if defined(__HIP_DEVICE_COMPILE__)
#define A2AV_DEVICE_CODE 1
#endif

__device__ inline float bf16_to_f32(uint32_t v) { return __uint_as_float(v << 16); }

// Round to bfloat16, nearest, ties to even; NaN stays NaN.
__device__ inline uint32_t f32_to_bf16(float f) { return __builtin_bit_cast(u16, (__bf16)f); }

// Two of them in one instruction, the first in the low half.
__device__ inline uint32_t f32_to_bf16_pair(float a, float b) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}

// Magnitude bits: as unsigned integers they order like the magnitudes, with NaN above
// infinity above every number, so an integer maximum keeps a NaN.
__device__ inline uint32_t abs_bits(float f) { return __float_as_uint(f) & 0x7FFFFFFFu; }

// Scale byte for a group whose largest magnitude has the bits `a`: the smallest power of
// two 2^e with max <= 448 * 2^e.  448 = 1.75 * 2^8, so e is the exponent minus 8, plus one
// when the fraction is past .75 (adding 0x1FFFFF carries into the exponent exactly then).
__device__ inline uint32_t mx_scale_byte(uint32_t a) {
    if (a >= 0x7F800000u) return 255u;
    const int e = (int)((a + 0x1FFFFFu) >> 23) - 8;
    return (uint32_t)(e < 0 ? 0 : e);
}

// 1 / 2^(byte - 127); byte <= 247 for every finite group, so it is a normal number.
__device__ inline float mx_inverse(uint32_t byte) { return __uint_as_float((254u - (byte > 253u ? 253u : byte)) << 23); }

// Four floats (already divided by their scale) as four e4m3 bytes.  A group whose scale is
// NaN holds 0x7F (NaN) everywhere.
__device__ inline uint32_t mx8_pack(float a, float b, float c, float d, bool bad) {
#ifdef A2AV_DEVICE_CODE
    int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    v = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
    return bad ? 0x7F7F7F7Fu : (uint32_t)v;
#else
    return 0;
#endif
}

}  // namespace a2av
