// E4M3 quantisation shared by the kernels that write codes with block or row scales.
//
// A scale group's codes are e4m3(v * f) with f = 448 / a and its scale a / 448, both in fp32, where
// a = max(amax, kFp8Floor).  The floor keeps f finite (448 / a overflows below a = 1.4e-36, where v * f
// would turn zeros into NaN); a group that small quantises to zeros and tiny codes.  Rounding happens
// once, from the fp32 product to the code (half a step: 2^-4 relative).
#pragma once

#include <type_traits>

#include "device_common.h"

namespace moe {

constexpr int kFp8Block = 128;               // columns under one scale
constexpr float kFp8Floor = 7.8886091e-31f;  // 2^-100

struct Fp8Scale {
    float factor;  // 448 / a
    float scale;   // a / 448
};

__device__ __forceinline__ Fp8Scale fp8_scale(float amax) {
    if (!(amax > 0.f)) return {1.f, 1.f};
    const float a = fmaxf(amax, kFp8Floor);
    return {448.0f / a, a / 448.0f};
}

// codes of 4 values, value 0 in the lowest byte
__device__ __forceinline__ uint32_t fp8_codes4(float v0, float v1, float v2, float v3) {
    int pk = __builtin_amdgcn_cvt_pk_fp8_f32(v0, v1, 0, false);
    return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(v2, v3, pk, true));
}

// max over the 16 lanes of a DPP row, in every one of them: rotations by 1, 2, 4 and 8.  16 lanes of
// 8 columns each are one block of 128.  fmaxf drops NaN.
__device__ __forceinline__ float row16_max(float v) {
    auto ror = [](float x, auto n) {
        return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x120 + decltype(n)::value, 0xF, 0xF, false));
    };
    v = fmaxf(v, ror(v, std::integral_constant<int, 1>{}));
    v = fmaxf(v, ror(v, std::integral_constant<int, 2>{}));
    v = fmaxf(v, ror(v, std::integral_constant<int, 4>{}));
    return fmaxf(v, ror(v, std::integral_constant<int, 8>{}));
}

// two codes of a word (its low or high half) as a pair of bf16 values; exact
__device__ __forceinline__ uint32_t fp8_pair(uint32_t w, bool hi) {
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    const bf16x2_t v = hi ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true)
                          : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false);
    return __builtin_bit_cast(uint32_t, v);
}

// eight codes as a bf16 MFMA operand
__device__ __forceinline__ bf16x8 fp8_to_bf16(uint32_t w0, uint32_t w1) {
    return __builtin_bit_cast(bf16x8, u32x4{fp8_pair(w0, false), fp8_pair(w0, true), fp8_pair(w1, false), fp8_pair(w1, true)});
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

}  // namespace moe
