// GPTQ int4 words as bf16 MFMA operands, shared by the kernels that stream them: OR-ing nibble pairs
// into bf16 0x4300 (= 128.0) gives the exact values 128 + q in a permuted k order, and the activation
// fragment takes the same order (gemm_int4.hip has the arithmetic).
#pragma once

#include "device_common.h"

namespace moe {

__device__ __forceinline__ bf16x8 as_bf16x8(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

// x fragment k order (k0..k7) -> (k0,k4,k1,k5,k2,k6,k3,k7), matching the nibble pairs: one
// v_perm_b32 per output word (byte selectors 0-3 pick from the second operand, 4-7 the first).
__device__ __forceinline__ u32x4 permute_k(u32x4 a) {
    u32x4 r;
    r[0] = __builtin_amdgcn_perm(a[2], a[0], 0x05040100u);
    r[1] = __builtin_amdgcn_perm(a[2], a[0], 0x07060302u);
    r[2] = __builtin_amdgcn_perm(a[3], a[1], 0x05040100u);
    r[3] = __builtin_amdgcn_perm(a[3], a[1], 0x07060302u);
    return r;
}

// One qweight word (8 nibbles of consecutive k) -> bf16 (128+q) in the permuted k order.  The
// mask and the bf16 exponent pattern come in registers (opaque to the compiler) so that each
// pair is one v_and_or_b32: a VOP3 instruction cannot take them as literals.
__device__ __forceinline__ u32x4 dequant_word(uint32_t w, uint32_t mask, uint32_t magic) {
    u32x4 r;
    r[0] = (w & mask) | magic;
    r[1] = ((w >> 4) & mask) | magic;
    r[2] = ((w >> 8) & mask) | magic;
    r[3] = ((w >> 12) & mask) | magic;
    return r;
}

}  // namespace moe
