// Matrix-core and LDS helpers of the product kernels (gfx950).
#pragma once

#include "device.h"

namespace moe_ep {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef short i16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// 16 x 16 x 128 E4M3 product from zero.  Operand lane l: row l % 16, 32 of the
// 128 k (the same ones in both operands).  Result lane l: column l % 16 (second
// operand's row), rows 4 * (l / 16) + i of the first.
__device__ __forceinline__ f32x4 mfma_fp8(const i32x8& a, const i32x8& b)
{
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, zero, 0, 0, 0, 0, 0, 0);
}

// Two fp32 -> packed bf16, round to nearest even (v_cvt_pk_bf16_f32).
__device__ __forceinline__ uint32_t pack2_bf16(float lo, float hi)
{
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{lo, hi}, bf16x2));
}

__device__ __forceinline__ i32x8 join(const u32x4& lo, const u32x4& hi)
{
    return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3], (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// Copy 16 bytes a lane from global memory to LDS without registers: lane i's
// bytes land at `lds` + 16 * i (`lds` the same in all lanes).
__device__ __forceinline__ void load_to_lds16(const void* g, void* lds)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)g,
                                     (__attribute__((address_space(3))) void*)lds, 16, 0, 0);
}

__device__ __forceinline__ void load_to_lds4(const void* g, void* lds)
{
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)g,
                                     (__attribute__((address_space(3))) void*)lds, 4, 0, 0);
}

// Transposed LDS read of 16-bit values: within 16 lanes, lane l names four
// values of row l / 4 at columns 4 * (l % 4) and gets column l of the four rows.
__device__ __forceinline__ i16x4 lds_read_tr16(const void* p)
{
    return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) i16x4*)p);
}

}  // namespace moe_ep
