// One FP8 block by eight lanes: each holds 16 of the block's 128 channels.
#pragma once

#include "device.h"

namespace moe_ep {

// Two fp32 values -> E4M3FN codes in bytes 0,1 (HI: 2,3) of `old`, with gfx950's
// converter (round to nearest even).  It agrees with f32_to_e4m3fn on every
// value of magnitude <= 448, and the callers' values reach 448 * (1 + 2^-23)
// at most, which still rounds to 448.
template <bool HI>
__device__ __forceinline__ uint32_t e4m3fn_pair(float a, float b, uint32_t old)
{
    return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, (int)old, HI);
}

// Maximum over the eight lanes of a block (lane ^ 1, ^ 2 and ^ 7 within rows of 16).
__device__ __forceinline__ float max8(float m)
{
    m = fmaxf(m, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(m), 0xB1, 0xF, 0xF, true)));   // quad_perm 1,0,3,2
    m = fmaxf(m, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(m), 0x4E, 0xF, 0xF, true)));   // quad_perm 2,3,0,1
    return fmaxf(m, __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(m), 0x141, 0xF, 0xF, true))); // row_half_mirror
}

// The block's codes (this lane's 16) and its scale: a = max(amax, 2^-64),
// codes = RNE(v * (448 / a)), scale = a / 448.  Called by all eight lanes.
__device__ __forceinline__ u32x4 encode_block(const float (&v)[16], float& scale)
{
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < 16; ++j)
        m = fmaxf(m, fabsf(v[j]));
    const float a = fmaxf(max8(m), 0x1p-64f);
    const float inv = 448.0f / a;
    scale = a / 448.0f;
    u32x4 q;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t c = e4m3fn_pair<false>(v[4 * j] * inv, v[4 * j + 1] * inv, 0u);
        q[j] = e4m3fn_pair<true>(v[4 * j + 2] * inv, v[4 * j + 3] * inv, c);
    }
    return q;
}

// 16 bf16 channels -> fp32
__device__ __forceinline__ void widen16(const u32x4& lo, const u32x4& hi, float (&v)[16])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = bf16_lo(lo[j]);
        v[2 * j + 1] = bf16_hi(lo[j]);
        v[8 + 2 * j] = bf16_lo(hi[j]);
        v[8 + 2 * j + 1] = bf16_hi(hi[j]);
    }
}

// 16 codes and their scale -> fp32
__device__ __forceinline__ void decode16(const u32x4& q, float scale, float (&v)[16])
{
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float a, b;
        e4m3fn_pair_to_f32<false>(q[j], a, b);
        v[4 * j] = a * scale;
        v[4 * j + 1] = b * scale;
        e4m3fn_pair_to_f32<true>(q[j], a, b);
        v[4 * j + 2] = a * scale;
        v[4 * j + 3] = b * scale;
    }
}

}  // namespace moe_ep
