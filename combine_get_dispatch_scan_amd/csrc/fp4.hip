// Expert weights in 4 bits on gfx950: E2M1 codes with one E8M0 scale (a power of two)
// for 32 weights along k, and back.
//   s = the smallest power of two with amax < 7 s:  amax rounded to one mantissa bit
//       is m * 2^e with m in {1, 3/2}, and s = 2^(e-2): an addition and a shift of the
//       float's bits.  amax / s lies in [3.5, 7); 6 is the largest code, so the largest
//       weight is off by at most half a step like every other one.
//   code = RNE_E2M1(w / s), by gfx950's converter, which divides by the scale's power
//       of two itself (a device test compares it with the formula).
//
// Memory bounds both: 32 x 4096 x 7168 in bf16 takes 371 us there and 363 us back, 6.4
// and 6.6 TB/s (a copy of 1 GiB: 5.1).  A thread takes two units of eight weights: both
// directions 825 us, with four units 889, with one 831 (all of it through the caches, before
// calls of this size went around them).  8 x 512 x 1024 from fp32 and back to bf16: 3.5 and
// 3.8 us.
#include "block_launch.h"

namespace moe_ep {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

// Four lanes hold the 32 weights of a scale, eight each.
constexpr int kFp4Units = 2;         // groups of eight weights that a thread has in flight

// Past the Infinity Cache's size nothing of a call's data is found there again, so it is
// read and written around the caches (32 x 4096 x 7168, both directions: 735 us, 830
// through them).  Below, who reads the result finds it there (8 x 2048 x 2048, there and
// back: 32.5 us around them, 30.3 through them).
constexpr int64_t kAroundBytes = (int64_t)256 << 20;

__device__ __forceinline__ uint32_t quad_max(uint32_t m)
{
    m = max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0xB1, 0xF, 0xF, true));     // lane ^ 1
    return max(m, (uint32_t)__builtin_amdgcn_mov_dpp((int)m, 0x4E, 0xF, 0xF, true));  // lane ^ 2
}

// The scale's byte from the bits of the largest magnitude (NaNs and infinities are
// the largest of all), and the scale itself.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits)
{
    if (amax_bits >= 0x7F800000u)
        return 255u;
    const int e = (int)((amax_bits + 0x00200000u) >> 23) - 2;
    return (uint32_t)max(e, 0);
}

__device__ __forceinline__ float scale_value(uint32_t byte)
{
    return __uint_as_float(byte == 255u ? 0x7FC00000u : byte ? byte << 23 : 0x00400000u);
}

template <bool F32, bool AROUND>
__global__ __launch_bounds__(256) void quantize_fp4_kernel(const void* __restrict__ w, int64_t units,
                                                           uint32_t* __restrict__ codes,
                                                           uint8_t* __restrict__ scales)
{
    const int64_t u0 = (int64_t)blockIdx.x * (256 * kFp4Units) + threadIdx.x;
    u32x4 d[kFp4Units][F32 ? 2 : 1];
#pragma unroll
    for (int i = 0; i < kFp4Units; ++i) {
        const int64_t u = u0 + 256 * i;
        if (u < units) {
#pragma unroll
            for (int j = 0; j < (F32 ? 2 : 1); ++j)
                d[i][j] = load16_hint<AROUND>(static_cast<const char*>(w) + u * (F32 ? 32 : 16) + 16 * j);
        } else {
#pragma unroll
            for (int j = 0; j < (F32 ? 2 : 1); ++j)
                d[i][j] = u32x4{0u, 0u, 0u, 0u};
        }
    }
#pragma unroll
    for (int i = 0; i < kFp4Units; ++i) {
        const int64_t u = u0 + 256 * i;
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < (F32 ? 2 : 1); ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                if (F32) {
                    m = max(m, d[i][j][c] & 0x7FFFFFFFu);
                } else {
                    m = max(m, d[i][j][c] & 0x7FFF0000u);
                    m = max(m, (d[i][j][c] << 16) & 0x7FFF0000u);
                }
            }
        const uint32_t byte = scale_byte(quad_max(m));
        const float s = scale_value(byte);
        uint32_t q = 0;
        if constexpr (F32) {
            const auto f = [&](int k) { return __uint_as_float(d[i][k >> 2][k & 3]); };
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f(0), f(1), s, 0);
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f(2), f(3), s, 1);
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f(4), f(5), s, 2);
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f(6), f(7), s, 3);
        } else {
            const auto f = [&](int k) {
                const uint32_t pair = d[i][0][k];       // a vector's element itself is cast wrongly
                return __builtin_bit_cast(bf16x2, pair);
            };
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, f(0), s, 0);
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, f(1), s, 1);
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, f(2), s, 2);
            q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, f(3), s, 3);
        }
        if (u < units) {
            if (AROUND)
                __builtin_nontemporal_store(q, codes + u);
            else
                codes[u] = q;
            if ((threadIdx.x & 3) == 0)
                scales[u >> 2] = (uint8_t)byte;
        }
    }
}

hipError_t launch_quantize_fp4(const void* w, bool w_f32, int64_t groups32, uint8_t* codes, uint8_t* scales,
                               hipStream_t stream)
{
    const int64_t units = groups32 * 4, per = 256 * kFp4Units;
    const dim3 grid((unsigned)((units + per - 1) / per));
    debug_launch("quantize_fp4", grid, dim3(256), 0);
    const bool around = groups32 * (w_f32 ? 128 : 64) > kAroundBytes;
    auto* kernel = w_f32 ? (around ? quantize_fp4_kernel<true, true> : quantize_fp4_kernel<true, false>)
                         : (around ? quantize_fp4_kernel<false, true> : quantize_fp4_kernel<false, false>);
    kernel<<<grid, 256, 0, stream>>>(w, units, reinterpret_cast<uint32_t*>(codes), scales);
    return hipGetLastError();
}

template <bool F32, bool AROUND>
__global__ __launch_bounds__(256) void dequantize_fp4_kernel(const uint32_t* __restrict__ codes,
                                                             const uint8_t* __restrict__ scales, int64_t units,
                                                             void* __restrict__ out)
{
    const int64_t u0 = (int64_t)blockIdx.x * (256 * kFp4Units) + threadIdx.x;
    uint32_t q[kFp4Units], b[kFp4Units];
#pragma unroll
    for (int i = 0; i < kFp4Units; ++i) {
        const int64_t u = u0 + 256 * i;
        q[i] = u < units ? codes[u] : 0u;
        b[i] = u < units ? scales[u >> 2] : 0u;
    }
#pragma unroll
    for (int i = 0; i < kFp4Units; ++i) {
        const int64_t u = u0 + 256 * i;
        if (u >= units)
            break;
        const float s = scale_value(b[i]);
        if constexpr (F32) {
            f32x2 v[4];
            v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], s, 0);
            v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], s, 1);
            v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], s, 2);
            v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[i], s, 3);
            u32x4 o[2];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                o[k >> 2][k & 3] = b[i] == 255u ? 0x7FC00000u : __float_as_uint(v[k >> 1][k & 1]);
            char* p = static_cast<char*>(out) + u * 32;
            store16_hint<AROUND>(p, o[0]);
            store16_hint<AROUND>(p + 16, o[1]);
        } else {
            u32x4 o;
            o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[i], s, 0));
            o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[i], s, 1));
            o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[i], s, 2));
            o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q[i], s, 3));
            if (b[i] == 255u)
                o = u32x4{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
            store16_hint<AROUND>(static_cast<char*>(out) + u * 16, o);
        }
    }
}

hipError_t launch_dequantize_fp4(const uint8_t* codes, const uint8_t* scales, int64_t groups32, void* out,
                                 bool out_f32, hipStream_t stream)
{
    const int64_t units = groups32 * 4, per = 256 * kFp4Units;
    const dim3 grid((unsigned)((units + per - 1) / per));
    debug_launch("dequantize_fp4", grid, dim3(256), 0);
    const bool around = groups32 * (out_f32 ? 128 : 64) > kAroundBytes;
    auto* kernel = out_f32 ? (around ? dequantize_fp4_kernel<true, true> : dequantize_fp4_kernel<true, false>)
                           : (around ? dequantize_fp4_kernel<false, true> : dequantize_fp4_kernel<false, false>);
    kernel<<<grid, 256, 0, stream>>>(reinterpret_cast<const uint32_t*>(codes), scales, units, out);
    return hipGetLastError();
}

}  // namespace moe_ep
