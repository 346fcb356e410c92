// Grouped weight gradient on gfx950: for every group g
//   dW[g][n][k] = sum over the group's rows r of dy[r][n] * x[r][k] * sx[r][k / 128]
// with dy in bf16 and x in the 8 bits it was dispatched in (the activation
// checkpoint of the product).  The scale belongs to a row, and rows are what is
// summed over, so it cannot be taken out of the sum: x is widened to bf16 on its
// way into LDS (a 4-bit code times the scale, one rounding of 2^-9 relative) and
// the product runs on the bf16 matrix cores with fp32 sums.
#include "expert_launch.h"
#include "mfma.h"

namespace moe_ep {

constexpr int kWgRows = 64;                    // rows of a step
constexpr int kWgLd = 128 + 16;                // LDS row in bf16 values: 32 bytes of padding

template <bool F32>
__global__ __launch_bounds__(256) void wgrad_kernel(WgradLaunch a)
{
    __shared__ __align__(16) uint16_t ldy[kWgRows * kWgLd];
    __shared__ __align__(16) uint16_t ldx[kWgRows * kWgLd];
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int N = a.N, K = a.K, KB = K / kQBlock;
    const int kb = blockIdx.x, nb = blockIdx.y, g = blockIdx.z;
    int begin, end;
    group_bounds(a.groups, g, begin, end);
    f32x4 acc[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int wn = (wave & 1) * 64, wk = (wave >> 1) * 64;
    for (int r0 = begin; r0 < end; r0 += kWgRows) {
        // dy: 16 chunks of 8 columns a row; x: 8 chunks of 16.  Rows past the group
        // are read from its last row, and their x is put to zero.
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int rr = i * 16 + tid / 16;
            const int r = r0 + rr < end ? r0 + rr : end - 1;
            *reinterpret_cast<u32x4*>(ldy + rr * kWgLd + (tid % 16) * 8) =
                load16_hint<false>(a.dy + (size_t)r * N + nb * 128 + (tid % 16) * 8);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int rr = i * 32 + tid / 8;
            const bool on = r0 + rr < end;
            const int r = on ? r0 + rr : end - 1;
            const u32x4 q = load16_hint<false>(a.x + (size_t)r * K + kb * kQBlock + (tid % 8) * 16);
            const float s = a.x_scales[scale_at(r, kb, KB, a.x_scale_ld)];
            u32x4 o[2];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float v0, v1, v2, v3;
                e4m3fn_pair_to_f32<false>(q[j], v0, v1);
                e4m3fn_pair_to_f32<true>(q[j], v2, v3);
                o[j / 2][(j % 2) * 2] = on ? pack_bf16x2(v0 * s, v1 * s) : 0u;
                o[j / 2][(j % 2) * 2 + 1] = on ? pack_bf16x2(v2 * s, v3 * s) : 0u;
            }
            *reinterpret_cast<u32x4*>(ldx + rr * kWgLd + (tid % 8) * 16) = o[0];
            *reinterpret_cast<u32x4*>(ldx + rr * kWgLd + (tid % 8) * 16 + 8) = o[1];
        }
        __syncthreads();
#pragma unroll
        for (int s = 0; s < kWgRows; s += 32) {
            i16x8 fy[4], fx[4];
            // lane group q = lane / 16 takes rows s + 8q .. s + 8q + 7
            const int at = (s + (lane >> 4) * 8 + ((lane & 15) >> 2)) * kWgLd + (lane & 3) * 4;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const i16x4 y0 = lds_read_tr16(ldy + at + wn + 16 * i), y1 = lds_read_tr16(ldy + at + 4 * kWgLd + wn + 16 * i);
                const i16x4 x0 = lds_read_tr16(ldx + at + wk + 16 * i), x1 = lds_read_tr16(ldx + at + 4 * kWgLd + wk + 16 * i);
                fy[i] = __builtin_shufflevector(y0, y1, 0, 1, 2, 3, 4, 5, 6, 7);
                fx[i] = __builtin_shufflevector(x0, x1, 0, 1, 2, 3, 4, 5, 6, 7);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, fx[j]),
                                                                        __builtin_bit_cast(bf16x8, fy[i]), acc[i][j], 0, 0, 0);
        }
        __syncthreads();
    }
    // lane: row n = lane % 16 of tile i, columns k = 4 * (lane / 16) .. + 3 of tile j
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const size_t n = (size_t)nb * 128 + wn + 16 * i + (lane & 15);
            const size_t at = ((size_t)g * N + n) * K + kb * kQBlock + wk + 16 * j + 4 * (lane >> 4);
            if (F32)
                *reinterpret_cast<f32x4*>(static_cast<float*>(a.dw) + at) = acc[i][j];
            else
                *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.dw) + at) =
                    uint2{pack_bf16x2(acc[i][j][0], acc[i][j][1]), pack_bf16x2(acc[i][j][2], acc[i][j][3])};
        }
}

hipError_t launch_grouped_wgrad(const WgradLaunch& L, hipStream_t stream)
{
    if (L.groups.num == 0)
        return hipSuccess;
    const dim3 grid(L.K / kQBlock, L.N / 128, L.groups.num);
    debug_launch("grouped_wgrad", grid, dim3(256), 0);
    if (L.dw_f32)
        wgrad_kernel<true><<<grid, 256, 0, stream>>>(L);
    else
        wgrad_kernel<false><<<grid, 256, 0, stream>>>(L);
    return hipGetLastError();
}

}  // namespace moe_ep
