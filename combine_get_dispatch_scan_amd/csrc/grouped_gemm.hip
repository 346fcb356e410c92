// Grouped FP8 product on gfx950: for the rows r of group g
//   y[r][n] = sum over 128-channel blocks b of
//             sx[r][b] * sw[g][n / 128][b] * (sum over k in b of x[r][k] * w[g][n][k])
// The inner sum is one matrix instruction (K = 128, E4M3, fp32 result); the two
// scales are arbitrary fp32 numbers, so every block's result is scaled on the
// vector unit and added in fp32.  The weights are the instruction's first
// operand: a lane then holds four neighbouring columns of one row and needs one
// scale for them.
#include "expert_launch.h"
#include "mfma.h"

namespace moe_ep {

constexpr int kXcds = 8;

// Skinny tiles, for few rows a group: a workgroup's four waves split the K
// blocks of a 16*RT x 16*CT tile between them (operands straight from memory to
// registers, each weight byte read by one lane) and add up through LDS.
template <int RT, int CT>
__global__ __launch_bounds__(256) void gemm_skinny_kernel(GemmLaunch a)
{
    constexpr int kRows = 16 * RT, kCols = 16 * CT, kStep = 2;
    extern __shared__ int prefix[];
    __shared__ f32x4 part[4][RT][CT][kWave];
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
    const int N = a.N, K = a.K, KB = K / kQBlock, NT = N / kCols;
    tile_prefix<kRows>(a.groups, prefix);
    __syncthreads();
    const int64_t total = (int64_t)prefix[a.groups.num] * NT;
    const int64_t per = (total + kXcds - 1) / kXcds;
    const int xcd = blockIdx.x % kXcds;
    for (int64_t i = blockIdx.x / kXcds; i < per; i += gridDim.x / kXcds) {
        const int64_t t = xcd * per + i;
        if (t >= total)
            break;
        const int g = find_group(prefix, a.groups.num, t, NT);
        int begin, end;
        group_bounds(a.groups, g, begin, end);
        const int mt = prefix[g + 1] - prefix[g];
        const int64_t local = t - (int64_t)prefix[g] * NT;
        const int m0 = begin + (int)(local % mt) * kRows, n0 = (int)(local / mt) * kCols;
        f32x4 acc[RT][CT];
        const uint8_t* xp[RT];
        const float* sp[RT];
        int64_t sstep = a.x_scale_ld ? a.x_scale_ld : 1;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            int row = m0 + 16 * r + (lane & 15);
            row = row < end ? row : end - 1;           // rows past the group: any of its rows, not stored
            xp[r] = a.x + (size_t)row * K + (lane >> 4) * 32;
            sp[r] = a.x_scales + scale_at(row, 0, KB, a.x_scale_ld);
#pragma unroll
            for (int c = 0; c < CT; ++c)
                acc[r][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        const uint8_t* wp = a.w + ((size_t)g * N + n0 + (lane & 15)) * K + (lane >> 4) * 32;
        const float* wsp = a.w_scales + ((size_t)g * (N / kQBlock) + n0 / kQBlock) * KB;
        for (int kb0 = wave; kb0 < KB; kb0 += 4 * kStep) {
            u32x4 w[kStep][CT][2], x[kStep][RT][2];
            float s[kStep][RT];
#pragma unroll
            for (int u = 0; u < kStep; ++u) {
                const bool on = kb0 + 4 * u < KB;
                const int kb = on ? kb0 + 4 * u : KB - 1;
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    const uint8_t* p = wp + (size_t)16 * c * K + (size_t)kb * kQBlock;
                    w[u][c][0] = load16_hint<false>(p);
                    w[u][c][1] = load16_hint<false>(p + 16);
                }
                const float sw = on ? wsp[kb] : 0.0f;
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const uint8_t* p = xp[r] + (size_t)kb * kQBlock;
                    x[u][r][0] = load16_hint<false>(p);
                    x[u][r][1] = load16_hint<false>(p + 16);
                    s[u][r] = sp[r][kb * sstep] * sw;
                }
            }
#pragma unroll
            for (int u = 0; u < kStep; ++u) {
                if (kb0 + 4 * u >= KB)
                    break;
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int c = 0; c < CT; ++c) {
                        const f32x4 d = mfma_fp8(join(w[u][c][0], w[u][c][1]), join(x[u][r][0], x[u][r][1]));
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            acc[r][c][q] = __builtin_fmaf(d[q], s[u][r], acc[r][c][q]);
                    }
            }
        }
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int c = 0; c < CT; ++c)
                part[wave][r][c][lane] = acc[r][c];
        __syncthreads();
        // wave w finishes tiles w, w + 4, ...: the four partial sums in wave order
        for (int q = wave; q < RT * CT; q += 4) {
            const int r = q / CT, c = q % CT;
            f32x4 v = part[0][r][c][lane];
#pragma unroll
            for (int w = 1; w < 4; ++w)
                v += part[w][r][c][lane];
            const int row = m0 + 16 * r + (lane & 15);
            if (row < end)
                *reinterpret_cast<uint2*>(a.out + (size_t)row * N + n0 + 16 * c + 4 * (lane >> 4)) =
                    uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        }
        __syncthreads();
    }
}

hipError_t launch_grouped_gemm(const GemmLaunch& L, hipStream_t stream)
{
    if (L.groups.rows == 0 || L.groups.num == 0)
        return hipSuccess;
    const size_t lds = (size_t)(L.groups.num + 1) * 4;
    const dim3 grid(256 * 4);
    debug_launch("grouped_gemm_skinny", grid, dim3(256), lds);
    gemm_skinny_kernel<2, 2><<<grid, 256, lds, stream>>>(L);
    return hipGetLastError();
}

}  // namespace moe_ep
