// Grouped product of FP8 rows with 4-bit weights on gfx950: for the rows r of group g
//   y[r][n] = sum over 128-channel blocks b of
//             sx[r][b] * (sum over k in b of x[r][k] * code[g][n][k] * s[g][n][k / 32])
// The inner sum is one matrix instruction (K = 128, E2M1 by E4M3), which applies the
// weights' scales itself: a lane of its first operand holds 32 neighbouring k of one
// column n, which is one scale.  Its second operand's lane holds k = 16 q .. + 15 and
// 64 + 16 q .. + 15 (q = lane / 16).  The rows' scales are arbitrary fp32 numbers, so
// every block's result is scaled on the vector unit and added in fp32.
#include "block_launch.h"
#include "mfma.h"

namespace moe_ep {

constexpr int kXcds = 8, kCus = 256;

// 16 x 16 x 128 product from zero: a: E2M1 (16 bytes), b: E4M3, s: the E8M0 scale of
// a's 32 weights in its low byte.
__device__ __forceinline__ f32x4 mfma_fp4_fp8(const u32x4& a, const i32x8& b, uint32_t s)
{
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    const i32x8 w = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, b, zero, 4, 0, 0, (int)s, 0, 0x7F7F7F7F);
}

// Skinny tiles: a workgroup's four waves split the K blocks of a 16*RT x 16*CT tile
// between them (operands straight from memory to registers, each weight byte read by
// one lane) and add up through LDS.
template <int RT, int CT>
__global__ __launch_bounds__(256) void gemm_fp4_skinny_kernel(GemmFp4Launch a)
{
    constexpr int kRows = 16 * RT, kCols = 16 * CT, kStep = 2;
    extern __shared__ int prefix[];
    __shared__ f32x4 part[4][RT][CT][kWave];
    const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave, q = lane >> 4;
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
        const int64_t sstep = a.x_scale_ld ? a.x_scale_ld : 1;
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            int row = m0 + 16 * r + (lane & 15);
            row = row < end ? row : end - 1;           // rows past the group: any of its rows, not stored
            xp[r] = a.x + (size_t)row * K + q * 16;
            sp[r] = a.x_scales + scale_at(row, 0, KB, a.x_scale_ld);
#pragma unroll
            for (int c = 0; c < CT; ++c)
                acc[r][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        const size_t col = (size_t)g * N + n0 + (lane & 15);
        const uint8_t* wp = a.w + col * (K / 2) + q * 16;
        const uint8_t* wsp = a.w_scales + col * (K / 32) + q;
        // a wave takes two neighbouring blocks at a time: 128 bytes of a column
        for (int kb0 = kStep * wave; kb0 < KB; kb0 += 4 * kStep) {
            u32x4 w[kStep][CT], x[kStep][RT][2];
            uint32_t ws[kStep][CT];
            float s[kStep][RT];
#pragma unroll
            for (int u = 0; u < kStep; ++u) {
                const int kb = kb0 + u < KB ? kb0 + u : KB - 1;
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    w[u][c] = load16_hint<false>(wp + (size_t)16 * c * (K / 2) + (size_t)kb * 64);
                    ws[u][c] = wsp[(size_t)16 * c * (K / 32) + (size_t)kb * 4];
                }
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const uint8_t* p = xp[r] + (size_t)kb * kQBlock;
                    x[u][r][0] = load16_hint<false>(p);
                    x[u][r][1] = load16_hint<false>(p + 64);
                    s[u][r] = sp[r][kb * sstep];
                }
            }
#pragma unroll
            for (int u = 0; u < kStep; ++u) {
                if (kb0 + u >= KB)
                    break;
#pragma unroll
                for (int r = 0; r < RT; ++r)
#pragma unroll
                    for (int c = 0; c < CT; ++c) {
                        const f32x4 d = mfma_fp4_fp8(w[u][c], join(x[u][r][0], x[u][r][1]), ws[u][c]);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            acc[r][c][j] = __builtin_fmaf(d[j], s[u][r], acc[r][c][j]);
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
        for (int i = wave; i < RT * CT; i += 4) {
            const int r = i / CT, c = i % CT;
            f32x4 v = part[0][r][c][lane];
#pragma unroll
            for (int w = 1; w < 4; ++w)
                v += part[w][r][c][lane];
            const int row = m0 + 16 * r + (lane & 15);
            if (row < end)
                *reinterpret_cast<uint2*>(a.out + (size_t)row * N + n0 + 16 * c + 4 * q) =
                    uint2{pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3])};
        }
        __syncthreads();
    }
}

template <int RT, int CT>
static void skinny_run(const GemmFp4Launch& L, hipStream_t stream)
{
    const size_t lds = (size_t)(L.groups.num + 1) * 4;
    const dim3 grid(kCus * 4);
    debug_launch("grouped_gemm_fp4_skinny", grid, dim3(256), lds);
    gemm_fp4_skinny_kernel<RT, CT><<<grid, 256, lds, stream>>>(L);
}

hipError_t launch_grouped_gemm_fp4(const GemmFp4Launch& L, hipStream_t stream)
{
    if (L.groups.rows == 0 || L.groups.num == 0)
        return hipSuccess;
    const int m = L.expected_rows;
    if (m <= 8)
        skinny_run<1, 4>(L, stream);
    else if (m <= 16)
        skinny_run<2, 4>(L, stream);
    else
        skinny_run<4, 4>(L, stream);
    return hipGetLastError();
}

}  // namespace moe_ep
