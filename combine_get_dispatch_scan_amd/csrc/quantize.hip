// FP8 quantisers of the expert layer on gfx950: rows (1 x 128 blocks, gradients
// on their way into a product) and weights (128 x 128 blocks, also transposed
// for the backward product).  The arithmetic is dispatch's: a = max(amax, 2^-64),
// codes = RNE_E4M3FN(x * (448 / a)), scale = a / 448, one fp32 rounding each.  Both
// are bound by HBM: 32768 x 7168 rows in 125 us (5.7 TB/s), 32 x 4096 x 7168 bf16
// weights with their transposes in 720 us (5.2 TB/s; a 1 GiB copy: 5.05).
#include "expert_launch.h"
#include "quant16.h"

namespace moe_ep {

// Rows: eight lanes per block, 16 channels a lane, so a wave holds eight blocks
// whatever the row's width; kRowUnits blocks per eight lanes are in flight.
constexpr int kRowUnits = 2;

__global__ __launch_bounds__(256) void quantize_rows_kernel(const uint16_t* __restrict__ x, int nb, Groups g,
                                                            int scale_ld, uint8_t* __restrict__ codes,
                                                            float* __restrict__ scales)
{
    const int lane8 = threadIdx.x & 7;
    const int64_t total = (int64_t)g.rows * nb;
    const int64_t u0 = (int64_t)blockIdx.x * (32 * kRowUnits) + (threadIdx.x >> 3);
    u32x4 lo[kRowUnits], hi[kRowUnits];
    bool act[kRowUnits];
#pragma unroll
    for (int i = 0; i < kRowUnits; ++i) {
        const int64_t u = u0 + 32 * i;
        act[i] = u < total && row_in_group(g, (int)(u / nb));
        lo[i] = hi[i] = u32x4{0u, 0u, 0u, 0u};
        if (act[i]) {
            const uint16_t* p = x + u * kQBlock + lane8 * 16;
            lo[i] = load16_hint<false>(p);
            hi[i] = load16_hint<false>(p + 8);
        }
    }
#pragma unroll
    for (int i = 0; i < kRowUnits; ++i) {
        const int64_t u = u0 + 32 * i;
        float v[16], scale;
        widen16(lo[i], hi[i], v);
        const u32x4 q = encode_block(v, scale);
        if (act[i]) {
            store16_hint<false>(codes + u * kQBlock + lane8 * 16, q);
            if (lane8 == 0)
                scales[scale_at((int)(u / nb), (int)(u % nb), nb, scale_ld)] = scale;
        }
    }
}

hipError_t launch_quantize_rows(const void* x, int H, const Groups& g, int scale_ld, void* codes,
                                float* scales, hipStream_t stream)
{
    const int nb = H / kQBlock;
    const int64_t units = (int64_t)g.rows * nb;
    if (units == 0)
        return hipSuccess;
    const dim3 grid((unsigned)((units + 32 * kRowUnits - 1) / (32 * kRowUnits)));
    debug_launch("quantize_rows", grid, dim3(256), 0);
    quantize_rows_kernel<<<grid, 256, 0, stream>>>(static_cast<const uint16_t*>(x), nb, g, scale_ld,
                                                   static_cast<uint8_t*>(codes), scales);
    return hipGetLastError();
}

// Weights: one workgroup per 128 x 128 block.  A thread reads 16 channels of
// four rows; the transposed codes go through LDS, 4 x 4 bytes at a time.
constexpr int kTileLd = kQBlock / 4 + 1;          // dwords per LDS row, padded by one

template <bool F32>
__global__ __launch_bounds__(256) void quantize_weights_kernel(const void* __restrict__ w, int N, int K,
                                                               uint8_t* __restrict__ codes,
                                                               float* __restrict__ scales,
                                                               uint8_t* __restrict__ codes_t,
                                                               float* __restrict__ scales_t)
{
    __shared__ float wave_max[4];
    __shared__ uint32_t tile[kQBlock * kTileLd];
    const int tid = threadIdx.x;
    const int kb = blockIdx.x, nblk = blockIdx.y;
    const size_t g = blockIdx.z;
    const int NB = N / kQBlock, KB = K / kQBlock;
    const int r0 = tid >> 3, c0 = (tid & 7) * 16;
    const size_t base = (g * N + (size_t)nblk * kQBlock) * K + (size_t)kb * kQBlock;
    float v[4][16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const size_t at = base + (size_t)(r0 + 32 * i) * K + c0;
        if (F32) {
            const float* p = static_cast<const float*>(w) + at;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const u32x4 d = load16_hint<false>(p + 4 * j);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    v[i][4 * j + c] = __uint_as_float(d[c]);
            }
        } else {
            const uint16_t* p = static_cast<const uint16_t*>(w) + at;
            widen16(load16_hint<false>(p), load16_hint<false>(p + 8), v[i]);
        }
    }
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j)
            m = fmaxf(m, fabsf(v[i][j]));
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1)
        m = fmaxf(m, __shfl_xor(m, d));
    if ((tid & (kWave - 1)) == 0)
        wave_max[tid / kWave] = m;
    __syncthreads();
    const float a = fmaxf(fmaxf(fmaxf(wave_max[0], wave_max[1]), fmaxf(wave_max[2], wave_max[3])), 0x1p-64f);
    const float inv = 448.0f / a;
    if (tid == 0) {
        scales[(g * NB + nblk) * KB + kb] = a / 448.0f;
        if (codes_t)
            scales_t[(g * KB + kb) * NB + nblk] = a / 448.0f;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        u32x4 q;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t c = e4m3fn_pair<false>(v[i][4 * j] * inv, v[i][4 * j + 1] * inv, 0u);
            q[j] = e4m3fn_pair<true>(v[i][4 * j + 2] * inv, v[i][4 * j + 3] * inv, c);
        }
        store16_hint<false>(codes + base + (size_t)(r0 + 32 * i) * K + c0, q);
        if (codes_t) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                tile[(r0 + 32 * i) * kTileLd + (c0 >> 2) + j] = q[j];
        }
    }
    if (!codes_t)
        return;
    __syncthreads();
    // this thread: 16 rows n of four columns k
    const int n0 = (tid & 7) * 16, k4 = tid >> 3;
    u32x4 o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t* t = tile + (n0 + 4 * j) * kTileLd + k4;
        const uint32_t a0 = t[0], a1 = t[kTileLd], a2 = t[2 * kTileLd], a3 = t[3 * kTileLd];
        // byte b of a0..a3 -> the four bytes of o[b][j] (__byte_perm counts the first operand's bytes 0-3)
        const uint32_t p01 = __byte_perm(a0, a1, 0x5140), p23 = __byte_perm(a2, a3, 0x5140);
        const uint32_t q01 = __byte_perm(a0, a1, 0x7362), q23 = __byte_perm(a2, a3, 0x7362);
        o[0][j] = __byte_perm(p01, p23, 0x5410);
        o[1][j] = __byte_perm(p01, p23, 0x7632);
        o[2][j] = __byte_perm(q01, q23, 0x5410);
        o[3][j] = __byte_perm(q01, q23, 0x7632);
    }
    const size_t tbase = (g * K + (size_t)kb * kQBlock) * N + (size_t)nblk * kQBlock;
#pragma unroll
    for (int b = 0; b < 4; ++b)
        store16_hint<false>(codes_t + tbase + (size_t)(4 * k4 + b) * N + n0, o[b]);
}

hipError_t launch_quantize_weights(const void* w, bool w_f32, int G, int N, int K, void* codes,
                                   float* scales, void* codes_t, float* scales_t, hipStream_t stream)
{
    const dim3 grid(K / kQBlock, N / kQBlock, G);
    debug_launch("quantize_weights", grid, dim3(256), 0);
    auto* kernel = w_f32 ? quantize_weights_kernel<true> : quantize_weights_kernel<false>;
    kernel<<<grid, 256, 0, stream>>>(w, N, K, static_cast<uint8_t*>(codes), scales,
                                     static_cast<uint8_t*>(codes_t), scales_t);
    return hipGetLastError();
}

}  // namespace moe_ep
