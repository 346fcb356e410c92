// Grouped product of FP8 rows with 4-bit weights on gfx950: for the rows r of group g
//   y[r][n] = sum over 128-channel blocks b of
//             sx[r][b] * (sum over k in b of x[r][k] * code[g][n][k] * s[g][n][k / 32])
// The inner sum is one matrix instruction (K = 128, E2M1 by E4M3), which applies the
// weights' scales itself: a lane of its first operand holds 32 neighbouring k of one
// column n, which is one scale.  Its second operand's lane holds k = 16 q .. + 15 and
// 64 + 16 q .. + 15 (q = lane / 16).  The rows' scales are arbitrary fp32 numbers, so
// every block's result is scaled on the vector unit and added in fp32.
#include <type_traits>

#include "block_launch.h"
#include "gemm_tile.h"

namespace moe_ep {

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

// Large tiles: 256 rows x 256 columns by eight waves, each 64 rows x 128 columns.  One
// K block is computed from LDS while the next one is copied in behind it: 32 KB of x a
// block; of w two blocks at a time (128 bytes of a column, a whole cache line), half of
// the columns with each of the two blocks before.  The scales of four blocks are fetched
// together: 16 bytes of a row of x, 16 of a column of w.
struct TileFp4Source {
    const uint8_t* x;             // first row of the tile
    const uint8_t* w;
    const float* xs;
    const uint8_t* ws;
    uint32_t xo[4], wo[4], so, wso;
    int sld;                      // column-major row scales: elements between blocks
    bool four;                    // row-major row scales whose rows are whole, aligned fours
    int tail;                     // subtracted in the last pair of blocks, where it is half of one
};

__device__ __forceinline__ void copy_x(const TileFp4Source& t, int kb, int wave, uint8_t* lx)
{
#pragma unroll
    for (int i = 0; i < 4; ++i)
        load_to_lds16(t.x + (t.xo[i] + kb * kQBlock), lx + (8 * i + wave) * 1024);
}

// Columns 128 * half .. + 127 of block pair p.
__device__ __forceinline__ void copy_w(const TileFp4Source& t, int p, int half, int pairs, int wave, uint8_t* lw)
{
    const int back = p == pairs - 1 ? t.tail : 0;
#pragma unroll
    for (int i = 0; i < 2; ++i)
        load_to_lds16(t.w + (t.wo[2 * half + i] + p * kQBlock - back), lw + (16 * half + 8 * i + wave) * 1024);
}

// The columns' scales of blocks kb .. kb + 3, by waves 4-7, 64 columns each: [column][block][four]
// or, one by one, [block][column][four].
template <bool FOUR>
__device__ __forceinline__ void copy_w_scales(const TileFp4Source& t, int kb, int KB, int wave, uint8_t* ls)
{
    if (wave < 4)
        return;
    if (FOUR) {
        load_to_lds16(t.ws + (t.wso + kb * 4), ls + (wave - 4) * 1024);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            load_to_lds4(t.ws + (t.wso + min(kb + i, KB - 1) * 4), ls + i * 1024 + (wave - 4) * 256);
    }
}

// One K block: the wave's 4 row tiles x 8 column tiles.  A matrix instruction's result is
// scaled and added three instructions later, while the next ones run; the order is
// pinned, since left alone the compiler waits for each result.
// x0, x1: where this lane's two chunks of its row of row tile 0 lie, w0: its chunk of its
// column of column tile 0.  The other tiles lie at fixed distances, since a chunk's
// permutation does not depend on them.
__device__ __forceinline__ int column_step(int c) { return 32 * (c >> 1) + 4 * (c & 1); }

__device__ __forceinline__ void compute_fp4(const uint8_t* x0, const uint8_t* x1, const uint8_t* w0,
                                            const float (&s)[4], const uint32_t (&ws)[8], f32x4 (&acc)[4][8])
{
    const auto read_w = [&](int c) { return *reinterpret_cast<const u32x4*>(w0 + column_step(c) * kQBlock); };
    i32x8 x[4];
    u32x4 w[3];
    f32x4 d[4];
    w[0] = read_w(0);
#pragma unroll
    for (int r = 0; r < 4; ++r)
        x[r] = join(*reinterpret_cast<const u32x4*>(x0 + 16 * r * kQBlock), *reinterpret_cast<const u32x4*>(x1 + 16 * r * kQBlock));
    w[1] = read_w(1);
#pragma unroll
    for (int i = 0; i < 32 + 3; ++i) {
        const int c = i >> 2, r = i & 3;
        if (i < 32)
            d[r] = mfma_fp4_fp8(w[c % 3], x[r], ws[c]);
        if (r == 0 && c + 2 < 8)
            w[(c + 2) % 3] = read_w(c + 2);
        if (i >= 3) {
            const int pc = (i - 3) >> 2, pr = (i - 3) & 3;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                acc[pr][pc][q] = __builtin_fmaf(d[pr][q], s[pr], acc[pr][pc][q]);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
}

// FOUR: the columns' scales are whole, aligned fours.
template <bool FOUR>
__global__ __launch_bounds__(512, 2) void gemm_fp4_tile_kernel(GemmFp4Launch a)
{
    __shared__ __align__(1024) uint8_t lx0[kStage], lx1[kStage], lw0[kStage], lw1[kStage];
    __shared__ __align__(16) float ls[2][4 * kTile];
    __shared__ __align__(16) uint8_t lws[2][16 * kTile];
    __shared__ int prefix[EP_MAX_EXPERTS + 1];
    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int N = a.N, K = a.K, KB = K / kQBlock, pairs = (KB + 1) / 2, NT = (N + kTile - 1) / kTile;
    tile_prefix<kTile>(a.groups, prefix);
    __syncthreads();
    const int64_t total = (int64_t)prefix[a.groups.num] * NT;
    const int row0 = (wave >> 1) * 64, col0 = (wave & 1) * 128;
    const int xbase = (row0 + (lane & 15)) * kQBlock + (((lane >> 4) ^ place_x(lane & 15)) << 4);
    const int col = column_of(col0, 0, lane);
    const int wbase = col * kQBlock + (((lane >> 4) ^ place_w(col)) << 4);
    const int wsbase = col * (FOUR ? 16 : 4) + (lane >> 4);
    const int64_t t0 = (int64_t)(blockIdx.x % kXcds) * (gridDim.x / kXcds) + blockIdx.x / kXcds;
    for (int64_t t = t0; t < total; t += gridDim.x) {
        const int g = __builtin_amdgcn_readfirstlane(find_group(prefix, a.groups.num, t, NT));
        int begin, end;
        group_bounds(a.groups, g, begin, end);
        const int mt = prefix[g + 1] - prefix[g];
        const int local = (int)(t - (int64_t)prefix[g] * NT);
        const int m0 = __builtin_amdgcn_readfirstlane(begin + (local % mt) * kTile);
        const int n0 = __builtin_amdgcn_readfirstlane((local / mt) * kTile);
        TileFp4Source src;
        src.x = a.x + (size_t)m0 * K;
        src.w = a.w + ((size_t)g * N + n0) * (K / 2);
        src.ws = a.w_scales + ((size_t)g * N + n0) * (K / 32);
        src.xs = a.x_scales + scale_at(m0, 0, KB, a.x_scale_ld);
        const int last_row = end - 1 - m0, last_col = N - 1 - n0;   // rows past the end: the last one again
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = (8 * i + wave) * 8 + (lane >> 3);
            src.xo[i] = (uint32_t)min(r, last_row) * K + ((lane & 7) ^ place_x(r)) * 16;
            src.wo[i] = (uint32_t)min(r, last_col) * (K / 2) + ((lane & 7) ^ place_w(r)) * 16;
        }
        // an odd number of blocks ends with half a pair: chunks 0-3 stand in for its chunks 4-7 (place_w's bit 2 is
        // bit 0 of the wave in each of its rows)
        src.tail = (KB & 1) && (((lane >> 2) ^ wave) & 1) ? 64 : 0;
        {
            const int r = (wave & 3) * 64 + lane;
            src.so = a.x_scale_ld ? min(r, last_row) : (uint32_t)min(r, last_row) * KB;
            src.sld = a.x_scale_ld;
            src.four = !a.x_scale_ld && KB % 4 == 0 && reinterpret_cast<uintptr_t>(a.x_scales) % 16 == 0;
            src.wso = (uint32_t)min(r, last_col) * (K / 32);
        }
        const bool on = row0 <= last_row && col0 <= last_col;
        f32x4 acc[4][8];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 8; ++c)
                acc[r][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        copy_x(src, 0, wave, lx0);
        copy_w(src, 0, 0, pairs, wave, lw0);
        copy_w(src, 0, 1, pairs, wave, lw0);
        copy_scales(src, 0, KB, wave, ls[0]);
        copy_w_scales<FOUR>(src, 0, KB, wave, lws[0]);
        __syncthreads();
        // block kb, the HALF of its pair: computed from lx, lw while block kb + 1 goes to nx and half of the next
        // pair's columns to nw.  The scales are read before the copies are issued: the compiler would wait for
        // those of a later group
        const auto stage = [&](auto HALF, int kb, const uint8_t* lx, const uint8_t* lw, uint8_t* nx, uint8_t* nw) {
            constexpr int half = decltype(HALF)::value;
            float s[4];
            uint32_t ws[8];
            const float* p = ls[(kb >> 2) & 1];
            const int first = src.four ? (row0 + (lane & 15)) * 4 + (kb & 3) : (kb & 3) * kTile + row0 + (lane & 15);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                s[r] = p[first + (src.four ? 64 : 16) * r];
            const uint8_t* q = lws[(kb >> 2) & 1] + wsbase + (kb & 3) * (FOUR ? 4 : 1024);
#pragma unroll
            for (int c = 0; c < 8; ++c)
                ws[c] = q[column_step(c) * (FOUR ? 16 : 4)];
            if (kb + 1 < KB) {
                copy_x(src, kb + 1, wave, nx);
                if ((kb + 1) % 4 == 0) {
                    copy_scales(src, kb + 1, KB, wave, ls[((kb + 1) >> 2) & 1]);
                    copy_w_scales<FOUR>(src, kb + 1, KB, wave, lws[((kb + 1) >> 2) & 1]);
                }
            }
            if ((kb >> 1) + 1 < pairs)
                copy_w(src, (kb >> 1) + 1, half, pairs, wave, nw);
            if (on)
                compute_fp4(lx + xbase, lx + (xbase ^ 64), lw + (wbase ^ (64 * half)), s, ws, acc);
            __syncthreads();
        };
        constexpr std::integral_constant<int, 0> even{};
        constexpr std::integral_constant<int, 1> odd{};
        for (int kb = 0; kb < KB; kb += 4) {
            stage(even, kb, lx0, lw0, lx1, lw1);
            if (kb + 1 < KB)
                stage(odd, kb + 1, lx1, lw0, lx0, lw1);
            if (kb + 2 < KB)
                stage(even, kb + 2, lx0, lw1, lx1, lw0);
            if (kb + 3 < KB)
                stage(odd, kb + 3, lx1, lw1, lx0, lw0);
        }
        if (on) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = row0 + 16 * r + (lane & 15);
                if (row > last_row)
                    continue;
                uint16_t* o = a.out + (size_t)(m0 + row) * N + n0 + col0 + 8 * (lane >> 4);
#pragma unroll
                for (int c = 0; c < 8; c += 2)
                    store16_hint<false>(o + 16 * c, u32x4{pack2_bf16(acc[r][c][0], acc[r][c][1]),
                                                          pack2_bf16(acc[r][c][2], acc[r][c][3]),
                                                          pack2_bf16(acc[r][c + 1][0], acc[r][c + 1][1]),
                                                          pack2_bf16(acc[r][c + 1][2], acc[r][c + 1][3])});
            }
        }
        // the last barrier lies behind every read of the stages and scales: the next tile may overwrite them
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
    else if (m <= 64)
        skinny_run<4, 4>(L, stream);
    else {
        debug_launch("grouped_gemm_fp4_tile", dim3(kCus), dim3(512), 0);
        const bool four = L.K % 512 == 0 && reinterpret_cast<uintptr_t>(L.w_scales) % 16 == 0;
        auto* kernel = four ? gemm_fp4_tile_kernel<true> : gemm_fp4_tile_kernel<false>;
        kernel<<<kCus, 512, 0, stream>>>(L);
    }
    return hipGetLastError();
}

}  // namespace moe_ep
