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
#include "moe_ep.h"

namespace moe_ep {

constexpr int kXcds = 8, kCus = 256;

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
                    uint2{pack2_bf16(v[0], v[1]), pack2_bf16(v[2], v[3])};
        }
        __syncthreads();
    }
}

// Large tiles: 256 rows x 256 columns by eight waves, each 64 rows x 128
// columns (one scale block of the weights).  One K block of both operands
// (2 x 32 KB and the rows' scales) is computed from LDS while the next one is
// copied in behind it.  LDS rows are the 128 bytes of a K block; a row's 16-byte
// chunks are permuted by its number, which the copy does for free (it chooses
// which global chunk lands where), so that eight rows read at the same chunk
// hit all banks once.
//
// 65536 rows in 32 groups, N = 4096, K = 7168: 1838-1899 us over five inputs on one card,
// 1949 on another, 1.97-2.09 PFLOP/s, where a library product of E4M3 matrices with one
// scale reaches 2.9 (8192^3) to 3.2 (16384^3).  The matrix cores are busy for 51% of the
// cycles, and the clock falls to 1.9 GHz.  In a run at 1883 us, copies of the kernel with
// parts taken out take 1612 us (no matrix instructions, scaled sums and LDS reads) and
// 1442 us (no copies after the first two blocks): the two do not overlap fully.  Forms
// with a stream of stages across tiles, copies one and a half stages ahead, or pinned
// fetches into L2 came out within 3% or slower.
constexpr int kTile = 256;
constexpr int kStage = kTile * kQBlock;

// Where a tile's operands come from, and this lane's offsets.  Wave w copies rows
// 8 * (8 * i + w) .. + 7 of both operands.
struct TileSource {
    const uint8_t* x;             // first row of the tile
    const uint8_t* w;
    const float* xs;
    uint32_t xo[4], wo[4], so;
    int sld;                      // column-major scales: elements between blocks
    bool four;                    // row-major scales whose rows are whole, aligned fours
};

__device__ __forceinline__ void copy_stage(const TileSource& t, int kb, int wave, uint8_t* lx, uint8_t* lw)
{
    const uint32_t k = kb * kQBlock;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        load_to_lds16(t.w + (t.wo[i] + k), lw + (8 * i + wave) * 1024);
        load_to_lds16(t.x + (t.xo[i] + k), lx + (8 * i + wave) * 1024);
    }
}

// The rows' scales of blocks kb .. kb + 3, by waves 0-3, 64 rows each.  In row-major
// scales every row is a cache line of its own, so the four are fetched together:
// one by one they were a third of all requests a tile makes (1950 against 1865 us
// at 65536 x 4096 x 7168).
__device__ __forceinline__ void copy_scales(const TileSource& t, int kb, int KB, int wave, float* ls)
{
    if (wave >= 4)
        return;
    if (t.four) {
        load_to_lds16(t.xs + (t.so + kb), ls + wave * 256);            // [row][block]
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {                                  // [block][row]
            const int k = min(kb + i, KB - 1);
            load_to_lds4(t.xs + (t.so + (t.sld ? (size_t)k * t.sld : k)), ls + i * kTile + wave * 64);
        }
    }
}

// The permutation of row r's chunks, w's and x's: the eight rows that lanes read
// together (see read_w, read_x) have eight different ones.
__device__ __forceinline__ int place_w(int r) { return (r & 3) | ((r >> 1) & 4); }
__device__ __forceinline__ int place_x(int r) { return r & 7; }

__device__ __forceinline__ i32x8 read_fragment(const uint8_t* row, int place, int lane)
{
    const int c = lane >> 4;
    const u32x4 lo = *reinterpret_cast<const u32x4*>(row + ((c ^ place) << 4));
    const u32x4 hi = *reinterpret_cast<const u32x4*>(row + (((c + 4) ^ place) << 4));
    return join(lo, hi);
}

__device__ __forceinline__ i32x8 read_x(const uint8_t* lds, int row0, int r, int lane)
{
    const int row = row0 + 16 * r + (lane & 15);
    return read_fragment(lds + row * kQBlock, place_x(row), lane);
}

// Column tiles 2i and 2i + 1 take every other four of 32 columns, so that a lane's
// results of both are eight neighbouring columns (one 16-byte store).
__device__ __forceinline__ i32x8 read_w(const uint8_t* lds, int col0, int c, int lane)
{
    const int row = col0 + 32 * (c >> 1) + ((lane & 12) << 1) + (lane & 3) + 4 * (c & 1);
    return read_fragment(lds + row * kQBlock, place_w(row), lane);
}

// One K block: the wave's 4 row tiles x 8 column tiles.  A matrix instruction's
// result is scaled and added three instructions later, while the next ones run;
// the order is pinned, since left alone the compiler waits for each result.
__device__ __forceinline__ void compute_stage(const uint8_t* lx, const uint8_t* lw, const float (&s)[4],
                                              int row0, int col0, int lane, f32x4 (&acc)[4][8])
{
    i32x8 x[4], w[3];
    f32x4 d[4];
    w[0] = read_w(lw, col0, 0, lane);
#pragma unroll
    for (int r = 0; r < 4; ++r)
        x[r] = read_x(lx, row0, r, lane);
    w[1] = read_w(lw, col0, 1, lane);
#pragma unroll
    for (int i = 0; i < 32 + 3; ++i) {
        const int c = i >> 2, r = i & 3;
        if (i < 32)
            d[r] = mfma_fp8(w[c % 3], x[r]);
        if (r == 0 && c + 2 < 8)
            w[(c + 2) % 3] = read_w(lw, col0, c + 2, lane);
        if (i >= 3) {
            const int pc = (i - 3) >> 2, pr = (i - 3) & 3;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                acc[pr][pc][q] = __builtin_fmaf(d[pr][q], s[pr], acc[pr][pc][q]);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
}

__global__ __launch_bounds__(512, 2) void gemm_tile_kernel(GemmLaunch a)
{
    __shared__ __align__(1024) uint8_t lx0[kStage], lx1[kStage], lw0[kStage], lw1[kStage];
    __shared__ __align__(16) float ls[2][4 * kTile];
    __shared__ float lsw[2][EP_MAX_HIDDEN / kQBlock];
    __shared__ int prefix[EP_MAX_EXPERTS + 1];
    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int N = a.N, K = a.K, KB = K / kQBlock, NB = N / kQBlock, NT = (N + kTile - 1) / kTile;
    tile_prefix<kTile>(a.groups, prefix);
    __syncthreads();
    const int64_t total = (int64_t)prefix[a.groups.num] * NT;
    const int row0 = (wave >> 1) * 64, col0 = (wave & 1) * 128;
    const int64_t t0 = (int64_t)(blockIdx.x % kXcds) * (gridDim.x / kXcds) + blockIdx.x / kXcds;
    for (int64_t t = t0; t < total; t += gridDim.x) {
        const int g = __builtin_amdgcn_readfirstlane(find_group(prefix, a.groups.num, t, NT));
        int begin, end;
        group_bounds(a.groups, g, begin, end);
        const int mt = prefix[g + 1] - prefix[g];
        const int local = (int)(t - (int64_t)prefix[g] * NT);
        const int m0 = __builtin_amdgcn_readfirstlane(begin + (local % mt) * kTile);
        const int n0 = __builtin_amdgcn_readfirstlane((local / mt) * kTile);
        TileSource src;
        src.x = a.x + (size_t)m0 * K;
        src.w = a.w + ((size_t)g * N + n0) * K;
        src.xs = a.x_scales + scale_at(m0, 0, KB, a.x_scale_ld);
        const int last_row = end - 1 - m0, last_col = N - 1 - n0;   // rows past the end: the last one again
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int r = (8 * i + wave) * 8 + (lane >> 3);
            src.xo[i] = (uint32_t)min(r, last_row) * K + ((lane & 7) ^ place_x(r)) * 16;
            src.wo[i] = (uint32_t)min(r, last_col) * K + ((lane & 7) ^ place_w(r)) * 16;
        }
        {
            const int r = min((wave & 3) * 64 + lane, last_row);
            src.so = a.x_scale_ld ? r : (uint32_t)r * KB;
            src.sld = a.x_scale_ld;
            src.four = !a.x_scale_ld && KB % 4 == 0 && reinterpret_cast<uintptr_t>(a.x_scales) % 16 == 0;
        }
        const bool on = row0 <= last_row && col0 <= last_col;
        for (int i = tid; i < 2 * KB; i += 512) {
            const int half = i >= KB, nb = min(n0 / kQBlock + half, NB - 1);
            lsw[half][i - half * KB] = a.w_scales[((size_t)g * NB + nb) * KB + i - half * KB];
        }
        const float* sw = lsw[wave & 1];
        f32x4 acc[4][8];
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
            for (int c = 0; c < 8; ++c)
                acc[r][c] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        copy_stage(src, 0, wave, lx0, lw0);
        copy_scales(src, 0, KB, wave, ls[0]);
        __syncthreads();
        // the stage's scales are read before its copies are issued: the compiler would
        // wait for those of a later group
        const auto scales = [&](int kb, float (&s)[4]) {
            const float* p = ls[(kb >> 2) & 1];
            const int first = src.four ? (row0 + (lane & 15)) * 4 + (kb & 3) : (kb & 3) * kTile + row0 + (lane & 15);
#pragma unroll
            for (int r = 0; r < 4; ++r)
                s[r] = p[first + (src.four ? 64 : 16) * r] * sw[kb];
        };
        for (int kb = 0; kb < KB; kb += 2) {
            float s[4];
            scales(kb, s);
            if (kb + 1 < KB)
                copy_stage(src, kb + 1, wave, lx1, lw1);
            if (on)
                compute_stage(lx0, lw0, s, row0, col0, lane, acc);
            __syncthreads();
            if (kb + 1 < KB) {
                scales(kb + 1, s);
                if (kb + 2 < KB) {
                    copy_stage(src, kb + 2, wave, lx0, lw0);
                    if ((kb + 2) % 4 == 0)
                        copy_scales(src, kb + 2, KB, wave, ls[((kb + 2) >> 2) & 1]);
                }
                if (on)
                    compute_stage(lx1, lw1, s, row0, col0, lane, acc);
                __syncthreads();
            }
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
        // the last barrier lies behind every read of lsw and the stages: the next tile may overwrite them
    }
}

template <int RT, int CT>
static void skinny_run(const GemmLaunch& L, hipStream_t stream)
{
    const size_t lds = (size_t)(L.groups.num + 1) * 4;
    const dim3 grid(kCus * 4);
    debug_launch("grouped_gemm_skinny", grid, dim3(256), lds);
    gemm_skinny_kernel<RT, CT><<<grid, 256, lds, stream>>>(L);
}

// The tile by the typical rows m of a group.  G = 32, N = 4096, K = 7168 (940 MB of
// weights; 188 us at the rate of a large copy), in us:
//   m                 2     8    16    32   128   512
//   16 x 64 skinny  142   164   227   344  1160  4420
//   32 x 64 skinny  158   176   187   284   787  2890
//   256 x 256       194   196   197   201   234   570
// The 64 x 64 skinny form is for products of few large tiles, which leave CUs idle: up to
// 512 of its own tiles (two a CU at once), 64 x 64 against 256 x 256 in us:
//   64 x 64 tiles    128        256        512        1024       2048
//   512 x 1024      9 : 15     9 : 16    15 : 18    26 : 25    46 : 25     16 groups at m = 64; 32 at 64 .. 512
//   512 x 4096     23 : 40    24 : 40    41 : 45    76 : 67   148 : 67     the same
//   4096 x 7168    36 : 62    37 : 63    67 : 69   128 : 73   254 : 108    2, 4, 8 groups at m = 64; 8 at 128, 256
// Over 223 cases (1 to 32 groups, m = 17 to 2048) this choice takes 0.5 % longer than the
// better form; with the border at 704 or 1024 tiles 0.9 %, at 352 4.3 %.
hipError_t launch_grouped_gemm(const GemmLaunch& L, hipStream_t stream)
{
    if (L.groups.rows == 0 || L.groups.num == 0)
        return hipSuccess;
    const int m = L.expected_rows;
    const int64_t small = (int64_t)L.groups.num * (((int64_t)m + 63) / 64) * (L.N / 64);    // tiles of 64 x 64
    if (m <= 8) {
        skinny_run<1, 4>(L, stream);
    } else if (m <= 16) {
        skinny_run<2, 4>(L, stream);
    } else if (small <= 512) {
        skinny_run<4, 4>(L, stream);
    } else {
        debug_launch("grouped_gemm_tile", dim3(kCus), dim3(512), 0);
        gemm_tile_kernel<<<kCus, 512, 0, stream>>>(L);
    }
    return hipGetLastError();
}

}  // namespace moe_ep
