// Grouped weight gradient on gfx950: for every group g
//   dW[g][n][k] = sum over the group's rows r of dy[r][n] * x[r][k] * sx[r][k / 128]
// with dy in bf16 and x in the 8 bits it was dispatched in (the activation
// checkpoint of the product).  The scale belongs to a row, and rows are what is
// summed over, so it cannot be taken out of the sum: x is widened to bf16 on its
// way into LDS (an 8-bit code times the scale in fp32, then one rounding by at most
// 2^-8 of the value, which is 1.7e-3 of the result's norm: with an out of bf16 as much
// as its own rounding, with one of fp32 all of the error) and the product runs on the
// bf16 matrix cores with fp32 sums.  fp32 products of the same numbers would cost the
// matrix cores sixteen times as much.
#include "expert_launch.h"
#include "mfma.h"

namespace moe_ep {

// A tile is 128 * NW columns of dy x 256 of x by 4 * NW waves, each 128 x 64, ROWS
// rows (a stage) at a time from two LDS buffers.  dy is copied straight into LDS;
// x's codes are fetched into registers a stage ahead, widened and written there.
// Both operands are needed with the rows, which LDS holds one behind the other,
// along a lane's values: the transposed LDS read does that.  An LDS row's 32-byte
// chunks (16 columns, what such a read takes of a row) are permuted by the row's
// number, so that the rows it spans lie in different banks.
//
// Two forms (G = 32, N = 4096, K = 7168, MI355X):
//   NW = 2, 64 rows   one workgroup a CU; 2262 us at 1024 rows a group (850 TFLOP/s),
//                     682 us at 128, 514 us at 16
//   NW = 1, 32 rows   two, so that one's first loads and last stores run beside the
//                     other's products: 429 us at 16 rows a group, 699 us at 128,
//                     2603 us at 1024
// What bounds the first is the time a stage's loads take to arrive (a copy without the
// matrix instructions takes 1916 us in a run at 2264) and the stores at a tile's end (one
// without them 1930); the matrix cores are busy for 37% of the cycles.  The second, with
// few rows, is bound by the stores: 1.9 GB of gradients.
constexpr int kTile = 256;                     // columns of x

// The permutation of row r's chunks: rows 0-3 and 8-11 (4-7 and 12-15), which the
// lanes 0-31 of a transposed read span, take eight different places.
__device__ __forceinline__ int place(int r) { return (r & 3) | ((r >> 1) & 4); }

// Eight rows (row + 8 * (lane / 16)) of a chunk's 16 columns, transposed.
template <int LD>
__device__ __forceinline__ bf16x8 read_chunk(const uint16_t* lds, int row, int chunk, int lane)
{
    const int r = row + (lane >> 4) * 8 + ((lane & 15) >> 2);
    const uint16_t* p = lds + r * LD + ((chunk ^ place(r)) << 4) + (lane & 3) * 4;
    const i16x4 a = lds_read_tr16(p), b = lds_read_tr16(p + 4 * LD);
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// ROWS rows: the wave's 8 tiles of dy's columns x 4 of x's.
template <int NW, int ROWS>
__device__ __forceinline__ void wgrad_stage(const uint16_t* ly, const uint16_t* lx, int wn, int wk, int lane,
                                            f32x4 (&acc)[8][4])
{
#pragma unroll
    for (int s = 0; s < ROWS; s += 32) {
        bf16x8 x[4], y[2];
        y[0] = read_chunk<128 * NW>(ly, s, wn / 16, lane);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            x[j] = read_chunk<kTile>(lx, s, wk / 16 + j, lane);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i + 1 < 8)
                y[(i + 1) & 1] = read_chunk<128 * NW>(ly, s, wn / 16 + i + 1, lane);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[j], y[i & 1], acc[i][j], 0, 0, 0);
        }
    }
}

struct WgradSource {
    const uint16_t* dy;           // first column of the tile
    const uint8_t* x;
    const float* s;
    int N, K, end;
    size_t srow;                  // elements between rows' scales
    int yrow, ycol, xrow, xcol;   // this lane's
};

template <int NW, int ROWS>
__device__ __forceinline__ void copy_dy(const WgradSource& t, int r0, int wave, uint16_t* to)
{
#pragma unroll
    for (int j = 0; j < ROWS / 16; ++j) {          // 4 * NW waves copy 4 / NW rows each
        const int r = min(r0 + 16 * j + t.yrow, t.end - 1);
        load_to_lds16(t.dy + (size_t)r * t.N + t.ycol, to + (4 * NW * j + wave) * 512);
    }
}

struct XRegs {
    u32x4 q[2];                   // rows xrow and xrow + ROWS / 2
    float s[2];
};

// Rows past the group: the group's last row, as zeros once written to LDS.
template <int ROWS>
__device__ __forceinline__ void fetch_x(const WgradSource& t, int r0, XRegs& o)
{
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int r = min(r0 + ROWS / 2 * j + t.xrow, t.end - 1);
        o.q[j] = load16_hint<false>(t.x + (size_t)r * t.K + t.xcol);
        o.s[j] = t.s[(size_t)r * t.srow];
    }
}

// Of every 32 columns, the chunk of tile j holds columns 8 * i + 0..3, i = 0..3, and that
// of tile j + 1 the others: a lane's results of both are then eight neighbouring columns.
template <int ROWS>
__device__ __forceinline__ void write_x(const WgradSource& t, int r0, const XRegs& x, uint16_t* to)
{
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int row = ROWS / 2 * j + t.xrow;
        const bool on = r0 + row < t.end;
        u32x4 o[2];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float a, b, c, d;
            e4m3fn_pair_to_f32<false>(x.q[j][k], a, b);
            e4m3fn_pair_to_f32<true>(x.q[j][k], c, d);
            o[k & 1][k & 2] = on ? pack2_bf16(a * x.s[j], b * x.s[j]) : 0u;
            o[k & 1][(k & 2) + 1] = on ? pack2_bf16(c * x.s[j], d * x.s[j]) : 0u;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
            *reinterpret_cast<u32x4*>(to + row * kTile + ((((threadIdx.x & 14) + h) ^ place(row)) << 4) +
                                      (threadIdx.x & 1) * 8) = o[h];
    }
}

template <int NW, int ROWS, bool F32>
__global__ __launch_bounds__(256 * NW, 2) void wgrad_kernel(WgradLaunch a)
{
    constexpr int kTileN = 128 * NW;
    __shared__ __align__(1024) uint16_t ly0[ROWS * kTileN], ly1[ROWS * kTileN], lx0[ROWS * kTile], lx1[ROWS * kTile];
    const int tid = threadIdx.x, lane = tid % kWave, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int N = a.N, K = a.K, NT = (N + kTileN - 1) / kTileN, KT = (K + kTile - 1) / kTile;
    // neighbouring tiles on one XCD, 32 of them in every 256
    int t = blockIdx.x;
    if (t / 256 * 256 + 256 <= (int)gridDim.x)
        t = t / 256 * 256 + t % 8 * 32 + t % 256 / 8;
    const int g = t / (NT * KT), n0 = t % NT * kTileN, k0 = t / NT % KT * kTile;
    int begin, end;
    group_bounds(a.groups, g, begin, end);
    const int wn = wave % NW * 128, wk = wave / NW * 64;
    // columns past the matrix: the last ones again, not stored
    WgradSource src;
    const int KB = K / kQBlock;
    constexpr int kRowLanes = 16 * NW;        // lanes that copy a row of dy
    src.yrow = wave * (4 / NW) + lane / kRowLanes;
    src.ycol = min((((lane % kRowLanes >> 1) ^ place(src.yrow)) << 4) + (lane & 1) * 8, N - 8 - n0);
    src.xrow = tid >> 4;
    src.xcol = min((tid & 15) * 16, K - 16 - k0);
    src.dy = a.dy + n0;
    src.x = a.x + k0;
    src.s = a.x_scales + scale_at(0, (k0 + src.xcol) / kQBlock, KB, a.x_scale_ld);
    src.srow = a.x_scale_ld ? 1 : KB;
    src.N = N;
    src.K = K;
    src.end = end;
    f32x4 acc[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (begin < end) {
        const bool on = n0 + wn < N && k0 + wk < K;
        XRegs x;
        copy_dy<NW, ROWS>(src, begin, wave, ly0);
        fetch_x<ROWS>(src, begin, x);
        write_x<ROWS>(src, begin, x, lx0);
        __syncthreads();
        for (int r = begin; r < end; r += 2 * ROWS) {
            if (r + ROWS < end) {
                copy_dy<NW, ROWS>(src, r + ROWS, wave, ly1);
                fetch_x<ROWS>(src, r + ROWS, x);
            }
            __builtin_amdgcn_sched_barrier(0);
            if (on)
                wgrad_stage<NW, ROWS>(ly0, lx0, wn, wk, lane, acc);
            __builtin_amdgcn_sched_barrier(0);
            if (r + ROWS < end)
                write_x<ROWS>(src, r + ROWS, x, lx1);
            __syncthreads();
            if (r + ROWS < end) {
                if (r + 2 * ROWS < end) {
                    copy_dy<NW, ROWS>(src, r + 2 * ROWS, wave, ly0);
                    fetch_x<ROWS>(src, r + 2 * ROWS, x);
                }
                __builtin_amdgcn_sched_barrier(0);
                if (on)
                    wgrad_stage<NW, ROWS>(ly1, lx1, wn, wk, lane, acc);
                __builtin_amdgcn_sched_barrier(0);
                if (r + 2 * ROWS < end)
                    write_x<ROWS>(src, r + 2 * ROWS, x, lx0);
                __syncthreads();
            }
        }
    }
    // lane: row n = lane % 16 of tile i, columns 8 * (lane / 16) .. + 7 of the pair of tiles j, j + 1
    if (n0 + wn >= N || k0 + wk >= K)
        return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const size_t at = ((size_t)g * N + n0 + wn + 16 * i + (lane & 15)) * K + k0 + wk + 8 * (lane >> 4);
#pragma unroll
        for (int j = 0; j < 4; j += 2) {
            if (F32) {
                float* o = static_cast<float*>(a.dw) + at + 16 * j;
                *reinterpret_cast<f32x4*>(o) = acc[i][j];
                *reinterpret_cast<f32x4*>(o + 4) = acc[i][j + 1];
            } else {
                u32x4 v;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    v[q] = pack2_bf16(acc[i][j + (q >> 1)][(q & 1) * 2], acc[i][j + (q >> 1)][(q & 1) * 2 + 1]);
                *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.dw) + at + 16 * j) = v;
            }
        }
    }
}

template <int NW, int ROWS>
static void wgrad_run(const WgradLaunch& L, hipStream_t stream)
{
    const int64_t tiles = (int64_t)L.groups.num * ((L.N + 128 * NW - 1) / (128 * NW)) * ((L.K + kTile - 1) / kTile);
    const dim3 grid((unsigned)tiles);
    debug_launch("grouped_wgrad", grid, dim3(256 * NW), 0);
    if (L.dw_f32)
        wgrad_kernel<NW, ROWS, true><<<grid, 256 * NW, 0, stream>>>(L);
    else
        wgrad_kernel<NW, ROWS, false><<<grid, 256 * NW, 0, stream>>>(L);
}

hipError_t launch_grouped_wgrad(const WgradLaunch& L, hipStream_t stream)
{
    if (L.groups.num == 0)
        return hipSuccess;
    // m: rows a group on average; tiles: 256 x 256 ones of one group.  With equal groups and
    // every CU busy the forms cross near 128 rows.  Groups differ in size, which the host does
    // not know, and a launch ends with its largest group's tiles: where those leave half of
    // the CUs idle, twice as many smaller ones end sooner; from 512 rows a group only while
    // all groups' tiles do not fill the CUs twice, since equal groups lose more there.  NW = 1 against NW = 2 in us, 16
    // groups, even sizes | zipf ones, (rank + 1)^-1.2:
    //   m                                128                         512                        1024
    //   1408 x 2048 (48)     33 : 35 |  36 : 47       76 :  69 |  103 :  116      127 :  115 |  193 :  218
    //   2048 x 4096 (128)    99 : 93 | 101 : 108     215 : 186 |  223 :  199      362 :  330 |  395 :  373
    //   2816 x 4096 (176)   130 : 129 | 138 : 142    293 : 271 |  322 :  305      491 :  441 |  525 :  508
    //   4096 x 7168 (448)   355 : 346 | 365 : 348    773 : 702 |  777 :  705     1289 : 1133 | 1297 : 1141
    // Over 572 cases (1 to 64 groups, 8 to 448 tiles, 48 to 2048 rows, both distributions) this
    // choice takes 1.5 % longer than the better form, always NW = 1 3.2 %, always NW = 2 7.5 %.
    const int m = L.groups.rows / L.groups.num;
    const int64_t tiles = (int64_t)((L.N + kTile - 1) / kTile) * ((L.K + kTile - 1) / kTile);
    if (m < 128 || (tiles <= 128 && (m < 512 || tiles * L.groups.num < 512)))
        wgrad_run<1, 32>(L, stream);
    else
        wgrad_run<2, 64>(L, stream);
    return hipGetLastError();
}

}  // namespace moe_ep
