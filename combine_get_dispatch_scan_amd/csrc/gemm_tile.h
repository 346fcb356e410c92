// Pieces of the 256 x 256 tiles that the grouped products share: eight waves, each
// with 64 rows x 128 columns; LDS rows of 128 bytes whose 16-byte chunks are permuted
// by the row's number, which the copy does for free (it chooses which global chunk
// lands where), so that eight rows read at the same chunk hit all banks once.
#pragma once

#include "mfma.h"

namespace moe_ep {

constexpr int kTile = 256;
constexpr int kStage = kTile * kQBlock;

// The rows' scales of blocks kb .. kb + 3, by waves 0-3, 64 rows each.  In row-major
// scales every row is a cache line of its own, so the four are fetched together:
// one by one they were a third of all requests a tile makes (1950 against 1865 us
// at 65536 x 4096 x 7168).  A source has xs, so (this lane's row), sld (column-major
// scales: elements between blocks, else 0) and four (row-major, whole, aligned fours).
template <typename Source>
__device__ __forceinline__ void copy_scales(const Source& t, int kb, int KB, int wave, float* ls)
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
// together (see column_of, read_x) have eight different ones.
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

// The column of a wave's 128 that this lane reads for column tile c.  Column tiles 2i
// and 2i + 1 take every other four of 32 columns, so that a lane's results of both are
// eight neighbouring columns (one 16-byte store).
__device__ __forceinline__ int column_of(int col0, int c, int lane)
{
    return col0 + 32 * (c >> 1) + ((lane & 12) << 1) + (lane & 3) + 4 * (c & 1);
}

}  // namespace moe_ep
