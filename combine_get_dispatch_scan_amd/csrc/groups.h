// Row groups (the experts' blocks of a receive buffer) as the kernels see them.
#pragma once

#include "device.h"

namespace moe_ep {

// Group g holds off[g+1] - off[g] rows: from row off[g] on, or, with a stride,
// from row g*stride on (the static layout, at most `stride` of them).  The
// offsets are device data that the host has not seen, so every bound taken
// from them is clamped to the `rows` that exist: no content of the array makes
// a kernel leave its buffers.
struct Groups {
    const int32_t* off;
    int num, stride, rows;
};

__device__ __forceinline__ void group_bounds(const Groups& g, int i, int& begin, int& end)
{
    const int o0 = g.off[i], o1 = g.off[i + 1];
    if (g.stride) {
        const int64_t b = (int64_t)i * g.stride;
        const int64_t n = (int64_t)o1 - o0;
        begin = (int)(b < g.rows ? b : g.rows);
        const int64_t e = begin + (n < 0 ? 0 : n > g.stride ? g.stride : n);
        end = (int)(e < g.rows ? e : g.rows);
    } else {
        begin = o0 < 0 ? 0 : o0 > g.rows ? g.rows : o0;
        end = o1 < begin ? begin : o1 > g.rows ? g.rows : o1;
    }
}

// Whether row r (0 <= r < rows) belongs to a group.
__device__ __forceinline__ bool row_in_group(const Groups& g, int r)
{
    if (!g.off)
        return true;
    if (g.stride) {
        const int i = r / g.stride;
        if (i >= g.num)
            return false;
        return r - i * g.stride < (int64_t)g.off[i + 1] - g.off[i];
    }
    return r >= g.off[0] && r < g.off[g.num];
}

// Running count of the groups' row tiles of TILE rows: prefix[i] = tiles of groups
// before i (LDS, num + 1 entries).  The first wave fills it; the caller
// synchronises.  Groups that do not overlap have at most rows / TILE + num tiles;
// offsets that make them overlap are cut off at 2^30.
template <int TILE>
__device__ __forceinline__ void tile_prefix(const Groups& g, int* prefix)
{
    if (threadIdx.x >= kWave)
        return;
    const int lane = threadIdx.x;
    int64_t run = 0;
    if (lane == 0)
        prefix[0] = 0;
    for (int base = 0; base < g.num; base += kWave) {
        int64_t n = 0;
        if (base + lane < g.num) {
            int b, e;
            group_bounds(g, base + lane, b, e);
            n = ((int64_t)e - b + TILE - 1) / TILE;
        }
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
            const int64_t o = __shfl_up((long long)n, d);
            if (lane >= d)
                n += o;
        }
        if (base + lane < g.num)
            prefix[base + lane + 1] = (int)(run + n < (1 << 30) ? run + n : 1 << 30);
        run += __shfl((long long)n, kWave - 1);
    }
}

// The group whose tiles [prefix[i], prefix[i+1]) * per hold tile t.
__device__ __forceinline__ int find_group(const int* prefix, int num, int64_t t, int per)
{
    int lo = 0, hi = num;           // prefix[lo]*per <= t < prefix[hi]*per
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((int64_t)prefix[mid] * per <= t)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// Address of row r's scale of 128-channel block b (ld 0: row-major [rows][nb],
// else column-major [nb][ld]).
__device__ __forceinline__ size_t scale_at(int r, int b, int nb, int ld)
{
    return ld ? (size_t)b * ld + r : (size_t)r * nb + b;
}

}  // namespace moe_ep
