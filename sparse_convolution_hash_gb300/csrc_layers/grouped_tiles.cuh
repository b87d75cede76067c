// grouped_tiles.cuh -- how the persistent tensor-core kernels walk the tiles of
// all segments.
//
// Segment sizes are device data.  Each CTA sums the tiles of every segment
// once (its share of the grid is then tiles first, first + stride, ...) and finds the
// segment of its next tile by walking on from the last one.  Entry 0 stands for the positions
// before the first segment, entry segments + 1 for those after the last: their
// rows are zeros.
#pragma once

#include "layers.cuh"

namespace spc {

struct TileWalk {
    const int32_t* start;  // shared: first tile of each of the segments + 2 entries, and the total
    const int32_t* seg;
    int64_t m;
    int32_t segments;
    int32_t rows;          // positions per tile
    int32_t cols;          // column tiles
    int32_t v;             // current entry

    // Positions of entry v, clamped to [0, m).
    __device__ __forceinline__ void bounds(int entry, int64_t& lo, int64_t& hi) const
    {
        if (entry == 0) {
            const int64_t f = fetch(seg);
            lo = 0;
            hi = f < 0 ? 0 : (f > m ? m : f);
        } else if (entry > segments) {
            const int64_t f = fetch(seg + segments);
            lo = f < 0 ? 0 : (f > m ? m : f);
            hi = m;
        } else {
            segment_bounds(seg, entry - 1, m, nullptr, lo, hi);
        }
    }

    struct Tile {
        int32_t g;        // segment, -1: rows of zeros
        int64_t lo, hi;   // positions
        int32_t col;      // column tile
    };

    // Tile t (t increases from call to call).  Within a segment, blocks of eight row tiles
    // go through the column tiles together, so the CTAs at work share rows and weights in L2.
    __device__ __forceinline__ Tile at(int32_t t)
    {
        while (t >= start[v + 1]) ++v;
        int64_t a, b;
        bounds(v, a, b);
        const int32_t u = t - start[v];
        const int32_t mt = (start[v + 1] - start[v]) / cols;
        const int32_t block = u / (8 * cols), in = u - block * 8 * cols;
        const int32_t high = mt - block * 8 < 8 ? mt - block * 8 : 8;
        Tile k;
        k.g = v == 0 || v > segments ? -1 : v - 1;
        k.lo = a + (int64_t)(block * 8 + in % high) * rows;
        k.hi = k.lo + rows < b ? k.lo + rows : b;
        k.col = in / high;
        return k;
    }
};

// Fills s_start [segments + 3] (every thread of the block calls it; `threads` of them,
// a multiple of 32, at most 1024) and returns the number of tiles.
__device__ __forceinline__ int32_t tile_starts(const int32_t* seg, int segments, int64_t m, int rows, int cols,
                                               int32_t* s_start, int32_t* status, int tid, int threads)
{
    __shared__ int32_t s_warp[32];
    const int lane = tid & 31, warp = tid >> 5;
    int32_t carry = 0;
    for (int v0 = 0; v0 < segments + 2; v0 += threads) {
        const int v = v0 + tid;
        int64_t a = 0, b = 0;
        if (v == 0) {
            const int64_t f = fetch(seg);
            b = f < 0 ? 0 : (f > m ? m : f);
        } else if (v <= segments) {
            segment_bounds(seg, v - 1, m, status, a, b);
        } else if (v == segments + 1) {
            const int64_t f = fetch(seg + segments);
            a = f < 0 ? 0 : (f > m ? m : f);
            b = m;
        }
        const int32_t tiles = (int32_t)((b - a + rows - 1) / rows) * cols;
        int32_t inc = tiles;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t u = __shfl_up_sync(FULL_MASK, inc, d);
            if (lane >= d) inc += u;
        }
        if (lane == 31) s_warp[warp] = inc;
        __syncthreads();
        int32_t base = carry;
        for (int w = 0; w < threads / 32; ++w) {
            if (w < warp) base += s_warp[w];
            carry += s_warp[w];
        }
        if (v < segments + 2) s_start[v] = base + inc - tiles;
        __syncthreads();
    }
    if (tid == 0) s_start[segments + 2] = carry;
    __syncthreads();
    return carry;
}

}  // namespace spc
