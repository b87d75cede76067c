// grouped_wgrad_plan.cuh -- which CTA sums up which rows of which tile of dW, and which parts
// belong together.  Everything is a function of `seg` and the grid alone; a test runs this file on the CPU.
#pragma once

#include "layers.cuh"

namespace spc {

namespace {

constexpr int kUnit = 64;  // rows of a unit
constexpr int kSplitFrom = 24;
constexpr int kMaxParts = 192;  // CTAs at most: one thread of the smaller block plans for each

// A part of one tile: units [k0, k1) of its `units`.
struct Piece {
    int32_t g, tile;
    int32_t k0, k1, units;
    int64_t lo, hi;  // positions of the segment
    int32_t slot;    // of a part: 0 at the start of its CTA's share, else 1
    __device__ __forceinline__ bool whole() const { return k0 == 0 && k1 == units; }
};

// The plan of a call, the same in every CTA: a function of `seg` and the grid alone.
// Segments are listed with those of at most an even share (total units / CTAs) first,
// the longer ones after them.  The tiles of that list in turn: the first `waves` x CTAs
// are whole tiles, tile c + i CTAs for CTA c, so that neighbouring tiles read the same
// rows at the same time; the units of the tiles after them go to the CTAs in
// contiguous shares, each as long as evens out what its whole tiles took.  Where no tile is
// longer than kSplitFrom units all of them stay whole: a cut costs two parts of 128 KB written and
// read again, as much as 20 units or so (4,096 rows of 8 segments, 512 x 2048: 25 us
// against 33).
struct Plan {
    int64_t m;                   // positions, 0 where the offsets cannot be used
    int64_t whole;               // tiles that stay whole
    int32_t longest;             // units of the longest tile
    int32_t parts;               // CTAs
    int64_t base;                // first unit of the shares
    int64_t first[kMaxParts + 1];  // share c: units base + first[c] .. base + first[c + 1)
    int32_t id[kMaxParts];       // number of CTA c among those that have a share
};

struct Walk {
    const int32_t* start;  // units of a tile of the listed segments before j, summed
    const int32_t* list;   // segment j of the list
    const int32_t* seg;
    const Plan* plan;
    int32_t segments, tiles;  // tiles of one segment
    int32_t wave, c;
    int64_t u, begin, end;

    __device__ __forceinline__ void piece(Piece& p, int j, int32_t tile) const
    {
        p.g = list[j];
        p.tile = tile;
        p.units = start[j + 1] - start[j];
        segment_bounds(seg, p.g, plan->m, nullptr, p.lo, p.hi);
    }
    __device__ __forceinline__ void reset(int32_t cta)
    {
        c = cta;
        wave = 0;
        u = begin = plan->base + plan->first[c];
        end = plan->base + plan->first[c + 1];
    }
    __device__ __forceinline__ int64_t tile_of(int w) const { return c + (int64_t)w * plan->parts; }
    __device__ __forceinline__ bool more() const { return tile_of(wave) < plan->whole || u < end; }
    __device__ __forceinline__ Piece next()
    {
        Piece p;
        if (tile_of(wave) < plan->whole) {
            const int64_t t = tile_of(wave);
            const int32_t j = (int32_t)((uint32_t)t / (uint32_t)tiles);
            piece(p, j, (int32_t)(t - (int64_t)j * tiles));
            p.k0 = p.slot = 0;
            p.k1 = p.units;
            ++wave;
            return p;
        }
        p = at(u);
        const int64_t left = end - u;
        p.slot = u == begin ? 0 : 1;
        p.k1 = p.units - p.k0 <= left ? p.units : p.k0 + (int32_t)left;
        u += p.k1 - p.k0;
        return p;
    }
    // The piece that begins at unit v and runs to its tile's end.
    __device__ __forceinline__ Piece at(int64_t v) const
    {
        const int32_t f = (int32_t)(v / tiles);
        int lo = 0, hi = segments;  // last j with start[j] <= f
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (start[mid] <= f) lo = mid;
            else hi = mid;
        }
        const int64_t in = v - (int64_t)start[lo] * tiles;
        const int32_t units = start[lo + 1] - start[lo], tile = (int32_t)(in / units);
        Piece p;
        piece(p, lo, tile);
        p.k0 = (int32_t)(in - (int64_t)tile * units);
        p.k1 = units;
        p.slot = 0;
        return p;
    }
};

template <typename V>
__device__ __forceinline__ V warp_add(V v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(FULL_MASK, v, d);
    return v;
}
template <typename V>
__device__ __forceinline__ V warp_before(V v, int lane)  // the sum of the lanes below
{
    const V own = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const V u = __shfl_up_sync(FULL_MASK, v, d);
        if (lane >= d) v += u;
    }
    return v - own;
}

// The whole tiles and the shares, by one warp; a lane speaks for kMaxParts / 32 CTAs in a row.
__device__ __forceinline__ void share_out(Plan* plan, const int32_t* s_start, int segments, int tiles, int parts, int shorter,
                                          int64_t total, int lane)
{
    constexpr int P = kMaxParts / 32;
    auto unit_of_tile = [&](int64_t t) -> int64_t {
        const int32_t j = (int32_t)((uint32_t)t / (uint32_t)tiles);
        if (j >= segments) return total;
        return (int64_t)s_start[j] * tiles + (t - (int64_t)j * tiles) * (s_start[j + 1] - s_start[j]);
    };
    // whole waves: all there are, less one where too little would be left to even out
    int32_t waves = (int32_t)((int64_t)shorter * tiles / parts);
    if (waves > 0 && (total - unit_of_tile((int64_t)waves * parts)) * 8 < total / waves) --waves;
    const bool all_whole = plan->longest <= kSplitFrom;
    const int64_t whole = all_whole ? (int64_t)segments * tiles : (int64_t)waves * parts;
    const int64_t base = unit_of_tile(whole), rest = total - base;
    int64_t took[P];
    bool below[P];
#pragma unroll
    for (int q = 0; q < P; ++q) {
        const int c = lane * P + q;
        took[q] = 0;
        below[q] = c < parts && rest > 0;
        if (below[q])
            for (int i = 0; i < waves; ++i) {
                const uint32_t j = (uint32_t)(c + i * parts) / (uint32_t)tiles;
                took[q] += s_start[j + 1] - s_start[j];
            }
    }
    // the level to which the shares fill every CTA that is below it.  A round takes out those above the level of
    // the others; the lowest is never above it, so there are at most `parts` rounds (a few, unless segments
    // differ by orders of magnitude) and the shares add up to the rest.
    int64_t level = 0, extra = 0;
    for (int round = 0; round < parts && rest > 0; ++round) {
        int64_t sum = 0;
        int32_t n = 0;
#pragma unroll
        for (int q = 0; q < P; ++q)
            if (below[q]) {
                sum += took[q];
                ++n;
            }
        sum = warp_add(sum) + rest;
        n = warp_add(n);
        level = sum / n;
        extra = sum - level * n;
        bool above = false;
#pragma unroll
        for (int q = 0; q < P; ++q) above |= below[q] && took[q] > level;
        if (!__any_sync(FULL_MASK, above)) break;
#pragma unroll
        for (int q = 0; q < P; ++q) below[q] = below[q] && took[q] <= level;
    }
    int32_t mine = 0;
#pragma unroll
    for (int q = 0; q < P; ++q) mine += below[q];
    int32_t rank = warp_before(mine, lane);
    int64_t share[P], sum = 0;
    int32_t some = 0;
#pragma unroll
    for (int q = 0; q < P; ++q) {
        share[q] = below[q] ? level - took[q] + (rank++ < extra ? 1 : 0) : 0;
        sum += share[q];
        some += share[q] > 0;
    }
    int64_t to = warp_before(sum, lane);
    int32_t id = warp_before(some, lane);
#pragma unroll
    for (int q = 0; q < P; ++q) {
        const int c = lane * P + q;
        to += share[q];
        if (c < parts) {
            plan->first[c + 1] = to;
            plan->id[c] = share[q] > 0 ? id : id - 1;
        }
        id += share[q] > 0;
    }
    if (lane == 0) {
        plan->first[0] = 0;
        plan->whole = whole;
        plan->parts = parts;
        plan->base = base;
    }
}

// Fills the list, its unit sums [segments + 1] and the plan; one warp does it all, which
// spares a dozen barriers of the block.
__device__ __forceinline__ void make_plan(const int32_t* seg, int segments, int64_t m, int tiles, int parts,
                                          int32_t* s_start, int32_t* s_list, int32_t* s_units, Plan* plan, int32_t* status,
                                          int lane)
{
    int64_t all = 0;
    int32_t longest = 0;
    for (int g = lane; g < segments; g += 32) {
        int64_t a, b;
        segment_bounds(seg, g, m, status, a, b);
        const int32_t units = b > a ? (int32_t)((b - a + kUnit - 1) / kUnit) : 1;
        s_units[g] = units;
        all += units;
        longest = longest > units ? longest : units;
    }
    all = warp_add(all);
    longest = __reduce_max_sync(FULL_MASK, longest);
    __syncwarp();
    if (all > INT32_MAX) {
        // only offsets out of order, which were reported, name that many: each segment is taken as empty, as
        // the sums of units below have 31 bits
        for (int g = lane; g < segments; g += 32) s_units[g] = 1;
        all = segments;
        longest = 1;
        m = 0;
        __syncwarp();
    }
    const int64_t total = all * tiles, even = total / parts;
    int32_t listed = 0, shorter = 0, carry = 0;
    for (int pass = 0; pass < 2; ++pass)
        for (int g0 = 0; g0 < segments; g0 += 32) {
            const int g = g0 + lane;
            const int32_t units = g < segments ? s_units[g] : 0;
            const bool mine = g < segments && (units <= even) == (pass == 0);
            const unsigned who = __ballot_sync(FULL_MASK, mine);
            const int32_t at = listed + __popc(who & ((1u << lane) - 1u)), own = mine ? units : 0;
            const int32_t before = carry + warp_before(own, lane);
            if (mine) {
                s_list[at] = g;
                s_start[at] = before;
            }
            listed += __popc(who);
            carry = __shfl_sync(FULL_MASK, before + own, 31);
            if (pass == 0) shorter = listed;
        }
    if (lane == 0) {
        s_start[segments] = carry;
        plan->longest = longest;
        plan->m = m;
    }
    __syncwarp();
    share_out(plan, s_start, segments, tiles, parts, shorter, total, lane);
}

// The tile that starts in the share of a CTA and ends in a later one: its parts are slot `slot`
// of that share and the first slots of the `more` shares after it (0: there is none).
struct Join {
    int32_t g, tile, slot, more;
};

__device__ __forceinline__ Join join_of(const Walk& walk, int c)
{
    const Plan* plan = walk.plan;
    const int64_t u0 = plan->base + plan->first[c], u1 = plan->base + plan->first[c + 1];
    Join j{0, 0, 0, 0};
    const Piece p = walk.at(u1 - 1);
    const int64_t first = u1 - 1 - p.k0, end = first + p.units;
    if (first < u0 || end <= u1) return j;
    j.g = p.g;
    j.tile = p.tile;
    j.slot = first == u0 ? 0 : 1;
    for (int q = c + 1; q < plan->parts && plan->base + plan->first[q] < end; ++q)
        if (plan->first[q + 1] > plan->first[q]) ++j.more;
    return j;
}

// CTA c's entry of `joins`, by one thread; a number that no share has gets an empty one.
__device__ __forceinline__ void write_join(const Walk& walk, int c, Join* joins)
{
    const Plan* plan = walk.plan;
    if (plan->first[c + 1] > plan->first[c]) joins[plan->id[c]] = join_of(walk, c);
    const int n = plan->id[plan->parts - 1] + 1;
    if (n + c < plan->parts) joins[n + c] = Join{0, 0, 0, 0};
}

}  // namespace

}  // namespace spc
