// Runs the plan of the gradient by the weights (csrc_layers/grouped_wgrad_plan.cuh) on the CPU: 32 threads
// stand for the lanes of a warp and exchange values where the warp does.
//
// Input, a case a line: segments, positions m, tiles of a segment, CTAs, then segments + 1 offsets.  For each case
// it walks every CTA's pieces and every join and prints "ok" and the number of joins, or what is wrong:
//   every unit of every tile belongs to one piece; parts of a cut tile have places of their own;
//   each join names a tile's parts in the order of its rows, and each part has one join.
#include <barrier>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <iostream>
#include <map>
#include <sstream>
#include <string>
#include <thread>
#include <vector>

static std::barrier<>* g_meet;
static uint64_t g_slot[32];
static thread_local int t_lane;

template <typename T>
static T exchange(T v, int from)
{
    uint64_t w = 0;
    std::memcpy(&w, &v, sizeof(v));
    g_slot[t_lane] = w;
    g_meet->arrive_and_wait();
    T r;
    std::memcpy(&r, &g_slot[from < 0 || from > 31 ? t_lane : from], sizeof(r));
    g_meet->arrive_and_wait();
    return r;
}
template <typename T> static T __shfl_sync(unsigned, T v, int from) { return exchange(v, from); }
template <typename T> static T __shfl_xor_sync(unsigned, T v, int d) { return exchange(v, t_lane ^ d); }
template <typename T> static T __shfl_up_sync(unsigned, T v, int d) { return exchange(v, t_lane - d); }
static unsigned __ballot_sync(unsigned, bool p)
{
    unsigned r = 0;
    g_slot[t_lane] = p;
    g_meet->arrive_and_wait();
    for (int i = 0; i < 32; ++i) r |= (unsigned)g_slot[i] << i;
    g_meet->arrive_and_wait();
    return r;
}
static bool __any_sync(unsigned m, bool p) { return __ballot_sync(m, p) != 0; }
static int __reduce_max_sync(unsigned, int v)
{
    int r = v;
    g_slot[t_lane] = (uint32_t)v;
    g_meet->arrive_and_wait();
    for (int i = 0; i < 32; ++i) r = (int)g_slot[i] > r ? (int)g_slot[i] : r;
    g_meet->arrive_and_wait();
    return r;
}
static void __syncwarp() { g_meet->arrive_and_wait(); }
static int __popc(unsigned v) { return __builtin_popcount(v); }
static int atomicCAS(int* p, int expected, int v)
{
    __atomic_compare_exchange_n(p, &expected, v, false, __ATOMIC_RELAXED, __ATOMIC_RELAXED);
    return expected;
}

#include "grouped_wgrad_plan.cuh"

using namespace spc;

struct Span {
    int32_t g, tile, k0, k1, units;
};

static std::string check(int segments, int64_t m, int tiles, int parts, const std::vector<int32_t>& seg)
{
    std::vector<int32_t> start(segments + 1), list(segments), units(segments);
    static Plan plan;
    std::memset(&plan, 0x5a, sizeof(plan));
    int32_t status = 0;
    std::vector<std::thread> lanes;
    for (int i = 0; i < 32; ++i)
        lanes.emplace_back([&, i] {
            t_lane = i;
            make_plan(seg.data(), segments, m, tiles, parts, start.data(), list.data(), units.data(), &plan, &status, i);
        });
    for (auto& t : lanes) t.join();

    char text[256];
    auto say = [&](const char* what, long a, long b) {
        std::snprintf(text, sizeof(text), "%s (%ld, %ld)", what, a, b);
        return std::string(text);
    };
    // what the tiles have, straight from the offsets
    std::vector<int64_t> want(segments), taken((size_t)segments * tiles, 0);
    for (int g = 0; g < segments; ++g) {
        int64_t lo, hi;
        segment_bounds(seg.data(), g, m, nullptr, lo, hi);
        want[g] = hi > lo ? (hi - lo + kUnit - 1) / kUnit : 1;
    }
    Walk walk{start.data(), list.data(), seg.data(), &plan, segments, tiles, 0, 0, 0, 0, 0};
    std::map<int64_t, Span> cut;  // by place: number of the share, slot
    const int64_t most = (int64_t)segments * tiles + 2 * parts;
    for (int c = 0; c < parts; ++c) {
        walk.reset(c);
        for (int64_t n = 0; walk.more(); ++n) {
            if (n > most) return say("a walk that does not end", c, n);
            const Piece p = walk.next();
            if (p.g < 0 || p.g >= segments || p.tile < 0 || p.tile >= tiles) return say("no such tile", p.g, p.tile);
            if (p.units != (p.lo == p.hi ? 1 : want[p.g]) || p.k0 < 0 || p.k0 >= p.k1 || p.k1 > p.units)
                return say("no such units", p.k0, p.k1);
            taken[(size_t)p.g * tiles + p.tile] += p.k1 - p.k0;
            if (p.whole()) continue;
            if (plan.id[c] < 0 || plan.id[c] >= parts) return say("a share without a number", c, plan.id[c]);
            if (!cut.emplace((int64_t)plan.id[c] * 2 + p.slot, Span{p.g, p.tile, p.k0, p.k1, p.units}).second)
                return say("two parts in one place", c, p.slot);
        }
    }
    if (status == 0)
        for (size_t i = 0; i < taken.size(); ++i)
            if (taken[i] != want[i / tiles]) return say("a tile's units are not each taken once", (long)i, taken[i]);
    std::vector<Join> joins(parts, Join{-7, -7, -7, 1 << 20});
    for (int c = 0; c < parts; ++c) write_join(walk, c, joins.data());
    long done = 0;
    for (int n = 0; n < parts; ++n) {
        const Join j = joins[n];
        if (j.more == 0) continue;
        if (j.more < 0 || j.more >= parts) return say("an entry that nobody wrote", n, j.more);
        int32_t k = 0, all = -1;
        for (int q = 0; q <= j.more; ++q) {
            const auto at = cut.find(q == 0 ? (int64_t)n * 2 + j.slot : (int64_t)(n + q) * 2);
            if (at == cut.end()) return say("a join of a part that is not there", n, q);
            const Span s = at->second;
            if (s.g != j.g || s.tile != j.tile || s.k0 != k) return say("a join of another tile's part", n, q);
            k = s.k1;
            all = s.units;
            cut.erase(at);
        }
        if (k != all) return say("a join that ends early", n, k);
        ++done;
    }
    if (!cut.empty()) return say("a part without a join", (long)cut.size(), 0);
    return say("ok", done, status);
}

int main()
{
    std::barrier<> meet(32);
    g_meet = &meet;
    std::string line;
    while (std::getline(std::cin, line)) {
        std::istringstream in(line);
        int segments, tiles, parts;
        int64_t m;
        in >> segments >> m >> tiles >> parts;
        std::vector<int32_t> seg(segments + 1);
        for (auto& v : seg) in >> v;
        std::cout << check(segments, m, tiles, parts, seg) << std::endl;
    }
}
