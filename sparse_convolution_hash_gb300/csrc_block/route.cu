// route.cu -- the experts of each token and their weights, and the gradient by the logits.
//
// A row of logits lies in the registers of L lanes (1 to 32), eight neighbouring experts to a lane (beyond 256
// experts four such chunks).  Each lane sorts its eight once; then the best of the lanes' firsts is taken k times and
// its lane moves up, so a round costs a reduction and a few moves whatever the number of experts.  Without a bias and groups
// the logits themselves are compared, which is exact; 16-bit ones are sorted together with their expert in one word.
// With a bias or groups the scores decide, p + bias, and fp32 is not enough for the last digit: the row's choice is made in fp32, and where
// two neighbours of the result lie closer than fp32's error, made again in 64 bits: about one row in a hundred or fewer where scores are
// spread out, most rows where sigmoids are saturated (16,000 rows of 256 experts bf16, 8 each, without bias: 23 us for logits of 0 +- 1.2, 215 of
// 0 +- 5).  The choice is therefore that of the formula in 64 bits, whatever the order of the sums.
//
// Bound by instructions: a row of 64 experts in 16 bits is 128 bytes and some 140 instructions, one of 256 in fp32 in groups 1,300.
#include <math.h>

#include "block.cuh"
#include "pairs.cuh"

namespace spc {

namespace {

constexpr int kBlock = 128;
constexpr int kPer = 8;  // experts of a lane's chunk
constexpr int kNone = INT32_MAX;

__device__ __forceinline__ float exp_of(float x) { return expf(x); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }

template <int L, typename S>
__device__ __forceinline__ S lanes_sum(S v)
{
#pragma unroll
    for (int o = L >> 1; o; o >>= 1) v += __shfl_xor_sync(FULL_MASK, v, o);
    return v;
}
template <int L, typename S>
__device__ __forceinline__ S lanes_max(S v)
{
#pragma unroll
    for (int o = L >> 1; o; o >>= 1) v = max(v, __shfl_xor_sync(FULL_MASK, v, o));
    return v;
}

// Logits of a row, -inf where there is no expert, and for one that is not available (-inf, NaN); +inf counts as
// the largest finite number, so that differences exist.
template <typename T, int C, int L>
__device__ __forceinline__ void load_logits(const T* row, int experts, int lane, bool whole, float (&l)[C][kPer])
{
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e0 = (c * L + lane) * kPer;
        if (whole && e0 < experts) {
            constexpr int V = 16 / sizeof(T);
#pragma unroll
            for (int q = 0; q < kPer / V; ++q) {
                const Vec<T, V> v = *reinterpret_cast<const Vec<T, V>*>(row + e0 + q * V);
#pragma unroll
                for (int j = 0; j < V; ++j) l[c][q * V + j] = elem<T>::to_f32(v.e[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kPer; ++j) l[c][j] = e0 + j < experts ? elem<T>::to_f32(fetch(row + e0 + j)) : -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) l[c][j] = l[c][j] > -INFINITY ? fminf(l[c][j], 3.402823466e38f) : -INFINITY;
    }
}

// Sum over the row of exp(l - most), `most` its largest logit (-inf: no expert is available).
template <typename S, int C, int L>
__device__ __forceinline__ S exp_sum(const float (&l)[C][kPer], float most)
{
    S s = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (l[c][j] > -INFINITY) s += exp_of((S)l[c][j] - (S)most);
    }
    return lanes_sum<L>(s);
}

template <typename S>
__device__ __forceinline__ S score_of(float l, bool sigmoid, float most, S sum)
{
    return sigmoid ? (S)1 / ((S)1 + exp_of(-(S)l)) : exp_of((S)l - (S)most) / sum;
}

// For the choice in fp32: off by less than 2^-21 (sigmoid) or 2^-18 of the largest score.
__device__ __forceinline__ float rough_score(float l, bool sigmoid, float most, float sum)
{
    return sigmoid ? __fdividef(1.f, 1.f + __expf(fminf(-l, 88.f))) : __fdividef(__expf(l - most), sum);
}

struct RouteShared {
    int32_t* expert;   // [k] of this row, and one more for the choice in fp32
    float* logit;      // the same
    void* c;           // [experts], then [groups], of 64 bits; groups only
};

// Scores as words that are ordered as they are (the least word for -inf and NaN, which are never chosen).
__device__ __forceinline__ uint32_t order_of(float v)
{
    const uint32_t b = __float_as_uint(v + 0.f);  // one zero
    return v > -INFINITY ? b ^ (b >> 31 ? 0xffffffffu : 0x80000000u) : 0u;
}
__device__ __forceinline__ float value_of(uint32_t w) { return w ? __uint_as_float(w >> 31 ? w ^ 0x80000000u : ~w) : -INFINITY; }

template <int L>
__device__ __forceinline__ uint32_t lanes_most(uint32_t v)
{
    if constexpr (L == 32) return __reduce_max_sync(FULL_MASK, v);
    else return lanes_max<L>(v);
}

// The best of a warp's values: (value, expert, logit), ties to the lowest expert; expert kNone where none is left.
__device__ __forceinline__ void best_of_warp(float& top, int& e, float& l)
{
    const uint32_t key = order_of(top), most = lanes_most<32>(key);
    const bool mine = key == most && e != kNone;
    const uint32_t least = ~lanes_most<32>(~(mine ? (uint32_t)e : (uint32_t)kNone));
    const int winner = __ffs(__ballot_sync(FULL_MASK, mine && (uint32_t)e == least)) - 1;
    const int from = max(winner, 0);
    e = __shfl_sync(FULL_MASK, e, from);
    l = __shfl_sync(FULL_MASK, l, from);
    top = value_of(most);
    if (winner < 0) e = kNone;
}

// ---- a lane's eight in falling order.  Words of 64 bits: order_of(value), then the larger for the lower expert; of 32
// bits, for 16-bit logits: their order in the high half.  0: not available.
__device__ __forceinline__ uint64_t rank_of(float v, int e)
{
    const uint32_t w = order_of(v);
    return w ? (uint64_t)w << 32 | (0xffffffffu - (uint32_t)e) : 0ull;
}
template <typename T>
__device__ __forceinline__ uint32_t rank16(T v, int e)
{
    constexpr uint32_t kInf = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
    uint16_t h;
    memcpy(&h, &v, 2);
    uint32_t b = h == 0x8000u ? 0u : h;
    const bool there = (b & 0x7fffu) <= kInf && b != (0x8000u | kInf);
    b = b & 0x8000u ? ~b & 0xffffu : b | 0x8000u;
    return there ? b << 16 | (0xffffu - (uint32_t)e) : 0u;
}
template <typename T>
__device__ __forceinline__ float logit16(uint32_t word)
{
    const uint32_t b = word >> 16;
    const uint16_t h = (uint16_t)(b & 0x8000u ? b & 0x7fffu : ~b);
    T v;
    memcpy(&v, &h, 2);
    return fminf(elem<T>::to_f32(v), 3.402823466e38f);
}

template <typename W>
__device__ __forceinline__ void sort8(W (&v)[8])
{
    // Batcher's odd-even merging network
    constexpr int kA[19] = {0, 2, 4, 6, 0, 1, 4, 5, 1, 5, 0, 1, 2, 3, 2, 3, 1, 3, 5};
    constexpr int kB[19] = {1, 3, 5, 7, 2, 3, 6, 7, 2, 6, 4, 5, 6, 7, 4, 5, 2, 4, 6};
#pragma unroll
    for (int x = 0; x < 19; ++x) {
        const W a = v[kA[x]], b = v[kB[x]];
        v[kA[x]] = max(a, b);
        v[kB[x]] = min(a, b);
    }
}

// The best of the lanes' firsts (0: none is left), which its lane drops; e: its expert.
template <int L>
__device__ __forceinline__ uint32_t take_best(uint32_t (&v)[8], int, int& e)
{
    const uint32_t most = lanes_most<L>(v[0]);  // no two are equal but 0
    e = 0xffff - (int)(most & 0xffffu);
    if (v[0] == most) {
#pragma unroll
        for (int j = 0; j < 7; ++j) v[j] = v[j + 1];
        v[7] = 0u;
    }
    return most;
}
template <int L>
__device__ __forceinline__ uint32_t take_best(uint64_t (&v)[8], int lane, int& e)
{
    const uint32_t most = lanes_most<L>((uint32_t)(v[0] >> 32));
    // lanes hold ascending experts, so the lowest lane has the lowest of equal ones
    const uint32_t at = (threadIdx.x & 31) - lane, votes = __ballot_sync(FULL_MASK, (uint32_t)(v[0] >> 32) == most) >> at;
    const int winner = __ffs(votes) - 1;
    e = (int)(0xffffffffu - __shfl_sync(FULL_MASK, (uint32_t)v[0], winner, L));
    if (lane == winner) {
#pragma unroll
        for (int j = 0; j < 7; ++j) v[j] = v[j + 1];
        v[7] = 0ull;
    }
    return most;
}

// A group's score from its two best.  What fp32 does not hold becomes its lowest number or infinity, which lie near every
// other such sum, so that 64 bits decide.
__device__ __forceinline__ float group_score(float first, float second)
{
    return second > -INFINITY ? fmaxf(first + second, -3.402823466e38f) : first;
}

// Scores in fp32 are compared without their last three bits, where the place among the lane's eight stands: sorting
// is a third of what it is with words of 64 bits.
__device__ __forceinline__ uint32_t rough_rank(float v, int j)
{
    const uint32_t w = order_of(v);
    return w ? (w & ~7u) | (uint32_t)(7 - j) : 0u;
}
template <int L>
__device__ __forceinline__ uint32_t take_rough_best(uint32_t (&v)[8], int lane, int& e)
{
    const uint32_t mine = v[0] & ~7u, most = lanes_most<L>(mine);
    const uint32_t at = (threadIdx.x & 31) - lane, votes = __ballot_sync(FULL_MASK, mine == most) >> at;
    const int winner = __ffs(votes) - 1;
    e = winner * kPer + 7 - (int)(__shfl_sync(FULL_MASK, v[0], winner, L) & 7u);
    if (lane == winner) {
#pragma unroll
        for (int j = 0; j < 7; ++j) v[j] = v[j + 1];
        v[7] = 0u;
    }
    return most;
}

// The row's k best, written to sh.expert and sh.logit by its lane 0.  By the logits, exactly
// (BY_LOGIT), or by the scores in fp32: returns whether two neighbours, or the border of the kept groups, lie
// within the error: scores are off by 2^-20, or 2^-16 of the largest one (softmax), and by 2^-20 of their own size, at most.
template <typename T, bool BY_LOGIT, int C, int L>
__device__ __forceinline__ bool choose(const RouteArgs& a, const T* row, const float (&l)[C][kPer], int lane, bool whole,
                                       const RouteShared& sh)
{
    constexpr float kLow = -INFINITY;
    bool near = false;
    float c[C][kPer], off = 0;
    const bool in_lanes = C == 1 && a.lanes_log2 >= 0;  // no shared memory
    if constexpr (BY_LOGIT) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) c[i][j] = l[i][j];
        }
    } else {
        const bool sigmoid = a.score == SPC_SCORE_SIGMOID;
        float most = -INFINITY;
#pragma unroll
        for (int i = 0; i < C; ++i) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) most = fmaxf(most, l[i][j]);
        }
        most = lanes_max<L>(most);
        const float sum = sigmoid ? 1.f : exp_sum<float, C, L>(l, most);
        off = sigmoid ? 0x1p-20f : 0x1p-16f / sum;
#pragma unroll
        for (int i = 0; i < C; ++i) {
            const int e0 = (i * L + lane) * kPer;
            float b[kPer];
            if (whole && a.bias && e0 < a.experts && (reinterpret_cast<uintptr_t>(a.bias) & 15) == 0) {
#pragma unroll
                for (int j = 0; j < kPer; j += 4) {
                    const float4 v = *reinterpret_cast<const float4*>(a.bias + e0 + j);
                    b[j] = v.x, b[j + 1] = v.y, b[j + 2] = v.z, b[j + 3] = v.w;
                }
            } else {
#pragma unroll
                for (int j = 0; j < kPer; ++j) b[j] = a.bias && e0 + j < a.experts ? fetch(a.bias + e0 + j) : 0.f;
            }
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                c[i][j] = l[i][j] > -INFINITY ? rough_score(l[i][j], sigmoid, most, sum) + b[j] : kLow;
                if (!(c[i][j] > kLow)) c[i][j] = kLow;  // a bias of NaN
            }
        }
        if (a.groups > 1 && !in_lanes) {
            // a group's score: the sum of its two best (its only one's, where it has one)
            float* by = static_cast<float*>(sh.c);
            float* best = by + a.experts;
            const int size = a.experts / a.groups;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < C; ++i) {
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    const int e = (i * L + lane) * kPer + j;
                    if (e < a.experts) by[e] = c[i][j];
                }
            }
            __syncwarp();
            // with fewer groups than lanes several lanes read a group, neighbours side by side
            const int share = a.groups >= L ? 1 : 1 << (31 - __clz(L / a.groups));
            float size_of = 0;  // of the numbers that are added, which may cancel
            for (int g0 = 0; g0 < a.groups; g0 += L / share) {
                const int g = g0 + lane / share;
                float first = kLow, second = kLow;
                if (g < a.groups) {
                    for (int e = lane & (share - 1); e < size; e += share) {
                        const float v = by[g * size + e], low = min(v, first);
                        first = max(v, first);
                        second = max(second, low);
                    }
                }
                for (int o = 1; o < share; o <<= 1) {
                    const float v = __shfl_xor_sync(FULL_MASK, first, o), w = __shfl_xor_sync(FULL_MASK, second, o);
                    second = max(max(second, w), min(first, v));
                    first = max(first, v);
                }
                if (g < a.groups && (lane & (share - 1)) == 0) best[g] = group_score(first, second);
                if (first > kLow) size_of = max(size_of, fabsf(first) + (second > kLow ? fabsf(second) : 0.f));
            }
            __syncwarp();
            float least_kept = INFINITY, best_left = kLow;
            uint32_t kept_mask = 0;  // of this lane's groups: 1,024 groups on 32 lanes are 32
            for (int g = lane, q = 0; g < a.groups; g += L, ++q) {
                const float mine = best[g];
                int better = 0;
                for (int o = 0; o < a.groups; ++o) {
                    const float other = best[o];
                    better += other > mine || (other == mine && o < g);
                }
                const bool keep = better < a.top_groups && mine > kLow;
                if (keep) least_kept = min(least_kept, mine);
                else best_left = max(best_left, mine);
                if (keep) kept_mask |= 1u << q;
            }
            least_kept = -lanes_max<L>(-least_kept);
            best_left = lanes_max<L>(best_left);
            const float largest = lanes_max<L>(size_of);
            near = best_left > kLow && !(least_kept - best_left > 4 * off + 0x1p-18f * largest);
            __syncwarp();
            for (int g = lane, q = 0; g < a.groups; g += L, ++q) best[g] = kept_mask >> q & 1 ? 1.f : 0.f;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < C; ++i) {
                // the group of each expert, by counting on from the first one's
                int e = (i * L + lane) * kPer, g = e / size, in = e - g * size;
#pragma unroll
                for (int j = 0; j < kPer; ++j, ++e) {
                    if (e < a.experts && best[g] == 0.f) c[i][j] = kLow;
                    if (++in == size) {
                        in = 0;
                        ++g;
                    }
                }
            }
        }
    }
    const int rounds = BY_LOGIT ? a.top_k : a.top_k + 1;  // one more than asked for shows the gap to the first that is left out
    float before = 0;
    int before_e = 0;
    auto logit_at = [&](int e) { return fminf(elem<T>::to_f32(fetch(row + e)), 3.402823466e38f); };
    auto bias_at = [&](int e) { return a.bias ? fetch(a.bias + e) : 0.f; };
    // equal logits and biases are a tie in any arithmetic
    auto tied = [&](int e0, int e1) { return logit_at(e0) == logit_at(e1) && bias_at(e0) == bias_at(e1); };
    auto as_one = [&](float top) { return before - top <= 2 * off + 0x1p-19f * (fabsf(before) + fabsf(top)); };  // for all that fp32 shows
    auto too_near = [&](float top, int e) { return as_one(top) && !tied(before_e, e); };
    if constexpr (C == 1 && BY_LOGIT) {
        uint64_t v[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) v[j] = rank_of(c[0][j], lane * kPer + j);
        sort8(v);
        for (int r = 0; r < a.top_k; ++r) {
            int e;
            const uint32_t most = take_best<L>(v, lane, e);
            if (lane == 0) {
                sh.expert[r] = most ? e : -1;
                sh.logit[r] = value_of(most);
            }
        }
    } else if constexpr (C == 1) {
        uint32_t v[kPer];
#pragma unroll
        for (int j = 0; j < kPer; ++j) v[j] = rough_rank(c[0][j], j);
        sort8(v);
        if (a.groups > 1 && in_lanes) {
            // a group's score: the sum of its two best (its only one's, where it has one)
            float first = value_of(v[0] & ~7u), second = value_of(v[1] & ~7u);
            for (int o = 1; o < 1 << a.lanes_log2; o <<= 1) {
                const float x = __shfl_xor_sync(FULL_MASK, first, o), y = __shfl_xor_sync(FULL_MASK, second, o);
                second = max(max(second, y), min(first, x));
                first = max(first, x);
            }
            const float best = group_score(first, second);
            const float size_of = best > kLow ? fabsf(first) + (second > kLow ? fabsf(second) : 0.f) : 0.f;  // the numbers may cancel
            const int mine = lane >> a.lanes_log2;
            int better = 0;
#pragma unroll 4
            for (int g = 0; g < a.groups; ++g) {
                const float other = __shfl_sync(FULL_MASK, best, g << a.lanes_log2, L);
                better += other > best || (other == best && g < mine);
            }
            const bool there = lane * kPer < a.experts && best > kLow, keep = there && better < a.top_groups;
            const float least_kept = -lanes_max<L>(keep ? -best : kLow), best_left = lanes_max<L>(there && !keep ? best : kLow);
            const float largest = lanes_max<L>(size_of);
            near = best_left > kLow && !(least_kept - best_left > 4 * off + 0x1p-18f * largest);
            if (!keep) {
#pragma unroll
                for (int j = 0; j < kPer; ++j) v[j] = 0u;
            }
        }
        for (int r = 0; r < rounds; ++r) {
            int e;
            const uint32_t most = take_rough_best<L>(v, lane, e);
            if (lane == 0) {
                sh.expert[r] = most ? e : -1;
                sh.logit[r] = __uint_as_float(most);
            }
        }
        __syncwarp();
        for (int r = lane; r < a.top_k; r += L) {
            const int e = sh.expert[r + 1];
            if (e < 0) break;
            before = value_of(__float_as_uint(sh.logit[r]));
            before_e = sh.expert[r];
            near |= too_near(value_of(__float_as_uint(sh.logit[r + 1])), e);
        }
        // A tie between the last that is chosen and the first that is left out says nothing of what lies behind it, where a larger
        // score may hide: all that is left has to be of the same tie, or clearly less.
        const int next = sh.expert[a.top_k];
        before = value_of(__float_as_uint(sh.logit[a.top_k - 1]));
        before_e = sh.expert[a.top_k - 1];
        if (next >= 0 && as_one(value_of(__float_as_uint(sh.logit[a.top_k]))) && tied(before_e, next)) {
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if (v[j]) near |= too_near(value_of(v[j] & ~7u), lane * kPer + 7 - (int)(v[j] & 7u));
        }
    } else {
        static_assert(L == 32, "several chunks to a lane, a warp to a row");
        bool at_border = false;  // the last that is chosen and the first that is left out are a tie
        for (int r = 0; r < rounds; ++r) {
            float top = kLow;
            int e_top = kNone;
            float l_top = 0.f;
#pragma unroll
            for (int i = 0; i < C; ++i) {
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    if (c[i][j] > top) {
                        top = c[i][j];
                        e_top = (i * L + lane) * kPer + j;
                        l_top = l[i][j];
                    }
            }
            best_of_warp(top, e_top, l_top);
            const bool found = e_top != kNone;
            if (!BY_LOGIT && found) {
                if (r > 0) near |= too_near(top, e_top);
                at_border = r == a.top_k && as_one(top) && tied(before_e, e_top);
            }
            if (!at_border) {
                before = top;
                before_e = found ? e_top : 0;
            }
            if (r < a.top_k && lane == 0) {
                sh.expert[r] = found ? e_top : -1;
                if (BY_LOGIT) sh.logit[r] = l_top;
            }
            if (found && e_top / kPer % L == lane) {
#pragma unroll
                for (int i = 0; i < C; ++i) {
#pragma unroll
                    for (int j = 0; j < kPer; ++j)
                        if ((i * L + lane) * kPer + j == e_top) c[i][j] = kLow;
                }
            }
        }
        if (at_border) {  // a tie there: as above
#pragma unroll
            for (int i = 0; i < C; ++i) {
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    if (c[i][j] > kLow) near |= too_near(c[i][j], (i * L + lane) * kPer + j);
            }
        }
    }
    if (!BY_LOGIT) {
        __syncwarp();
        for (int r = lane; r < a.top_k; r += L) sh.logit[r] = sh.expert[r] >= 0 ? logit_at(sh.expert[r]) : 0.f;
    }
    return near;
}

// 16-bit logits by themselves: expert and logit in one word.
template <typename T, int L>
__device__ __forceinline__ void choose16(const RouteArgs& a, const T* row, int lane, bool whole, const RouteShared& sh)
{
    uint32_t v[kPer];
    const int e0 = lane * kPer;
    if (whole && e0 < a.experts) {
        const Vec<T, kPer> raw = *reinterpret_cast<const Vec<T, kPer>*>(row + e0);
#pragma unroll
        for (int j = 0; j < kPer; ++j) v[j] = rank16(raw.e[j], e0 + j);
    } else {
#pragma unroll
        for (int j = 0; j < kPer; ++j) v[j] = e0 + j < a.experts ? rank16(fetch(row + e0 + j), e0 + j) : 0u;
    }
    sort8(v);
    for (int r = 0; r < a.top_k; ++r) {
        int e;
        const uint32_t most = take_best<L>(v, lane, e);
        if (lane == 0) {
            sh.expert[r] = most ? e : -1;
            sh.logit[r] = logit16<T>(most);
        }
    }
}

// The same choice in 64 bits, for the rows that need it.  Only the scores and the groups' sums are computed in
// floating point, as it is slow (2 a cycle on an SM): comparisons are of words that are ordered as the scores are, 0 for
// what is not available.  One such row is alone at the end of many a call: with comparisons of doubles it took 17 us.
__device__ __forceinline__ uint64_t order_of(double v)
{
    const uint64_t b = (uint64_t)__double_as_longlong(v + 0.0);  // one zero
    return v > -INFINITY ? b ^ (b >> 63 ? ~0ull : 1ull << 63) : 0ull;
}
__device__ __forceinline__ double value_of(uint64_t w) { return __longlong_as_double((long long)(w >> 63 ? w ^ (1ull << 63) : ~w)); }

template <typename T, int C, int L>
__device__ __noinline__ void choose_exactly(const RouteArgs& a, const T* row, int lane, bool whole, const RouteShared& sh)
{
    uint64_t w[C][kPer];
    {
        float l[C][kPer];
        load_logits<T, C, L>(row, a.experts, lane, whole, l);
        const bool sigmoid = a.score == SPC_SCORE_SIGMOID;
        float most = -INFINITY;
#pragma unroll
        for (int i = 0; i < C; ++i) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) most = fmaxf(most, l[i][j]);
        }
        most = lanes_max<L>(most);
        const double sum = sigmoid ? 1.0 : exp_sum<double, C, L>(l, most);
#pragma unroll
        for (int i = 0; i < C; ++i) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int e = (i * L + lane) * kPer + j;
                w[i][j] = l[i][j] > -INFINITY ? order_of(score_of<double>(l[i][j], sigmoid, most, sum) + (a.bias ? (double)fetch(a.bias + e) : 0.0)) : 0ull;
            }
        }
    }
    if (a.groups > 1) {
        uint64_t* by = static_cast<uint64_t*>(sh.c);
        uint64_t* best = by + a.experts;
        const int size = a.experts / a.groups;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < C; ++i) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int e = (i * L + lane) * kPer + j;
                if (e < a.experts) by[e] = w[i][j];
            }
        }
        __syncwarp();
        const int share = a.groups >= L ? 1 : 1 << (31 - __clz(L / a.groups));
        for (int g0 = 0; g0 < a.groups; g0 += L / share) {
            const int g = g0 + lane / share;
            uint64_t first = 0, second = 0;
            if (g < a.groups) {
                for (int e = lane & (share - 1); e < size; e += share) {
                    const uint64_t v = by[g * size + e], low = min(v, first);
                    first = max(v, first);
                    second = max(second, low);
                }
            }
            for (int o = 1; o < share; o <<= 1) {
                const uint64_t x = __shfl_xor_sync(FULL_MASK, first, o), y = __shfl_xor_sync(FULL_MASK, second, o);
                second = max(max(second, y), min(first, x));
                first = max(first, x);
            }
            if (g < a.groups && (lane & (share - 1)) == 0) best[g] = second ? order_of(value_of(first) + value_of(second)) : first;
        }
        __syncwarp();
        uint32_t kept = 0;  // of this lane's groups: 1,024 groups on 32 lanes are 32
        for (int g = lane, q = 0; g < a.groups; g += L, ++q) {
            const uint64_t mine = best[g];
            int better = 0;
            for (int o = 0; o < a.groups; ++o) {
                const uint64_t other = best[o];
                better += other > mine || (other == mine && o < g);
            }
            if (better < a.top_groups && mine) kept |= 1u << q;
        }
        __syncwarp();
        for (int g = lane, q = 0; g < a.groups; g += L, ++q) best[g] = kept >> q & 1;
        __syncwarp();
#pragma unroll
        for (int i = 0; i < C; ++i) {
            int e = (i * L + lane) * kPer, g = e / size, in = e - g * size;
#pragma unroll
            for (int j = 0; j < kPer; ++j, ++e) {
                if (e < a.experts && !best[g]) w[i][j] = 0;
                if (++in == size) {
                    in = 0;
                    ++g;
                }
            }
        }
    }
    for (int r = 0; r < a.top_k; ++r) {
        uint64_t top = 0;
        int e = kNone;
#pragma unroll
        for (int i = 0; i < C; ++i) {
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if (w[i][j] > top) {
                    top = w[i][j];
                    e = (i * L + lane) * kPer + j;
                }
        }
        // the largest word, high half first, then the lowest expert that has it
        const uint32_t high = lanes_most<L>((uint32_t)(top >> 32));
        bool mine = top && (uint32_t)(top >> 32) == high;
        const uint32_t low = lanes_most<L>(mine ? (uint32_t)top : 0u);
        mine = mine && (uint32_t)top == low;
        e = (int)~lanes_most<L>(~(uint32_t)(mine ? e : kNone));
        if (lane == 0) {
            sh.expert[r] = e != kNone ? e : -1;
            sh.logit[r] = e != kNone ? fminf(elem<T>::to_f32(fetch(row + e)), 3.402823466e38f) : 0.f;
        }
#pragma unroll
        for (int i = 0; i < C; ++i) {
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if ((i * L + lane) * kPer + j == e) w[i][j] = 0;
        }
    }
}

// An expert's weight from its logit: its score, or its share of the chosen ones' scores.
struct Weights {
    float most, total;
    bool sigmoid;
    __device__ __forceinline__ float of(float l) const { return score_of<float>(l, sigmoid, most, 1.f) / total; }
};

// most and sum: of the whole row (softmax without renorm).  Lanes take the chosen experts in turn.
template <int L>
__device__ __forceinline__ Weights weights_of(const RouteShared& sh, int k, bool sigmoid, bool renorm, float most, float sum, int lane)
{
    Weights w{most, sum, sigmoid};
    if (!renorm) return w;
    w.most = -INFINITY;
    for (int r = lane; r < k; r += L)
        if (sh.expert[r] >= 0) w.most = fmaxf(w.most, sh.logit[r]);
    w.most = lanes_max<L>(w.most);
    auto add_up = [&]() {
        float s = 0.f;
        for (int r = lane; r < k; r += L)
            if (sh.expert[r] >= 0) s += score_of<float>(sh.logit[r], w.sigmoid, w.most, 1.f);
        return lanes_sum<L>(s);
    };
    w.total = add_up();
    if (sigmoid) {
        // scores that fp32 does not hold: sigmoid(l) is exp(l) there, to the last bit
        const bool tiny = w.total < 1e-30f;
        if (__any_sync(FULL_MASK, tiny)) {
            w.sigmoid = !tiny;
            const float total = add_up();
            if (tiny) w.total = total;
        }
    }
    return w;
}

template <typename T, int C, int L>
__global__ void __launch_bounds__(kBlock)
k_route(RouteArgs a, bool whole)
{
    extern __shared__ double room[];
    wait_for_kernel_before();
    const int lane = threadIdx.x & (L - 1), rows = kBlock / L, mine = threadIdx.x / L;
    const int64_t row = (int64_t)blockIdx.x * rows + mine, at = min(row, a.n - 1);
    RouteShared sh;
    const int grouped = a.groups > 1 ? a.experts + a.groups : 0;
    sh.c = room + mine * grouped;
    sh.logit = reinterpret_cast<float*>(room + rows * grouped) + mine * 2 * (a.top_k + 1);
    sh.expert = reinterpret_cast<int32_t*>(sh.logit + a.top_k + 1);
    const T* logits = static_cast<const T*>(a.logits) + at * a.experts;
    const bool sigmoid = a.score == SPC_SCORE_SIGMOID, by_logit = !a.bias && a.groups == 1, all = !sigmoid && !a.renorm;
    float most = -INFINITY, sum = 1.f;
    constexpr bool kWords = sizeof(T) == 2 && C == 1;  // by_logit: expert and logit in one word
    bool chosen = false;
    if constexpr (kWords) {
        if (by_logit) {
            choose16<T, L>(a, logits, lane, whole, sh);
            chosen = true;
        }
    }
    if (!chosen || all) {
        float l[C][kPer];
        load_logits<T, C, L>(logits, a.experts, lane, whole, l);
        if (chosen) {
        } else if (!kWords && by_logit) {
            if constexpr (!kWords) choose<T, true, C, L>(a, logits, l, lane, whole, sh);
        } else if (__any_sync(FULL_MASK, choose<T, false, C, L>(a, logits, l, lane, whole, sh))) {
            __syncwarp();
            choose_exactly<T, C, L>(a, logits, lane, whole, sh);
        }
        if (all) {
#pragma unroll
            for (int c = 0; c < C; ++c) {
#pragma unroll
                for (int j = 0; j < kPer; ++j) most = fmaxf(most, l[c][j]);
            }
            most = lanes_max<L>(most);
            sum = exp_sum<float, C, L>(l, most);
        }
    }
    __syncwarp();
    const Weights w = weights_of<L>(sh, a.top_k, sigmoid, a.renorm, most, sum, lane);
    if (row >= a.n) return;
    for (int r = lane; r < a.top_k; r += L) {
        a.expert[row * a.top_k + r] = sh.expert[r];
        a.gate[row * a.top_k + r] = sh.expert[r] >= 0 ? w.of(sh.logit[r]) * a.scale : 0.f;
    }
}

// With s the scale, G the chosen experts and p the scores:
//   softmax  dl_e = p_e ([e in G] s dg_e - sum_G s dg p),           sigmoid  dl_e = [e in G] s dg_e p_e (1 - p_e)
// and with weights g = p / sum_G p:  dl_e = [e in G] s g_e (dg_e - sum_G g dg), times (1 - p_e) for sigmoid.
template <typename T, int C, int L>
__global__ void __launch_bounds__(kBlock)
k_route_grad(RouteGradArgs a, bool whole)
{
    wait_for_kernel_before();
    extern __shared__ double room[];
    const int lane = threadIdx.x & (L - 1), rows = kBlock / L, mine = threadIdx.x / L;
    const int64_t row = (int64_t)blockIdx.x * rows + mine, at = min(row, a.n - 1);
    const T* logits = static_cast<const T*>(a.logits) + at * a.experts;
    const bool sigmoid = a.score == SPC_SCORE_SIGMOID;
    RouteShared sh;
    sh.logit = reinterpret_cast<float*>(room) + mine * 2 * a.top_k;
    sh.expert = reinterpret_cast<int32_t*>(sh.logit + a.top_k);
    // the chosen experts' logits, -1 where there is none
    for (int r = lane; r < a.top_k; r += L) {
        int e = fetch(a.expert + at * a.top_k + r);
        if (e < -1 || e >= a.experts) set_status(a.status, SPC_ERR_ROW_INDEX);
        float l = e >= 0 && e < a.experts ? elem<T>::to_f32(fetch(logits + e)) : -INFINITY;
        l = l > -INFINITY ? fminf(l, 3.402823466e38f) : -INFINITY;
        sh.logit[r] = l;
        sh.expert[r] = l > -INFINITY ? e : -1;
    }
    float dl[C][kPer];
    float most = -INFINITY, sum = 1.f;
    const bool full = !sigmoid && !a.renorm;
    if (full) {
        load_logits<T, C, L>(logits, a.experts, lane, whole, dl);
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) most = fmaxf(most, dl[c][j]);
        }
        most = lanes_max<L>(most);
        // exponentials stand in for the logits from here on
        float s = 0.f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                dl[c][j] = dl[c][j] > -INFINITY ? expf(dl[c][j] - most) : 0.f;
                s += dl[c][j];
            }
        }
        sum = lanes_sum<L>(s);
    }
    __syncwarp();
    const Weights w = weights_of<L>(sh, a.top_k, sigmoid, a.renorm, most, sum, lane);
    float dot = 0.f;
    for (int r = lane; r < a.top_k; r += L)
        if (sh.expert[r] >= 0) dot += w.of(sh.logit[r]) * fetch(a.dgate + at * a.top_k + r);
    dot = a.renorm || !sigmoid ? lanes_sum<L>(dot) : 0.f;
    const float rest = full && sum > 0.f ? -a.scale * dot / sum : 0.f;  // sum 0: no expert is available
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) dl[c][j] = full ? rest * dl[c][j] : 0.f;
    }
    __syncwarp();
    // what the chosen ones add, in the place of their logits
    for (int r = lane; r < a.top_k; r += L) {
        const float l = sh.logit[r];
        const float g = w.of(l) * (sigmoid ? 1.f / (1.f + expf(l)) : 1.f);
        sh.logit[r] = a.scale * g * (fetch(a.dgate + at * a.top_k + r) - (a.renorm ? dot : 0.f));
    }
    __syncwarp();
    for (int r = 0; r < a.top_k; ++r) {
        const int e = sh.expert[r];
        if (e < 0 || e / kPer % L != lane) continue;
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if ((c * L + lane) * kPer + j == e) dl[c][j] += sh.logit[r];
        }
    }
    if (row >= a.n) return;
    T* out = static_cast<T*>(a.dlogits) + row * a.experts;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e0 = (c * L + lane) * kPer;
        if (whole) {
            if (e0 >= a.experts) continue;
            constexpr int V = 16 / sizeof(T);
#pragma unroll
            for (int q = 0; q < kPer / V; ++q) {
                Vec<T, V> v;
#pragma unroll
                for (int j = 0; j < V; ++j) v.e[j] = elem<T>::from_f32(dl[c][q * V + j]);
                *reinterpret_cast<Vec<T, V>*>(out + e0 + q * V) = v;
            }
        } else {
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if (e0 + j < a.experts) out[e0 + j] = elem<T>::from_f32(dl[c][j]);
        }
    }
}

// Lanes to a row: eight experts each, up to a warp; beyond 256 experts four chunks of eight.  One lane for 8 experts and
// two for 16 take a bf16 call of 498,145 rows 11 and 21 us where four take 47; 2,000 rows are 2.5 us with either (the gradient
// of 2,000 rows of 8 experts 4.3 us with one lane, 3.2 with four; of 498,145 rows 14 and 31).
int lanes_for(int experts)
{
    int L = 1;
    while (L < 32 && L * kPer < experts) L *= 2;
    return L;
}

template <auto KERNEL, typename A>
spc_status start(const A& a, int L, size_t smem, bool whole, cudaStream_t st)
{
    const int64_t blocks = ceil_div(a.n, (int64_t)(kBlock / L));
    if (blocks > INT32_MAX) return SPC_ERR_UNSUPPORTED;
    if (smem > 32 * 1024) {  // 48 KB with the static part need no leave
        const spc_status s = allow_smem<KERNEL>();
        if (s != SPC_OK) return s;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kBlock);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1] = {beside_the_kernel_before()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    SPC_CUDA_TRY(cudaLaunchKernelEx(&cfg, KERNEL, a, whole));
    return SPC_OK;
}

// Of groups that are whole lanes, a power of two of them: that power, else -1.
int lanes_log2_of(int experts, int groups)
{
    int p = 0;
    while (groups * (kPer << p) < experts) ++p;
    return groups * (kPer << p) == experts ? p : -1;
}

template <typename T>
spc_status fwd(RouteArgs a, cudaStream_t st)
{
    a.lanes_log2 = lanes_log2_of(a.experts, a.groups);
    const bool whole = a.experts % kPer == 0 && aligned16(a.logits);
    const int L = lanes_for(a.experts);
    const size_t smem = (size_t)(kBlock / L) * ((a.groups > 1 ? 8 * (size_t)(a.experts + a.groups) : 0) + 8 * (size_t)(a.top_k + 1));
    if (a.experts > 256) return start<k_route<T, 4, 32>>(a, L, smem, whole, st);
    switch (L) {
    case 1: return start<k_route<T, 1, 1>>(a, L, smem, whole, st);
    case 2: return start<k_route<T, 1, 2>>(a, L, smem, whole, st);
    case 4: return start<k_route<T, 1, 4>>(a, L, smem, whole, st);
    case 8: return start<k_route<T, 1, 8>>(a, L, smem, whole, st);
    case 16: return start<k_route<T, 1, 16>>(a, L, smem, whole, st);
    default: return start<k_route<T, 1, 32>>(a, L, smem, whole, st);
    }
}

template <typename T>
spc_status bwd(const RouteGradArgs& a, cudaStream_t st)
{
    const bool whole = a.experts % kPer == 0 && aligned16(a.logits) && aligned16(a.dlogits);
    const int L = lanes_for(a.experts);
    const size_t smem = 8 * (size_t)(kBlock / L) * a.top_k;
    if (a.experts > 256) return start<k_route_grad<T, 4, 32>>(a, L, smem, whole, st);
    switch (L) {
    case 1: return start<k_route_grad<T, 1, 1>>(a, L, smem, whole, st);
    case 2: return start<k_route_grad<T, 1, 2>>(a, L, smem, whole, st);
    case 4: return start<k_route_grad<T, 1, 4>>(a, L, smem, whole, st);
    case 8: return start<k_route_grad<T, 1, 8>>(a, L, smem, whole, st);
    case 16: return start<k_route_grad<T, 1, 16>>(a, L, smem, whole, st);
    default: return start<k_route_grad<T, 1, 32>>(a, L, smem, whole, st);
    }
}

}  // namespace

spc_status route(const RouteArgs& a, spc_dtype dt, cudaStream_t st)
{
    if (a.n == 0) return SPC_OK;
    switch (dt) {
    case SPC_F32: return fwd<float>(a, st);
    case SPC_F16: return fwd<__half>(a, st);
    default: return fwd<__nv_bfloat16>(a, st);
    }
}

spc_status route_grad(const RouteGradArgs& a, spc_dtype dt, cudaStream_t st)
{
    if (a.n == 0) return SPC_OK;
    switch (dt) {
    case SPC_F32: return bwd<float>(a, st);
    case SPC_F16: return bwd<__half>(a, st);
    default: return bwd<__nv_bfloat16>(a, st);
    }
}

}  // namespace spc
