// group_norm.cuh -- group norm with an activation over the rows of each segment,
// and its gradients; one translation unit per element type instantiates it.
//
// Both passes need sums over a segment before they can write a row, so each reads its
// rows twice: a first kernel forms sums, a second applies them, walking its rows
// backwards so that it meets the ones the first kernel read last while they are still in
// L2 (498,145 x 64 bf16: 47 of the forward's 64 MB, 64 of the gradients' 128).  One CTA per SM owns a run of consecutive positions in both.  A thread owns
// V neighbouring channels (16 bytes where the row length allows) of every rt-th row, keeps
// their parameters in registers and works on them in pairs (f32x2 instructions: the loops are
// bound by issue slots before anything else).  The CTAs' sums over a segment
// that several share go to the workspace, and every CTA that needs them
// adds them in the order of the rows; a segment inside one CTA's run is finished there.
//
// Statistics: a thread sums d = x - p and d^2 around its own first value p, so a mean far
// from zero costs no digits; threads, channels and CTAs are merged as (count, mean,
// sum of squares around the mean), M2 = sum M2_i + sum n_i (mean_i - mean)^2.
// Gradients: with dz = dy act'(z), sums of dz and dz (x - mean) per channel give dgamma,
// dbeta and, weighted by gamma, the two means of a group; dx = A dz + B + D (x - mean).
//
// Large inputs take 2.2 times what one reading of their rows would (498,145 x 64 bf16, 4 samples, SILU: forward
// 40 us, gradients 64).  With few rows every instruction is run once and costs
// about 10 cycles whatever it does, so the code around the loops over rows is kept short: sums and
// statistics go through the same code in turn, short runs take one row body (2,000 x 16 fp32: with that
// unrolled forward 9.5 us for 9.1, gradients 10.8 for 9.6; a launch beside the kernel before: 8.8 and 9.2).
#pragma once

#include "kernels.cuh"
#include "layers.cuh"
#include "pairs.cuh"
#include "ptx.cuh"

namespace spc {

namespace {

constexpr int kBlock = 256;      // of the kernels for very long rows
constexpr int kThreads = 512;    // of the others
constexpr uint64_t kDrainNs = 200000000ull;  // bound of the wait for a CTA's own copies
constexpr int kMinRows = 64;     // positions of a CTA, at least

// a / b for 0 <= a < 2^20, 1 <= b: the half keeps the product's rounding off the whole numbers, and the
// division's own code, some 25 instructions, out of kernels that run it once.
__device__ __forceinline__ int quotient(int a, int b) { return (int)(((float)a + 0.5f) * __fdividef(1.f, (float)b)); }

// A per-channel table as pairs.
template <int V, typename F>
__device__ __forceinline__ void gather_pairs(F2 (&f)[kPairs<V>], F value)
{
#pragma unroll
    for (int j = 0; j < kPairs<V>; ++j) f[j] = F2{value(2 * j), 2 * j + 1 < V ? value(2 * j + 1) : 0.f};
}

// ------------------------------------------------------------------- activations
// 1 / (1 + exp(-z)) with the hardware's exp2 and reciprocal: within 2^-19 for the |z| of a
// normalised feature, a small part of the rounding of a 16-bit output.  fp32 rows take it too: 20,000 x 64 come
// out 9.3e-8 from 64 bits by the norm, 5.8e-8 without the activation (with the exact functions
// 498,145 x 64 bf16 takes 73 us forward for 37.5 and 185 for 63 in its gradients, repeated calls).  The special-function unit has a
// quarter of the rate that this needs, so the pair shares one reciprocal, 1 / a = b / (a b);
// exp is held to 2^57 for that, where the sigmoid is 0 to 17 digits.
__device__ __forceinline__ F2 sigmoid(F2 z)
{
    const F2 t = mul(z, both(-1.4426950408889634f));
    F2 e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(fminf(t.x, 57.f)));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(fminf(t.y, 57.f)));
    e = add(e, both(1.f));
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e.x * e.y));
    return mul(both(r), F2{e.y, e.x});
}

// SILU, or max(z, floor): floor 0 for RELU, -infinity for none (a NaN passes).
template <bool SILU>
__device__ __forceinline__ F2 activate(F2 z, float floor)
{
    if (SILU) return mul(z, sigmoid(z));
    return F2{z.x < floor ? floor : z.x, z.y < floor ? floor : z.y};
}

// dy act'(z); least: the smallest z of slope 1 (RELU: the least positive number).
template <bool SILU>
__device__ __forceinline__ F2 through(F2 dy, F2 z, float least)
{
    if (SILU) {
        const F2 s = sigmoid(z);
        const F2 rest = fma(s, both(-1.f), both(1.f));
        return mul(dy, mul(s, fma(z, rest, both(1.f))));
    }
    return F2{z.x < least ? 0.f : z.x != z.x ? z.x : dy.x, z.y < least ? 0.f : z.y != z.y ? z.y : dy.y};
}
__device__ __forceinline__ float floor_of(int act) { return act == SPC_ACT_RELU ? 0.f : -INFINITY; }
__device__ __forceinline__ float least_of(int act) { return act == SPC_ACT_RELU ? __int_as_float(1) : -INFINITY; }

// The same for the kernels that take one element at a time.
__device__ __forceinline__ float activate(float z, int act)
{
    return act == SPC_ACT_SILU ? activate<true>(both(z), 0.f).x : activate<false>(both(z), floor_of(act)).x;
}
__device__ __forceinline__ float slope(float z, int act)
{
    return act == SPC_ACT_SILU ? through<true>(both(1.f), both(z), 0.f).x : through<false>(both(1.f), both(z), least_of(act)).x;
}

__device__ __forceinline__ float block_sum(float v)
{
    __shared__ float s[kBlock / 32];
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(FULL_MASK, v, d);
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < kBlock / 32; ++w) t += s[w];
    __syncthreads();
    return t;
}

// ------------------------------------------------- runs of consecutive positions
// The offsets, in shared memory, inside [0, n]; what is out of range or order is reported.
__device__ __forceinline__ void load_offsets(const NormArgs& a, int32_t* s_seg, bool report)
{
    for (int s = threadIdx.x; s <= a.segments; s += (int)blockDim.x) {
        const int32_t v = fetch(a.seg + s);
        s_seg[s] = v < 0 ? 0 : (v > a.n ? (int32_t)a.n : v);
        if (report && (v < 0 || v > a.n || (s < a.segments && fetch(a.seg + s + 1) < v)))
            set_status(a.status, SPC_ERR_ROW_INDEX);
    }
    __syncthreads();
}

// The last s with seg[s] <= r: the segment of position r, -1 before the first, `segments` from
// the last offset on.
__device__ __forceinline__ int find_segment(const int32_t* s_seg, int segments, int64_t r)
{
    int lo = 0, hi = segments + 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (s_seg[mid] > r) hi = mid;
        else lo = mid + 1;
    }
    return lo - 1;
}

struct Run {
    int s;           // segment, -1: none
    int64_t lo, hi;  // its positions in this CTA's share
    // Whether the share [begin, end) holds all of the segment.
    __device__ __forceinline__ bool whole(const int32_t* s_seg) const { return lo == s_seg[s] && hi >= s_seg[s + 1]; }
    // Where its part goes: a share's first slot if it begins with the share, else its second.
    __device__ __forceinline__ int slot(int64_t begin) const { return 2 * (int)blockIdx.x + (lo > begin ? 1 : 0); }
};

// The run that begins at position r of a share that ends at `end`.
__device__ __forceinline__ Run run_at(const NormArgs& a, const int32_t* s_seg, int64_t r, int64_t end)
{
    Run k;
    k.s = find_segment(s_seg, a.segments, r);
    int64_t to = k.s >= a.segments ? a.n : s_seg[k.s + 1];
    if (k.s >= a.segments) k.s = -1;
    to = to > r ? to : r + 1;  // offsets out of order: still forward
    k.lo = r;
    k.hi = to < end ? to : end;
    return k;
}

// The run that ends before position `end` of a share that begins at `begin`.
__device__ __forceinline__ Run run_before(const NormArgs& a, const int32_t* s_seg, int64_t begin, int64_t end)
{
    Run k;
    k.s = find_segment(s_seg, a.segments, end - 1);
    int64_t from = k.s < 0 ? 0 : s_seg[k.s >= a.segments ? a.segments : k.s];
    if (k.s >= a.segments) k.s = -1;
    from = from < end ? from : end - 1;
    k.hi = end;
    k.lo = from > begin ? from : begin;
    return k;
}

// Segment s over shares of `rows` positions: shares first .. last hold a part of it.
struct Span {
    int64_t lo, hi;
    int first, last;
    __device__ __forceinline__ Span(const int32_t* s_seg, int s, int64_t rows)
    {
        lo = s_seg[s];
        hi = s_seg[s + 1] > lo ? s_seg[s + 1] : lo;
        first = (int)((uint32_t)lo / (uint32_t)rows);
        last = hi > lo ? (int)((uint32_t)(hi - 1) / (uint32_t)rows) : first;
    }
    __device__ __forceinline__ int64_t count(int c, int64_t rows) const
    {
        const int64_t b = c * rows > lo ? c * rows : lo, e = (c + 1) * rows < hi ? (c + 1) * rows : hi;
        return e - b;
    }
    // a share's part stands in its first slot if it begins with the share, else in its second
    __device__ __forceinline__ int slot(int c, int64_t rows) const { return 2 * c + (c == first && lo > c * rows ? 1 : 0); }
};

// ------------------------------------------------------------ rows in flight
// Barrier of the threads that work on rows (the loading warp has its own way).
__device__ __forceinline__ void sync_workers() { ptx::bar_sync_named(1, kThreads); }

// Rows in order (DENSE): a run is one contiguous piece of each of the N tensors.  A warp of its
// own brings it in stages of kRowsOf rows a thread by bulk copies, kStages ahead of their use and on
// into the next run, so neither addresses nor latencies cost the others anything.
// Rows through a list, or not a multiple of 16 bytes: each thread loads its own.
template <typename T, int V, int N, bool DENSE>
struct Feed {
    // rows of a thread per stage: two stages of 64 KB (498,145 x 64 bf16 forward 41.9 us; five of
    // 32 KB 43.3, five of 16 KB 46.4)
    static constexpr int kRowsOf = DENSE ? 8 / N : 4;
    static constexpr int kStage = kRowsOf * N * kThreads * (int)sizeof(T) * V;  // bytes
    static constexpr int kStages = 2;
    static constexpr size_t kSmem = DENSE ? (size_t)kStages * kStage + 2 * kStages * sizeof(uint64_t) : 0;
    static constexpr int kBlockThreads = DENSE ? kThreads + 32 : kThreads;

    const NormArgs& a;
    const T* base[N];        // this thread's vector of row 0
    uint8_t* stages;
    uint64_t* full;
    uint64_t* empty;
    uint64_t wait_ns;
    uint32_t it;             // stages used so far
    int vpr, rt, tr;
    int step;                // 1 forwards, -1 backwards
    int64_t lo, hi;          // the run
    int32_t next[DENSE ? 1 : kRowsOf];
    bool ok;

    __device__ __forceinline__ Feed(const NormArgs& args, void* smem, uint64_t limit, int vpr_, int rt_, int tr_)
        : a(args), stages(static_cast<uint8_t*>(smem)), wait_ns(limit), it(0), vpr(vpr_), rt(rt_), tr(tr_), ok(true)
    {
        full = reinterpret_cast<uint64_t*>(stages + (size_t)kStages * kStage);
        empty = full + kStages;
        if (DENSE && threadIdx.x == 0) {
            for (int s = 0; s < kStages; ++s) {
                ptx::mbar_init(&full[s], 1);
                ptx::mbar_init(&empty[s], kThreads / 32);
            }
            ptx::mbar_init_fence();
        }
    }
    __device__ __forceinline__ int stage_rows() const { return kRowsOf * rt; }
    // The share's first rows on their way into L2 before its runs are known.
    __device__ __forceinline__ void ahead(int64_t begin, int64_t end, const T* const (&tensor)[N])
    {
        if (!DENSE || threadIdx.x != kThreads || begin >= end) return;
        const int64_t rows = stage_rows(), count = end - begin < rows ? end - begin : rows;
        const int64_t r = step > 0 ? begin : end - count;
#pragma unroll
        for (int t = 0; t < N; ++t)
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(tensor[t] + r * a.c),
                         "r"((uint32_t)(count * a.c * (int64_t)sizeof(T)))
                         : "memory");
    }

    // The loading thread: the run's stages in turn.
    __device__ __forceinline__ void load(const Run& k, const T* const (&tensor)[N])
    {
        const int64_t rows = stage_rows();
        const uint32_t row_bytes = (uint32_t)a.c * (uint32_t)sizeof(T);
        for (int64_t done = 0; done < k.hi - k.lo && ok; done += rows, ++it) {
            const int s = it % kStages;
            if (it >= kStages) ok = ptx::mbar_wait(&empty[s], ((it / kStages) - 1) & 1, wait_ns);
            if (!ok) break;
            const int64_t count = k.hi - k.lo - done < rows ? k.hi - k.lo - done : rows;
            const int64_t r = step > 0 ? k.lo + done : k.hi - done - count;
            ptx::mbar_arrive_expect_tx(&full[s], (uint32_t)(N * count) * row_bytes);
#pragma unroll
            for (int t = 0; t < N; ++t)
                asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                                 ptx::smem_u32(stages + (size_t)s * kStage + t * (kStage / N))),
                             "l"(tensor[t] + r * a.c), "r"((uint32_t)count * row_bytes), "r"(ptx::smem_u32(&full[s]))
                             : "memory");
        }
    }
    // ... and at the end whatever it still has in flight.
    __device__ __forceinline__ void drain()
    {
        if (!ok) set_status(a.status, SPC_ERR_TIMEOUT);
        const uint32_t first = it > kStages ? it - kStages : 0;
        for (uint32_t j = first; j < it; ++j) ptx::mbar_wait(&full[j % kStages], (j / kStages) & 1, kDrainNs);
    }

    // The working threads.
    __device__ __forceinline__ void begin(const Run& k)
    {
        lo = k.lo;
        hi = k.hi;
        if constexpr (!DENSE) list_rows(lo + tr);
    }
    // The list's entries for this thread's next rows, from position p on: read a turn ahead.
    __device__ __forceinline__ void list_rows(int64_t p)
    {
#pragma unroll
        for (int q = 0; q < kRowsOf; ++q, p += rt) next[q] = p >= hi ? -1 : a.order ? fetch(a.order + p) : (int32_t)p;
    }
    __device__ __forceinline__ void wait_full()
    {
        if (!DENSE || !ok) return;
        const bool came = ptx::mbar_wait(&full[it % kStages], (it / kStages) & 1, wait_ns);
        if (!came) set_status(a.status, SPC_ERR_TIMEOUT);
        ok = came;
    }
    __device__ __forceinline__ const Vec<T, V>* slot(int q, int t) const
    {
        return reinterpret_cast<const Vec<T, V>*>(stages + (size_t)(it % kStages) * kStage + t * (kStage / N)) + q * rt * vpr + (int)threadIdx.x;
    }
    // This thread's first row of a run that goes forwards (0 where its entry is out of range) and
    // the run's first one; nothing is used up.
    __device__ __forceinline__ void first(F2 (&mine)[kPairs<V>], F2 (&lead)[kPairs<V>])
    {
        if constexpr (DENSE) {
            wait_full();
            if (lo + tr < hi) unpack<T, V>(*slot(0, 0), mine);
            unpack<T, V>(*(slot(0, 0) - tr * vpr), lead);
        } else {
            const int64_t r0 = row_at(a.order, lo, a.n, nullptr), r1 = next[0] < a.n ? next[0] : -1;
            if (r0 >= 0) unpack<T, V>(*reinterpret_cast<const Vec<T, V>*>(base[0] + r0 * a.c), lead);
            if (r1 >= 0) unpack<T, V>(*reinterpret_cast<const Vec<T, V>*>(base[0] + r1 * a.c), mine);
        }
    }
    // body(values, row) for each of this thread's rows; every working thread calls it, `works`
    // says whether it has rows at all.
    template <typename B>
    __device__ __forceinline__ void run(bool works, B body)
    {
        if constexpr (DENSE) {
            const int64_t rows = stage_rows();
            for (int64_t done = 0; done < hi - lo; done += rows, ++it) {
                wait_full();
                const int64_t left = hi - lo - done;
                const int count = (int)(left < rows ? left : rows);
                const int64_t r = (step > 0 ? lo + done : hi - done - count) + tr;
                if (ok && works) {
                    if (count == rows) {
                        F2 f[kRowsOf][N][kPairs<V>];
#pragma unroll
                        for (int q = 0; q < kRowsOf; ++q)
#pragma unroll
                            for (int t = 0; t < N; ++t) unpack<T, V>(*slot(q, t), f[q][t]);
#pragma unroll
                        for (int q = 0; q < kRowsOf; ++q) body(f[q], r + q * rt);
                    } else {
                        for (int q = 0; q * rt + tr < count; ++q) {
                            F2 f[N][kPairs<V>];
#pragma unroll
                            for (int t = 0; t < N; ++t) unpack<T, V>(*slot(q, t), f[t]);
                            body(f, r + q * rt);
                        }
                    }
                }
                __syncwarp();
                if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(&empty[it % kStages]);
            }
        } else if (works) {
            for (int64_t p = lo + tr; p < hi; p += kRowsOf * rt) {
                int32_t row[kRowsOf];
#pragma unroll
                for (int q = 0; q < kRowsOf; ++q) {
                    row[q] = next[q];
                    if (p + q * rt < hi && (row[q] < 0 || row[q] >= a.n)) {
                        set_status(a.status, SPC_ERR_ROW_INDEX);
                        row[q] = -1;
                    }
                }
                Vec<T, V> v[kRowsOf][N];
#pragma unroll
                for (int q = 0; q < kRowsOf; ++q)
                    if (row[q] >= 0)
#pragma unroll
                        for (int t = 0; t < N; ++t) v[q][t] = *reinterpret_cast<const Vec<T, V>*>(base[t] + (int64_t)row[q] * a.c);
                list_rows(p + kRowsOf * rt);
                if (p + (kRowsOf - 1) * rt >= hi) {
                    // the last rows, or a short run's: one after the other through the same code
#pragma unroll 1
                    for (int q = 0; q < kRowsOf; ++q) {
                        if (row[0] >= 0) {
                            F2 f[N][kPairs<V>];
#pragma unroll
                            for (int t = 0; t < N; ++t) unpack<T, V>(v[0][t], f[t]);
                            body(f, row[0]);
                        }
#pragma unroll
                        for (int i = 0; i + 1 < kRowsOf; ++i) {
                            row[i] = row[i + 1];
#pragma unroll
                            for (int t = 0; t < N; ++t) v[i][t] = v[i + 1][t];
                        }
                        row[kRowsOf - 1] = -1;
                    }
                    break;
                }
#pragma unroll
                for (int q = 0; q < kRowsOf; ++q)
                    if (row[q] >= 0) {
                        F2 f[N][kPairs<V>];
#pragma unroll
                        for (int t = 0; t < N; ++t) unpack<T, V>(v[q][t], f[t]);
                        body(f, row[q]);
                    }
            }
        }
    }
};

// ------------------------------------------------------------------ column sums
// A sum that carries the rounding errors of its additions along (Knuth's two-sum).
struct Exact {
    float s = 0.f, e = 0.f;
    __device__ __forceinline__ void add(float v)
    {
        const float t = s + v, z = t - s;
        e += (s - (t - z)) + (v - z);
        s = t;
    }
    __device__ __forceinline__ float value() const { return e == e ? s + e : s; }  // s itself once it is not finite
};

// Values from, from + stride, ... (count of them), four loads at a time.  The additions are
// exact to twice the digits, so that a mean hardly depends on how rows were dealt out to threads.
__device__ __forceinline__ float stretch(const float* from, int stride, int count)
{
    Exact all;
#pragma unroll 1
    for (int r = 0; r < count; r += 4, from += 4 * stride) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = r + i < count ? from[i * stride] : 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) all.add(v[i]);
    }
    return all.value();
}

// Sums over the rt row threads of N values per channel, into s_out [N][c].  The threads
// lay their values out by row and channel; each then adds a stretch of one channel's rows, and
// the stretches are added in turn: two short steps whatever c is, with their indexes worked
// out once.  s: kSums<V, N> floats.
template <int V, int N> constexpr int kSums = N * kThreads * (V + 1);
struct Columns {
    int c, rt, parts, len, part, ch;
    __device__ __forceinline__ Columns(int c_, int rt_) : c(c_), rt(rt_)
    {
        parts = c < kThreads ? quotient(kThreads, c) : 1;
        len = quotient(rt + parts - 1, parts);
        part = quotient((int)threadIdx.x, c);
        ch = (int)threadIdx.x - part * c;
    }
};
template <int V, int N>
__device__ __forceinline__ void column_sums(const Columns& k, const F2 (&v)[N][kPairs<V>], float* s, float* s_out, int tr, int tv)
{
    constexpr int P = V >= 4 ? 4 : V;
    using W = Vec<float, P>;
    const int plane = k.rt * k.c;
    if (tr < k.rt)
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
            for (int h = 0; h < V / P; ++h) {
                W u;
#pragma unroll
                for (int j = 0; j < P; ++j) {
                    const F2 f = v[n][(h * P + j) / 2];
                    u.e[j] = (h * P + j) % 2 ? f.y : f.x;
                }
                *reinterpret_cast<W*>(s + n * plane + tr * k.c + tv * V + h * P) = u;
            }
    sync_workers();
    if (k.parts == 1) {
#pragma unroll 1
        for (int ch = threadIdx.x; ch < k.c; ch += kThreads)
#pragma unroll 1
            for (int n = 0; n < N; ++n) s_out[n * k.c + ch] = stretch(s + n * plane + ch, k.c, k.rt);
        sync_workers();
        return;
    }
    // first [N][rt][c] to [N][parts][c], a part to each thread, then that to [N][c]
    const int r0 = k.part * k.len, left = k.rt - r0;
    const float* from = s + r0 * k.c + k.ch;
    float* to = s + N * plane + k.part * k.c + k.ch;
    int count = left < k.len ? left : k.len, step = plane, step_to = k.parts * k.c;
    bool mine = k.part < k.parts;
#pragma unroll 1
    for (int turn = 0; turn < 2; ++turn) {
        if (mine)
#pragma unroll 1
            for (int n = 0; n < N; ++n) to[n * step_to] = stretch(from + n * step, k.c, count);
        sync_workers();
        from = s + N * plane + (int)threadIdx.x;
        to = s_out + (int)threadIdx.x;
        count = k.parts;
        step = step_to;
        step_to = k.c;
        mine = (int)threadIdx.x < k.c;
    }
}

// Who sums up a group: a thread for itself, or a warp's lanes together where groups are wide.
constexpr int kNarrow = 16;
__device__ __forceinline__ float warp_sum(float v);
__device__ __forceinline__ float group_sum(float v, int per) { return per <= kNarrow ? v : warp_sum(v); }
struct GroupLoop {
    int g, step, lane, lanes;
    __device__ __forceinline__ explicit GroupLoop(int per)
    {
        const bool narrow = per <= kNarrow;
        g = narrow ? threadIdx.x : threadIdx.x >> 5;
        step = narrow ? kThreads : kThreads / 32;
        lane = narrow ? 0 : threadIdx.x & 31;
        lanes = narrow ? 1 : 32;
    }
};

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(FULL_MASK, v, d);
    return v;
}

// What the two kernels of a pass hand over.
struct Ws {
    float2* part;   // [2 shares][groups] sums over a shared segment's parts
    float2* coef;   // [segments][groups] sums over the segments inside one share
    float* total;   // [shares][2][c] sums over a share
};

// Thread tid's place: vector tv of every rt-th row from row tr on.
template <int V>
struct Place {
    int vpr, rt, tr, tv, per, warp, lane;
    int group[V];        // of each of its channels
    int64_t begin, end;  // positions of this CTA
    __device__ __forceinline__ Place(const NormArgs& a, int64_t rows)
    {
        const int tid = threadIdx.x;
        vpr = a.c / V;
        rt = quotient(kThreads, vpr);
        tr = quotient(tid, vpr);
        tv = tid - tr * vpr;
        per = quotient(a.c, a.groups);
        warp = tid >> 5;
        lane = tid & 31;
        int g = quotient(tv * V, per), r = tv * V - g * per;
#pragma unroll
        for (int j = 0; j < V; ++j) {
            group[j] = g;
            if (++r == per) {
                r = 0;
                ++g;
            }
        }
        begin = blockIdx.x * rows;
        end = begin + rows < a.n ? begin + rows : a.n;
    }
};

// ------------------------------------------------------------------- statistics
// part[slot][g] = (mean, M2) of a shared segment's part; whole segments end in mean, rstd.
template <typename T, int V, bool DENSE>
__global__ void __launch_bounds__(Feed<T, V, 1, DENSE>::kBlockThreads, 1) k_norm_stats(NormArgs a, int64_t rows, Ws w, uint64_t wait_ns)
{
    extern __shared__ __align__(16) uint8_t s_raw[];
    using S = Feed<T, V, 1, DENSE>;
    float* s_sum = reinterpret_cast<float*>(s_raw + S::kSmem);
    float* s_mean = s_sum + kSums<V, 1>;  // channel means, and sums of squares around them
    float* s_m2 = s_mean + a.c;
    int32_t* s_seg = reinterpret_cast<int32_t*>(s_m2 + a.c);
    const Place<V> at(a, rows);
    const bool works = at.tr < at.rt;
    S in(a, s_raw, wait_ns, at.vpr, at.rt, at.tr);
    const T* const tensor[1] = {static_cast<const T*>(a.x)};
    in.step = 1;
#pragma unroll
    for (int t = 0; t < 1; ++t) in.base[t] = tensor[t] + at.tv * V;
    wait_for_kernel_before();
    in.ahead(at.begin, at.end, tensor);
    load_offsets(a, s_seg, blockIdx.x == 0);
    if (DENSE && at.warp == kThreads / 32) {
        if (at.lane == 0) {
            for (int64_t r0 = at.begin; r0 < at.end;) {
                const Run k = run_at(a, s_seg, r0, at.end);
                r0 = k.hi;
                if (k.s >= 0) in.load(k, tensor);
            }
            in.drain();
        }
        return;
    }
    const Columns columns(a.c, at.rt);
    // empty segments are finished here, a block each in turn
    for (int s = blockIdx.x; s < a.segments; s += gridDim.x)
        if (s_seg[s] >= s_seg[s + 1])
            for (int g = threadIdx.x; g < a.groups; g += kThreads) {
                a.mean[(int64_t)s * a.groups + g] = 0.f;
                a.rstd[(int64_t)s * a.groups + g] = 1.f / sqrtf(a.eps);
            }
    for (int64_t r0 = at.begin; r0 < at.end;) {
        const Run k = run_at(a, s_seg, r0, at.end);
        r0 = k.hi;
        if (k.s < 0) continue;
        F2 pivot[1][kPairs<V>], s1[kPairs<V>], s2[kPairs<V>], lead[kPairs<V>];
#pragma unroll
        for (int j = 0; j < kPairs<V>; ++j) pivot[0][j] = s1[j] = s2[j] = lead[j] = both(0.f);
        int count = 0;
        in.begin(k);
        // the run's first row is what the threads' sums are brought together around
        if (works) in.first(pivot[0], lead);
        F2 minus[kPairs<V>];
#pragma unroll
        for (int j = 0; j < kPairs<V>; ++j) minus[j] = F2{-pivot[0][j].x, -pivot[0][j].y};
        in.run(works, [&](const F2 (&f)[1][kPairs<V>], int64_t) {
            ++count;
#pragma unroll
            for (int j = 0; j < kPairs<V>; ++j) {
                const F2 d = add(f[0][j], minus[j]);
                s1[j] = add(s1[j], d);
                s2[j] = fma(d, d, s2[j]);
            }
        });
        // channel means around the run's first row, then squares around the channel means
        const float n = (float)(int)(k.hi - k.lo), mine = (float)count, inverse = 1.f / mine;
#pragma unroll 1
        for (int turn = 0; turn < 2; ++turn) {
            F2 v[1][kPairs<V>];
            if (turn == 0) {
#pragma unroll
                for (int j = 0; j < kPairs<V>; ++j)
                    v[0][j] = F2{fmaf(mine, pivot[0][j].x - lead[j].x, s1[j].x), fmaf(mine, pivot[0][j].y - lead[j].y, s1[j].y)};
            } else {
                auto square = [&](float p, float a1, float a2, int ch) -> float {
                    const float m = a1 * inverse, d = (p - s_mean[ch]) + m, m2 = fmaf(-m, a1, a2);
                    return works && count ? (m2 < 0.f ? 0.f : m2) + mine * d * d : 0.f;
                };
#pragma unroll
                for (int j = 0; j < kPairs<V>; ++j) {
                    v[0][j].x = square(pivot[0][j].x, s1[j].x, s2[j].x, at.tv * V + 2 * j);
                    v[0][j].y = 2 * j + 1 < V ? square(pivot[0][j].y, s1[j].y, s2[j].y, at.tv * V + 2 * j + 1) : 0.f;
                }
            }
            column_sums<V, 1>(columns, v, s_sum, turn == 0 ? s_mean : s_m2, at.tr, at.tv);
            if (turn == 0) {
                if (at.tr == 0)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float b = j % 2 ? lead[j / 2].y : lead[j / 2].x;
                        s_mean[at.tv * V + j] = b + s_mean[at.tv * V + j] / n;
                    }
                sync_workers();
            }
        }
        // channels to groups
        const bool whole = k.whole(s_seg);
        const int slot = k.slot(at.begin);
        const GroupLoop way(at.per);
        for (int g = way.g; g < a.groups; g += way.step) {
            const int ch0 = g * at.per;
            const float lead0 = s_mean[ch0];
            float m = 0.f;
            for (int j = way.lane; j < at.per; j += way.lanes) m += s_mean[ch0 + j] - lead0;
            const float mean = lead0 + group_sum(m, at.per) / (float)at.per;
            float q = 0.f;
            for (int j = way.lane; j < at.per; j += way.lanes) {
                const float d = s_mean[ch0 + j] - mean;
                q += s_m2[ch0 + j] + n * d * d;
            }
            q = group_sum(q, at.per);
            if (way.lane == 0) {
                if (whole) {
                    a.mean[(int64_t)k.s * a.groups + g] = mean;
                    a.rstd[(int64_t)k.s * a.groups + g] = 1.f / sqrtf(q / (n * (float)at.per) + a.eps);
                } else {
                    w.part[(int64_t)slot * a.groups + g] = make_float2(mean, q);
                }
            }
        }
        sync_workers();
    }
}

// Sixteen lanes join the parts of a group; sums over them.
constexpr int kJoin = 16;
__device__ __forceinline__ float join_sum(float v)
{
#pragma unroll
    for (int d = kJoin / 2; d; d >>= 1) v += __shfl_xor_sync(FULL_MASK, v, d);
    return v;
}

// The parts of a shared segment, as their shares left them.
struct Parts {
    const float2* at;        // part of share `first`, group 0
    int first, last, groups;
    int odd;                 // the first part stands in its share's second slot
    float rows, rows_first, rows_last;
    __device__ __forceinline__ Parts(const Span& span, const float2* part, int64_t rows_, int groups_)
        : first(span.first), last(span.last), groups(groups_)
    {
        const int slot = span.slot(first, rows_);
        odd = slot & 1;
        at = part + (int64_t)slot * groups;
        rows = (float)(int)rows_;
        rows_first = (float)(int)span.count(first, rows_);
        rows_last = (float)(int)span.count(last, rows_);
    }
    // Part of share first + i.
    __device__ __forceinline__ float2 get(int i, int g) const { return at[(2 * i - (i ? odd : 0)) * groups + g]; }
    __device__ __forceinline__ int count() const { return last - first + 1; }
    __device__ __forceinline__ float rows_of(int i) const { return i == 0 ? rows_first : first + i == last ? rows_last : rows; }
    // One of the parts with the most rows; the first and the last may be a single one.
    __device__ __forceinline__ int longest() const { return count() > 2 || rows_last > rows_first ? 1 : 0; }
};

// (mean, rstd) of segment s into s_stat [groups], from the parts where several CTAs
// share it; the CTA that holds its first position also writes them out.  Parts are taken around the first one's
// mean p: M2 = sum (M2_i + n_i (mean_i - p)^2) - n (mean - p)^2.  Their means lie close together as a rule; where
// the difference would cancel more than a sixteenth (a first part of one row far from the others cost the
// rstd of 40,000 rows of 1000 +- 1 2e-3), a second pass takes squares around the joint mean.  (A second pass
// at all times: 498,145 x 64 bf16 38.2 us for 37.4.)
__device__ __forceinline__ void join_stats(const NormArgs& a, const int32_t* s_seg, int s, int64_t rows, const float2* part,
                                           float2* s_stat)
{
    const Span span(s_seg, s, rows);
    const int lane = threadIdx.x % kJoin;
    const float per = (float)(a.c / a.groups);
    sync_workers();
    // all lanes of a warp go round as often: the shuffles are the warp's
    for (int g0 = 0; g0 < a.groups; g0 += kThreads / kJoin) {
        const int g = g0 + (int)threadIdx.x / kJoin, gr = g < a.groups ? g : 0;
        float mean = a.mean[(int64_t)s * a.groups + gr], rstd = a.rstd[(int64_t)s * a.groups + gr];
        if (span.first != span.last) {
            const Parts parts(span, part, rows, a.groups);
            const float base = parts.get(0, gr).x;
            float m = 0.f, q = 0.f;
#pragma unroll 5
            for (int i = lane; i < parts.count(); i += kJoin) {
                const float2 v = parts.get(i, gr);
                const float n = parts.rows_of(i), d = v.x - base;
                m = fmaf(n, d, m);
                q += fmaf(n * per, d * d, v.y);
            }
            const float n = (float)(int)(span.hi - span.lo), shift = join_sum(m) / n;
            mean = base + shift;
            q = join_sum(q);
            const bool near = n * per * shift * shift <= 0.0625f * q;
            q = fmaf(-n * per * shift, shift, q);
            if (!__all_sync(FULL_MASK, near)) {
                // around the mean of one of the longest parts, then around the joint mean
                const float middle = parts.get(parts.longest(), gr).x;
                float m2 = 0.f, q2 = 0.f;
#pragma unroll 1
                for (int i = lane; i < parts.count(); i += kJoin) m2 = fmaf(parts.rows_of(i), parts.get(i, gr).x - middle, m2);
                const float joint = middle + join_sum(m2) / n;
#pragma unroll 1
                for (int i = lane; i < parts.count(); i += kJoin) {
                    const float2 v = parts.get(i, gr);
                    const float d = v.x - joint;
                    q2 += fmaf(parts.rows_of(i) * per, d * d, v.y);
                }
                q2 = join_sum(q2);
                // a group that was near keeps its sums: they do not depend on its neighbours'
                mean = near ? mean : joint;
                q = near ? q : q2;
            }
            rstd = 1.f / sqrtf((q < 0.f ? 0.f : q) / (n * per) + a.eps);
            if (g < a.groups && lane == 0 && (int)blockIdx.x == span.first) {
                a.mean[(int64_t)s * a.groups + g] = mean;
                a.rstd[(int64_t)s * a.groups + g] = rstd;
            }
        }
        if (g < a.groups && lane == 0) s_stat[g] = make_float2(mean, rstd);
    }
    sync_workers();
}

template <typename T, int V, bool DENSE, bool SILU>
__global__ void __launch_bounds__(Feed<T, V, 1, DENSE>::kBlockThreads, 1) k_norm_apply(NormArgs a, int64_t rows, Ws w, uint64_t wait_ns)
{
    extern __shared__ __align__(16) uint8_t s_raw[];
    using S = Feed<T, V, 1, DENSE>;
    float2* s_stat = reinterpret_cast<float2*>(s_raw + S::kSmem);
    int32_t* s_seg = reinterpret_cast<int32_t*>(s_stat + a.groups);
    const Place<V> at(a, rows);
    const bool works = at.tr < at.rt;
    T* y = static_cast<T*>(a.out) + at.tv * V;
    S in(a, s_raw, wait_ns, at.vpr, at.rt, at.tr);
    const T* const tensor[1] = {static_cast<const T*>(a.x)};
    in.step = -1;
#pragma unroll
    for (int t = 0; t < 1; ++t) in.base[t] = tensor[t] + at.tv * V;
    in.ahead(at.begin, at.end, tensor);
    load_offsets(a, s_seg, false);
    if (DENSE && at.warp == kThreads / 32) {
        if (at.lane == 0) {
            for (int64_t r0 = at.end; r0 > at.begin;) {
                const Run k = run_before(a, s_seg, at.begin, r0);
                r0 = k.lo;
                if (k.s >= 0) in.load(k, tensor);
            }
            in.drain();
        }
        return;
    }
    F2 gamma[kPairs<V>], beta[kPairs<V>];
    gather_pairs<V>(gamma, [&](int j) { return works && a.gamma ? fetch(a.gamma + at.tv * V + j) : 1.f; });
    gather_pairs<V>(beta, [&](int j) { return works && a.beta ? fetch(a.beta + at.tv * V + j) : 0.f; });
    const float floor = floor_of(a.act);
    bool waited = false;
    for (int64_t r0 = at.end; r0 > at.begin;) {
        const Run k = run_before(a, s_seg, at.begin, r0);
        r0 = k.lo;
        if (k.s < 0) {
            F2 zero[kPairs<V>];
#pragma unroll
            for (int j = 0; j < kPairs<V>; ++j) zero[j] = both(0.f);
            if (works)
                for (int64_t r = k.lo + at.tr; r < k.hi; r += at.rt) {
                    const int64_t row = row_at(a.order, r, a.n, a.status);
                    if (row >= 0) *reinterpret_cast<Vec<T, V>*>(y + row * a.c) = pack<T, V>(zero);
                }
            continue;
        }
        in.begin(k);
        if (!waited) wait_for_kernel_before();
        waited = true;
        join_stats(a, s_seg, k.s, rows, w.part, s_stat);
        F2 minus[kPairs<V>], scale[kPairs<V>];
        gather_pairs<V>(scale, [&](int j) {
            return s_stat[at.group[j]].y;
        });
#pragma unroll
        for (int j = 0; j < kPairs<V>; ++j) scale[j] = mul(scale[j], gamma[j]);
        // the mean is taken off first: a constant channel gives beta exactly
        gather_pairs<V>(minus, [&](int j) { return -s_stat[at.group[j]].x; });
        in.run(works, [&](F2 (&f)[1][kPairs<V>], int64_t row) {
#pragma unroll
            for (int j = 0; j < kPairs<V>; ++j) f[0][j] = activate<SILU>(fma(add(f[0][j], minus[j]), scale[j], beta[j]), floor);
            *reinterpret_cast<Vec<T, V>*>(y + row * a.c) = pack<T, V>(f[0]);
        });
    }
    if (!waited) wait_for_kernel_before();
}

// -------------------------------------------------------------------- gradients
// Sums over the rows of this CTA: total[c][0] of dz and [1] of dz xh per channel, and per segment
// and group (sum gamma dz, sum gamma dz xh): whole segments' in coef[s], parts in part[slot].
template <typename T, int V, bool DENSE, bool SILU>
__global__ void __launch_bounds__(Feed<T, V, 2, DENSE>::kBlockThreads, 1) k_norm_bwd_sums(NormArgs a, int64_t rows, Ws w, uint64_t wait_ns)
{
    extern __shared__ __align__(16) uint8_t s_raw[];
    using S = Feed<T, V, 2, DENSE>;
    float* s_sum = reinterpret_cast<float*>(s_raw + S::kSmem);
    float* s_dz = s_sum + kSums<V, 2>;  // [2][c]
    int32_t* s_seg = reinterpret_cast<int32_t*>(s_dz + 2 * a.c);
    const Place<V> at(a, rows);
    const bool works = at.tr < at.rt;
    S in(a, s_raw, wait_ns, at.vpr, at.rt, at.tr);
    const T* const tensor[2] = {static_cast<const T*>(a.x), static_cast<const T*>(a.dy)};
    in.step = 1;
#pragma unroll
    for (int t = 0; t < 2; ++t) in.base[t] = tensor[t] + at.tv * V;
    wait_for_kernel_before();
    in.ahead(at.begin, at.end, tensor);
    load_offsets(a, s_seg, blockIdx.x == 0);
    if (DENSE && at.warp == kThreads / 32) {
        if (at.lane == 0) {
            for (int64_t r0 = at.begin; r0 < at.end;) {
                const Run k = run_at(a, s_seg, r0, at.end);
                r0 = k.hi;
                if (k.s >= 0) in.load(k, tensor);
            }
            in.drain();
        }
        return;
    }
    const Columns columns(a.c, at.rt);
    F2 gamma[kPairs<V>], beta[kPairs<V>];
    gather_pairs<V>(gamma, [&](int j) { return works && a.gamma ? fetch(a.gamma + at.tv * V + j) : 1.f; });
    gather_pairs<V>(beta, [&](int j) { return works && a.beta ? fetch(a.beta + at.tv * V + j) : 0.f; });
    const float least = least_of(a.act);
    float all[2][V];
#pragma unroll
    for (int j = 0; j < V; ++j) all[0][j] = all[1][j] = 0.f;
    for (int64_t r0 = at.begin; r0 < at.end;) {
        const Run k = run_at(a, s_seg, r0, at.end);
        r0 = k.hi;
        if (k.s < 0) continue;
        F2 minus[kPairs<V>], scale[kPairs<V>], sum[2][kPairs<V>];
#pragma unroll
        for (int j = 0; j < kPairs<V>; ++j) sum[0][j] = sum[1][j] = both(0.f);
        in.begin(k);
        const float* mean = a.mean + (int64_t)k.s * a.groups;
        const float* rstd = a.rstd + (int64_t)k.s * a.groups;
        gather_pairs<V>(minus, [&](int j) { return works ? -fetch(mean + at.group[j]) : 0.f; });
        gather_pairs<V>(scale, [&](int j) {
            return works ? fetch(rstd + at.group[j]) : 0.f;
        });
#pragma unroll
        for (int j = 0; j < kPairs<V>; ++j) scale[j] = mul(scale[j], gamma[j]);
        in.run(works, [&](const F2 (&f)[2][kPairs<V>], int64_t) {
#pragma unroll
            for (int j = 0; j < kPairs<V>; ++j) {
                const F2 e = add(f[0][j], minus[j]);
                const F2 dz = through<SILU>(f[1][j], fma(e, scale[j], beta[j]), least);
                sum[0][j] = add(sum[0][j], dz);
                sum[1][j] = fma(dz, e, sum[1][j]);
            }
        });
        if (works) {
            F2 r[kPairs<V>];
            gather_pairs<V>(r, [&](int j) { return fetch(rstd + at.group[j]); });
#pragma unroll
            for (int j = 0; j < kPairs<V>; ++j) sum[1][j] = mul(sum[1][j], r[j]);
        }
        column_sums<V, 2>(columns, sum, s_sum, s_dz, at.tr, at.tv);
        if (at.tr == 0)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                all[0][j] += s_dz[at.tv * V + j];
                all[1][j] += s_dz[a.c + at.tv * V + j];
            }
        const bool whole = k.whole(s_seg);
        const int slot = k.slot(at.begin);
        const GroupLoop way(at.per);
        for (int g = way.g; g < a.groups; g += way.step) {
            float m0 = 0.f, m1 = 0.f;
            for (int j = way.lane; j < at.per; j += way.lanes) {
                const int ch = g * at.per + j;
                const float u = a.gamma ? fetch(a.gamma + ch) : 1.f;
                m0 = fmaf(u, s_dz[ch], m0);
                m1 = fmaf(u, s_dz[a.c + ch], m1);
            }
            m0 = group_sum(m0, at.per);
            m1 = group_sum(m1, at.per);
            if (way.lane == 0) {
                if (whole) w.coef[(int64_t)k.s * a.groups + g] = make_float2(m0, m1);
                else w.part[(int64_t)slot * a.groups + g] = make_float2(m0, m1);
            }
        }
        sync_workers();
    }
    if (at.tr == 0)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            w.total[(int64_t)blockIdx.x * 2 * a.c + at.tv * V + j] = all[0][j];
            w.total[((int64_t)blockIdx.x * 2 + 1) * a.c + at.tv * V + j] = all[1][j];
        }
}

template <typename T, int V, bool DENSE, bool SILU>
__global__ void __launch_bounds__(Feed<T, V, 2, DENSE>::kBlockThreads, 1) k_norm_bwd_apply(NormArgs a, int64_t rows, Ws w, uint64_t wait_ns)
{
    extern __shared__ __align__(16) uint8_t s_raw[];
    using S = Feed<T, V, 2, DENSE>;
    float2* s_stat = reinterpret_cast<float2*>(s_raw + S::kSmem);
    int32_t* s_seg = reinterpret_cast<int32_t*>(s_stat + a.groups);
    const Place<V> at(a, rows);
    const bool works = at.tr < at.rt;
    T* dx = static_cast<T*>(a.out) + at.tv * V;
    S in(a, s_raw, wait_ns, at.vpr, at.rt, at.tr);
    const T* const tensor[2] = {static_cast<const T*>(a.x), static_cast<const T*>(a.dy)};
    in.step = -1;
#pragma unroll
    for (int t = 0; t < 2; ++t) in.base[t] = tensor[t] + at.tv * V;
    in.ahead(at.begin, at.end, tensor);
    load_offsets(a, s_seg, false);
    if (DENSE && at.warp == kThreads / 32) {
        if (at.lane == 0) {
            for (int64_t r0 = at.end; r0 > at.begin;) {
                const Run k = run_before(a, s_seg, at.begin, r0);
                r0 = k.lo;
                if (k.s >= 0) in.load(k, tensor);
            }
            in.drain();
        }
        return;
    }
    F2 gamma[kPairs<V>], beta[kPairs<V>];
    gather_pairs<V>(gamma, [&](int j) { return works && a.gamma ? fetch(a.gamma + at.tv * V + j) : 1.f; });
    gather_pairs<V>(beta, [&](int j) { return works && a.beta ? fetch(a.beta + at.tv * V + j) : 0.f; });
    const float least = least_of(a.act);
    bool waited = false;
    for (int64_t r0 = at.end; r0 > at.begin;) {
        const Run k = run_before(a, s_seg, at.begin, r0);
        r0 = k.lo;
        if (k.s < 0) {
            F2 zero[kPairs<V>];
#pragma unroll
            for (int j = 0; j < kPairs<V>; ++j) zero[j] = both(0.f);
            if (works)
                for (int64_t r = k.lo + at.tr; r < k.hi; r += at.rt) {
                    const int64_t row = row_at(a.order, r, a.n, a.status);
                    if (row >= 0) *reinterpret_cast<Vec<T, V>*>(dx + row * a.c) = pack<T, V>(zero);
                }
            continue;
        }
        in.begin(k);
        if (!waited) wait_for_kernel_before();
        waited = true;
        const Span span(s_seg, k.s, rows);
        sync_workers();
        for (int g0 = 0; g0 < a.groups; g0 += kThreads / kJoin) {
            const int g = g0 + (int)threadIdx.x / kJoin, lane = threadIdx.x % kJoin;
            const bool real = g < a.groups;
            float2 m = make_float2(0.f, 0.f);
            if (span.first == span.last) {
                if (real && lane == 0) m = w.coef[(int64_t)k.s * a.groups + g];
            } else {
                const Parts parts(span, w.part, rows, a.groups);
#pragma unroll 5
                for (int i = lane; i < parts.count(); i += kJoin) {
                    const float2 v = parts.get(i, real ? g : 0);
                    m.x += v.x;
                    m.y += v.y;
                }
                m.x = join_sum(m.x);
                m.y = join_sum(m.y);
            }
            const float n = (float)(int)(span.hi - span.lo) * (float)at.per;
            if (real && lane == 0) s_stat[g] = make_float2(m.x / n, m.y / n);
        }
        sync_workers();
        F2 minus[kPairs<V>], scale[kPairs<V>], lift[kPairs<V>], tilt[kPairs<V>];
        const float* mean = a.mean + (int64_t)k.s * a.groups;
        const float* rstd = a.rstd + (int64_t)k.s * a.groups;
        gather_pairs<V>(minus, [&](int j) { return -fetch(mean + at.group[j]); });
        gather_pairs<V>(scale, [&](int j) {
            return works ? fetch(rstd + at.group[j]) : 0.f;
        });
#pragma unroll
        for (int j = 0; j < kPairs<V>; ++j) scale[j] = mul(scale[j], gamma[j]);
        gather_pairs<V>(lift, [&](int j) {
            const int g = at.group[j];
            return -fetch(rstd + g) * s_stat[g].x;
        });
        gather_pairs<V>(tilt, [&](int j) {
            const int g = at.group[j];
            const float r = fetch(rstd + g);
            return -r * r * s_stat[g].y;
        });
        in.run(works, [&](F2 (&f)[2][kPairs<V>], int64_t row) {
#pragma unroll
            for (int j = 0; j < kPairs<V>; ++j) {
                const F2 e = add(f[0][j], minus[j]);
                const F2 dz = through<SILU>(f[1][j], fma(e, scale[j], beta[j]), least);
                f[0][j] = fma(dz, scale[j], fma(e, tilt[j], lift[j]));
            }
            *reinterpret_cast<Vec<T, V>*>(dx + row * a.c) = pack<T, V>(f[0]);
        });
    }
    if (!waited) wait_for_kernel_before();
    // dgamma and dbeta: a warp for each channel
    if (a.dgamma || a.dbeta)
        for (int ch = blockIdx.x * (kThreads / 32) + at.warp; ch < a.c; ch += gridDim.x * (kThreads / 32)) {
            float s0 = 0.f, s1 = 0.f;
            for (int c = at.lane; c < (int)gridDim.x; c += 32) {
                s0 += w.total[(int64_t)c * 2 * a.c + ch];
                s1 += w.total[((int64_t)c * 2 + 1) * a.c + ch];
            }
            s0 = warp_sum(s0);
            s1 = warp_sum(s1);
            if (at.lane == 0 && a.dbeta) a.dbeta[ch] = s0;
            if (at.lane == 0 && a.dgamma) a.dgamma[ch] = s1;
        }
}

// ------------------------------------------- rows of more than kThreads vectors
// One block per (group, segment), then a thread per element: a simple form for rows that are rare.  40,000 x 1030
// fp32, 10 groups, 2 samples: forward 13.5 ms, gradients 1.8, of 49 and 73 us that the bytes would take.  The
// twenty blocks of the statistics, each dividing for every element's place, are nearly all of the forward.
template <typename T>
__global__ void __launch_bounds__(kBlock) k_norm_stats_wide(NormArgs a)
{
    const int g = blockIdx.x, s = blockIdx.y, per = a.c / a.groups;
    int64_t lo, hi;
    segment_bounds(a.seg, s, a.n, a.status, lo, hi);
    const T* x = static_cast<const T*>(a.x);
    const int64_t total = (hi - lo) * per;
    const float count = (float)(total > 0 ? total : 1);
    auto at = [&](int64_t e) -> float {
        const int64_t row = row_at(a.order, lo + e / per, a.n, a.status);
        return row < 0 ? 0.f : elem<T>::to_f32(x[row * a.c + g * per + e % per]);
    };
    // a thread's sums are long (a 256th of the group): around the group's first value, carrying their rounding
    const float pivot = total > 0 ? at(0) : 0.f;
    Exact sum, squares;
    for (int64_t e = threadIdx.x; e < total; e += kBlock) sum.add(at(e) - pivot);
    const float mean = pivot + block_sum(sum.value()) / count;
    for (int64_t e = threadIdx.x; e < total; e += kBlock) {
        const float d = at(e) - mean;
        squares.add(d * d);
    }
    const float var = block_sum(squares.value()) / count;
    if (threadIdx.x == 0) {
        a.mean[s * a.groups + g] = mean;
        a.rstd[s * a.groups + g] = 1.f / sqrtf(var + a.eps);
    }
}

template <typename T>
__global__ void __launch_bounds__(kBlock) k_norm_apply_wide(NormArgs a)
{
    const int64_t t = (int64_t)blockIdx.x * kBlock + threadIdx.x;
    const int64_t r = t / a.c;
    const int c = (int)(t % a.c);
    if (r >= a.n) return;
    const int64_t row = row_at(a.order, r, a.n, a.status);
    if (row < 0) return;
    const int s = segment_of(a.seg, a.segments, r);
    float y = 0.f;
    if (s >= 0 && s < a.segments) {
        const int i = s * a.groups + c / (a.c / a.groups);
        const float xh = (elem<T>::to_f32(static_cast<const T*>(a.x)[row * a.c + c]) - a.mean[i]) * a.rstd[i];
        y = activate(xh * (a.gamma ? a.gamma[c] : 1.f) + (a.beta ? a.beta[c] : 0.f), a.act);
    }
    static_cast<T*>(a.out)[row * a.c + c] = elem<T>::from_f32(y);
}

// part[s][0][c] = sum of dz, part[s][1][c] = sum of dz xh over segment s
template <typename T>
__global__ void __launch_bounds__(kBlock) k_norm_bwd_sums_wide(NormArgs a, float* __restrict__ part)
{
    const int c = blockIdx.x, s = blockIdx.y;
    const int i = s * a.groups + c / (a.c / a.groups);
    int64_t lo, hi;
    segment_bounds(a.seg, s, a.n, a.status, lo, hi);
    const float mean = a.mean[i], rstd = a.rstd[i];
    const float gamma = a.gamma ? a.gamma[c] : 1.f, beta = a.beta ? a.beta[c] : 0.f;
    float s0 = 0.f, s1 = 0.f;
    for (int64_t r = lo + threadIdx.x; r < hi; r += kBlock) {
        const int64_t row = row_at(a.order, r, a.n, a.status);
        if (row < 0) continue;
        const float xh = (elem<T>::to_f32(static_cast<const T*>(a.x)[row * a.c + c]) - mean) * rstd;
        const float dz = elem<T>::to_f32(static_cast<const T*>(a.dy)[row * a.c + c]) * slope(xh * gamma + beta, a.act);
        s0 += dz;
        s1 += dz * xh;
    }
    s0 = block_sum(s0);
    s1 = block_sum(s1);
    if (threadIdx.x == 0) {
        part[(int64_t)s * 2 * a.c + c] = s0;
        part[(int64_t)s * 2 * a.c + a.c + c] = s1;
    }
}

__global__ void __launch_bounds__(kBlock) k_norm_bwd_params_wide(NormArgs a, const float* __restrict__ part)
{
    const int c = blockIdx.x * kBlock + threadIdx.x;
    if (c >= a.c) return;
    float s0 = 0.f, s1 = 0.f;
    for (int s = 0; s < a.segments; ++s) {
        s0 += part[(int64_t)s * 2 * a.c + c];
        s1 += part[(int64_t)s * 2 * a.c + a.c + c];
    }
    if (a.dbeta) a.dbeta[c] = s0;
    if (a.dgamma) a.dgamma[c] = s1;
}

template <typename T>
__global__ void __launch_bounds__(kBlock) k_norm_bwd_apply_wide(NormArgs a, const float* __restrict__ part)
{
    const int64_t t = (int64_t)blockIdx.x * kBlock + threadIdx.x;
    const int64_t r = t / a.c;
    const int c = (int)(t % a.c), per = a.c / a.groups;
    if (r >= a.n) return;
    const int64_t row = row_at(a.order, r, a.n, a.status);
    if (row < 0) return;
    const int s = segment_of(a.seg, a.segments, r);
    float dx = 0.f;
    if (s >= 0 && s < a.segments) {
        const int g = c / per, i = s * a.groups + g;
        int64_t lo, hi;
        segment_bounds(a.seg, s, a.n, a.status, lo, hi);
        const float count = (float)((hi - lo) * per);
        float m0 = 0.f, m1 = 0.f;
        for (int j = g * per; j < (g + 1) * per; ++j) {
            const float w = a.gamma ? a.gamma[j] : 1.f;
            m0 += w * part[(int64_t)s * 2 * a.c + j];
            m1 += w * part[(int64_t)s * 2 * a.c + a.c + j];
        }
        const float gamma = a.gamma ? a.gamma[c] : 1.f, beta = a.beta ? a.beta[c] : 0.f;
        const float xh = (elem<T>::to_f32(static_cast<const T*>(a.x)[row * a.c + c]) - a.mean[i]) * a.rstd[i];
        const float dz = elem<T>::to_f32(static_cast<const T*>(a.dy)[row * a.c + c]) * slope(xh * gamma + beta, a.act);
        dx = a.rstd[i] * (gamma * dz - m0 / count - xh * (m1 / count));
    }
    static_cast<T*>(a.out)[row * a.c + c] = elem<T>::from_f32(dx);
}

template <typename T>
spc_status fwd_wide(const NormArgs& a, cudaStream_t st)
{
    const int64_t blocks = ceil_div(a.n * a.c, kBlock);
    if (blocks > INT32_MAX) return SPC_ERR_UNSUPPORTED;
    k_norm_stats_wide<T><<<dim3(a.groups, a.segments), kBlock, 0, st>>>(a);
    SPC_LAUNCH_CHECK();
    if (a.n == 0) return SPC_OK;
    k_norm_apply_wide<T><<<(unsigned)blocks, kBlock, 0, st>>>(a);
    SPC_LAUNCH_CHECK();
    return SPC_OK;
}

template <typename T>
spc_status bwd_wide(const NormArgs& a, float* part, cudaStream_t st)
{
    const int64_t blocks = ceil_div(a.n * a.c, kBlock);
    if (blocks > INT32_MAX) return SPC_ERR_UNSUPPORTED;
    k_norm_bwd_sums_wide<T><<<dim3(a.c, a.segments), kBlock, 0, st>>>(a, part);
    SPC_LAUNCH_CHECK();
    if (a.dgamma || a.dbeta) {
        k_norm_bwd_params_wide<<<(unsigned)ceil_div(a.c, kBlock), kBlock, 0, st>>>(a, part);
        SPC_LAUNCH_CHECK();
    }
    if (a.n == 0) return SPC_OK;
    k_norm_bwd_apply_wide<T><<<(unsigned)blocks, kBlock, 0, st>>>(a, part);
    SPC_LAUNCH_CHECK();
    return SPC_OK;
}

// ----------------------------------------------------------------------- launch
// Channels of a thread: as many as divide the row and stand aligned in it.
template <typename T>
int vector_of(const NormArgs& a)
{
    const uintptr_t low = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.out) |
                          reinterpret_cast<uintptr_t>(a.dy);
    int v = 16 / (int)sizeof(T);
    while (v > 1 && (a.c % v != 0 || (low & (v * sizeof(T) - 1)) != 0)) v /= 2;
    return v;
}

int shares_of(int64_t n) { return (int)std::max<int64_t>(1, std::min<int64_t>(sm_count(), ceil_div(n, kMinRows))); }

size_t carve(int64_t n, int32_t c, int32_t segments, int32_t groups, char* base, Ws* w)
{
    size_t off = 0;
    auto take = [&](size_t bytes) {
        char* p = base ? base + off : nullptr;
        off = align_up(off + bytes, 256);
        return p;
    };
    const size_t shares = (size_t)shares_of(n);
    char* part = take(sizeof(float2) * 2 * shares * groups);
    char* coef = take(sizeof(float2) * (size_t)segments * groups);
    char* total = take(sizeof(float) * 2 * shares * c);
    if (w) *w = Ws{reinterpret_cast<float2*>(part), reinterpret_cast<float2*>(coef), reinterpret_cast<float*>(total)};
    return off;
}

template <auto KERNEL>
spc_status launch(int shares, int threads, size_t smem, cudaStream_t st, const NormArgs& a, int64_t rows, const Ws& w)
{
    const spc_status allowed = allow_smem<KERNEL>();
    if (allowed != SPC_OK) return allowed;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)shares);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    // the first kernel of a pass waits before it touches memory, the second where it needs the first one's sums
    cudaLaunchAttribute attr[1] = {beside_the_kernel_before()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    SPC_CUDA_TRY(cudaLaunchKernelEx(&cfg, KERNEL, a, rows, w, wait_limit_ns()));
    return SPC_OK;
}

template <typename T, int V, bool DENSE, bool SILU>
spc_status rows_pass(const NormArgs& a, const Ws& w, bool backward, cudaStream_t st)
{
    const int shares = shares_of(a.n);
    const int64_t rows = std::max<int64_t>(1, ceil_div(a.n, shares));
    const size_t offsets = sizeof(int32_t) * (a.segments + 1), stat = sizeof(float2) * a.groups;
    if (backward) {
        using F = Feed<T, V, 2, DENSE>;
        const size_t base = F::kSmem + offsets;
        const spc_status s = launch<k_norm_bwd_sums<T, V, DENSE, SILU>>(shares, F::kBlockThreads,
                                    base + sizeof(float) * (kSums<V, 2> + 2 * a.c), st, a, rows, w);
        return s != SPC_OK ? s : launch<k_norm_bwd_apply<T, V, DENSE, SILU>>(shares, F::kBlockThreads, base + stat, st, a, rows, w);
    }
    using F = Feed<T, V, 1, DENSE>;
    const size_t base = F::kSmem + offsets;
    const spc_status s = launch<k_norm_stats<T, V, DENSE>>(shares, F::kBlockThreads,
                                base + sizeof(float) * (kSums<V, 1> + 2 * a.c), st, a, rows, w);
    return s != SPC_OK || a.n == 0
               ? s
               : launch<k_norm_apply<T, V, DENSE, SILU>>(shares, F::kBlockThreads, base + stat, st, a, rows, w);
}

template <typename T, int V>
spc_status rows_pass(const NormArgs& a, const Ws& w, bool backward, cudaStream_t st)
{
    const bool silu = a.act == SPC_ACT_SILU;
    // the form for rows in order exists for whole 16-byte vectors; the other takes any
    if constexpr (V * sizeof(T) == 16)
        if (!a.order) return silu ? rows_pass<T, V, true, true>(a, w, backward, st) : rows_pass<T, V, true, false>(a, w, backward, st);
    return silu ? rows_pass<T, V, false, true>(a, w, backward, st) : rows_pass<T, V, false, false>(a, w, backward, st);
}

template <typename T>
spc_status norm_pass(const NormArgs& a, void* ws, bool backward, cudaStream_t st)
{
    const int v = vector_of<T>(a);
    Ws w;
    carve(a.n, a.c, a.segments, a.groups, static_cast<char*>(ws), &w);
    if (a.c / v > kThreads) return backward ? bwd_wide<T>(a, static_cast<float*>(ws), st) : fwd_wide<T>(a, st);
    if constexpr (sizeof(T) == 2)
        if (v == 8) return rows_pass<T, 8>(a, w, backward, st);
    if (v == 4) return rows_pass<T, 4>(a, w, backward, st);
    if (v == 2) return rows_pass<T, 2>(a, w, backward, st);
    return rows_pass<T, 1>(a, w, backward, st);
}

}  // namespace

}  // namespace spc
