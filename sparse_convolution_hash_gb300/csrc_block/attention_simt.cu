// attention_simt.cu -- attention over segments on CUDA cores: fp32 (full fp32 products), and 16-bit heads that the
// tensor-core kernels do not take (channels not a multiple of 8, rows off a 16-byte boundary, no rows on one side).
//
// 64 x 64 tiles of scores by 256 threads, 4 x 4 a thread, operands as fp32 in shared memory.  The forward pass
// keeps a running maximum and sum per row; the gradients take the probabilities from the forward's
// log-sum and are two kernels, one that walks over the queries for dk and dv and one over the keys for dq, so every
// sum has its place and its order and there are no atomics.  A tile's walk may be split (see attention.cu);
// then fp32 parts go to the workspace.
// Bound by shared memory: 64 multiply-adds (32 instructions, two at a time) stand against eight reads of 16 bytes, which
// take four cycles each.  8 heads of 64, 6,000 rows: 1.95 ms forward (38 TFLOP/s), 6.5 ms backward.
//
// The forward pass of fp32 heads of up to 16 channels has a kernel of its own: a thread keeps its rows' queries and sums in
// registers, so that shared memory holds keys and values only and no score passes through it.  2,000 rows, 4 heads
// of 16: 37 us with the join against 64 with tiles; 30,000 rows in 600 segments, 8 heads of 16: 61 against 92.
#include "attention.cuh"
#include "pairs.cuh"
#include "ptx.cuh"

namespace spc {

namespace {

constexpr int kThreads = 256, kTile = 64, kPad = 4;
constexpr float kLazy = 8.f;  // a maximum may grow by this much (log2) before sums are rescaled

template <int DP> struct Mat { float v[kTile][DP + kPad]; };
// blocks that share an SM
template <int DP> constexpr int kBlocks = DP <= 64 ? 2 : 1;
// (two blocks of 128 registers: 30,000 rows in 600 segments, 8 heads of 32: 174 us against 140 of three)
template <int DP> constexpr int kFwdBlocks = DP <= 32 ? 3 : kBlocks<DP>;
struct Probs { float v[kTile][kTile + kPad]; };

// Rows [row, end) of one head as fp32, zeros past the end and past d: four channels at once where fp32 rows allow it.
template <typename T, int DP>
__device__ __forceinline__ void load(Mat<DP>& m, const void* base, int64_t ld, int head, int d, int64_t row, int64_t end)
{
    const T* p = static_cast<const T*>(base) + (int64_t)head * d;
    if (sizeof(T) == 4 && ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)(ld * 4) | (uintptr_t)(d * 4)) & 15) == 0) {
#pragma unroll
        for (int i = threadIdx.x; i < kTile * DP / 4; i += kThreads) {
            const int r = i / (DP / 4), c = i % (DP / 4) * 4;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (row + r < end && c < d) v = *reinterpret_cast<const float4*>(p + (row + r) * ld + c);
            *reinterpret_cast<float4*>(&m.v[r][c]) = v;
        }
        return;
    }
    for (int i = threadIdx.x; i < kTile * DP; i += kThreads) {
        const int r = i / DP, c = i % DP;
        m.v[r][c] = row + r < end && c < d ? elem<T>::to_f32(p[(row + r) * ld + c]) : 0.f;
    }
}

// s[i][j] = a[4 ty + i] . b[tx + 16 j]
template <int DP, bool PAIRS>
__device__ __forceinline__ void dot(const Mat<DP>& a, const Mat<DP>& b, int ty, int tx, float (&s)[4][4])
{
    F2 two[4][4];  // even channels, odd channels
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) two[i][j] = F2{0.f, 0.f};
    }
#pragma unroll 2
    for (int c = 0; c < DP; c += 4) {
        float4 x[4], y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(&a.v[4 * ty + i][c]);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(&b.v[tx + 16 * j][c]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if constexpr (PAIRS) {
                    two[i][j] = fma(F2{x[i].x, x[i].y}, F2{y[j].x, y[j].y}, two[i][j]);
                    two[i][j] = fma(F2{x[i].z, x[i].w}, F2{y[j].z, y[j].w}, two[i][j]);
                } else {  // half the registers, for a third block on the SM
                    two[i][j].x = fmaf(x[i].x, y[j].x, two[i][j].x);
                    two[i][j].x = fmaf(x[i].y, y[j].y, two[i][j].x);
                    two[i][j].x = fmaf(x[i].z, y[j].z, two[i][j].x);
                    two[i][j].x = fmaf(x[i].w, y[j].w, two[i][j].x);
                }
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = PAIRS ? two[i][j].x + two[i][j].y : two[i][j].x;
    }
}

// A thread's share of the second products: four rows by four channels (eight for DP = 128, in two quads), so that a read of 16
// bytes feeds eight multiply-adds or more; where 16 threads then hold more than the DP channels, each part of them takes its share
// of the other side's rows, and the parts' sums join at the end.
template <int DP>
struct Out {
    static constexpr int kQuads = DP > 64 ? 2 : 1, kGroups = DP / (4 * kQuads), kParts = 16 / kGroups;
    F2 v[4][2 * kQuads];
    int group, part;

    __device__ __forceinline__ explicit Out(int tx) : group(tx % kGroups), part(tx / kGroups)
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int c = 0; c < 2 * kQuads; ++c) v[i][c] = F2{0.f, 0.f};
        }
    }
    __device__ __forceinline__ int channel(int quad) const { return 4 * group + 64 * quad; }
    __device__ __forceinline__ void add_row(const Mat<DP>& b, int row, const float (&w)[4])
    {
#pragma unroll
        for (int q = 0; q < kQuads; ++q) {
            const float4 y = *reinterpret_cast<const float4*>(&b.v[row][channel(q)]);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                v[i][2 * q] = fma(both(w[i]), F2{y.x, y.y}, v[i][2 * q]);
                v[i][2 * q + 1] = fma(both(w[i]), F2{y.z, y.w}, v[i][2 * q + 1]);
            }
        }
    }
    // += sum over k of p[4 ty + i][k] b[k][:]
    __device__ __forceinline__ void rows_times(const Probs& p, const Mat<DP>& b, int ty)
    {
#pragma unroll 2
        for (int k = 4 * part; k < kTile; k += 4 * kParts) {
            float4 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(&p.v[4 * ty + i][k]);
            add_row(b, k, {w[0].x, w[1].x, w[2].x, w[3].x});
            add_row(b, k + 1, {w[0].y, w[1].y, w[2].y, w[3].y});
            add_row(b, k + 2, {w[0].z, w[1].z, w[2].z, w[3].z});
            add_row(b, k + 3, {w[0].w, w[1].w, w[2].w, w[3].w});
        }
    }
    // += sum over r of p[r][4 ty + i] b[r][:]
    __device__ __forceinline__ void cols_times(const Probs& p, const Mat<DP>& b, int ty)
    {
#pragma unroll 4
        for (int r = part; r < kTile; r += kParts) {
            const float4 w = *reinterpret_cast<const float4*>(&p.v[r][4 * ty]);
            add_row(b, r, {w.x, w.y, w.z, w.w});
        }
    }
    __device__ __forceinline__ void join()
    {
#pragma unroll
        for (int o = kGroups; o < 16; o <<= 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
#pragma unroll
                for (int c = 0; c < 2 * kQuads; ++c) {
                    v[i][c].x += __shfl_xor_sync(FULL_MASK, v[i][c].x, o);
                    v[i][c].y += __shfl_xor_sync(FULL_MASK, v[i][c].y, o);
                }
            }
        }
    }
    // Joined sums of four rows from row + 4 ty on, scaled, as T or (split) as fp32; the parts take the rows in turn.
    template <typename T>
    __device__ __forceinline__ void store(const float (&mul)[4], T* out, int64_t ld, float* to_part, int64_t part_ld, int d, int64_t row,
                                          int64_t end, int ty)
    {
        join();
        // whole quads at once, in parts or where fp32 rows allow it (parts begin on 256 bytes)
        const bool quads = d % 4 == 0 && (to_part || (sizeof(T) == 4 && ((reinterpret_cast<uintptr_t>(out) | (uintptr_t)(ld * 4)) & 15) == 0));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int64_t r = row + 4 * ty + i;
            if (i % kParts != part || r >= end) continue;
#pragma unroll
            for (int q = 0; q < kQuads; ++q) {
                const int col = channel(q);
                const F2 lo = v[i][2 * q], hi = v[i][2 * q + 1];
                const float x[4] = {lo.x * mul[i], lo.y * mul[i], hi.x * mul[i], hi.y * mul[i]};
                if (quads && col < d) {
                    float* to = to_part ? to_part + r * part_ld : reinterpret_cast<float*>(out) + r * ld;
                    *reinterpret_cast<float4*>(to + col) = make_float4(x[0], x[1], x[2], x[3]);
                    continue;
                }
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (col + c >= d) break;
                    if (to_part) to_part[r * part_ld + col + c] = x[c];
                    else out[r * ld + col + c] = elem<T>::from_f32(x[c]);
                }
            }
        }
    }
};

// grid: slots of 64 queries, query heads, splits of the keys
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads, kFwdBlocks<DP>)
k_attn_simt(AttnArgs a)
{
    extern __shared__ float4 raw[];
    Mat<DP>& q = *reinterpret_cast<Mat<DP>*>(raw);
    Mat<DP>& k = *(&q + 1);
    Mat<DP>& v = *(&q + 2);
    Probs& p = *reinterpret_cast<Probs*>(&q + 3);
    wait_for_kernel_before();
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) {
        attn_check(a.seg_q, a.segments, a.nq, a.status, threadIdx.x, kThreads);
        if (a.seg_k != a.seg_q) attn_check(a.seg_k, a.segments, a.nk, a.status, threadIdx.x, kThreads);
    }
    AttnTile t;
    if (!attn_tile(a.seg_q, a.seg_k, a.segments, a.nq, a.nk, kTile, blockIdx.x, t)) return;
    const int head = blockIdx.y, kv = head / (a.hq / a.hk), tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    int64_t lo, hi;
    attn_share(t.lo, t.hi, kTile, blockIdx.z, a.splits, lo, hi);
    const float to_log2 = a.scale * kLog2e;
    float m[4], l[4];
    Out<DP> o(tx);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
    }
    if (lo < hi) load<T, DP>(q, a.q, a.ldq, head, a.d, t.row, t.end);
    for (int64_t at = lo; at < hi; at += kTile) {
        __syncthreads();
        load<T, DP>(k, a.k, a.ldk, kv, a.d, at, hi);
        load<T, DP>(v, a.v, a.ldv, kv, a.d, at, hi);
        __syncthreads();
        float s[4][4];
        dot<DP, (DP > 32)>(q, k, ty, tx, s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float most = m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = at + tx + 16 * j < hi ? s[i][j] : -INFINITY;
                most = fmaxf(most, s[i][j]);
            }
#pragma unroll
            for (int x = 8; x; x >>= 1) most = fmaxf(most, __shfl_xor_sync(FULL_MASK, most, x));
            // the rounding of the base is the row's sums' and its log-sum's alike
            const float base = most == -INFINITY ? 0.f : -most * to_log2, shrink = ptx::ex2((m[i] - (most == -INFINITY ? 0.f : most)) * to_log2);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float e = ptx::ex2(fmaf(s[i][j], to_log2, base));
                sum += e;
                p.v[4 * ty + i][tx + 16 * j] = e;
            }
            l[i] = l[i] * shrink + sum;  // of this thread's columns: they join at the end
            m[i] = most;
#pragma unroll
            for (int c = 0; c < 2 * Out<DP>::kQuads; ++c) o.v[i][c] = mul(o.v[i][c], both(shrink));
        }
        __syncwarp();  // a row of p is written and read by the same half warp
        o.rows_times(p, v, ty);
    }
    float inv[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int x = 8; x; x >>= 1) l[i] += __shfl_xor_sync(FULL_MASK, l[i], x);
        inv[i] = l[i] == 0.f ? 0.f : 1.f / l[i];
        if (l[i] == 0.f) {  // no keys: a zero, whatever stands in the sums
#pragma unroll
            for (int c = 0; c < 2 * Out<DP>::kQuads; ++c) o.v[i][c] = F2{0.f, 0.f};
        }
        const int64_t r = t.row + 4 * ty + i;
        if (tx == 0 && r < t.end) {
            const float lse = l[i] == 0.f ? -INFINITY : (m[i] * to_log2 + log2f(l[i])) * kLn2;
            if (a.splits > 1) a.part_lse[(blockIdx.z * a.nq + r) * a.hq + head] = lse;
            else a.lse[r * a.hq + head] = lse;
        }
    }
    const int64_t width = (int64_t)a.hq * a.d;
    o.template store<T>(inv, static_cast<T*>(a.o) + (int64_t)head * a.d, a.ldo,
                        a.splits > 1 ? a.part + blockIdx.z * a.nq * width + (int64_t)head * a.d : nullptr, width, a.d, t.row, t.end, ty);
}

// ---- narrow heads in fp32: a thread keeps R whole rows, queries and sums in registers, and reads keys and values
// as its warp does, all lanes the same 16 bytes.  The block's warps walk over different keys and join at the end.
constexpr int kNarrow = kAttnNarrow, kRowWarps = 4, kRowFields = kNarrow + 2;
template <int R>
struct Rows {
    static constexpr int kTile = 32 * R, kKeys = 32 * R;  // queries of a block, keys of a step
    static constexpr size_t kBuffers = sizeof(float) * 2 * 2 * kKeys * kNarrow, kJoin = sizeof(float) * kRowWarps * kRowFields * kTile;
    static constexpr size_t kSmem = kBuffers > kJoin ? kBuffers : kJoin;
};

// grid: slots of 32 R queries, query heads, splits of the keys
template <int R>
__global__ void __launch_bounds__(32 * kRowWarps, R == 4 ? 2 : 4)
k_attn_rows_simt(AttnArgs a)
{
    extern __shared__ float4 raw[];
    constexpr int kRowTile = Rows<R>::kTile, kRowKeys = Rows<R>::kKeys, kStep = kRowKeys / kRowWarps, kRowsEach = R;
    wait_for_kernel_before();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) {
        attn_check(a.seg_q, a.segments, a.nq, a.status, tid, 32 * kRowWarps);
        if (a.seg_k != a.seg_q) attn_check(a.seg_k, a.segments, a.nk, a.status, tid, 32 * kRowWarps);
    }
    AttnTile t;
    if (!attn_tile(a.seg_q, a.seg_k, a.segments, a.nq, a.nk, kRowTile, blockIdx.x, t)) return;
    const int head = blockIdx.y, kv = head / (a.hq / a.hk);
    int64_t lo, hi;
    attn_share(t.lo, t.hi, kRowKeys, blockIdx.z, a.splits, lo, hi);
    const float* keys = static_cast<const float*>(a.k) + (int64_t)kv * a.d;
    const float* values = static_cast<const float*>(a.v) + (int64_t)kv * a.d;
    const uint32_t base_s = (uint32_t)__cvta_generic_to_shared(raw);
    // keys then values of a buffer, zeros past the share's end and past d
    auto load = [&](int64_t at, int buffer) {
        for (int x = tid; x < 2 * kRowKeys * (kNarrow / 4); x += 32 * kRowWarps) {
            const int which = x / (kRowKeys * (kNarrow / 4)), row = x / (kNarrow / 4) % kRowKeys, c = x % (kNarrow / 4) * 4;
            const bool there = at + row < hi && c < a.d;
            const float* from = which ? values : keys;
            ptx::cp_async16(base_s + ((buffer * 2 + which) * kRowKeys + row) * (kNarrow * 4) + c * 4,
                       there ? from + (at + row) * (which ? a.ldv : a.ldk) + c : from, there ? 16 : 0);
        }
        ptx::cp_async_commit();
    };
    F2 q[kRowsEach][kNarrow / 2], o[kRowsEach][kNarrow / 2];
    float m[kRowsEach], l[kRowsEach];
#pragma unroll
    for (int i = 0; i < kRowsEach; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
        const int64_t row = t.row + lane + 32 * i;
        const float* from = static_cast<const float*>(a.q) + row * a.ldq + (int64_t)head * a.d;
#pragma unroll
        for (int c = 0; c < kNarrow; c += 4) {
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (row < t.end && c < a.d) x = *reinterpret_cast<const float4*>(from + c);
            q[i][c / 2] = F2{x.x, x.y};
            q[i][c / 2 + 1] = F2{x.z, x.w};
            o[i][c / 2] = o[i][c / 2 + 1] = F2{0.f, 0.f};
        }
    }
    const float c = a.scale * kLog2e;
    if (lo < hi) load(lo, 0);
    int buffer = 0;
    for (int64_t at = lo; at < hi; at += kRowKeys, buffer ^= 1) {
        if (at + kRowKeys < hi) {
            load(at + kRowKeys, buffer ^ 1);
            ptx::cp_async_wait<1>();
        } else {
            ptx::cp_async_wait<0>();
        }
        __syncthreads();
        const float4* k4 = raw + (buffer * 2 * kRowKeys + warp * kStep) * (kNarrow / 4);
        const float4* v4 = k4 + kRowKeys * (kNarrow / 4);
        const int valid = (int)min((int64_t)kStep, hi - at - warp * kStep);
#pragma unroll 1
        for (int x = 0; x < valid; x += 4) {
            float s[kRowsEach][4];
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                float4 k[kNarrow / 4];
#pragma unroll
                for (int z = 0; z < kNarrow / 4; ++z) k[z] = k4[(x + y) * (kNarrow / 4) + z];
#pragma unroll
                for (int i = 0; i < kRowsEach; ++i) {
                    F2 two{0.f, 0.f};
#pragma unroll
                    for (int z = 0; z < kNarrow / 4; ++z) {
                        two = fma(q[i][2 * z], F2{k[z].x, k[z].y}, two);
                        two = fma(q[i][2 * z + 1], F2{k[z].z, k[z].w}, two);
                    }
                    s[i][y] = x + y < valid ? two.x + two.y : -INFINITY;
                }
            }
            float top[kRowsEach];
            bool grow = false;
#pragma unroll
            for (int i = 0; i < kRowsEach; ++i) {
                top[i] = fmaxf(fmaxf(fmaxf(m[i], s[i][0]), fmaxf(s[i][1], s[i][2])), s[i][3]);
                grow |= (top[i] - m[i]) * c > kLazy;  // false where both are -inf
            }
            if (__any_sync(FULL_MASK, grow)) {
#pragma unroll
                for (int i = 0; i < kRowsEach; ++i) {
                    const float shrink = top[i] > m[i] ? ptx::ex2((m[i] - top[i]) * c) : 1.f;
                    m[i] = top[i];
                    l[i] *= shrink;
#pragma unroll
                    for (int z = 0; z < kNarrow / 2; ++z) o[i][z] = mul(o[i][z], both(shrink));
                }
            }
#pragma unroll
            for (int i = 0; i < kRowsEach; ++i) {
                const float base = m[i] == -INFINITY ? 0.f : -m[i] * c;
#pragma unroll
                for (int y = 0; y < 4; ++y) s[i][y] = ptx::ex2(fmaf(s[i][y], c, base));
                l[i] += (s[i][0] + s[i][1]) + (s[i][2] + s[i][3]);
            }
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                float4 v[kNarrow / 4];
#pragma unroll
                for (int z = 0; z < kNarrow / 4; ++z) v[z] = v4[(x + y) * (kNarrow / 4) + z];
#pragma unroll
                for (int i = 0; i < kRowsEach; ++i) {
#pragma unroll
                    for (int z = 0; z < kNarrow / 4; ++z) {
                        o[i][2 * z] = fma(both(s[i][y]), F2{v[z].x, v[z].y}, o[i][2 * z]);
                        o[i][2 * z + 1] = fma(both(s[i][y]), F2{v[z].z, v[z].w}, o[i][2 * z + 1]);
                    }
                }
            }
        }
        __syncthreads();
    }
    // each warp's maximum, sum and sums of values, [warp][field][row]; then a thread to a row
    float* box = reinterpret_cast<float*>(raw);
#pragma unroll
    for (int i = 0; i < kRowsEach; ++i) {
        float* to = box + warp * kRowFields * kRowTile + lane + 32 * i;
        to[0] = m[i];
        to[kRowTile] = l[i];
#pragma unroll
        for (int z = 0; z < kNarrow; ++z) to[(2 + z) * kRowTile] = z & 1 ? o[i][z / 2].y : o[i][z / 2].x;
    }
    __syncthreads();
    const int64_t row = t.row + tid;
    if (tid >= kRowTile || row >= t.end) return;
    float most = -INFINITY, total = 0.f, sum[kNarrow];
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) most = fmaxf(most, box[w * kRowFields * kRowTile + tid]);
#pragma unroll
    for (int z = 0; z < kNarrow; ++z) sum[z] = 0.f;
#pragma unroll
    for (int w = 0; w < kRowWarps; ++w) {
        const float* from = box + w * kRowFields * kRowTile + tid;
        const float f = from[0] == most ? 1.f : ptx::ex2((from[0] - most) * c);
        total = fmaf(f, from[kRowTile], total);
#pragma unroll
        for (int z = 0; z < kNarrow; ++z) sum[z] = fmaf(f, from[(2 + z) * kRowTile], sum[z]);
    }
    const float inv = total == 0.f ? 0.f : 1.f / total, lse = total == 0.f ? -INFINITY : (most * c + log2f(total)) * kLn2;
    const int64_t at = ((int64_t)blockIdx.z * a.nq + row) * a.hq + head;
    float* to = a.splits > 1 ? a.part + at * a.d : static_cast<float*>(a.o) + row * a.ldo + (int64_t)head * a.d;
    (a.splits > 1 ? a.part_lse[at] : a.lse[row * a.hq + head]) = lse;
#pragma unroll
    for (int z = 0; z < kNarrow; z += 4)
        if (z < a.d)  // no keys: a zero, whatever stands in the sums
            *reinterpret_cast<float4*>(to + z) = total == 0.f ? make_float4(0.f, 0.f, 0.f, 0.f)
                                                              : make_float4(sum[z] * inv, sum[z + 1] * inv, sum[z + 2] * inv, sum[z + 3] * inv);
}

// The scores' probabilities and their gradients of a tile, from s (and dp = do v^T), written to p and ds.
template <int DP, bool BY_Q>
__device__ __forceinline__ void tile_grad(const AttnArgs& a, const Mat<DP>& q, const Mat<DP>& k, const Mat<DP>& v, const Mat<DP>& g,
                                          int head, int64_t row, int64_t row_end, int64_t key, int64_t key_end, int ty, int tx,
                                          Probs* p, Probs& ds)
{
    float s[4][4], dp[4][4];
    dot<DP, true>(q, k, ty, tx, s);
    dot<DP, true>(g, v, ty, tx, dp);
    const float to_log2 = a.scale * kLog2e;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = row + 4 * ty + i;
        const bool there = r < row_end;
        const float lse = there ? fetch(a.lse2 + head * a.nq + r) : -INFINITY, delta = there ? fetch(a.delta + head * a.nq + r) : 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool in = there && key + tx + 16 * j < key_end && lse != -INFINITY;
            const float e = in ? ptx::ex2(s[i][j] * to_log2 + lse) : 0.f;
            if (!BY_Q) p->v[4 * ty + i][tx + 16 * j] = e;
            ds.v[4 * ty + i][tx + 16 * j] = in ? e * (dp[i][j] + delta) : 0.f;
        }
    }
}

// grid: slots of 64 queries, query heads, splits of the keys
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads, kBlocks<DP>)
k_attn_dq_simt(AttnArgs a)
{
    extern __shared__ float4 raw[];
    Mat<DP>& q = *reinterpret_cast<Mat<DP>*>(raw);
    Mat<DP>& k = *(&q + 1);
    Mat<DP>& v = *(&q + 2);
    Mat<DP>& g = *(&q + 3);
    Probs& ds = *reinterpret_cast<Probs*>(&q + 4);
    wait_for_kernel_before();
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) attn_check(a.seg_q, a.segments, a.nq, a.status, threadIdx.x, kThreads);
    AttnTile t;
    if (!attn_tile(a.seg_q, a.seg_k, a.segments, a.nq, a.nk, kTile, blockIdx.x, t)) return;
    const int head = blockIdx.y, kv = head / (a.hq / a.hk), tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    int64_t lo, hi;
    attn_share(t.lo, t.hi, kTile, blockIdx.z, a.splits, lo, hi);
    Out<DP> dq(tx);
    if (lo < hi) {
        load<T, DP>(q, a.q, a.ldq, head, a.d, t.row, t.end);
        load<T, DP>(g, a.dout, a.lddo, head, a.d, t.row, t.end);
    }
    for (int64_t at = lo; at < hi; at += kTile) {
        __syncthreads();
        load<T, DP>(k, a.k, a.ldk, kv, a.d, at, hi);
        load<T, DP>(v, a.v, a.ldv, kv, a.d, at, hi);
        __syncthreads();
        tile_grad<DP, true>(a, q, k, v, g, head, t.row, t.end, at, hi, ty, tx, nullptr, ds);
        __syncwarp();
        dq.rows_times(ds, k, ty);
    }
    const float mul[4] = {a.scale, a.scale, a.scale, a.scale};
    const int64_t width = (int64_t)a.hq * a.d;
    dq.template store<T>(mul, static_cast<T*>(a.dq) + (int64_t)head * a.d, a.lddq,
                         a.splits > 1 ? a.part + blockIdx.z * a.nq * width + (int64_t)head * a.d : nullptr, width, a.d, t.row, t.end, ty);
}

// grid: slots of 64 keys, key heads, splits of the queries (of all heads that share the keys, one after the other)
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads, kBlocks<DP>)
k_attn_dkv_simt(AttnArgs a)
{
    extern __shared__ float4 raw[];
    Mat<DP>& q = *reinterpret_cast<Mat<DP>*>(raw);
    Mat<DP>& k = *(&q + 1);
    Mat<DP>& v = *(&q + 2);
    Mat<DP>& g = *(&q + 3);
    Probs& p = *reinterpret_cast<Probs*>(&q + 4);
    Probs& ds = *(&p + 1);
    wait_for_kernel_before();
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) attn_check(a.seg_k, a.segments, a.nk, a.status, threadIdx.x, kThreads);
    AttnTile t;
    if (!attn_tile(a.seg_k, a.seg_q, a.segments, a.nk, a.nq, kTile, blockIdx.x, t)) return;
    const int kv = blockIdx.y, per = a.hq / a.hk, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    Out<DP> dk(tx), dv(tx);
    // the share of the tiles of all heads
    const int64_t tiles = (t.hi - t.lo + kTile - 1) / kTile, all = tiles * per;
    const int64_t from = all * blockIdx.z / a.splits_kv, to = all * (blockIdx.z + 1) / a.splits_kv;
    if (from < to) {
        load<T, DP>(k, a.k, a.ldk, kv, a.d, t.row, t.end);
        load<T, DP>(v, a.v, a.ldv, kv, a.d, t.row, t.end);
    }
    for (int64_t i = from; i < to; ++i) {
        const int head = kv * per + (int)(i / tiles);
        const int64_t at = t.lo + i % tiles * kTile;
        __syncthreads();
        load<T, DP>(q, a.q, a.ldq, head, a.d, at, t.hi);
        load<T, DP>(g, a.dout, a.lddo, head, a.d, at, t.hi);
        __syncthreads();
        tile_grad<DP, false>(a, q, k, v, g, head, at, t.hi, t.row, t.end, ty, tx, &p, ds);
        __syncthreads();
        dv.cols_times(p, g, ty);
        dk.cols_times(ds, q, ty);
    }
    const int64_t width = (int64_t)a.hk * a.d, part = (int64_t)a.nk * width;
    const float one[4] = {1.f, 1.f, 1.f, 1.f}, mul[4] = {a.scale, a.scale, a.scale, a.scale};
    float* part_k = a.splits_kv > 1 ? a.part_kv + blockIdx.z * part + (int64_t)kv * a.d : nullptr;
    dk.template store<T>(mul, static_cast<T*>(a.dk) + (int64_t)kv * a.d, a.lddk, part_k, width, a.d, t.row, t.end, ty);
    dv.template store<T>(one, static_cast<T*>(a.dv) + (int64_t)kv * a.d, a.lddv, part_k ? part_k + part * a.splits_kv : nullptr, width, a.d,
                         t.row, t.end, ty);
}

template <int DP> constexpr size_t kMat = sizeof(Mat<DP>);

template <typename T, int DP>
spc_status fwd(const AttnArgs& a, cudaStream_t st)
{
    const int64_t slots = attn_slots(a.nq, a.segments, kTile);
    if (slots > INT32_MAX) return SPC_ERR_UNSUPPORTED;
    return attn_start_kernel<k_attn_simt<T, DP>>(dim3((unsigned)slots, a.hq, a.splits), kThreads, 3 * kMat<DP> + sizeof(Probs), st, a);
}

template <typename T, int DP>
spc_status bwd(const AttnArgs& a, cudaStream_t st)
{
    const int64_t slots_q = attn_slots(a.nq, a.segments, kTile), slots_k = attn_slots(a.nk, a.segments, kTile);
    if (slots_q > INT32_MAX || slots_k > INT32_MAX) return SPC_ERR_UNSUPPORTED;
    if (a.nk > 0) {
        const spc_status s = attn_start_kernel<k_attn_dkv_simt<T, DP>>(dim3((unsigned)slots_k, a.hk, a.splits_kv), kThreads,
                                                                       4 * kMat<DP> + 2 * sizeof(Probs), st, a);
        if (s != SPC_OK) return s;
    }
    if (a.nq == 0) return SPC_OK;
    return attn_start_kernel<k_attn_dq_simt<T, DP>>(dim3((unsigned)slots_q, a.hq, a.splits), kThreads, 4 * kMat<DP> + sizeof(Probs), st, a);
}

// Whether the kernel of whole rows takes a forward call.
bool by_rows(const AttnArgs& a)
{
    const uintptr_t low = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
                          reinterpret_cast<uintptr_t>(a.o);
    return a.d <= kNarrow && a.d % 4 == 0 && low % 16 == 0 && (a.ldq | a.ldk | a.ldv | a.ldo) % 4 == 0 && a.nk > 0;
}

template <int R>
spc_status fwd_rows(const AttnArgs& a, cudaStream_t st)
{
    const int64_t slots = attn_slots(a.nq, a.segments, Rows<R>::kTile);
    if (slots > INT32_MAX) return SPC_ERR_UNSUPPORTED;
    return attn_start_kernel<k_attn_rows_simt<R>>(dim3((unsigned)slots, a.hq, a.splits), 32 * kRowWarps, Rows<R>::kSmem, st, a);
}

template <typename T>
spc_status any(const AttnArgs& a, bool backward, cudaStream_t st)
{
    if (sizeof(T) == 4 && !backward && by_rows(a)) return attn_rows_each(a.nq, a.nk, a.segments, a.hq) == 4 ? fwd_rows<4>(a, st) : fwd_rows<2>(a, st);
    if (a.d <= 16) return backward ? bwd<T, 16>(a, st) : fwd<T, 16>(a, st);
    if (a.d <= 32) return backward ? bwd<T, 32>(a, st) : fwd<T, 32>(a, st);
    if (a.d <= 64) return backward ? bwd<T, 64>(a, st) : fwd<T, 64>(a, st);
    return backward ? bwd<T, 128>(a, st) : fwd<T, 128>(a, st);
}

spc_status typed(const AttnArgs& a, spc_dtype dt, bool backward, cudaStream_t st)
{
    switch (dt) {
    case SPC_F32: return any<float>(a, backward, st);
    case SPC_F16: return any<__half>(a, backward, st);
    default: return any<__nv_bfloat16>(a, backward, st);
    }
}

}  // namespace

spc_status attention_fwd_simt(const AttnArgs& a, spc_dtype dt, cudaStream_t st) { return typed(a, dt, false, st); }
spc_status attention_bwd_simt(const AttnArgs& a, spc_dtype dt, cudaStream_t st) { return typed(a, dt, true, st); }

}  // namespace spc
