// attention_simt.cu -- attention over segments on CUDA cores: fp32 (full fp32 products), and 16-bit heads that the
// tensor-core kernels do not take (channels not a multiple of 8, rows off a 16-byte boundary, no rows on one side).
//
// 64 x 64 tiles of scores by 256 threads, 4 x 4 a thread, operands as fp32 in shared memory.  The forward pass
// keeps a running maximum and sum per row; the gradients take the probabilities from the forward's
// log-sum and are two kernels, one that walks over the queries for dk and dv and one over the keys for dq, so every
// sum has its place and its order and there are no atomics.  A tile's walk may be split (see attention.cu);
// then fp32 parts go to the workspace.
// Bound by the FMA units and shared memory together: 64 multiply-adds stand against eight 16-byte reads.
#include "attention.cuh"

namespace spc {

namespace {

constexpr int kThreads = 256, kTile = 64, kPad = 4;

template <int DP> struct Mat { float v[kTile][DP + kPad]; };
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
template <int DP>
__device__ __forceinline__ void dot(const Mat<DP>& a, const Mat<DP>& b, int ty, int tx, float (&s)[4][4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
    }
#pragma unroll 4
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
                s[i][j] = fmaf(x[i].x, y[j].x, s[i][j]);
                s[i][j] = fmaf(x[i].y, y[j].y, s[i][j]);
                s[i][j] = fmaf(x[i].z, y[j].z, s[i][j]);
                s[i][j] = fmaf(x[i].w, y[j].w, s[i][j]);
            }
        }
    }
}

// acc[i][:] += sum over k of p[4 ty + i][k] b[k][this thread's channels]: DP / 16 neighbouring ones
template <int DP>
__device__ __forceinline__ void rows_times(const Probs& p, const Mat<DP>& b, int ty, int tx, float (&acc)[4][DP / 16])
{
    constexpr int W = DP / 16;
#pragma unroll 2
    for (int k = 0; k < kTile; k += 4) {
        float4 w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(&p.v[4 * ty + i][k]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float y[W];
#pragma unroll
            for (int c = 0; c < W; ++c) y[c] = b.v[k + q][tx * W + c];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float u = q == 0 ? w[i].x : q == 1 ? w[i].y : q == 2 ? w[i].z : w[i].w;
#pragma unroll
                for (int c = 0; c < W; ++c) acc[i][c] = fmaf(u, y[c], acc[i][c]);
            }
        }
    }
}

// acc[i][:] += sum over r of p[r][4 ty + i] b[r][this thread's channels]
template <int DP>
__device__ __forceinline__ void cols_times(const Probs& p, const Mat<DP>& b, int ty, int tx, float (&acc)[4][DP / 16])
{
    constexpr int W = DP / 16;
#pragma unroll 4
    for (int r = 0; r < kTile; ++r) {
        const float4 w = *reinterpret_cast<const float4*>(&p.v[r][4 * ty]);
        float y[W];
#pragma unroll
        for (int c = 0; c < W; ++c) y[c] = b.v[r][tx * W + c];
#pragma unroll
        for (int c = 0; c < W; ++c) {
            acc[0][c] = fmaf(w.x, y[c], acc[0][c]);
            acc[1][c] = fmaf(w.y, y[c], acc[1][c]);
            acc[2][c] = fmaf(w.z, y[c], acc[2][c]);
            acc[3][c] = fmaf(w.w, y[c], acc[3][c]);
        }
    }
}

// Four rows of results from row + 4 ty on, scaled, as T or (split) as fp32.
template <typename T, int W>
__device__ __forceinline__ void store(const float (&acc)[4][W], const float (&mul)[4], T* out, int64_t ld, float* part,
                                      int64_t part_ld, int d, int64_t row, int64_t end, int ty, int tx)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = row + 4 * ty + i;
        if (r >= end) break;
#pragma unroll
        for (int c = 0; c < W; ++c) {
            const int col = tx * W + c;
            if (col >= d) break;
            const float v = acc[i][c] * mul[i];
            if (part) part[r * part_ld + col] = v;
            else out[r * ld + col] = elem<T>::from_f32(v);
        }
    }
}

// grid: slots of 64 queries, query heads, splits of the keys
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads)
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
    float m[4], l[4], o[4][DP / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.f;
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) o[i][c] = 0.f;
    }
    if (lo < hi) load<T, DP>(q, a.q, a.ldq, head, a.d, t.row, t.end);
    for (int64_t at = lo; at < hi; at += kTile) {
        __syncthreads();
        load<T, DP>(k, a.k, a.ldk, kv, a.d, at, hi);
        load<T, DP>(v, a.v, a.ldv, kv, a.d, at, hi);
        __syncthreads();
        float s[4][4];
        dot<DP>(q, k, ty, tx, s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float most = m[i];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                s[i][j] = at + tx + 16 * j < hi ? s[i][j] * to_log2 : -INFINITY;
                most = fmaxf(most, s[i][j]);
            }
#pragma unroll
            for (int x = 8; x; x >>= 1) most = fmaxf(most, __shfl_xor_sync(FULL_MASK, most, x));
            const float base = most == -INFINITY ? 0.f : most, shrink = ptx::ex2(m[i] - base);
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float e = ptx::ex2(s[i][j] - base);
                sum += e;
                p.v[4 * ty + i][tx + 16 * j] = e;
            }
            l[i] = l[i] * shrink + sum;  // of this thread's columns: they join at the end
            m[i] = most;
#pragma unroll
            for (int c = 0; c < DP / 16; ++c) o[i][c] *= shrink;
        }
        __syncwarp();  // a row of p is written and read by the same half warp
        rows_times<DP>(p, v, ty, tx, o);
    }
    float mul[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int x = 8; x; x >>= 1) l[i] += __shfl_xor_sync(FULL_MASK, l[i], x);
        mul[i] = l[i] == 0.f ? 0.f : 1.f / l[i];
        if (l[i] == 0.f) {  // no keys: a zero, whatever stands in the sums
#pragma unroll
            for (int c = 0; c < DP / 16; ++c) o[i][c] = 0.f;
        }
        const int64_t r = t.row + 4 * ty + i;
        if (tx == 0 && r < t.end) {
            const float lse = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
            if (a.splits > 1) a.part_lse[(blockIdx.z * a.nq + r) * a.hq + head] = lse;
            else a.lse[r * a.hq + head] = lse;
        }
    }
    const int64_t width = (int64_t)a.hq * a.d;
    store<T, DP / 16>(o, mul, static_cast<T*>(a.o) + (int64_t)head * a.d, a.ldo,
                      a.splits > 1 ? a.part + blockIdx.z * a.nq * width + (int64_t)head * a.d : nullptr, width, a.d, t.row, t.end,
                      ty, tx);
}

// The scores' probabilities and their gradients of a tile, from s (and dp = do v^T), written to p and ds.
template <int DP, bool BY_Q>
__device__ __forceinline__ void tile_grad(const AttnArgs& a, const Mat<DP>& q, const Mat<DP>& k, const Mat<DP>& v, const Mat<DP>& g,
                                          int head, int64_t row, int64_t row_end, int64_t key, int64_t key_end, int ty, int tx,
                                          Probs* p, Probs& ds)
{
    float s[4][4], dp[4][4];
    dot<DP>(q, k, ty, tx, s);
    dot<DP>(g, v, ty, tx, dp);
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
__global__ void __launch_bounds__(kThreads)
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
    float dq[4][DP / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) dq[i][c] = 0.f;
    }
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
        rows_times<DP>(ds, k, ty, tx, dq);
    }
    const float mul[4] = {a.scale, a.scale, a.scale, a.scale};
    const int64_t width = (int64_t)a.hq * a.d;
    store<T, DP / 16>(dq, mul, static_cast<T*>(a.dq) + (int64_t)head * a.d, a.lddq,
                      a.splits > 1 ? a.part + blockIdx.z * a.nq * width + (int64_t)head * a.d : nullptr, width, a.d, t.row, t.end,
                      ty, tx);
}

// grid: slots of 64 keys, key heads, splits of the queries (of all heads that share the keys, one after the other)
template <typename T, int DP>
__global__ void __launch_bounds__(kThreads)
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
    float dk[4][DP / 16], dv[4][DP / 16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int c = 0; c < DP / 16; ++c) dk[i][c] = dv[i][c] = 0.f;
    }
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
        cols_times<DP>(p, g, ty, tx, dv);
        cols_times<DP>(ds, q, ty, tx, dk);
    }
    const int64_t width = (int64_t)a.hk * a.d, part = (int64_t)a.nk * width;
    const float one[4] = {1.f, 1.f, 1.f, 1.f}, mul[4] = {a.scale, a.scale, a.scale, a.scale};
    float* part_k = a.splits_kv > 1 ? a.part_kv + blockIdx.z * part + (int64_t)kv * a.d : nullptr;
    store<T, DP / 16>(dk, mul, static_cast<T*>(a.dk) + (int64_t)kv * a.d, a.lddk, part_k, width, a.d, t.row, t.end, ty, tx);
    store<T, DP / 16>(dv, one, static_cast<T*>(a.dv) + (int64_t)kv * a.d, a.lddv, part_k ? part_k + part * a.splits_kv : nullptr, width,
                      a.d, t.row, t.end, ty, tx);
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

template <typename T>
spc_status any(const AttnArgs& a, bool backward, cudaStream_t st)
{
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
