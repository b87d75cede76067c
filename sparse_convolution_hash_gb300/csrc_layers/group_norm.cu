// group_norm.cu -- group norm with an activation over the rows of each segment,
// and its gradients.
//
// Both passes need sums over a segment before they can write a row, so each reads its
// rows twice: a first kernel forms sums, a second applies them, walking its rows
// backwards so that it meets the ones the first kernel read last while they are still in
// L2.  One CTA per SM owns a run of consecutive positions in both.  A thread owns
// V neighbouring channels (16 bytes where the row length allows) of every RT-th row and
// keeps their parameters in registers.  The CTAs' sums over a segment
// that several share go to the workspace, and every CTA that needs them
// adds them in the order of the rows; a segment inside one CTA's run is finished there.
//
// Statistics: a thread sums d = x - p and d^2 around its own first value p, so a mean far
// from zero costs no digits; threads, channels and CTAs are merged as (count, mean,
// sum of squares around the mean), M2 = sum M2_i + sum n_i (mean_i - mean)^2.
// Gradients: with dz = dy act'(z), sums of dz and dz (x - mean) per channel give dgamma,
// dbeta and, weighted by gamma, the two means of a group; dx = A dz + B + D (x - mean).
#include "layers.cuh"

namespace spc {

namespace {

constexpr int kBlock = 256;      // of the kernels for very long rows
constexpr int kThreads = 512;    // of the others
constexpr int kUnroll = 4;       // rows of a thread in flight
constexpr int kMinRows = 64;     // positions of a CTA, at least

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T e[V];
};

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

__device__ __forceinline__ float activate(float z, int act)
{
    if (act == SPC_ACT_RELU) return z > 0.f || z != z ? z : 0.f;
    if (act == SPC_ACT_SILU) return z / (1.f + expf(-z));
    return z;
}

// act'(z)
__device__ __forceinline__ float slope(float z, int act)
{
    if (act == SPC_ACT_RELU) return z > 0.f ? 1.f : (z != z ? z : 0.f);
    if (act == SPC_ACT_SILU) {
        const float s = 1.f / (1.f + expf(-z));
        return s * (1.f + z * (1.f - s));
    }
    return 1.f;
}

// ------------------------------------------------- runs of consecutive positions
struct Run {
    int s;           // segment, -1: none
    int64_t lo, hi;  // its positions in this CTA's share
};

// The run that begins at position r of a share that ends at `end`.
__device__ __forceinline__ Run run_at(const NormArgs& a, int64_t r, int64_t end)
{
    Run k;
    k.s = segment_of(a.seg, a.segments, r);
    int64_t to = k.s >= a.segments ? a.n : __ldg(a.seg + k.s + 1);
    if (k.s >= a.segments) k.s = -1;
    to = to > r ? to : r + 1;  // offsets out of order: still forward
    k.lo = r;
    k.hi = to < end ? to : end;
    return k;
}

// The run that ends before position `end` of a share that begins at `begin`.
__device__ __forceinline__ Run run_before(const NormArgs& a, int64_t begin, int64_t end)
{
    Run k;
    k.s = segment_of(a.seg, a.segments, end - 1);
    int64_t from = k.s < 0 ? 0 : __ldg(a.seg + (k.s >= a.segments ? a.segments : k.s));
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
    __device__ __forceinline__ Span(const NormArgs& a, int s, int64_t rows)
    {
        segment_bounds(a.seg, s, a.n, nullptr, lo, hi);
        first = (int)(lo / rows);
        last = hi > lo ? (int)((hi - 1) / rows) : first;
    }
    __device__ __forceinline__ int64_t count(int c, int64_t rows) const
    {
        const int64_t b = c * rows > lo ? c * rows : lo, e = (c + 1) * rows < hi ? (c + 1) * rows : hi;
        return e - b;
    }
    // a share's part stands in its first slot if it begins with the share, else in its second
    __device__ __forceinline__ int slot(int c, int64_t rows) const { return 2 * c + (c == first && lo > c * rows ? 1 : 0); }
};

// Column sums over the RT row threads: v[j] of channel tv V + j ends in s[channel].
template <int V, int N>
__device__ __forceinline__ void column_sums(const float (&v)[N][V], float* s, int c, int tr, int tv, int rt)
{
    const int plane = rt * c;
    __syncthreads();
    if (tr < rt)
#pragma unroll
        for (int k = 0; k < N; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) s[k * plane + tr * c + tv * V + j] = v[k][j];
    int h = 1;
    while (h < rt) h <<= 1;
    for (h >>= 1; h; h >>= 1) {
        __syncthreads();
        if (tr < h && tr + h < rt)
#pragma unroll
            for (int k = 0; k < N; ++k)
#pragma unroll
                for (int j = 0; j < V; ++j)
                    s[k * plane + tr * c + tv * V + j] += s[k * plane + (tr + h) * c + tv * V + j];
    }
    __syncthreads();
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int d = 16; d; d >>= 1) v += __shfl_xor_sync(FULL_MASK, v, d);
    return v;
}

// Row of each of a thread's next kUnroll positions (-1: past the run, or out of range).
__device__ __forceinline__ void rows_of(const NormArgs& a, int64_t r, int rt, int64_t lo, int64_t hi, int64_t (&row)[kUnroll])
{
    int32_t v[kUnroll];
#pragma unroll
    for (int q = 0; q < kUnroll; ++q) {
        const int64_t p = r + (int64_t)q * rt;
        const bool in = p >= lo && p < hi;
        row[q] = in ? p : -1;
        v[q] = in && a.order ? __ldg(a.order + p) : 0;
    }
    if (!a.order) return;
#pragma unroll
    for (int q = 0; q < kUnroll; ++q)
        if (row[q] >= 0) {
            const bool good = v[q] >= 0 && v[q] < a.n;
            if (!good) set_status(a.status, SPC_ERR_ROW_INDEX);
            row[q] = good ? v[q] : -1;
        }
}

// ------------------------------------------------------------------- statistics
// part[slot][g] = (mean, M2) of a shared segment's part; whole segments end in mean, rstd.
template <typename T, int V>
__global__ void __launch_bounds__(kThreads, 1) k_norm_stats(NormArgs a, int64_t rows, float2* __restrict__ part)
{
    extern __shared__ float s_sum[];
    const int tid = threadIdx.x, vpr = a.c / V, rt = kThreads / vpr, tr = tid / vpr, tv = tid % vpr;
    const int per = a.c / a.groups, warp = tid >> 5, lane = tid & 31;
    float* s_mean = s_sum + rt * a.c;  // channel means
    const T* x = static_cast<const T*>(a.x) + tv * V;
    // offsets are checked, and empty segments finished, once
    for (int s = blockIdx.x * kThreads + tid; s < a.segments; s += gridDim.x * kThreads) {
        int64_t lo, hi;
        segment_bounds(a.seg, s, a.n, a.status, lo, hi);
        if (lo == hi)
            for (int g = 0; g < a.groups; ++g) {
                a.mean[(int64_t)s * a.groups + g] = 0.f;
                a.rstd[(int64_t)s * a.groups + g] = 1.f / sqrtf(a.eps);
            }
    }
    const int64_t begin = blockIdx.x * rows, end = begin + rows < a.n ? begin + rows : a.n;
    for (int64_t r0 = begin; r0 < end;) {
        const Run k = run_at(a, r0, end);
        r0 = k.hi;
        if (k.s < 0) continue;
        float pivot[V], s1[V], s2[V];
        int64_t count = 0;
#pragma unroll
        for (int j = 0; j < V; ++j) pivot[j] = s1[j] = s2[j] = 0.f;
        if (tr < rt)
            for (int64_t r = k.lo + tr; r < k.hi; r += (int64_t)kUnroll * rt) {
                int64_t row[kUnroll];
                rows_of(a, r, rt, k.lo, k.hi, row);
                Vec<T, V> v[kUnroll];
#pragma unroll
                for (int q = 0; q < kUnroll; ++q)
                    if (row[q] >= 0) v[q] = *reinterpret_cast<const Vec<T, V>*>(x + row[q] * a.c);
#pragma unroll
                for (int q = 0; q < kUnroll; ++q)
                    if (row[q] >= 0) {
                        if (count == 0)
#pragma unroll
                            for (int j = 0; j < V; ++j) pivot[j] = elem<T>::to_f32(v[q].e[j]);
                        ++count;
#pragma unroll
                        for (int j = 0; j < V; ++j) {
                            const float d = elem<T>::to_f32(v[q].e[j]) - pivot[j];
                            s1[j] += d;
                            s2[j] = fmaf(d, d, s2[j]);
                        }
                    }
            }
        // channel means around the run's first row, then squares around the channel means
        const float n = (float)(k.hi - k.lo), mine = (float)count;
        const int64_t row0 = row_at(a.order, k.lo, a.n, nullptr);
        float base[V], v1[1][V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            base[j] = tr < rt && row0 >= 0 ? elem<T>::to_f32(x[row0 * a.c + j]) : 0.f;
            v1[0][j] = fmaf(mine, pivot[j] - base[j], s1[j]);
        }
        column_sums<V, 1>(v1, s_sum, a.c, tr, tv, rt);
        if (tr == 0)
#pragma unroll
            for (int j = 0; j < V; ++j) s_mean[tv * V + j] = base[j] + s_sum[tv * V + j] / n;
        __syncthreads();
        if (tr < rt)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float m = count ? s1[j] / mine : 0.f, d = (pivot[j] - s_mean[tv * V + j]) + m;
                const float m2 = fmaf(-m, s1[j], s2[j]);
                v1[0][j] = count ? (m2 < 0.f ? 0.f : m2) + mine * d * d : 0.f;
            }
        column_sums<V, 1>(v1, s_sum, a.c, tr, tv, rt);
        // channels to groups, a warp each
        const Span span(a, k.s, rows);
        const bool whole = span.first == span.last;
        for (int g = warp; g < a.groups; g += kThreads / 32) {
            const float first = s_mean[g * per];
            float m = 0.f;
            for (int j = lane; j < per; j += 32) m += s_mean[g * per + j] - first;
            const float mean = first + warp_sum(m) / (float)per;
            float q = 0.f;
            for (int j = lane; j < per; j += 32) {
                const float d = s_mean[g * per + j] - mean;
                q += s_sum[g * per + j] + n * d * d;
            }
            q = warp_sum(q);
            if (lane == 0) {
                if (whole) {
                    a.mean[(int64_t)k.s * a.groups + g] = mean;
                    a.rstd[(int64_t)k.s * a.groups + g] = 1.f / sqrtf(q / (n * (float)per) + a.eps);
                } else {
                    part[(int64_t)span.slot(blockIdx.x, rows) * a.groups + g] = make_float2(mean, q);
                }
            }
        }
    }
}

// (mean, rstd) of segment s into s_stat [groups], from the parts where several CTAs
// share it; the CTA that holds its first position also writes them out.
__device__ __forceinline__ void join_stats(const NormArgs& a, int s, int64_t rows, const float2* part, float2* s_stat)
{
    const Span span(a, s, rows);
    const int per = a.c / a.groups, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    for (int g = warp; g < a.groups; g += kThreads / 32) {
        float mean, rstd;
        if (span.first == span.last) {
            mean = a.mean[(int64_t)s * a.groups + g];
            rstd = a.rstd[(int64_t)s * a.groups + g];
        } else {
            const float base = part[(int64_t)span.slot(span.first, rows) * a.groups + g].x;
            float m = 0.f;
            for (int c = span.first + lane; c <= span.last; c += 32)
                m += (float)span.count(c, rows) * (part[(int64_t)span.slot(c, rows) * a.groups + g].x - base);
            const float n = (float)(span.hi - span.lo);
            mean = base + warp_sum(m) / n;
            float q = 0.f;
            for (int c = span.first + lane; c <= span.last; c += 32) {
                const float2 v = part[(int64_t)span.slot(c, rows) * a.groups + g];
                const float d = v.x - mean;
                q += v.y + (float)span.count(c, rows) * (float)per * d * d;
            }
            rstd = 1.f / sqrtf(warp_sum(q) / (n * (float)per) + a.eps);
            if (lane == 0 && (int)blockIdx.x == span.first) {
                a.mean[(int64_t)s * a.groups + g] = mean;
                a.rstd[(int64_t)s * a.groups + g] = rstd;
            }
        }
        if (lane == 0) s_stat[g] = make_float2(mean, rstd);
    }
    __syncthreads();
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads, 1) k_norm_apply(NormArgs a, int64_t rows, const float2* __restrict__ part)
{
    extern __shared__ float2 s_stat[];
    const int tid = threadIdx.x, vpr = a.c / V, rt = kThreads / vpr, tr = tid / vpr, tv = tid % vpr;
    const int per = a.c / a.groups;
    const T* x = static_cast<const T*>(a.x) + tv * V;
    T* y = static_cast<T*>(a.out) + tv * V;
    const int64_t begin = blockIdx.x * rows, end = begin + rows < a.n ? begin + rows : a.n;
    for (int64_t r0 = end; r0 > begin;) {
        const Run k = run_before(a, begin, r0);
        r0 = k.lo;
        float mean[V], scale[V], shift[V];
        if (k.s >= 0) {
            join_stats(a, k.s, rows, part, s_stat);
            if (tr < rt)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const int ch = tv * V + j;
                    const float2 st = s_stat[ch / per];
                    mean[j] = st.x;
                    scale[j] = st.y * (a.gamma ? __ldg(a.gamma + ch) : 1.f);
                    shift[j] = a.beta ? __ldg(a.beta + ch) : 0.f;
                }
        }
        if (tr >= rt) continue;
        for (int64_t r = k.hi - 1 - tr; r >= k.lo; r -= (int64_t)kUnroll * rt) {
            int64_t row[kUnroll];
            rows_of(a, r, -rt, k.lo, k.hi, row);
            Vec<T, V> v[kUnroll];
            if (k.s >= 0)
#pragma unroll
                for (int q = 0; q < kUnroll; ++q)
                    if (row[q] >= 0) v[q] = *reinterpret_cast<const Vec<T, V>*>(x + row[q] * a.c);
#pragma unroll
            for (int q = 0; q < kUnroll; ++q)
                if (row[q] >= 0) {
                    Vec<T, V> o;
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        float z = 0.f;
                        if (k.s >= 0) z = activate(fmaf(elem<T>::to_f32(v[q].e[j]) - mean[j], scale[j], shift[j]), a.act);
                        o.e[j] = elem<T>::from_f32(z);
                    }
                    *reinterpret_cast<Vec<T, V>*>(y + row[q] * a.c) = o;
                }
        }
    }
}

// -------------------------------------------------------------------- gradients
// Sums over the rows of this CTA: total[c][0] of dz and [1] of dz xh per channel, and per segment
// and group (sum gamma dz, sum gamma dz xh): whole segments' in coef[s], parts in part[slot].
template <typename T, int V>
__global__ void __launch_bounds__(kThreads, 1)
k_norm_bwd_sums(NormArgs a, int64_t rows, float2* __restrict__ part, float2* __restrict__ coef, float* __restrict__ total)
{
    extern __shared__ float s_sum[];
    const int tid = threadIdx.x, vpr = a.c / V, rt = kThreads / vpr, tr = tid / vpr, tv = tid % vpr;
    const int per = a.c / a.groups, warp = tid >> 5, lane = tid & 31, plane = rt * a.c;
    const T* x = static_cast<const T*>(a.x) + tv * V;
    const T* dy = static_cast<const T*>(a.dy) + tv * V;
    for (int s = blockIdx.x * kThreads + tid; s < a.segments; s += gridDim.x * kThreads) {
        int64_t lo, hi;
        segment_bounds(a.seg, s, a.n, a.status, lo, hi);
    }
    const int64_t begin = blockIdx.x * rows, end = begin + rows < a.n ? begin + rows : a.n;
    float all[2][V];
#pragma unroll
    for (int j = 0; j < V; ++j) all[0][j] = all[1][j] = 0.f;
    for (int64_t r0 = begin; r0 < end;) {
        const Run k = run_at(a, r0, end);
        r0 = k.hi;
        if (k.s < 0) continue;
        float mean[V], scale[V], shift[V], rstd[V], sum[2][V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const int ch = tr < rt ? tv * V + j : 0;
            const int64_t i = (int64_t)k.s * a.groups + ch / per;
            mean[j] = __ldg(a.mean + i);
            rstd[j] = __ldg(a.rstd + i);
            scale[j] = rstd[j] * (a.gamma ? __ldg(a.gamma + ch) : 1.f);
            shift[j] = a.beta ? __ldg(a.beta + ch) : 0.f;
            sum[0][j] = sum[1][j] = 0.f;
        }
        if (tr < rt)
            for (int64_t r = k.lo + tr; r < k.hi; r += (int64_t)kUnroll * rt) {
                int64_t row[kUnroll];
                rows_of(a, r, rt, k.lo, k.hi, row);
                Vec<T, V> v[kUnroll], d[kUnroll];
#pragma unroll
                for (int q = 0; q < kUnroll; ++q)
                    if (row[q] >= 0) {
                        v[q] = *reinterpret_cast<const Vec<T, V>*>(x + row[q] * a.c);
                        d[q] = *reinterpret_cast<const Vec<T, V>*>(dy + row[q] * a.c);
                    }
#pragma unroll
                for (int q = 0; q < kUnroll; ++q)
                    if (row[q] >= 0)
#pragma unroll
                        for (int j = 0; j < V; ++j) {
                            const float e = elem<T>::to_f32(v[q].e[j]) - mean[j];
                            const float dz = elem<T>::to_f32(d[q].e[j]) * slope(fmaf(e, scale[j], shift[j]), a.act);
                            sum[0][j] += dz;
                            sum[1][j] = fmaf(dz, e, sum[1][j]);
                        }
            }
#pragma unroll
        for (int j = 0; j < V; ++j) sum[1][j] *= rstd[j];
        column_sums<V, 2>(sum, s_sum, a.c, tr, tv, rt);
        if (tr == 0)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                all[0][j] += s_sum[tv * V + j];
                all[1][j] += s_sum[plane + tv * V + j];
            }
        const Span span(a, k.s, rows);
        for (int g = warp; g < a.groups; g += kThreads / 32) {
            float m0 = 0.f, m1 = 0.f;
            for (int j = lane; j < per; j += 32) {
                const float w = a.gamma ? __ldg(a.gamma + g * per + j) : 1.f;
                m0 = fmaf(w, s_sum[g * per + j], m0);
                m1 = fmaf(w, s_sum[plane + g * per + j], m1);
            }
            m0 = warp_sum(m0);
            m1 = warp_sum(m1);
            if (lane == 0) {
                if (span.first == span.last) coef[(int64_t)k.s * a.groups + g] = make_float2(m0, m1);
                else part[(int64_t)span.slot(blockIdx.x, rows) * a.groups + g] = make_float2(m0, m1);
            }
        }
    }
    if (tr == 0)
#pragma unroll
        for (int j = 0; j < V; ++j) {
            total[(int64_t)blockIdx.x * 2 * a.c + tv * V + j] = all[0][j];
            total[((int64_t)blockIdx.x * 2 + 1) * a.c + tv * V + j] = all[1][j];
        }
}

template <typename T, int V>
__global__ void __launch_bounds__(kThreads, 1)
k_norm_bwd_apply(NormArgs a, int64_t rows, const float2* __restrict__ part, const float2* __restrict__ coef,
                 const float* __restrict__ total)
{
    extern __shared__ float2 s_stat[];
    const int tid = threadIdx.x, vpr = a.c / V, rt = kThreads / vpr, tr = tid / vpr, tv = tid % vpr;
    const int per = a.c / a.groups, warp = tid >> 5, lane = tid & 31;
    const T* x = static_cast<const T*>(a.x) + tv * V;
    const T* dy = static_cast<const T*>(a.dy) + tv * V;
    T* dx = static_cast<T*>(a.out) + tv * V;
    const int64_t begin = blockIdx.x * rows, end = begin + rows < a.n ? begin + rows : a.n;
    for (int64_t r0 = end; r0 > begin;) {
        const Run k = run_before(a, begin, r0);
        r0 = k.lo;
        float mean[V], scale[V], shift[V], lift[V], tilt[V];
        if (k.s >= 0) {
            const Span span(a, k.s, rows);
            __syncthreads();
            for (int g = warp; g < a.groups; g += kThreads / 32) {
                float2 m = make_float2(0.f, 0.f);
                if (span.first == span.last) {
                    m = coef[(int64_t)k.s * a.groups + g];
                } else {
                    for (int c = span.first + lane; c <= span.last; c += 32) {
                        const float2 v = part[(int64_t)span.slot(c, rows) * a.groups + g];
                        m.x += v.x;
                        m.y += v.y;
                    }
                    m.x = warp_sum(m.x);
                    m.y = warp_sum(m.y);
                }
                const float n = (float)(span.hi - span.lo) * (float)per;
                if (lane == 0) s_stat[g] = make_float2(m.x / n, m.y / n);
            }
            __syncthreads();
            if (tr < rt)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const int ch = tv * V + j;
                    const int64_t i = (int64_t)k.s * a.groups + ch / per;
                    const float rstd = __ldg(a.rstd + i);
                    const float2 m = s_stat[ch / per];
                    mean[j] = __ldg(a.mean + i);
                    scale[j] = rstd * (a.gamma ? __ldg(a.gamma + ch) : 1.f);
                    shift[j] = a.beta ? __ldg(a.beta + ch) : 0.f;
                    lift[j] = -rstd * m.x;
                    tilt[j] = -rstd * rstd * m.y;
                }
        }
        if (tr >= rt) continue;
        for (int64_t r = k.hi - 1 - tr; r >= k.lo; r -= (int64_t)kUnroll * rt) {
            int64_t row[kUnroll];
            rows_of(a, r, -rt, k.lo, k.hi, row);
            Vec<T, V> v[kUnroll], d[kUnroll];
            if (k.s >= 0)
#pragma unroll
                for (int q = 0; q < kUnroll; ++q)
                    if (row[q] >= 0) {
                        v[q] = *reinterpret_cast<const Vec<T, V>*>(x + row[q] * a.c);
                        d[q] = *reinterpret_cast<const Vec<T, V>*>(dy + row[q] * a.c);
                    }
#pragma unroll
            for (int q = 0; q < kUnroll; ++q)
                if (row[q] >= 0) {
                    Vec<T, V> o;
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        float g = 0.f;
                        if (k.s >= 0) {
                            const float e = elem<T>::to_f32(v[q].e[j]) - mean[j];
                            const float dz = elem<T>::to_f32(d[q].e[j]) * slope(fmaf(e, scale[j], shift[j]), a.act);
                            g = fmaf(dz, scale[j], fmaf(e, tilt[j], lift[j]));
                        }
                        o.e[j] = elem<T>::from_f32(g);
                    }
                    *reinterpret_cast<Vec<T, V>*>(dx + row[q] * a.c) = o;
                }
        }
    }
    // dgamma and dbeta: a warp for each channel
    if (a.dgamma || a.dbeta)
        for (int ch = blockIdx.x * (kThreads / 32) + warp; ch < a.c; ch += gridDim.x * (kThreads / 32)) {
            float s0 = 0.f, s1 = 0.f;
            for (int c = lane; c < (int)gridDim.x; c += 32) {
                s0 += total[(int64_t)c * 2 * a.c + ch];
                s1 += total[((int64_t)c * 2 + 1) * a.c + ch];
            }
            s0 = warp_sum(s0);
            s1 = warp_sum(s1);
            if (lane == 0 && a.dbeta) a.dbeta[ch] = s0;
            if (lane == 0 && a.dgamma) a.dgamma[ch] = s1;
        }
}

// ------------------------------------------- rows of more than kThreads vectors
// One block per (group, segment), then a thread per element.
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
    float v = 0.f;
    for (int64_t e = threadIdx.x; e < total; e += kBlock) v += at(e);
    const float mean = block_sum(v) / count;
    v = 0.f;
    for (int64_t e = threadIdx.x; e < total; e += kBlock) {
        const float d = at(e) - mean;
        v += d * d;
    }
    const float var = block_sum(v) / count;
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
    const uintptr_t bits = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.out) |
                           reinterpret_cast<uintptr_t>(a.dy);
    int v = 16 / (int)sizeof(T);
    while (v > 1 && (a.c % v != 0 || (bits & (v * sizeof(T) - 1)) != 0)) v /= 2;
    return v;
}

int shares_of(int64_t n) { return (int)std::max<int64_t>(1, std::min<int64_t>(sm_count(), ceil_div(n, kMinRows))); }

struct Ws {
    float2* part;   // [2 shares][groups]
    float2* coef;   // [segments][groups]
    float* total;   // [shares][2][c]
};

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

template <typename T, int V>
spc_status fwd_rows(const NormArgs& a, const Ws& w, cudaStream_t st)
{
    const int shares = shares_of(a.n), rt = kThreads / (a.c / V);
    const int64_t rows = std::max<int64_t>(1, ceil_div(a.n, shares));
    k_norm_stats<T, V><<<shares, kThreads, sizeof(float) * (rt + 1) * a.c, st>>>(a, rows, w.part);
    SPC_LAUNCH_CHECK();
    if (a.n == 0) return SPC_OK;
    k_norm_apply<T, V><<<shares, kThreads, sizeof(float2) * a.groups, st>>>(a, rows, w.part);
    SPC_LAUNCH_CHECK();
    return SPC_OK;
}

template <typename T, int V>
spc_status bwd_rows(const NormArgs& a, const Ws& w, cudaStream_t st)
{
    const int shares = shares_of(a.n), rt = kThreads / (a.c / V);
    const int64_t rows = std::max<int64_t>(1, ceil_div(a.n, shares));
    k_norm_bwd_sums<T, V><<<shares, kThreads, sizeof(float) * 2 * rt * a.c, st>>>(a, rows, w.part, w.coef, w.total);
    SPC_LAUNCH_CHECK();
    k_norm_bwd_apply<T, V><<<shares, kThreads, sizeof(float2) * a.groups, st>>>(a, rows, w.part, w.coef, w.total);
    SPC_LAUNCH_CHECK();
    return SPC_OK;
}

template <typename T>
spc_status run(const NormArgs& a, void* ws, bool backward, cudaStream_t st)
{
    const int v = vector_of<T>(a);
    Ws w;
    carve(a.n, a.c, a.segments, a.groups, static_cast<char*>(ws), &w);
    if (a.c / v > kThreads) return backward ? bwd_wide<T>(a, static_cast<float*>(ws), st) : fwd_wide<T>(a, st);
    if constexpr (sizeof(T) == 2)
        if (v == 8) return backward ? bwd_rows<T, 8>(a, w, st) : fwd_rows<T, 8>(a, w, st);
    if (v == 4) return backward ? bwd_rows<T, 4>(a, w, st) : fwd_rows<T, 4>(a, w, st);
    if (v == 2) return backward ? bwd_rows<T, 2>(a, w, st) : fwd_rows<T, 2>(a, w, st);
    return backward ? bwd_rows<T, 1>(a, w, st) : fwd_rows<T, 1>(a, w, st);
}

spc_status dispatch(const NormArgs& a, spc_dtype dt, void* ws, bool backward, cudaStream_t st)
{
    switch (dt) {
    case SPC_F32: return run<float>(a, ws, backward, st);
    case SPC_F16: return run<__half>(a, ws, backward, st);
    default: return run<__nv_bfloat16>(a, ws, backward, st);
    }
}

}  // namespace

size_t group_norm_ws_bytes(int64_t n, int32_t c, int32_t segments, int32_t groups, spc_dtype dt)
{
    (void)dt;
    // rows of more than kThreads vectors keep two sums per segment and channel instead
    const size_t wide = c > kThreads ? align_up(sizeof(float) * 2 * (size_t)c * (size_t)segments, 256) : 0;
    return std::max(carve(n, c, segments, groups, nullptr, nullptr), wide);
}

spc_status group_norm_fwd(const NormArgs& a, spc_dtype dt, void* ws, cudaStream_t st)
{
    return dispatch(a, dt, ws, false, st);
}

spc_status group_norm_bwd(const NormArgs& a, spc_dtype dt, void* ws, cudaStream_t st)
{
    return dispatch(a, dt, ws, true, st);
}

}  // namespace spc
