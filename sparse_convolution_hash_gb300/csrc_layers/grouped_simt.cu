// grouped_simt.cu -- products grouped by segment on CUDA cores: fp32 in full fp32
// multiplies, and the 16-bit shapes that the tensor-core kernels do not take.
//
// A block computes 64 positions x 64 columns of one segment, 4 x 4 per thread,
// 16 of the reduction at a time through shared memory.  Segment sizes are known
// on the device only, so the grid covers the most row tiles there can be (one
// partial tile per segment) and each block finds its segment in `seg`.
#include "layers.cuh"

namespace spc {

namespace {

constexpr int kTile = 64, kStep = 16, kBlock = 256;

// Row tile t of the positions: those of the segments in turn, between them the
// positions before the first and after the last (segment -1).  False past the last tile.
__device__ bool find_tile(const int32_t* seg, int segments, int64_t m, int64_t t, int32_t* status,
                          int& g, int64_t& lo, int64_t& hi)
{
    const int lane = threadIdx.x & 31;
    int64_t done = 0;
    for (int v0 = 0; v0 < segments + 2; v0 += 32) {
        const int v = v0 + lane;
        int64_t a = 0, b = 0;
        if (v == 0) {
            const int64_t f = __ldg(seg);
            b = f < 0 ? 0 : (f > m ? m : f);
        } else if (v <= segments) {
            segment_bounds(seg, v - 1, m, status, a, b);
        } else if (v == segments + 1) {
            const int64_t f = __ldg(seg + segments);
            a = f < 0 ? 0 : (f > m ? m : f);
            b = m;
        }
        const int64_t tiles = (b - a + kTile - 1) / kTile;
        int64_t inc = tiles;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t u = __shfl_up_sync(FULL_MASK, inc, d);
            if (lane >= d) inc += u;
        }
        const unsigned hit = __ballot_sync(FULL_MASK, t < done + inc);
        if (hit) {
            const int src = __ffs(hit) - 1;
            const int64_t first = __shfl_sync(FULL_MASK, done + inc - tiles, src);
            a = __shfl_sync(FULL_MASK, a, src);
            b = __shfl_sync(FULL_MASK, b, src);
            const int w = v0 + src;
            g = w == 0 || w == segments + 1 ? -1 : w - 1;
            lo = a + (t - first) * kTile;
            hi = lo + kTile < b ? lo + kTile : b;
            return true;
        }
        done += __shfl_sync(FULL_MASK, inc, 31);
    }
    return false;
}

template <typename T>
__global__ void __launch_bounds__(kBlock) k_grouped_simt(GroupedArgs a)
{
    __shared__ float s_a[kStep][kTile + 4], s_b[kStep][kTile + 4];
    __shared__ int32_t s_row[kTile];
    int g;
    int64_t lo, hi;
    if (!find_tile(a.seg, a.segments, a.m, blockIdx.x, a.status, g, lo, hi)) return;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int n0 = blockIdx.y * kTile;
    if (tid < kTile) s_row[tid] = lo + tid < hi ? (int32_t)row_at(a.in_rows, lo + tid, a.in_n, a.status) : -1;
    __syncthreads();
    const T* in = static_cast<const T*>(a.in);
    const T* w = static_cast<const T*>(a.w) + (int64_t)(g < 0 ? 0 : g) * a.k * a.n;
    float acc[4][4] = {};
    for (int k0 = 0; k0 < (g < 0 ? 0 : a.k); k0 += kStep) {
#pragma unroll
        for (int e = tid; e < kTile * kStep; e += kBlock) {
            const int r = e / kStep, k = k0 + e % kStep;
            const int32_t row = s_row[r];
            s_a[e % kStep][r] = row >= 0 && k < a.k ? elem<T>::to_f32(in[(int64_t)row * a.k + k]) : 0.f;
        }
#pragma unroll
        for (int e = tid; e < kTile * kStep; e += kBlock) {
            if (a.w_transposed) {
                const int j = e / kStep, k = k0 + e % kStep;
                s_b[e % kStep][j] = n0 + j < a.n && k < a.k ? elem<T>::to_f32(w[(int64_t)(n0 + j) * a.k + k]) : 0.f;
            } else {
                const int j = e % kTile, k = k0 + e / kTile;
                s_b[e / kTile][j] = n0 + j < a.n && k < a.k ? elem<T>::to_f32(w[(int64_t)k * a.n + n0 + j]) : 0.f;
            }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kStep; ++k) {
            float u[4], v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                u[i] = s_a[k][ty * 4 + i];
                v[i] = s_b[k][tx * 4 + i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(u[i], v[j], acc[i][j]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = lo + ty * 4 + i;
        if (r >= hi) break;
        const int64_t row = row_at(a.out_rows, r, a.m, a.status);
        if (row < 0) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = n0 + tx * 4 + j;
            if (n < a.n) static_cast<T*>(a.out)[row * a.n + n] = elem<T>::from_f32(acc[i][j]);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kBlock) k_grouped_wgrad_simt(GroupedWgradArgs a)
{
    __shared__ float s_a[kStep][kTile + 4], s_b[kStep][kTile + 4];
    __shared__ int32_t s_row[2][kStep];
    const int g = blockIdx.z, c0 = blockIdx.y * kTile, n0 = blockIdx.x * kTile;
    int64_t lo, hi;
    segment_bounds(a.seg, g, a.m, a.status, lo, hi);
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const T* x = static_cast<const T*>(a.x);
    const T* dy = static_cast<const T*>(a.dy);
    float acc[4][4] = {};
    for (int64_t r0 = lo; r0 < hi; r0 += kStep) {
        if (tid < 2 * kStep) {
            const int64_t r = r0 + tid % kStep;
            const bool first = tid < kStep;
            s_row[first ? 0 : 1][tid % kStep] =
                r < hi ? (int32_t)row_at(first ? a.x_rows : a.y_rows, r, first ? a.n_x : a.n_y, a.status) : -1;
        }
        __syncthreads();
#pragma unroll
        for (int e = tid; e < kTile * kStep; e += kBlock) {
            const int q = e / kTile, j = e % kTile;
            const int32_t xr = s_row[0][q], yr = s_row[1][q];
            const bool both = xr >= 0 && yr >= 0;
            s_a[q][j] = both && c0 + j < a.cin ? elem<T>::to_f32(x[(int64_t)xr * a.cin + c0 + j]) : 0.f;
            s_b[q][j] = both && n0 + j < a.cout ? elem<T>::to_f32(dy[(int64_t)yr * a.cout + n0 + j]) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kStep; ++k) {
            float u[4], v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                u[i] = s_a[k][ty * 4 + i];
                v[i] = s_b[k][tx * 4 + i];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(u[i], v[j], acc[i][j]);
        }
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = c0 + ty * 4 + i, n = n0 + tx * 4 + j;
            if (c < a.cin && n < a.cout) a.dw[((int64_t)g * a.cin + c) * a.cout + n] = acc[i][j];
        }
}

}  // namespace

spc_status grouped_simt(const GroupedArgs& a, spc_dtype dt, cudaStream_t st)
{
    const int64_t tiles = a.m / kTile + a.segments + 2, cols = ceil_div(a.n, kTile);
    if (cols > 65535) return SPC_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)tiles, (unsigned)cols);
    switch (dt) {
    case SPC_F32: k_grouped_simt<float><<<grid, kBlock, 0, st>>>(a); break;
    case SPC_F16: k_grouped_simt<__half><<<grid, kBlock, 0, st>>>(a); break;
    default: k_grouped_simt<__nv_bfloat16><<<grid, kBlock, 0, st>>>(a); break;
    }
    SPC_LAUNCH_CHECK();
    return SPC_OK;
}

spc_status grouped_wgrad_simt(const GroupedWgradArgs& a, spc_dtype dt, cudaStream_t st)
{
    const int64_t rows = ceil_div(a.cin, kTile);
    if (rows > 65535) return SPC_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)ceil_div(a.cout, kTile), (unsigned)rows, (unsigned)a.segments);
    switch (dt) {
    case SPC_F32: k_grouped_wgrad_simt<float><<<grid, kBlock, 0, st>>>(a); break;
    case SPC_F16: k_grouped_wgrad_simt<__half><<<grid, kBlock, 0, st>>>(a); break;
    default: k_grouped_wgrad_simt<__nv_bfloat16><<<grid, kBlock, 0, st>>>(a); break;
    }
    SPC_LAUNCH_CHECK();
    return SPC_OK;
}

}  // namespace spc
