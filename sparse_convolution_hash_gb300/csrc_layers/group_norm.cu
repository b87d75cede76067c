// group_norm.cu -- group norm with an activation over the rows of each segment,
// and its gradients.
//
// One block per (group, segment) forms the sums, then a thread per element
// applies them.  The variance is summed around the mean, so features far from
// zero lose nothing.
#include "layers.cuh"

namespace spc {

namespace {

constexpr int kBlock = 256;

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

template <typename T>
__global__ void __launch_bounds__(kBlock) k_norm_stats(NormArgs a)
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
__global__ void __launch_bounds__(kBlock) k_norm_apply(NormArgs a)
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
__global__ void __launch_bounds__(kBlock) k_norm_bwd_sums(NormArgs a, float* __restrict__ part)
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

__global__ void __launch_bounds__(kBlock) k_norm_bwd_params(NormArgs a, const float* __restrict__ part)
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
__global__ void __launch_bounds__(kBlock) k_norm_bwd_apply(NormArgs a, const float* __restrict__ part)
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
spc_status fwd(const NormArgs& a, cudaStream_t st)
{
    k_norm_stats<T><<<dim3(a.groups, a.segments), kBlock, 0, st>>>(a);
    SPC_LAUNCH_CHECK();
    if (a.n == 0) return SPC_OK;
    const int64_t blocks = ceil_div(a.n * a.c, kBlock);
    if (blocks > INT32_MAX) return SPC_ERR_UNSUPPORTED;
    k_norm_apply<T><<<(unsigned)blocks, kBlock, 0, st>>>(a);
    SPC_LAUNCH_CHECK();
    return SPC_OK;
}

template <typename T>
spc_status bwd(const NormArgs& a, float* part, cudaStream_t st)
{
    k_norm_bwd_sums<T><<<dim3(a.c, a.segments), kBlock, 0, st>>>(a, part);
    SPC_LAUNCH_CHECK();
    if (a.dgamma || a.dbeta) {
        k_norm_bwd_params<<<(unsigned)ceil_div(a.c, kBlock), kBlock, 0, st>>>(a, part);
        SPC_LAUNCH_CHECK();
    }
    if (a.n == 0) return SPC_OK;
    const int64_t blocks = ceil_div(a.n * a.c, kBlock);
    if (blocks > INT32_MAX) return SPC_ERR_UNSUPPORTED;
    k_norm_bwd_apply<T><<<(unsigned)blocks, kBlock, 0, st>>>(a, part);
    SPC_LAUNCH_CHECK();
    return SPC_OK;
}

}  // namespace

size_t group_norm_ws_bytes(int64_t n, int32_t c, int32_t segments, int32_t groups, spc_dtype dt)
{
    (void)n;
    (void)groups;
    (void)dt;
    return align_up(sizeof(float) * 2 * (size_t)c * (size_t)segments, 256);
}

spc_status group_norm_fwd(const NormArgs& a, spc_dtype dt, void* ws, cudaStream_t st)
{
    (void)ws;
    switch (dt) {
    case SPC_F32: return fwd<float>(a, st);
    case SPC_F16: return fwd<__half>(a, st);
    default: return fwd<__nv_bfloat16>(a, st);
    }
}

spc_status group_norm_bwd(const NormArgs& a, spc_dtype dt, void* ws, cudaStream_t st)
{
    float* part = static_cast<float*>(ws);
    switch (dt) {
    case SPC_F32: return bwd<float>(a, part, st);
    case SPC_F16: return bwd<__half>(a, part, st);
    default: return bwd<__nv_bfloat16>(a, part, st);
    }
}

}  // namespace spc
