// dropout.cu -- y = residual + keep(x) / (1 - p) with a mask that is a function
// of the element's index.
//
// Word i % 4 of block i / 4 of Philox4x32-10 (Salmon, Moraes, Dror, Shaw, SC
// 2011) decides element i: ten rounds of two 32 x 32 -> 64 multiplications, a
// Feistel exchange of their halves, and two round keys that advance by the
// published constants.  Four elements share one block, so a thread owns whole
// groups of four.
#include <math.h>

#include "layers.cuh"

namespace spc {

namespace {

constexpr int kBlock = 256;

struct Words {
    uint32_t w[4];
};

__device__ __forceinline__ Words philox10(uint64_t block, uint64_t offset, uint64_t seed)
{
    uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32);
    uint32_t c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t p0 = (uint64_t)0xD2511F53u * c0, p1 = (uint64_t)0xCD9E8D57u * c2;
        c0 = (uint32_t)(p1 >> 32) ^ c1 ^ k0;
        c2 = (uint32_t)(p0 >> 32) ^ c3 ^ k1;
        c1 = (uint32_t)p1;
        c3 = (uint32_t)p0;
        k0 += 0x9E3779B9u;
        k1 += 0xBB67AE85u;
    }
    return Words{{c0, c1, c2, c3}};
}

// any: the drop probability is not 0; last: the largest word that drops.
template <typename T>
__global__ void __launch_bounds__(kBlock)
k_dropout(const T* x, const T* residual, int64_t n, uint32_t last, bool any, float scale,
          const uint64_t* __restrict__ rng, T* y)
{
    const int64_t q = (int64_t)blockIdx.x * kBlock + threadIdx.x;
    if (q * 4 >= n) return;
    const Words r = philox10((uint64_t)q, rng[1], rng[0]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t i = q * 4 + j;
        if (i >= n) break;
        const bool drop = any && r.w[j] <= last;
        float v = drop ? 0.f : elem<T>::to_f32(x[i]) * scale;
        if (residual) v += elem<T>::to_f32(residual[i]);
        y[i] = elem<T>::from_f32(v);
    }
}

template <typename T>
spc_status launch(const void* x, const void* residual, int64_t n, uint32_t last, bool any, float scale,
                  const uint64_t* rng, void* y, cudaStream_t st)
{
    const int64_t blocks = ceil_div(ceil_div(n, 4), kBlock);
    if (blocks > INT32_MAX) return SPC_ERR_UNSUPPORTED;
    k_dropout<T><<<(unsigned)blocks, kBlock, 0, st>>>(
        static_cast<const T*>(x), static_cast<const T*>(residual), n, last, any, scale, rng,
        static_cast<T*>(y));
    SPC_LAUNCH_CHECK();
    return SPC_OK;
}

}  // namespace

spc_status dropout(const void* x, const void* residual, int64_t n, double p, const uint64_t* rng,
                   spc_dtype dt, void* y, cudaStream_t st)
{
    if (n == 0) return SPC_OK;
    // drop when word < round(p 2^32), a number up to 2^32: kept as the last word
    // that drops, so that p = 1 fits 32 bits
    const uint64_t threshold = (uint64_t)nearbyint(p * 4294967296.0);
    const bool any = threshold > 0;
    const uint32_t last = any ? (uint32_t)(threshold - 1) : 0u;
    const float scale = p < 1.0 ? (float)(1.0 / (1.0 - p)) : 0.f;
    switch (dt) {
    case SPC_F32: return launch<float>(x, residual, n, last, any, scale, rng, y, st);
    case SPC_F16: return launch<__half>(x, residual, n, last, any, scale, rng, y, st);
    default: return launch<__nv_bfloat16>(x, residual, n, last, any, scale, rng, y, st);
    }
}

}  // namespace spc
