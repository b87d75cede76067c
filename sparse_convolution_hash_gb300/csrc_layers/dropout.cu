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
struct Rule {
    uint32_t last;
    bool any;
    float scale;
};

template <typename T>
struct alignas(16) Pack {
    T e[16 / sizeof(T)];
};

// Elements 4 b .. 4 b + 3 of a pack (v, and r where there is a residual) under block `block`.
template <typename T>
__device__ __forceinline__ void four(const T* v, const T* r, T* o, uint64_t block, uint64_t seed, uint64_t offset, const Rule& k)
{
    const Words w = philox10(block, offset, seed);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const bool drop = k.any && w.w[j] <= k.last;
        float f = drop ? 0.f : elem<T>::to_f32(v[j]) * k.scale;
        if (r) f += elem<T>::to_f32(r[j]);
        o[j] = elem<T>::from_f32(f);
    }
}

// Whole 16-byte vectors: kVectors of them in flight a thread, a block's neighbours together.
// The generator takes about 15 issue slots an element beside the 4 to 12 bytes, so memory and arithmetic are
// near each other's pace; nothing but the vectors is read or written.
constexpr int kVectors = 4;
template <typename T, bool RESIDUAL>
__global__ void __launch_bounds__(kBlock)
k_dropout(const T* x, const T* residual, int64_t n, Rule k, const uint64_t* __restrict__ rng, T* y)
{
    constexpr int E = 16 / sizeof(T);
    const uint64_t seed = __ldg(rng), offset = __ldg(rng + 1);
    const int64_t vectors = n / E, first = (int64_t)blockIdx.x * (kBlock * kVectors) + threadIdx.x;
    Pack<T> v[kVectors], r[kVectors];
#pragma unroll
    for (int q = 0; q < kVectors; ++q) {
        const int64_t i = first + q * kBlock;
        if (i < vectors) {
            v[q] = reinterpret_cast<const Pack<T>*>(x)[i];
            if (RESIDUAL) r[q] = reinterpret_cast<const Pack<T>*>(residual)[i];
        }
    }
#pragma unroll
    for (int q = 0; q < kVectors; ++q) {
        const int64_t i = first + q * kBlock;
        if (i >= vectors) break;
        Pack<T> o;
#pragma unroll
        for (int h = 0; h < E / 4; ++h)
            four<T>(v[q].e + 4 * h, RESIDUAL ? r[q].e + 4 * h : nullptr, o.e + 4 * h, (uint64_t)i * (E / 4) + h, seed, offset, k);
        reinterpret_cast<Pack<T>*>(y)[i] = o;
    }
    // the rest of a last, partial vector
    const int64_t t = vectors * E + threadIdx.x * 4;
    if (blockIdx.x == 0 && t < n) {
        const Words w = philox10((uint64_t)t / 4, offset, seed);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (t + j < n) {
                float f = k.any && w.w[j] <= k.last ? 0.f : elem<T>::to_f32(x[t + j]) * k.scale;
                if (RESIDUAL) f += elem<T>::to_f32(residual[t + j]);
                y[t + j] = elem<T>::from_f32(f);
            }
    }
}

// Tensors off a 16-byte boundary: four elements a thread, one by one.
template <typename T>
__global__ void __launch_bounds__(kBlock)
k_dropout_unaligned(const T* x, const T* residual, int64_t n, Rule k, const uint64_t* __restrict__ rng, T* y)
{
    const int64_t q = (int64_t)blockIdx.x * kBlock + threadIdx.x;
    if (q * 4 >= n) return;
    const Words w = philox10((uint64_t)q, rng[1], rng[0]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t i = q * 4 + j;
        if (i >= n) break;
        float f = k.any && w.w[j] <= k.last ? 0.f : elem<T>::to_f32(x[i]) * k.scale;
        if (residual) f += elem<T>::to_f32(residual[i]);
        y[i] = elem<T>::from_f32(f);
    }
}

template <typename T>
spc_status launch(const void* xv, const void* rv, int64_t n, const Rule& k, const uint64_t* rng, void* yv, cudaStream_t st)
{
    const T* x = static_cast<const T*>(xv);
    const T* r = static_cast<const T*>(rv);
    T* y = static_cast<T*>(yv);
    const bool whole = aligned16(x) && aligned16(r) && aligned16(y);
    const int64_t blocks = whole ? std::max<int64_t>(1, ceil_div(n / (16 / (int64_t)sizeof(T)), kBlock * kVectors))
                                 : ceil_div(ceil_div(n, 4), kBlock);
    if (blocks > INT32_MAX) return SPC_ERR_UNSUPPORTED;
    if (!whole) k_dropout_unaligned<T><<<(unsigned)blocks, kBlock, 0, st>>>(x, r, n, k, rng, y);
    else if (r) k_dropout<T, true><<<(unsigned)blocks, kBlock, 0, st>>>(x, r, n, k, rng, y);
    else k_dropout<T, false><<<(unsigned)blocks, kBlock, 0, st>>>(x, r, n, k, rng, y);
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
    Rule k;
    k.any = threshold > 0;
    k.last = k.any ? (uint32_t)(threshold - 1) : 0u;
    k.scale = p < 1.0 ? (float)(1.0 / (1.0 - p)) : 0.f;
    switch (dt) {
    case SPC_F32: return launch<float>(x, residual, n, k, rng, y, st);
    case SPC_F16: return launch<__half>(x, residual, n, k, rng, y, st);
    default: return launch<__nv_bfloat16>(x, residual, n, k, rng, y, st);
    }
}

}  // namespace spc
