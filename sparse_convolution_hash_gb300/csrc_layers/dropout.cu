// dropout.cu -- y = residual + keep(x) / (1 - p) with a mask that is a function
// of the element's index.
//
// Word i % 4 of block i / 4 of Philox4x32-10 (Salmon, Moraes, Dror, Shaw, SC
// 2011) decides element i: ten rounds of two 32 x 32 -> 64 multiplications, a
// Feistel exchange of their halves, and two round keys that advance by the
// published constants.  Four elements share one block, so a thread owns whole
// groups of four.
//
// The product with 1 / (1 - p) and the sum with the residual are each rounded to fp32, in every form
// of the kernel, so that an element's bits do not depend on which side of a 16-byte boundary it stands.
#include <math.h>

#include "layers.cuh"
#include "pairs.cuh"

namespace spc {

namespace {

constexpr int kBlock = 128;

struct Words {
    uint32_t w[4];
};

// Seed and offset of a call.  A warp-wide reduction of equal values leaves them in uniform
// registers, so the key schedule runs beside the lanes' arithmetic and not in it.
struct Keys {
    uint32_t k0, k1, c2, c3;
    __device__ __forceinline__ explicit Keys(const uint64_t* rng)
    {
        const uint64_t seed = fetch(rng), offset = fetch(rng + 1);
        k0 = __reduce_or_sync(FULL_MASK, (uint32_t)seed);
        k1 = __reduce_or_sync(FULL_MASK, (uint32_t)(seed >> 32));
        c2 = __reduce_or_sync(FULL_MASK, (uint32_t)offset);
        c3 = __reduce_or_sync(FULL_MASK, (uint32_t)(offset >> 32));
    }
};

__device__ __forceinline__ Words philox10(uint64_t block, const Keys& k)
{
    uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32), c2 = k.c2, c3 = k.c3, k0 = k.k0, k1 = k.k1;
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

// last: the largest word that drops (where the probability is not 0: ANY).
struct Rule {
    uint32_t last;
    float scale;
};

// Whole 16-byte vectors, kVectors of them in flight a thread, a block's neighbours together;
// nothing but the vectors is read or written.  The generator's 20 wide multiplications for four
// elements stand against 16 to 48 bytes: 398,833 x 128 bf16 with a residual takes 48.5 us (6.3 TB/s)
// and 44 with one of the ten rounds.  Four vectors hide most of it (two: 52, eight: 50; two and the key
// schedule in every lane: 56).  498,145 x 64 fp16: 30 us, with two vectors 33.
constexpr int kVectors = 4;
template <typename T, bool RESIDUAL, bool ANY>
__global__ void __launch_bounds__(kBlock)
k_dropout(const T* x, const T* residual, int64_t n, Rule k, const uint64_t* rng, T* y)
{
    constexpr int E = 16 / sizeof(T);
    using P = Vec<T, E>;
    wait_for_kernel_before();
    const Keys keys(rng);
    const int64_t vectors = n / E, first = (int64_t)blockIdx.x * (kBlock * kVectors) + threadIdx.x;
    P v[kVectors], r[kVectors];
#pragma unroll
    for (int q = 0; q < kVectors; ++q) {
        const int64_t i = first + q * kBlock;
        if (i < vectors) {
            v[q] = reinterpret_cast<const P*>(x)[i];
            if (RESIDUAL) r[q] = reinterpret_cast<const P*>(residual)[i];
        }
    }
#pragma unroll
    for (int q = 0; q < kVectors; ++q) {
        const int64_t i = first + q * kBlock;
        if (i >= vectors) break;
        F2 f[E / 2], g[E / 2];
        unpack<T, E>(v[q], f);
        if (RESIDUAL) unpack<T, E>(r[q], g);
#pragma unroll
        for (int h = 0; h < E / 4; ++h) {
            const Words w = philox10((uint64_t)i * (E / 4) + h, keys);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                // a dropped element is 0 whatever it holds
                F2 e = f[2 * h + j];
                e.x = ANY && w.w[2 * j] <= k.last ? 0.f : e.x;
                e.y = ANY && w.w[2 * j + 1] <= k.last ? 0.f : e.y;
                // the products one by one: a product of pairs and a sum of pairs would be made one instruction
                e = F2{__fmul_rn(e.x, k.scale), __fmul_rn(e.y, k.scale)};
                f[2 * h + j] = RESIDUAL ? add(e, g[2 * h + j]) : e;
            }
        }
        reinterpret_cast<P*>(y)[i] = pack<T, E>(f);
    }
    // the rest of a last, partial vector
    const int64_t t = vectors * E + threadIdx.x * 4;
    if (blockIdx.x == 0 && t < n) {
        const Words w = philox10((uint64_t)t / 4, keys);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (t + j < n) {
                const float f = ANY && w.w[j] <= k.last ? 0.f : __fmul_rn(elem<T>::to_f32(x[t + j]), k.scale);
                y[t + j] = elem<T>::from_f32(RESIDUAL ? __fadd_rn(f, elem<T>::to_f32(residual[t + j])) : f);
            }
    }
}

// Tensors off a 16-byte boundary: four elements a thread, one by one.
template <typename T, bool ANY>
__global__ void __launch_bounds__(kBlock)
k_dropout_unaligned(const T* x, const T* residual, int64_t n, Rule k, const uint64_t* rng, T* y)
{
    wait_for_kernel_before();
    const Keys keys(rng);
    const int64_t q = (int64_t)blockIdx.x * kBlock + threadIdx.x;
    if (q * 4 >= n) return;
    const Words w = philox10((uint64_t)q, keys);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t i = q * 4 + j;
        if (i >= n) break;
        const float f = ANY && w.w[j] <= k.last ? 0.f : __fmul_rn(elem<T>::to_f32(x[i]), k.scale);
        y[i] = elem<T>::from_f32(residual ? __fadd_rn(f, elem<T>::to_f32(residual[i])) : f);
    }
}

template <typename T, bool ANY>
spc_status launch(const void* xv, const void* rv, int64_t n, const Rule& k, const uint64_t* rng, void* yv, cudaStream_t st)
{
    const T* x = static_cast<const T*>(xv);
    const T* r = static_cast<const T*>(rv);
    T* y = static_cast<T*>(yv);
    const bool whole = aligned16(x) && aligned16(r) && aligned16(y);
    const int64_t blocks = whole ? std::max<int64_t>(1, ceil_div(n / (16 / (int64_t)sizeof(T)), kBlock * kVectors))
                                 : ceil_div(ceil_div(n, 4), kBlock);
    if (blocks > INT32_MAX) return SPC_ERR_UNSUPPORTED;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kBlock);
    cfg.stream = st;
    cudaLaunchAttribute attr[1] = {beside_the_kernel_before()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto* kernel = !whole ? k_dropout_unaligned<T, ANY> : r ? k_dropout<T, true, ANY> : k_dropout<T, false, ANY>;
    SPC_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, x, r, n, k, rng, y));
    return SPC_OK;
}

template <typename T>
spc_status launch(const void* x, const void* r, int64_t n, bool any, const Rule& k, const uint64_t* rng, void* y, cudaStream_t st)
{
    return any ? launch<T, true>(x, r, n, k, rng, y, st) : launch<T, false>(x, r, n, k, rng, y, st);
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
    const bool any = threshold > 0;
    k.last = any ? (uint32_t)(threshold - 1) : 0u;
    k.scale = p < 1.0 ? (float)(1.0 / (1.0 - p)) : 0.f;
    switch (dt) {
    case SPC_F32: return launch<float>(x, residual, n, any, k, rng, y, st);
    case SPC_F16: return launch<__half>(x, residual, n, any, k, rng, y, st);
    default: return launch<__nv_bfloat16>(x, residual, n, any, k, rng, y, st);
    }
}

}  // namespace spc
