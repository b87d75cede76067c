// pairs.cuh -- vectors of a row as pairs of fp32, and the two-at-a-time instructions on them.
#pragma once

#include <string.h>

#include <type_traits>

#include "common.cuh"

namespace spc {

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
    T e[V];
};

// ------------------------------------------------------------------ pairs of fp32
struct F2 {
    float x, y;
};
__device__ __forceinline__ uint64_t bits(F2 a)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
    return r;
}
__device__ __forceinline__ F2 pair(uint64_t r)
{
    F2 a;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a.x), "=f"(a.y) : "l"(r));
    return a;
}
__device__ __forceinline__ F2 both(float v) { return F2{v, v}; }
__device__ __forceinline__ F2 add(F2 a, F2 b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
    return pair(r);
}
__device__ __forceinline__ F2 mul(F2 a, F2 b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)));
    return pair(r);
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
    return pair(r);
}

template <int V> constexpr int kPairs = (V + 1) / 2;  // a single channel is the first of a pair

template <typename T, int V>
__device__ __forceinline__ void unpack(const Vec<T, V>& v, F2 (&f)[kPairs<V>])
{
    if constexpr (V == 1) {
        f[0] = F2{elem<T>::to_f32(v.e[0]), 0.f};
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) f[j] = F2{elem<T>::to_f32(v.e[2 * j]), elem<T>::to_f32(v.e[2 * j + 1])};
    } else {
        uint32_t w[V / 2];
        memcpy(w, v.e, sizeof(w));
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                f[j] = F2{__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u)};
            } else {
                __half2 h;
                memcpy(&h, &w[j], 4);
                const float2 g = __half22float2(h);
                f[j] = F2{g.x, g.y};
            }
        }
    }
}

template <typename T, int V>
__device__ __forceinline__ Vec<T, V> pack(const F2 (&f)[kPairs<V>])
{
    Vec<T, V> v;
    if constexpr (V == 1) {
        v.e[0] = elem<T>::from_f32(f[0].x);
    } else if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            v.e[2 * j] = elem<T>::from_f32(f[j].x);
            v.e[2 * j + 1] = elem<T>::from_f32(f[j].y);
        }
    } else {
        uint32_t w[V / 2];
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            if constexpr (std::is_same<T, __nv_bfloat16>::value) {
                const __nv_bfloat162 h = __floats2bfloat162_rn(f[j].x, f[j].y);
                memcpy(&w[j], &h, 4);
            } else {
                const __half2 h = __floats2half2_rn(f[j].x, f[j].y);
                memcpy(&w[j], &h, 4);
            }
        }
        memcpy(v.e, w, sizeof(w));
    }
    return v;
}

}  // namespace spc
