// attention_tc.cuh -- what the tensor-core attention kernels share: tensor maps of rows of heads, products whose
// first operand lies in tensor memory, and the wider moves between tensor memory and registers.
//
// All three kernels have one form.  The operand whose rows a block keeps (queries, or keys for dk and dv) gives
// the 128 lanes of a product S in tensor memory; four warps, a thread to a lane, turn S into 16-bit
// probabilities (or their gradients) there; and those are the first operand, from tensor memory, of the second product,
// whose other operand is the streamed tile read along its rows (an MN-major operand).  So nothing is transposed and the
// probabilities never pass through shared memory.
#pragma once

#include "attention.cuh"
#include "kernels.cuh"
#include "pairs.cuh"
#include "tc2.cuh"
#include "tmap.cuh"

namespace spc {

constexpr uint64_t kAttnDrainNs = 200000000ull;  // bound of the waits for a block's own copies and products

template <typename T> struct AttnFmt;
template <> struct AttnFmt<__half> { static constexpr uint32_t v = 0; static constexpr CUtensorMapDataType t = CU_TENSOR_MAP_DATA_TYPE_FLOAT16; };
template <> struct AttnFmt<__nv_bfloat16> { static constexpr uint32_t v = 1; static constexpr CUtensorMapDataType t = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16; };

// Rows of [heads, d], ld elements apart; boxes of 64 channels (zeros past d) x box_heads x box_rows, 128-byte swizzle.
template <typename T>
bool attn_tmap(CUtensorMap* m, const void* base, int64_t ld, int64_t rows, int heads, int d, int box_heads, int box_rows)
{
    EncodeFn enc = tmap_encoder();
    if (!enc) return false;
    const cuuint64_t dim[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t stride[2] = {(cuuint64_t)d * 2, (cuuint64_t)ld * 2};
    const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows}, one[3] = {1, 1, 1};
    return enc(m, AttnFmt<T>::t, 3, const_cast<void*>(base), dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

namespace ptx {

// D[tmem] (+)= A[tmem] B, 16-bit operands, K = 16: A's row is a lane, two values to a column.
__device__ __forceinline__ void mma_f16_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p;\n\t"
                 "setp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(tmem_d),
                 "r"(tmem_a), "l"(bdesc), "r"(idesc), "r"(accumulate)
                 : "memory");
}

// 32 lanes x 8 (16, 32) consecutive 32-bit columns, from thread i's registers to lane base + i.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]),
                 "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
                 "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
                 "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
                 : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
                 "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
                 "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
                 "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
                 "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
                 "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
                 "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The largest of three; a NaN among them is passed over.
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

}  // namespace ptx

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint32_t w;
    if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        memcpy(&w, &h, 4);
    } else {
        const __half2 h = __floats2half2_rn(lo, hi);
        memcpy(&w, &h, 4);
    }
    return w;
}

// The tensor warps run their loops as whole warps and elect a lane where they issue: what a loop computes then stays in
// uniform registers, from which products and copies take their operands.  With a loop of one lane each product took
// about 100 cycles to issue, and the products, not the exponentials, set the pace (d = 64: 385 TFLOP/s).
__device__ __forceinline__ bool attn_elect()
{
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}
__device__ __forceinline__ bool attn_wait(uint64_t* bar, uint32_t parity, uint64_t wait_ns)
{
    return __all_sync(FULL_MASK, ptx::mbar_wait(bar, parity, wait_ns));
}

// A product of rows of up to 128 channels in shared memory, both K-major, by one lane; boxes of 64 channels lie a_box / b_box
// bytes apart.  a, b: descriptors of the first box; `steps` of 16 channels, at most MOST.
template <int MOST>
__device__ __forceinline__ void attn_mma_ss(uint32_t d, uint64_t a, uint32_t a_box, uint64_t b, uint32_t b_box, uint32_t idesc, int steps)
{
#pragma unroll
    for (int q = 0; q < MOST; ++q)
        if (q < steps) ptx::mma_f16<1>(d, a + (q >> 2) * (a_box >> 4) + 2 * (q & 3), b + (q >> 2) * (b_box >> 4) + 2 * (q & 3), idesc, q != 0);
}

// Zeroes the rows [from, rows) of a tile in shared memory (NB boxes of `rows` lines of 128 bytes): what belongs to
// another segment may be NaN, and a zero probability does not silence that.  By `threads` threads, thread i.
template <int NB>
__device__ __forceinline__ void attn_clear_rows(uint32_t base, int rows, int from, int i, int threads)
{
    const int lines = (rows - from) * 8;
    for (int x = i; x < lines * NB; x += threads) {
        const uint32_t at = base + (uint32_t)(x / lines) * rows * 128 + from * 128 + (x % lines) * 16;
        asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
    }
    ptx::fence_proxy_async_smem();
}

}  // namespace spc
