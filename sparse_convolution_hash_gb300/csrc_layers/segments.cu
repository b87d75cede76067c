// segments.cu -- rows grouped by a small key: a stable counting sort.
//
// A block owns a run of consecutive rows and a warp a run within it.  The first
// kernel counts the keys of each block; the second sums the counts of the blocks
// before its own and of all blocks (a key's first position), counts the keys of
// its warps, and writes each row's position: the key's first position, plus the
// rows with that key in earlier blocks, earlier warps, earlier rounds of 32 rows and
// lower lanes (found with a warp-wide match).  Keys out of range count as one
// more key after the last.
#include "layers.cuh"

namespace spc {

namespace {

constexpr int kMaxBlocks = 152;
constexpr int kWarps = 8;
constexpr int kBlock = kWarps * 32;
constexpr int kMinRows = 1024;  // rows of a block, at least

__device__ __forceinline__ int key_of(const int32_t* ids, int64_t stride, int64_t i, int segments)
{
    const int32_t k = __ldg(ids + i * stride);
    return k < 0 || k >= segments ? segments : k;
}

// counts[b][k]: rows of block b with key k.
__global__ void __launch_bounds__(kBlock)
k_seg_count(const int32_t* __restrict__ ids, int64_t stride, int64_t n, int segments, int64_t rows,
            int32_t* __restrict__ counts)
{
    extern __shared__ int32_t s_count[];
    const int bins = segments + 1;
    for (int k = threadIdx.x; k < bins; k += kBlock) s_count[k] = 0;
    __syncthreads();
    const int64_t lo = (int64_t)blockIdx.x * rows, hi = lo + rows < n ? lo + rows : n;
    for (int64_t i = lo + threadIdx.x; i < hi; i += kBlock) {
        const int k = key_of(ids, stride, i, segments);
        const unsigned active = __activemask();
        const unsigned same = __match_any_sync(active, k);
        if ((int)(threadIdx.x & 31) == __ffs(same) - 1) atomicAdd(&s_count[k], __popc(same));
    }
    __syncthreads();
    for (int k = threadIdx.x; k < bins; k += kBlock) counts[(int64_t)blockIdx.x * bins + k] = s_count[k];
}

__global__ void __launch_bounds__(kBlock)
k_seg_place(const int32_t* __restrict__ ids, int64_t stride, int64_t n, int segments, int64_t rows,
            int blocks, const int32_t* __restrict__ counts, int32_t* __restrict__ seg,
            int32_t* __restrict__ order)
{
    extern __shared__ int32_t s_mem[];
    __shared__ int32_t s_scan[kWarps];
    const int bins = segments + 1;
    int32_t* s_first = s_mem;         // [bins] the key's first position for this block
    int32_t* s_warp = s_mem + bins;   // [kWarps][bins] next position of each warp
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // first positions: an exclusive scan of the keys' totals, kBlock keys at a time
    int32_t carry = 0;
    for (int k0 = 0; k0 < bins; k0 += kBlock) {
        const int k = k0 + tid;
        int32_t total = 0, before = 0;
        if (k < bins) {
#pragma unroll 8
            for (int b = 0; b < blocks; ++b) {
                const int32_t v = __ldg(counts + (int64_t)b * bins + k);
                total += v;
                if (b < (int)blockIdx.x) before += v;
            }
        }
        int32_t inc = total;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t v = __shfl_up_sync(FULL_MASK, inc, d);
            if (lane >= d) inc += v;
        }
        if (lane == 31) s_scan[warp] = inc;
        __syncthreads();
        int32_t base = carry, all = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) base += s_scan[w];
            all += s_scan[w];
        }
        if (k < bins) {
            const int32_t first = base + inc - total;
            s_first[k] = first + before;
            if (blockIdx.x == 0) seg[k] = first;
        }
        carry += all;
        __syncthreads();
    }
    if (!order) return;

    for (int k = tid; k < kWarps * bins; k += kBlock) s_warp[k] = 0;
    __syncthreads();
    const int64_t lo = (int64_t)blockIdx.x * rows, hi = lo + rows < n ? lo + rows : n;
    const int64_t per = rows / kWarps, w_lo = lo + warp * per, w_hi = w_lo + per < hi ? w_lo + per : hi;
    int32_t* mine = s_warp + warp * bins;
    for (int64_t r = w_lo; r < w_hi; r += 32) {
        const int64_t i = r + lane;
        const int k = i < w_hi ? key_of(ids, stride, i, segments) : -1;
        const unsigned same = __match_any_sync(FULL_MASK, k);
        if (k >= 0 && lane == __ffs(same) - 1) mine[k] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    for (int k = tid; k < bins; k += kBlock) {
        int32_t at = s_first[k];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const int32_t v = s_warp[w * bins + k];
            s_warp[w * bins + k] = at;
            at += v;
        }
    }
    __syncthreads();
    for (int64_t r = w_lo; r < w_hi; r += 32) {
        const int64_t i = r + lane;
        const int k = i < w_hi ? key_of(ids, stride, i, segments) : -1;
        const unsigned same = __match_any_sync(FULL_MASK, k);
        if (k >= 0) order[mine[k] + __popc(same & ((1u << lane) - 1u))] = (int32_t)i;
        __syncwarp();
        if (k >= 0 && lane == __ffs(same) - 1) mine[k] += __popc(same);
        __syncwarp();
    }
}

int block_count(int64_t n) { return (int)std::max<int64_t>(1, std::min<int64_t>(kMaxBlocks, ceil_div(n, kMinRows))); }

}  // namespace

size_t row_segments_ws_bytes(int64_t n, int32_t segments)
{
    return align_up(sizeof(int32_t) * (size_t)block_count(n) * (size_t)(segments + 1), 256);
}

spc_status row_segments(const int32_t* ids, int64_t id_stride, int64_t n, int32_t segments,
                        int32_t* seg, int32_t* order, void* ws, cudaStream_t st)
{
    const int bins = segments + 1;
    // whole rounds of 32 rows for each warp
    const int64_t rows = std::max<int64_t>(1, ceil_div(ceil_div(n, block_count(n)), kBlock)) * kBlock;
    const int blocks = (int)std::max<int64_t>(1, ceil_div(n, rows));
    int32_t* counts = static_cast<int32_t*>(ws);
    const size_t place_smem = sizeof(int32_t) * (size_t)bins * (1 + kWarps);
    const spc_status allowed = allow_smem<k_seg_place>();
    if (allowed != SPC_OK) return allowed;
    k_seg_count<<<blocks, kBlock, sizeof(int32_t) * bins, st>>>(ids, id_stride, n, segments, rows, counts);
    SPC_LAUNCH_CHECK();
    k_seg_place<<<order ? blocks : 1, kBlock, place_smem, st>>>(ids, id_stride, n, segments, rows, blocks,
                                                               counts, seg, order);
    SPC_LAUNCH_CHECK();
    return SPC_OK;
}

}  // namespace spc
