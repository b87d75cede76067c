// segments.cu -- rows grouped by a small key: a stable counting sort.
//
// A block owns a run of consecutive rows and a warp a run within it.  A row's position is its
// key's first position, plus the rows with that key in earlier blocks, earlier warps, earlier
// rounds of 32 rows and lower lanes.  Which lanes hold the same key follows from one ballot for each of the
// key's bits (the warp-wide match instruction takes several times that when the keys differ).
// Keys out of range count as one more key after the last.
//
// One kernel counts the keys of each block; the other finds its rows' places among its own
// meanwhile, then adds up the counts of all blocks (a warp for a key: its lanes take the blocks)
// and writes the positions.  Few rows go through one launch instead, in a cluster of blocks that read each
// other's counts in shared memory.  (All rows through that: 131,072 slots by 64 experts 30 us, as 8 SMs write
// the scattered positions; through two kernels 9.8.)
#include "layers.cuh"
#include "tc2.cuh"

namespace spc {

namespace {

constexpr int kMaxBlocks = 304;
constexpr int kWarps = 8;
constexpr int kBlock = kWarps * 32;
constexpr int kMinRows = 1024;  // rows of a block, at least
constexpr int kKeep = 8;        // rounds of a warp whose rows stay in registers

__device__ __forceinline__ int key_of(const int32_t* ids, int64_t stride, int64_t i, int segments)
{
    const int32_t k = __ldg(ids + i * stride);
    return k < 0 || k >= segments ? segments : k;
}

// The lanes of the warp whose key agrees with this one's in its low `bits` bits.
__device__ __forceinline__ unsigned same_key(int k, int bits)
{
    unsigned same = FULL_MASK;
    for (int b = 0; b < bits; ++b) {
        const bool one = (k >> b) & 1;
        const unsigned ones = __ballot_sync(FULL_MASK, one);
        same &= one ? ones : ~ones;
    }
    return same;
}

// A row with its key and the number of this warp's rows with that key before it.
struct Ranked {
    int32_t key, before;
};

// Takes a round of 32 rows into the warp's counts.
__device__ __forceinline__ Ranked take_round(int key, int bins, int bits, int32_t* mine)
{
    const int lane = threadIdx.x & 31;
    const unsigned same = same_key(key, bits);
    Ranked r{key, 0};
    if (key < bins) {
        const int had = mine[key];
        r.before = had + __popc(same & ((1u << lane) - 1u));
        __syncwarp(same);
        if (lane == __ffs(same) - 1) mine[key] = had + __popc(same);
    }
    __syncwarp();
    return r;
}

// counts[k][b]: rows of block b with key k.
__global__ void __launch_bounds__(kBlock)
k_seg_count(const int32_t* __restrict__ ids, int64_t stride, int64_t n, int segments, int bits, int64_t rows,
            int32_t* __restrict__ counts)
{
    extern __shared__ int32_t s_count[];
    const int bins = segments + 1;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    for (int k = threadIdx.x; k < bins; k += kBlock) s_count[k] = 0;
    __syncthreads();
    const int64_t lo = (int64_t)blockIdx.x * rows, hi = lo + rows < n ? lo + rows : n;
    // a key past the last one stands for no row
#pragma unroll 4
    for (int64_t i0 = lo; i0 < hi; i0 += kBlock) {
        const int64_t i = i0 + threadIdx.x;
        const int k = i < hi ? key_of(ids, stride, i, segments) : bins;
        const unsigned same = same_key(k, bits);
        if (k < bins && (int)(threadIdx.x & 31) == __ffs(same) - 1) atomicAdd(&s_count[k], __popc(same));
    }
    __syncthreads();
    for (int k = threadIdx.x; k < bins; k += kBlock) counts[(int64_t)k * gridDim.x + blockIdx.x] = s_count[k];
}

// KEEP: a warp's rows fit its registers, else it reads them again.
template <bool KEEP>
__global__ void __launch_bounds__(kBlock)
k_seg_place(const int32_t* __restrict__ ids, int64_t stride, int64_t n, int segments, int bits, int64_t rows,
            int blocks, const int32_t* counts, int32_t* __restrict__ seg, int32_t* __restrict__ order)
{
    extern __shared__ int32_t s_mem[];
    __shared__ int32_t s_scan[kWarps];
    const int bins = segments + 1;
    int32_t* s_first = s_mem;          // [bins] total of the key, then its first position for this block
    int32_t* s_prev = s_mem + bins;    // [bins] rows with the key in earlier blocks
    int32_t* s_warp = s_prev + bins;   // [kWarps][bins] rows of each warp, then the position of its first
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t lo = (int64_t)blockIdx.x * rows, hi = lo + rows < n ? lo + rows : n;
    const int64_t per = rows / kWarps, w_lo = lo + warp * per, w_hi = w_lo + per < hi ? w_lo + per : hi;
    int32_t* mine = s_warp + warp * bins;
    Ranked kept[KEEP ? kKeep : 1];
    if (order) {
        for (int k = lane; k < bins; k += 32) mine[k] = 0;
        __syncwarp();
        if constexpr (KEEP) {
#pragma unroll
            for (int r = 0; r < kKeep; ++r) {
                const int64_t i = w_lo + r * 32 + lane;
                kept[r].key = r * 32 < per && i < w_hi ? key_of(ids, stride, i, segments) : bins;
            }
#pragma unroll
            for (int r = 0; r < kKeep; ++r)
                if (r * 32 < per) kept[r] = take_round(kept[r].key, bins, bits, mine);
        } else {
            for (int64_t r = w_lo; r < w_hi; r += 32) {
                const int64_t i = r + lane;
                take_round(i < w_hi ? key_of(ids, stride, i, segments) : bins, bins, bits, mine);
            }
        }
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the counts of all blocks are there

#pragma unroll 4
    for (int k = warp; k < bins; k += kWarps) {
        int32_t total = 0, before = 0;
        for (int b = lane; b < blocks; b += 32) {
            const int32_t v = counts[(int64_t)k * blocks + b];
            total += v;
            if (b < (int)blockIdx.x) before += v;
        }
        total = __reduce_add_sync(FULL_MASK, total);
        before = __reduce_add_sync(FULL_MASK, before);
        if (lane == 0) {
            s_first[k] = total;
            s_prev[k] = before;
        }
    }
    __syncthreads();
    // first positions: an exclusive scan of the keys' totals, kBlock keys at a time
    int32_t carry = 0;
    for (int k0 = 0; k0 < bins; k0 += kBlock) {
        const int k = k0 + tid;
        const int32_t total = k < bins ? s_first[k] : 0;
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
            if (blockIdx.x == 0) seg[k] = first;
            int32_t at = first + s_prev[k];
            if (order)
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const int32_t v = s_warp[w * bins + k];
                    s_warp[w * bins + k] = at;
                    at += v;
                }
        }
        carry += all;
        __syncthreads();
    }
    if (!order) return;
    if constexpr (KEEP) {
#pragma unroll
        for (int r = 0; r < kKeep; ++r) {
            const int64_t i = w_lo + r * 32 + lane;
            if (r * 32 < per && i < w_hi) order[mine[kept[r].key] + kept[r].before] = (int32_t)i;
        }
    } else {
        // once more, with each key's next position in place of its count
        for (int64_t r = w_lo; r < w_hi; r += 32) {
            const int64_t i = r + lane;
            const Ranked row = take_round(i < w_hi ? key_of(ids, stride, i, segments) : bins, bins, bits, mine);
            if (i < w_hi) order[row.before] = (int32_t)i;
        }
    }
}

// ----------------------------------------------------------- one cluster of blocks
constexpr int kCluster = 8;
constexpr int kBigWarps = 32, kBigBlock = kBigWarps * 32;
constexpr int kRounds = 2;  // of 32 rows for each warp
constexpr int64_t kClusterRows = (int64_t)kCluster * kBigBlock * kRounds;

__global__ void __launch_bounds__(kBigBlock, 1)
k_seg_cluster(const int32_t* __restrict__ ids, int64_t stride, int n, int segments, int bits, int rows,
              int32_t* __restrict__ seg, int32_t* __restrict__ order)
{
    extern __shared__ int32_t s_mem[];
    __shared__ int32_t s_scan[kBigWarps];
    const int bins = segments + 1;
    int32_t* s_total = s_mem;          // [bins] rows of this block, read by the others
    int32_t* s_warp = s_mem + bins;    // [kBigWarps][bins] rows of each warp, then the position of its first
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = (int)ptx::cluster_rank(), blocks = gridDim.x;
    const int lo = rank * rows, hi = lo + rows < n ? lo + rows : n;
    const int per = rows / kBigWarps, w_lo = lo + warp * per, w_hi = w_lo + per < hi ? w_lo + per : hi;
    int32_t* mine = s_warp + warp * bins;
    Ranked kept[kRounds];
#pragma unroll
    for (int r = 0; r < kRounds; ++r) {
        const int i = w_lo + r * 32 + lane;
        kept[r].key = r * 32 < per && i < w_hi ? key_of(ids, stride, i, segments) : bins;
    }
    for (int k = lane; k < bins; k += 32) mine[k] = 0;
    __syncwarp();
#pragma unroll
    for (int r = 0; r < kRounds; ++r)
        if (r * 32 < per) kept[r] = take_round(kept[r].key, bins, bits, mine);
    __syncthreads();
    // a warp's counts become the rows of the warps before it
    for (int k = tid; k < bins; k += kBigBlock) {
        int32_t at = 0;
#pragma unroll 8
        for (int w = 0; w < kBigWarps; ++w) {
            const int32_t v = s_warp[w * bins + k];
            s_warp[w * bins + k] = at;
            at += v;
        }
        s_total[k] = at;
    }
    ptx::cluster_sync();
    int32_t carry = 0;
    for (int k0 = 0; k0 < bins; k0 += kBigBlock) {
        const int k = k0 + tid;
        int32_t total = 0, before = 0;
        if (k < bins) {
            const uint32_t here = ptx::smem_u32(s_total + k);
#pragma unroll
            for (int b = 0; b < kCluster; ++b)
                if (b < blocks) {
                    int32_t v;
                    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(ptx::map_rank(here, b)) : "memory");
                    total += v;
                    if (b < rank) before += v;
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
        // the warps' sums, scanned by every warp for itself
        int32_t all = s_scan[lane];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t v = __shfl_up_sync(FULL_MASK, all, d);
            if (lane >= d) all += v;
        }
        const int32_t below = __shfl_sync(FULL_MASK, all, warp ? warp - 1 : 0);
        const int32_t first = carry + (warp ? below : 0) + inc - total;
        if (k < bins) {
            if (rank == 0) seg[k] = first;
            for (int w = 0; w < kBigWarps; ++w) s_warp[w * bins + k] += first + before;
        }
        carry += __shfl_sync(FULL_MASK, all, 31);
        __syncthreads();
    }
    if (order)
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const int i = w_lo + r * 32 + lane;
            if (r * 32 < per && i < w_hi) order[mine[kept[r].key] + kept[r].before] = i;
        }
    ptx::cluster_sync();  // nobody's counts go while another block may read them
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
    const int bins = segments + 1, bits = ceil_log2((uint64_t)bins + 1);
    if (n <= kClusterRows) {
        const spc_status allowed = allow_smem<k_seg_cluster>();
        if (allowed != SPC_OK) return allowed;
        const int blocks = (int)std::max<int64_t>(1, std::min<int64_t>(kCluster, ceil_div(n, kBigBlock)));
        const int64_t rows = std::max<int64_t>(1, ceil_div(ceil_div(n, blocks), kBigBlock)) * kBigBlock;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)blocks);
        cfg.blockDim = dim3(kBigBlock);
        cfg.dynamicSmemBytes = sizeof(int32_t) * (size_t)bins * (1 + kBigWarps);
        cfg.stream = st;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)blocks;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        SPC_CUDA_TRY(cudaLaunchKernelEx(&cfg, k_seg_cluster, ids, id_stride, (int)n, (int)segments, bits, (int)rows, seg, order));
        return SPC_OK;
    }
    // whole rounds of 32 rows for each warp
    const int64_t rows = ceil_div(ceil_div(n, block_count(n)), kBlock) * kBlock;
    const int blocks = (int)ceil_div(n, rows);
    int32_t* counts = static_cast<int32_t*>(ws);
    const bool keep = rows <= kKeep * kBlock;
    const spc_status allowed = keep ? allow_smem<k_seg_place<true>>() : allow_smem<k_seg_place<false>>();
    if (allowed != SPC_OK) return allowed;
    k_seg_count<<<blocks, kBlock, sizeof(int32_t) * bins, st>>>(ids, id_stride, n, segments, bits, rows, counts);
    SPC_LAUNCH_CHECK();
    // the second kernel may start beside the first: it waits for it where it needs the counts
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(order ? blocks : 1));
    cfg.blockDim = dim3(kBlock);
    cfg.dynamicSmemBytes = sizeof(int32_t) * (size_t)bins * (2 + kWarps);
    cfg.stream = st;
    cudaLaunchAttribute attr[1] = {beside_the_kernel_before()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    SPC_CUDA_TRY(cudaLaunchKernelEx(&cfg, keep ? k_seg_place<true> : k_seg_place<false>, ids, id_stride, n, (int)segments,
                                    bits, rows, blocks, (const int32_t*)counts, seg, order));
    return SPC_OK;
}

}  // namespace spc
