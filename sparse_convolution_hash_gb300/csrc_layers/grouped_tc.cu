// grouped_tc.cu -- products grouped by segment on the 5th-generation tensor
// cores: out[out_rows(r)] = in[in_rows(r)] B[g], the forward (B[g] = W[g] as stored,
// an MN-major operand) and the gradient by the input (B[g] = W[g]^T, K-major as stored).
//
// Persistent: one CTA (or one pair of CTAs that share each tile, CG = 2) per SM
// walks over 128 CG x BN tiles of all segments.  In a CTA
//   warp 0 loads the stages: 64 of the reduction at a time, the rows as one TMA box,
//     the weights as 3-D TMA boxes, so that what lies past a segment's weights
//     reads as zeros, not as its neighbour's;
//   with a row list, warps 10-17 copy the rows instead, 16 bytes per cp.async
//     (a TMA gather of four rows takes about 85 cycles whatever the rows, 128 rows per 1.4 us,
//     a third of the pace of the MMAs; the copies keep up with them);
//   warp 1 issues the MMAs into one of two fp32 accumulators in tensor memory;
//   warps 2-9 empty the other one: round once, transpose through shared memory,
//     store 64-byte row pieces (two warps for each quarter of the rows: four did not keep up
//     with reductions of 512).  Rows past the segment's end are not stored.
// Every output row is written once, so results are run-to-run identical.
//
// Every wait is bounded by the library's wait limit; one that runs out sets
// SPC_ERR_TIMEOUT, and each role then waits (bounded) for what it has in flight
// itself before the CTA frees its tensor memory and returns.
#include "grouped_tiles.cuh"
#include "kernels.cuh"
#include "tc2.cuh"
#include "tmap.cuh"

namespace spc {

namespace {

constexpr int kEpilogueWarps = 8;
constexpr int kThreads = 64 + kEpilogueWarps * 32;
constexpr int kGatherWarps = 8, kGatherThreads = kGatherWarps * 32;
constexpr int kChunk = 64;  // reduction elements per stage: 128-byte rows
constexpr uint64_t kDrainNs = 200000000ull;  // bound of the waits for a CTA's own copies and MMAs

template <int CG, int BN>
struct Shape {
    static constexpr int kRows = 128 * CG;              // positions per tile
    static constexpr int kHalfN = BN / CG;              // columns of B that a CTA loads
    static constexpr int kABytes = 128 * 128;
    static constexpr int kBBytes = kHalfN * 128;
    static constexpr int kStage = kABytes + kBBytes;
    static constexpr int kStages = 196608 / kStage;     // 192 KB of stages
    static constexpr int kTmemCols = 2 * BN;
    static constexpr int kStaging = kEpilogueWarps * 32 * 64;  // a 32-row x 64-byte box per epilogue warp
    static size_t smem(int segments)
    {
        return 1024 + (size_t)kStages * kStage + kStaging + 8 * (2 * kStages + 4) + 16 + 4 * ((size_t)segments + 3);
    }
};

template <typename T> struct Fmt;
template <> struct Fmt<__half> { static constexpr uint32_t v = 0; static constexpr CUtensorMapDataType t = CU_TENSOR_MAP_DATA_TYPE_FLOAT16; };
template <> struct Fmt<__nv_bfloat16> { static constexpr uint32_t v = 1; static constexpr CUtensorMapDataType t = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16; };

// BMN: B as stored is [k][n] (the forward).  GATHER: rows come through in_rows.
template <typename T, int CG, int BN, bool BMN, bool GATHER>
__global__ void __launch_bounds__(GATHER ? kThreads + kGatherThreads : kThreads, 1)
k_grouped_tc(GroupedArgs a, uint64_t wait_ns, const __grid_constant__ CUtensorMap map_in,
             const __grid_constant__ CUtensorMap map_w)
{
    using S = Shape<CG, BN>;
    constexpr int kAll = GATHER ? kThreads + kGatherThreads : kThreads;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* staging = smem + (size_t)S::kStages * S::kStage;
    uint64_t* full = reinterpret_cast<uint64_t*>(staging + S::kStaging);
    uint64_t* empty = full + S::kStages;
    uint64_t* acc_full = empty + S::kStages;
    uint64_t* acc_empty = acc_full + 2;
    uint32_t* s_ctrl = reinterpret_cast<uint32_t*>(acc_empty + 2);  // tensor memory base
    int32_t* s_start = reinterpret_cast<int32_t*>(s_ctrl + 4);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = CG == 2 ? ptx::cluster_rank() : 0;

    if (tid == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            ptx::mbar_init(&full[s], GATHER ? 1 + kGatherThreads : 1);  // the TMA loads, each gather thread
            ptx::mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(&acc_full[b], 1);
            ptx::mbar_init(&acc_empty[b], kEpilogueWarps * CG);
        }
        ptx::mbar_init_fence();
        ptx::prefetch_tmap(&map_in);
        ptx::prefetch_tmap(&map_w);
    }
    // tensor memory only after the wait: a kernel before this one that lets it start early may still have to
    // allocate its own, and neither would end
    wait_for_kernel_before();
    if (warp == 1) ptx::tmem_alloc_cg<CG>(s_ctrl, S::kTmemCols);
    const int cols = (a.n + BN - 1) / BN;
    const int32_t tiles = tile_starts(a.seg, a.segments, a.m, S::kRows, cols, s_start,
                                      blockIdx.x == 0 ? a.status : nullptr, tid, kAll);
    ptx::tc_fence_before();
    if constexpr (CG == 2) ptx::cluster_sync();
    else __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = s_ctrl[0];
    TileWalk walk{s_start, a.seg, a.m, a.segments, S::kRows, cols, 0};
    const int first = blockIdx.x / CG, step = gridDim.x / CG;
    const int chunks = (a.k + kChunk - 1) / kChunk;
    bool ok = true;

    if (warp == 0) {
        // ------------------------------------------------------------ loads
        uint32_t it = 0;
        for (int32_t t = first; t < tiles && ok; t += step) {
            const TileWalk::Tile k = walk.at(t);
            if (k.g < 0) continue;
            const int64_t row0 = k.lo + rank * 128;
            const int n0 = k.col * BN + (int)rank * S::kHalfN;
            for (int c = 0; c < chunks; ++c, ++it) {
                const int s = it % S::kStages;
                if (it >= S::kStages) {
                    ok = ptx::mbar_wait(&empty[s], ((it / S::kStages) - 1) & 1, wait_ns);
                    ok = __all_sync(FULL_MASK, ok);
                    if (!ok) break;
                }
                const uint32_t base = ptx::smem_u32(smem + (size_t)s * S::kStage);
                uint32_t bar = ptx::smem_u32(&full[s]);
                if constexpr (CG == 2) bar = ptx::map_rank(bar, 0);
                if (rank == 0 && lane == 0) ptx::mbar_arrive_expect_tx(&full[s], CG * (GATHER ? S::kBBytes : S::kStage));
                __syncwarp();
                if constexpr (!GATHER) {
                    if (lane == 0) ptx::tma_load2d<CG>(base, &map_in, c * kChunk, (int32_t)row0, bar);
                }
                if (lane == 0) {
                    if constexpr (BMN) {
#pragma unroll
                        for (int j = 0; j < S::kHalfN / 64; ++j)
                            ptx::tma_load3d<CG>(base + S::kABytes + j * (kChunk * 128), &map_w, n0 + 64 * j, c * kChunk,
                                                k.g, bar);
                    } else {
                        ptx::tma_load3d<CG>(base + S::kABytes, &map_w, c * kChunk, n0, k.g, bar);
                    }
                }
                __syncwarp();
            }
        }
        if (!ok && lane == 0) set_status(a.status, SPC_ERR_TIMEOUT);
        // what is in flight has to land before the CTA's shared memory goes: the
        // leader's barriers count both CTAs' bytes, and the MMAs' commits arrive in both
        const uint32_t from = it > S::kStages ? it - S::kStages : 0;
        for (uint32_t j = from; j < it; ++j)
            ptx::mbar_wait(rank == 0 ? &full[j % S::kStages] : &empty[j % S::kStages], (j / S::kStages) & 1, kDrainNs);
    } else if (warp == 1) {
        // ------------------------------------------------------------- MMAs
        if (rank == 0 && lane == 0) {
            const uint32_t idesc = ptx::idesc_make(Fmt<T>::v, S::kRows, BN) | (BMN ? 1u << 16 : 0u);
            uint32_t it = 0, n = 0;
            for (int32_t t = first; t < tiles && ok; t += step) {
                const TileWalk::Tile k = walk.at(t);
                if (k.g < 0) continue;
                const uint32_t b = n & 1;
                if (n >= 2) ok = ptx::mbar_wait(&acc_empty[b], ((n >> 1) - 1) & 1, wait_ns);
                if (!ok) break;
                ptx::tc_fence_after();
                const uint32_t d = tmem + b * BN;
                for (int c = 0; c < chunks; ++c, ++it) {
                    const int s = it % S::kStages;
                    ok = ptx::mbar_wait(&full[s], (it / S::kStages) & 1, wait_ns);
                    if (!ok) break;
                    // gathered rows came through the generic proxy: order them before the
                    // tensor core's reads
                    if constexpr (GATHER) ptx::fence_proxy_async_smem();
                    ptx::tc_fence_after();
                    const uint32_t base = ptx::smem_u32(smem + (size_t)s * S::kStage);
                    const uint64_t ad = ptx::desc_k_sw128(base);
                    const uint64_t bd = BMN ? ptx::desc_mn_sw128(base + S::kABytes, kChunk * 128)
                                            : ptx::desc_k_sw128(base + S::kABytes);
                    constexpr uint64_t kBStep = BMN ? 2048 >> 4 : 2;
#pragma unroll
                    for (int q = 0; q < kChunk / 16; ++q)
                        ptx::mma_f16<CG>(d, ad + 2 * q, bd + kBStep * q, idesc, (c | q) != 0);
                    ptx::mma_commit_cg<CG>(&empty[s]);
                }
                if (!ok) break;
                ptx::mma_commit_cg<CG>(&acc_full[b]);
                ++n;
            }
            if (!ok) set_status(a.status, SPC_ERR_TIMEOUT);
            // MMAs in flight read shared memory: wait for the last stages' commits
            const uint32_t from = it > S::kStages ? it - S::kStages : 0;
            for (uint32_t j = from; j < it; ++j) ptx::mbar_wait(&empty[j % S::kStages], (j / S::kStages) & 1, kDrainNs);
        }
    } else if (warp >= kThreads / 32) {
        // ------------------------------------------------------ row copies
        // thread e copies piece e % 8 of rows e / 8 + 32 j: a warp instruction takes four
        // whole 128-byte pieces of rows
        if constexpr (GATHER) {
            static_assert(CG == 1, "a pair's rows would have to arrive on the leader's barrier");
            const int e = tid - kThreads, piece = e & 7, r0 = e >> 3;
            const uint8_t* in_base = static_cast<const uint8_t*>(a.in);
            const uint32_t off = (uint32_t)r0 * 128 + ((uint32_t)(piece ^ (r0 & 7)) << 4);
            uint32_t it = 0;
            // the list entries of tile t, read one tile ahead and checked when they are used
            // (-1 past the segment's end)
            TileWalk ahead = walk;
            auto entries = [&](int32_t t, int32_t (&v)[4], TileWalk::Tile& k) {
                k = ahead.at(t);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int64_t p = k.lo + r0 + 32 * j;
                    v[j] = p < k.hi && k.g >= 0 ? fetch(a.in_rows + p) : -1;
                }
            };
            int32_t entry[4] = {-1, -1, -1, -1}, after[4];
            TileWalk::Tile k, k_after;
            if (first < tiles) entries(first, entry, k);
            for (int32_t t = first; t < tiles && ok; t += step, k = k_after) {
                if (t + step < tiles) entries(t + step, after, k_after);
                const uint8_t* src[4];
                bool there[4], inside[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const bool in = inside[j] = k.lo + r0 + 32 * j < k.hi && k.g >= 0;
                    there[j] = in && entry[j] >= 0 && entry[j] < a.in_n;
                    if (in && !there[j]) set_status(a.status, SPC_ERR_ROW_INDEX);
                    src[j] = in_base + ((int64_t)(there[j] ? entry[j] : 0) * a.k + piece * 8) * 2;
                    entry[j] = after[j];
                }
                if (k.g < 0) continue;
                for (int c = 0; c < chunks; ++c, ++it) {
                    const int s = it % S::kStages;
                    if (it >= S::kStages) ok = ptx::mbar_wait(&empty[s], ((it / S::kStages) - 1) & 1, wait_ns);
                    if (!ok) break;
                    const uint32_t dst = ptx::smem_u32(smem + (size_t)s * S::kStage) + off;
                    const bool column = c * kChunk + piece * 8 < a.k;
                    // rows past the segment's end are not stored: whatever stands in the stage will do
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const bool take = there[j] && column;
                        if (inside[j]) ptx::cp_async16(dst + j * 32 * 128, take ? src[j] + (int64_t)c * kChunk * 2 : in_base, take ? 16u : 0u);
                    }
                    ptx::cp_async_arrive_noinc(&full[s]);
                }
            }
            if (!ok) set_status(a.status, SPC_ERR_TIMEOUT);
            ptx::cp_async_wait_all();  // nothing of ours may still land when the CTA ends
        }
    } else {
        // --------------------------------------------------------- epilogue
        const int quarter = warp & 3;
        uint8_t* box = staging + (warp - 2) * (32 * 64);
        T* out = static_cast<T*>(a.out);
        uint32_t n = 0;
        for (int32_t t = first; t < tiles && ok; t += step) {
            const TileWalk::Tile k = walk.at(t);
            const int64_t p = k.lo + rank * 128 + quarter * 32 + lane;
            int32_t row = -1;
            if (p < k.hi) row = (int32_t)row_at(a.out_rows, p, a.m, a.status);
            const uint32_t b = n & 1;
            if (k.g >= 0) {
                ok = ptx::mbar_wait(&acc_full[b], (n >> 1) & 1, wait_ns);
                ok = __all_sync(FULL_MASK, ok);
                if (!ok) break;
                ptx::tc_fence_after();
                ++n;
            }
#pragma unroll 1
            for (int c = (warp - 2) >> 2; c < BN / 32; c += kEpilogueWarps / 4) {
                const int n0 = k.col * BN + c * 32;
                if (n0 >= a.n) break;
                uint32_t v[32];
                if (k.g >= 0) {
                    ptx::tmem_ld32(tmem + ((uint32_t)(quarter * 32) << 16) + b * BN + c * 32, v);
                    ptx::tmem_ld_wait();
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0u;
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    alignas(16) T o[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) o[i] = elem<T>::from_f32(__uint_as_float(v[j * 8 + i]));
                    *reinterpret_cast<uint4*>(box + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) = *reinterpret_cast<uint4*>(o);
                }
                __syncwarp();
                const int piece = lane & 3;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int rr = j * 8 + (lane >> 2);
                    const int32_t to = __shfl_sync(FULL_MASK, row, rr);
                    const uint4 w = *reinterpret_cast<const uint4*>(box + rr * 64 + ((piece ^ ((rr >> 1) & 3)) << 4));
                    if (to >= 0 && n0 + piece * 8 < a.n)
                        __stcs(reinterpret_cast<uint4*>(out + (int64_t)to * a.n + n0 + piece * 8), w);
                }
                __syncwarp();
            }
            if (k.g >= 0) {
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if constexpr (CG == 2) ptx::mbar_arrive_cluster(ptx::map_rank(ptx::smem_u32(&acc_empty[b]), 0));
                    else ptx::mbar_arrive(&acc_empty[b]);
                }
            }
        }
        if (!ok && lane == 0) set_status(a.status, SPC_ERR_TIMEOUT);
    }
    __syncwarp();
    ptx::tc_fence_before();
    if constexpr (CG == 2) ptx::cluster_sync();
    else __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc_cg<CG>(tmem, S::kTmemCols);
    }
}

// Tensor [depth][rows][cols] of 16-bit elements, boxes of box_cols x box_rows, 128-byte swizzle.
template <typename T>
bool tmap(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint64_t depth, uint32_t box_cols,
          uint32_t box_rows, int dims)
{
    EncodeFn enc = tmap_encoder();
    if (!enc) return false;
    const cuuint64_t dim[3] = {cols, rows, depth};
    const cuuint64_t stride[2] = {cols * 2, cols * rows * 2};
    const cuuint32_t box[3] = {box_cols, box_rows, 1}, one[3] = {1, 1, 1};
    return enc(m, Fmt<T>::t, dims, const_cast<void*>(base), dim, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int CG, int BN, bool BMN, bool GATHER>
spc_status launch(const GroupedArgs& a, cudaStream_t st)
{
    using S = Shape<CG, BN>;
    CUtensorMap map_in, map_w;
    if (!tmap<T>(&map_in, a.in, (uint64_t)a.k, (uint64_t)a.in_n, 1, kChunk, 128, 2)) return SPC_ERR_CUDA;
    const bool w_ok = BMN ? tmap<T>(&map_w, a.w, (uint64_t)a.n, (uint64_t)a.k, (uint64_t)a.segments, 64, kChunk, 3)
                          : tmap<T>(&map_w, a.w, (uint64_t)a.k, (uint64_t)a.n, (uint64_t)a.segments, kChunk, S::kHalfN, 3);
    if (!w_ok) return SPC_ERR_CUDA;
    auto* kernel = k_grouped_tc<T, CG, BN, BMN, GATHER>;
    const size_t smem = S::smem(a.segments);
    const spc_status allowed = allow_smem<k_grouped_tc<T, CG, BN, BMN, GATHER>>();
    if (allowed != SPC_OK) return allowed;
    const int64_t most = (a.m / S::kRows + a.segments + 2) * ceil_div(a.n, BN);
    const int groups = (int)std::min<int64_t>(sm_count() / CG, most);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(groups * CG));
    cfg.blockDim = dim3(GATHER ? kThreads + kGatherThreads : kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2] = {beside_the_kernel_before()};
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = CG;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = CG == 2 ? 2 : 1;
    SPC_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, a, wait_limit_ns(), map_in, map_w));
    return SPC_OK;
}

template <typename T, int CG, int BN>
spc_status pick_operands(const GroupedArgs& a, cudaStream_t st)
{
    if constexpr (CG == 1)
        if (a.in_rows) return a.w_transposed ? launch<T, CG, BN, false, true>(a, st) : launch<T, CG, BN, true, true>(a, st);
    return a.w_transposed ? launch<T, CG, BN, false, false>(a, st) : launch<T, CG, BN, true, false>(a, st);
}

// The tile.  256 x 256 by a pair of CTAs halves what each loads of the weights, but half a
// tile of every segment is empty and its two epilogues have less time: it pays from about 2048 rows
// a segment and reductions of 512 on (bf16, 16 segments of 2048, 1024 -> 4096: 186 us
// against 199; one segment of 32,768: 168 against 186; 64 of 780, 1024 -> 256: 38 against 33; one of
// 398,833, 128 -> 256: 75 against 59).  128 x 128 where 128 x 256 would leave columns empty or
// make fewer tiles than there are SMs (398,833 x 128 -> 128: 40 us against 48; 8 segments of 256,
// 512 -> 512: 7.8 against 9.1); a segment has a tile however few its rows, and few rows of many
// segments run at the pace of the weights, better in wide tiles (32 rows of 64: 40 against 48).
template <typename T>
spc_status pick(const GroupedArgs& a, cudaStream_t st)
{
    const int64_t row_tiles = std::max<int64_t>(ceil_div(a.m, 128), std::min<int64_t>(a.m, a.segments));
    if (a.n <= 128 || ceil_div(a.n, 256) * row_tiles < sm_count()) return pick_operands<T, 1, 128>(a, st);
    if (!a.in_rows && a.k >= 512 && a.m / a.segments >= 2048) return pick_operands<T, 2, 256>(a, st);
    return pick_operands<T, 1, 256>(a, st);
}

}  // namespace

bool grouped_tc_supported(int32_t k, int32_t n, int64_t in_n, spc_dtype dt)
{
    // TMA rows start on 16-byte boundaries; an empty tensor has no map
    return (dt == SPC_F16 || dt == SPC_BF16) && k % 8 == 0 && n % 8 == 0 && in_n > 0;
}

spc_status grouped_tc(const GroupedArgs& a, spc_dtype dt, cudaStream_t st)
{
    if (ceil_div(a.n, 64) * (a.m / 128 + a.segments + 2) > INT32_MAX) return SPC_ERR_UNSUPPORTED;
    return dt == SPC_F16 ? pick<__half>(a, st) : pick<__nv_bfloat16>(a, st);
}

}  // namespace spc
