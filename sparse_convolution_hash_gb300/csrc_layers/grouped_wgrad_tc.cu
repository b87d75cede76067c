// grouped_wgrad_tc.cu -- dW[g] = sum over g's positions of x[x_rows(r)]^T dy[y_rows(r)]
// on the 5th-generation tensor cores, fp32 result.
//
// The reduction runs over rows, so both operands are MN-major: a row of a stage
// is 64 channels (M or N) of one reduction index, and a tile is 128 input x BN
// output channels.  Segments differ in length and there may be fewer tiles than SMs,
// so whole tiles go round the CTAs as far as they fill them evenly and the rest is cut by units
// of 64 rows (Plan).  A whole tile is written to dW as it is; the parts of the others go to the
// workspace and a second kernel adds them in the order of the rows: no atomics, run-to-run
// identical.
//
// The tensor core truncates where it adds to an accumulator, so sums over long segments would
// drift (4096 rows: 5 10^-6 of the result).  An accumulator takes 512 rows; eight warps then add it,
// rounding, to the piece's sums in their registers while the other one fills (5 10^-7).
//
// In a CTA, as in the forward: warp 0 loads dense rows by TMA, eight more copy listed
// rows by cp.async, warp 1 issues the MMAs into one of two accumulators and
// first clears the rows of a last, partial unit past the segment's end (they hold the
// next segment's rows: a zero weight would not do, as 0 x NaN is NaN).
// Wide tiles are bound by what comes from L2 (a 128 x 256 x 64 unit: 48 KB).  Every wait is bounded
// (SPC_ERR_TIMEOUT).
#include "grouped_wgrad_plan.cuh"
#include "kernels.cuh"
#include "layers.cuh"
#include "tc2.cuh"
#include "tmap.cuh"

namespace spc {

namespace {

constexpr int kEpilogueWarps = 8;
constexpr int kThreads = 64 + kEpilogueWarps * 32;
constexpr int kGatherThreads = 256;
constexpr int kFlush = 8;    // units that an accumulator in tensor memory sums up
constexpr int kTileM = 128;  // input channels of a tile
constexpr int kJoinRows = 4;
constexpr int kAtom = kUnit * 128;  // 64 rows x 64 channels
constexpr uint64_t kDrainNs = 200000000ull;

template <int BN>
struct Shape {
    static constexpr int kABytes = kTileM / 64 * kAtom;
    static constexpr int kBBytes = BN / 64 * kAtom;
    static constexpr int kStage = kABytes + kBBytes;
    static constexpr int kStages = 196608 / kStage;
    static constexpr int kTmemCols = 2 * BN;
    static constexpr int kWarpCols = BN / 2;  // columns of an epilogue warp
    static constexpr int kStaging = kEpilogueWarps * 32 * 64;
    static size_t smem(int segments)
    {
        return 1024 + (size_t)kStages * kStage + kStaging + 8 * (2 * kStages + 4) + 16 + 4 * (3 * (size_t)segments + 1);
    }
};

template <typename T> struct Fmt;
template <> struct Fmt<__half> { static constexpr uint32_t v = 0; static constexpr CUtensorMapDataType t = CU_TENSOR_MAP_DATA_TYPE_FLOAT16; };
template <> struct Fmt<__nv_bfloat16> { static constexpr uint32_t v = 1; static constexpr CUtensorMapDataType t = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16; };

template <typename T, int BN, bool GATHER>
__global__ void __launch_bounds__(GATHER ? kThreads + kGatherThreads : kThreads, 1)
k_grouped_wgrad_tc(GroupedWgradArgs a, float* __restrict__ part, Join* __restrict__ joins, uint64_t wait_ns,
                   const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_dy)
{
    using S = Shape<BN>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* staging = smem + (size_t)S::kStages * S::kStage;
    uint64_t* full = reinterpret_cast<uint64_t*>(staging + S::kStaging);
    uint64_t* empty = full + S::kStages;
    uint64_t* acc_full = empty + S::kStages;
    uint64_t* acc_empty = acc_full + 2;
    uint32_t* s_ctrl = reinterpret_cast<uint32_t*>(acc_empty + 2);
    int32_t* s_start = reinterpret_cast<int32_t*>(s_ctrl + 4);
    int32_t* s_list = s_start + a.segments + 1;
    __shared__ Plan plan;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int me = (int)blockIdx.x;

    if (tid == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            ptx::mbar_init(&full[s], GATHER ? kGatherThreads : 1);
            ptx::mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(&acc_full[b], 1);
            ptx::mbar_init(&acc_empty[b], kEpilogueWarps);
        }
        ptx::mbar_init_fence();
        if (!GATHER) {
            ptx::prefetch_tmap(&map_x);
            ptx::prefetch_tmap(&map_dy);
        }
    }
    wait_for_kernel_before();  // before tensor memory, as in the forward
    if (warp == 1) ptx::tmem_alloc_cg<1>(s_ctrl, S::kTmemCols);
    const int cols = (a.cout + BN - 1) / BN, tiles = (a.cin + kTileM - 1) / kTileM * cols;
    if (warp == 0)
        make_plan(a.seg, a.segments, a.m, tiles, gridDim.x, s_start, s_list, s_list + a.segments, &plan,
                  blockIdx.x == 0 ? a.status : nullptr, lane);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = s_ctrl[0];
    Walk walk{s_start, s_list, a.seg, &plan, a.segments, tiles, 0, 0, 0, 0, 0};
    walk.reset(me);
    bool ok = true;
    if (blockIdx.x == 0 && tid < plan.parts) write_join(walk, tid, joins);

    if (warp == 0) {
        // ------------------------------------------------------ dense loads
        if (!GATHER && lane == 0) {
            uint32_t it = 0;
            while (walk.more() && ok) {
                const Piece p = walk.next();
                if (p.lo == p.hi) continue;
                const int c0 = p.tile / cols * kTileM, n0 = p.tile % cols * BN;
                for (int k = p.k0; k < p.k1; ++k, ++it) {
                    const int s = it % S::kStages;
                    if (it >= S::kStages) ok = ptx::mbar_wait(&empty[s], ((it / S::kStages) - 1) & 1, wait_ns);
                    if (!ok) break;
                    const uint32_t base = ptx::smem_u32(smem + (size_t)s * S::kStage), bar = ptx::smem_u32(&full[s]);
                    const int32_t row = (int32_t)(p.lo + (int64_t)k * kUnit);
                    ptx::mbar_arrive_expect_tx(&full[s], S::kStage);
#pragma unroll
                    for (int j = 0; j < kTileM / 64; ++j) ptx::tma_load2d<1>(base + j * kAtom, &map_x, c0 + 64 * j, row, bar);
#pragma unroll
                    for (int j = 0; j < BN / 64; ++j)
                        ptx::tma_load2d<1>(base + S::kABytes + j * kAtom, &map_dy, n0 + 64 * j, row, bar);
                }
            }
            if (!ok) set_status(a.status, SPC_ERR_TIMEOUT);
            const uint32_t from = it > S::kStages ? it - S::kStages : 0;
            for (uint32_t j = from; j < it; ++j) ptx::mbar_wait(&full[j % S::kStages], (j / S::kStages) & 1, kDrainNs);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------- MMAs
        const uint32_t idesc = ptx::idesc_make(Fmt<T>::v, kTileM, BN) | (1u << 15) | (1u << 16);
        uint32_t it = 0, n = 0;
        while (walk.more() && ok) {
            const Piece p = walk.next();
            if (p.lo == p.hi) continue;
            for (int k0 = p.k0; k0 < p.k1 && ok; k0 += kFlush, ++n) {
                const uint32_t b = n & 1, d = tmem + b * BN;
                if (n >= 2) ok = __all_sync(FULL_MASK, ptx::mbar_wait(&acc_empty[b], ((n >> 1) - 1) & 1, wait_ns));
                if (!ok) break;
                ptx::tc_fence_after();
                const int k_end = k0 + kFlush < p.k1 ? k0 + kFlush : p.k1;
                for (int k = k0; k < k_end; ++k, ++it) {
                    const int s = it % S::kStages;
                    ok = __all_sync(FULL_MASK, ptx::mbar_wait(&full[s], (it / S::kStages) & 1, wait_ns));
                    if (!ok) break;
                    uint8_t* stage = smem + (size_t)s * S::kStage;
                    const int64_t left = p.hi - p.lo - (int64_t)k * kUnit;  // rows of this unit
                    if (!GATHER && left < kUnit) {
                        for (int e = (int)left * 8 + lane; e < kUnit * 8; e += 32)
#pragma unroll
                            for (int j = 0; j < kTileM / 64 + BN / 64; ++j)
                                *reinterpret_cast<uint4*>(stage + j * kAtom + e * 16) = make_uint4(0, 0, 0, 0);
                        ptx::fence_proxy_async_smem();
                        __syncwarp();
                    }
                    if (GATHER) ptx::fence_proxy_async_smem();
                    if (lane == 0) {
                        ptx::tc_fence_after();
                        const uint32_t base = ptx::smem_u32(stage);
                        const uint64_t ad = ptx::desc_mn_sw128(base, kAtom), bd = ptx::desc_mn_sw128(base + S::kABytes, kAtom);
#pragma unroll
                        for (int q = 0; q < kUnit / 16; ++q)
                            ptx::mma_f16<1>(d, ad + (uint64_t)(q * (2048 >> 4)), bd + (uint64_t)(q * (2048 >> 4)), idesc,
                                            k != k0 || q != 0);
                        ptx::mma_commit(&empty[s]);
                    }
                    __syncwarp();
                }
                if (!ok) break;
                if (lane == 0) ptx::mma_commit(&acc_full[b]);
            }
        }
        if (!ok && lane == 0) set_status(a.status, SPC_ERR_TIMEOUT);
        const uint32_t from = it > S::kStages ? it - S::kStages : 0;
        for (uint32_t j = from; j < it; ++j) ptx::mbar_wait(&empty[j % S::kStages], (j / S::kStages) & 1, kDrainNs);
    } else if (warp >= kThreads / 32) {
        // ------------------------------------------------------ row copies
        if constexpr (GATHER) {
            const int e = tid - kThreads, piece = e & 7, r0 = e >> 3;
            const uint8_t* x = static_cast<const uint8_t*>(a.x);
            const uint8_t* dy = static_cast<const uint8_t*>(a.dy);
            const uint32_t off = (uint32_t)r0 * 128 + ((uint32_t)(piece ^ (r0 & 7)) << 4);
            uint32_t it = 0;
            while (walk.more() && ok) {
                const Piece p = walk.next();
                if (p.lo == p.hi) continue;
                const int c0 = p.tile / cols * kTileM + piece * 8;
                const int n0 = p.tile % cols * BN + piece * 8;
                // the list entries of thread e's two reduction indices of unit k, read one
                // unit ahead and checked when they are used
                auto entries = [&](int k, int32_t (&xe)[2], int32_t (&ye)[2]) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int64_t r = p.lo + (int64_t)k * kUnit + r0 + 32 * j;
                        const bool in = k < p.k1 && r < p.hi;
                        xe[j] = !in ? -1 : a.x_rows ? fetch(a.x_rows + r) : (int32_t)r;
                        ye[j] = !in ? -1 : a.y_rows ? fetch(a.y_rows + r) : (int32_t)r;
                    }
                };
                int32_t xe[2], ye[2], xn[2], yn[2];
                entries(p.k0, xe, ye);
                for (int k = p.k0; k < p.k1; ++k, ++it) {
                    entries(k + 1, xn, yn);
                    const int s = it % S::kStages;
                    if (it >= S::kStages) ok = ptx::mbar_wait(&empty[s], ((it / S::kStages) - 1) & 1, wait_ns);
                    if (!ok) break;
                    int64_t xr[2], yr[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const bool in = p.lo + (int64_t)k * kUnit + r0 + 32 * j < p.hi;
                        const bool good = xe[j] >= 0 && xe[j] < a.n_x && ye[j] >= 0 && ye[j] < a.n_y;
                        if (in && !good) set_status(a.status, SPC_ERR_ROW_INDEX);
                        xr[j] = good ? xe[j] : -1;
                        yr[j] = good ? ye[j] : -1;
                    }
                    const uint32_t dst = ptx::smem_u32(smem + (size_t)s * S::kStage) + off;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
#pragma unroll
                        for (int q = 0; q < kTileM / 64; ++q) {
                            const bool take = xr[j] >= 0 && c0 + 64 * q < a.cin;
                            ptx::cp_async16(dst + q * kAtom + j * 32 * 128, take ? x + (xr[j] * a.cin + c0 + 64 * q) * 2 : x,
                                            take ? 16u : 0u);
                        }
#pragma unroll
                        for (int q = 0; q < BN / 64; ++q) {
                            const bool take = yr[j] >= 0 && n0 + 64 * q < a.cout;
                            ptx::cp_async16(dst + S::kABytes + q * kAtom + j * 32 * 128,
                                            take ? dy + (yr[j] * a.cout + n0 + 64 * q) * 2 : dy, take ? 16u : 0u);
                        }
                        xe[j] = xn[j];
                        ye[j] = yn[j];
                    }
                    ptx::cp_async_arrive_noinc(&full[s]);
                }
            }
            if (!ok) set_status(a.status, SPC_ERR_TIMEOUT);
            ptx::cp_async_wait_all();  // nothing of ours may still land when the CTA ends
        }
    } else {
        // --------------------------------------------------------- epilogue
        // warp w holds rows 32 (w % 4) .. of the tile's half and one half of its columns
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        uint8_t* box = staging + (warp - 2) * (32 * 64);
        uint32_t n = 0;
        while (walk.more() && ok) {
            const Piece p = walk.next();
            float sum[S::kWarpCols];
#pragma unroll
            for (int j = 0; j < S::kWarpCols; ++j) sum[j] = 0.f;
            for (int k0 = p.k0; k0 < p.k1 && p.lo != p.hi; k0 += kFlush, ++n) {
                const uint32_t b = n & 1;
                ok = __all_sync(FULL_MASK, ptx::mbar_wait(&acc_full[b], (n >> 1) & 1, wait_ns));
                if (!ok) break;
                ptx::tc_fence_after();
                const uint32_t ta = tmem + ((uint32_t)(quarter * 32) << 16) + b * BN + half * S::kWarpCols;
#pragma unroll
                for (int c = 0; c < S::kWarpCols; c += 16) {
                    uint32_t v[16];
                    ptx::tmem_ld16(ta + c, v);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j) sum[c + j] += __uint_as_float(v[j]);
                }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&acc_empty[b]);
            }
            if (!ok) break;
            const int c0 = p.tile / cols * kTileM + quarter * 32;
            const int n0 = p.tile % cols * BN + half * S::kWarpCols;
            // a whole tile goes to dW, a part to this CTA's first or last slot
            float* dst;
            int64_t pitch;
            int rows, width;
            if (p.whole()) {
                dst = a.dw + ((int64_t)p.g * a.cin + c0) * a.cout + n0;
                pitch = a.cout;
                rows = a.cin - c0;
                width = a.cout - n0;
            } else {
                dst = part + ((int64_t)plan.id[me] * 2 + p.slot) * (kTileM * BN) + quarter * 32 * BN + half * S::kWarpCols;
                pitch = BN;
                rows = 32;
                width = S::kWarpCols;
            }
            const int piece = lane & 3;
#pragma unroll
            for (int c = 0; c < S::kWarpCols; c += 16) {
                if (c >= width) break;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    *reinterpret_cast<float4*>(box + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) =
                        make_float4(sum[c + 4 * j], sum[c + 4 * j + 1], sum[c + 4 * j + 2], sum[c + 4 * j + 3]);
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int rr = j * 8 + (lane >> 2);
                    const uint4 w = *reinterpret_cast<const uint4*>(box + rr * 64 + ((piece ^ ((rr >> 1) & 3)) << 4));
                    if (rr < rows && c + piece * 4 < width) *reinterpret_cast<uint4*>(dst + rr * pitch + c + piece * 4) = w;
                }
                __syncwarp();
            }
        }
        if (!ok && lane == 0) set_status(a.status, SPC_ERR_TIMEOUT);
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc_cg<1>(tmem, S::kTmemCols);
    }
}

// Block (c, q): rows kJoinRows q .. of the tile that share c's plan names become the sum
// of its parts, in the order of the shares.
template <int BN>
__global__ void __launch_bounds__(kJoinRows * BN / 4)
k_grouped_wgrad_join(GroupedWgradArgs a, const float* part, const Join* joins)
{
    wait_for_kernel_before();  // set up while the blocks that write the parts end
    const int c = blockIdx.x;
    const Join j = joins[c];
    if (j.more == 0) return;
    const int cols = (a.cout + BN - 1) / BN;
    const int r = blockIdx.y * kJoinRows + threadIdx.x / (BN / 4), n = threadIdx.x % (BN / 4) * 4;
    const int row = j.tile / cols * kTileM + r, col = j.tile % cols * BN + n;
    if (row >= a.cin || col >= a.cout) return;
    constexpr int64_t kSlot = kTileM * BN;
    const float* src = part + r * BN + n;
    float4 s = fetch(reinterpret_cast<const float4*>(src + ((int64_t)c * 2 + j.slot) * kSlot));
    src += (int64_t)(c + 1) * 2 * kSlot;
#pragma unroll 8
    for (int q = 0; q < j.more; ++q) {
        const float4 v = fetch(reinterpret_cast<const float4*>(src + q * 2 * kSlot));
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
    }
    *reinterpret_cast<float4*>(a.dw + ((int64_t)j.g * a.cin + row) * a.cout + col) = s;
}

int grouped_wgrad_ctas() { return std::min(sm_count(), kMaxParts); }

// Two parts of a tile for each CTA, and the joins.
size_t parts_bytes()
{
    return align_up((sizeof(float) * 2 * kTileM * 256 + sizeof(Join)) * (size_t)grouped_wgrad_ctas(), 256);
}

template <typename T, int BN, bool GATHER>
spc_status launch(const GroupedWgradArgs& a, float* part, cudaStream_t st)
{
    using S = Shape<BN>;
    CUtensorMap mx, my;
    if (!tmap_2d(&mx, Fmt<T>::t, 2, a.x, (uint64_t)a.cin, (uint64_t)a.n_x, 64, kUnit, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !tmap_2d(&my, Fmt<T>::t, 2, a.dy, (uint64_t)a.cout, (uint64_t)a.n_y, 64, kUnit, CU_TENSOR_MAP_SWIZZLE_128B))
        return SPC_ERR_CUDA;
    const spc_status allowed = allow_smem<k_grouped_wgrad_tc<T, BN, GATHER>>();
    if (allowed != SPC_OK) return allowed;
    const int parts = grouped_wgrad_ctas();
    Join* joins = reinterpret_cast<Join*>(part + (int64_t)parts * 2 * kTileM * 256);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)parts);
    cfg.blockDim = dim3(GATHER ? kThreads + kGatherThreads : kThreads);
    cfg.dynamicSmemBytes = S::smem(a.segments);
    cfg.stream = st;
    cudaLaunchAttribute attr[1] = {beside_the_kernel_before()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    SPC_CUDA_TRY(cudaLaunchKernelEx(&cfg, k_grouped_wgrad_tc<T, BN, GATHER>, a, part, joins, wait_limit_ns(), mx, my));
    cfg.gridDim = dim3((unsigned)parts, kTileM / kJoinRows);
    cfg.blockDim = dim3(kJoinRows * BN / 4);
    cfg.dynamicSmemBytes = 0;
    SPC_CUDA_TRY(cudaLaunchKernelEx(&cfg, k_grouped_wgrad_join<BN>, a, (const float*)part, (const Join*)joins));
    return SPC_OK;
}

// Rows of one operand, `words` 16-byte words each, to their positions, a warp for a row; an entry
// out of range gives zeros.
constexpr int kBringWarps = 8;
__global__ void __launch_bounds__(kBringWarps * 32)
k_bring_rows(const uint4* __restrict__ from, const int32_t* __restrict__ list, int64_t rows, int64_t m, int words,
             uint4* __restrict__ to, int32_t* status)
{
    const int lane = threadIdx.x & 31;
    const int64_t r = (int64_t)blockIdx.x * kBringWarps + (threadIdx.x >> 5);
    if (r >= m) return;
    const int32_t i = fetch(list + r);
    const bool good = i >= 0 && i < rows;
    if (!good) set_status(status, SPC_ERR_ROW_INDEX);
    const uint4* src = from + (good ? i : 0) * (int64_t)words;
    uint4* dst = to + r * words;
#pragma unroll 4
    for (int w = lane; w < words; w += 32) dst[w] = good ? fetch(src + w) : make_uint4(0, 0, 0, 0);
}

spc_status bring(const void* from, const int32_t* list, int64_t rows, int64_t m, int32_t c, void* to, int32_t* status, cudaStream_t st)
{
    k_bring_rows<<<(unsigned)ceil_div(m, kBringWarps), kBringWarps * 32, 0, st>>>(
        static_cast<const uint4*>(from), list, rows, m, c / 8, static_cast<uint4*>(to), status);
    SPC_LAUNCH_CHECK();
    return SPC_OK;
}

// Listed rows of wide operands are brought into order first: every tile row (column) of weights would copy
// each of them again (bf16, 8 segments of 4096, 512 x 2048: 134 us against 194 by copies in the
// kernel; 398,833 rows of 128 x 128, where each is copied once: 75 in the kernel).  128 x 128 tiles where 128 x 256
// would be empty by half.
bool brings_rows(int32_t cin, int32_t cout) { return cin > kTileM && cout > kTileM; }

template <typename T>
spc_status pick(GroupedWgradArgs a, float* part, cudaStream_t st)
{
    // tiles are counted in 31 bits
    if (ceil_div(a.cin, 128) * ceil_div(a.cout, 128) * a.segments > INT32_MAX) return SPC_ERR_UNSUPPORTED;
    if ((a.x_rows || a.y_rows) && !brings_rows(a.cin, a.cout)) return launch<T, 128, true>(a, part, st);
    if (a.x_rows || a.y_rows) {
        uint8_t* x = reinterpret_cast<uint8_t*>(part) + parts_bytes();
        uint8_t* dy = x + align_up((size_t)a.m * a.cin * 2, 256);
        if (a.x_rows) {
            const spc_status s = bring(a.x, a.x_rows, a.n_x, a.m, a.cin, x, a.status, st);
            if (s != SPC_OK) return s;
            a.x = x;
            a.n_x = a.m;
        }
        if (a.y_rows) {
            const spc_status s = bring(a.dy, a.y_rows, a.n_y, a.m, a.cout, dy, a.status, st);
            if (s != SPC_OK) return s;
            a.dy = dy;
            a.n_y = a.m;
        }
        a.x_rows = a.y_rows = nullptr;
    }
    return a.cout <= 128 ? launch<T, 128, false>(a, part, st) : launch<T, 256, false>(a, part, st);
}

}  // namespace

size_t grouped_wgrad_tc_ws_bytes(int64_t m, int32_t cin, int32_t cout, bool listed)
{
    const size_t rows = listed && brings_rows(cin, cout)
                            ? align_up((size_t)m * cin * 2, 256) + align_up((size_t)m * cout * 2, 256)
                            : 0;
    return parts_bytes() + rows;
}

bool grouped_wgrad_tc_supported(const GroupedWgradArgs& a, spc_dtype dt)
{
    // an empty tensor has no tensor map
    return (dt == SPC_F16 || dt == SPC_BF16) && a.cin % 8 == 0 && a.cout % 8 == 0 && a.m > 0 && a.n_x > 0 && a.n_y > 0;
}

spc_status grouped_wgrad_tc(const GroupedWgradArgs& a, spc_dtype dt, void* ws, cudaStream_t st)
{
    float* part = static_cast<float*>(ws);
    return dt == SPC_F16 ? pick<__half>(a, part, st) : pick<__nv_bfloat16>(a, part, st);
}

}  // namespace spc
