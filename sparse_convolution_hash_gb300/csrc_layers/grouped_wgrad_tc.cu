// grouped_wgrad_tc.cu -- dW[g] = sum over g's positions of x[x_rows(r)]^T dy[y_rows(r)]
// on the 5th-generation tensor cores, fp32 result.
//
// The reduction runs over rows, so both operands are MN-major: a row of a stage
// is 64 channels (M or N) of one reduction index, and a tile is 128 input x BN output
// channels.  Segments differ in length and there may be fewer tiles than SMs,
// so the work is cut by units of 64 rows of one tile: all units of all tiles in a row, in equal
// shares, one for each CTA.  A tile inside one share is written to dW as it
// is; the parts of the others go to the workspace and a second kernel adds them in the
// order of the rows: no atomics, run-to-run identical.
//
// In a CTA, as in the forward: warp 0 loads dense rows by TMA, warps 6-13 copy listed
// rows by cp.async, warp 1 issues the MMAs into one of two accumulators and
// first clears the rows of a last, partial unit past the segment's end (they hold the
// next segment's rows: a zero weight would not do, as 0 x NaN is NaN), warps 2-5 store
// the other accumulator.  Every wait is bounded (SPC_ERR_TIMEOUT).
#include "kernels.cuh"
#include "layers.cuh"
#include "tc2.cuh"
#include "tmap.cuh"

namespace spc {

namespace {

constexpr int kThreads = 192;
constexpr int kGatherThreads = 256;
constexpr int kUnit = 64;    // rows of a unit
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
    static constexpr int kStaging = 4 * 32 * 128;
    static size_t smem(int segments)
    {
        return 1024 + (size_t)kStages * kStage + kStaging + 8 * (2 * kStages + 4) + 16 + 4 * ((size_t)segments + 1);
    }
};

template <typename T> struct Fmt;
template <> struct Fmt<__half> { static constexpr uint32_t v = 0; static constexpr CUtensorMapDataType t = CU_TENSOR_MAP_DATA_TYPE_FLOAT16; };
template <> struct Fmt<__nv_bfloat16> { static constexpr uint32_t v = 1; static constexpr CUtensorMapDataType t = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16; };

// A part of one tile: units [k0, k1) of its `units`.
struct Piece {
    int32_t g, tile;
    int32_t k0, k1, units;
    int64_t lo, hi;  // positions of the segment
    __device__ __forceinline__ bool whole() const { return k0 == 0 && k1 == units; }
};

// The shares: s_start[g] = units (of 64 rows, at least one) of the segments before g.
struct Shares {
    const int32_t* start;
    const int32_t* seg;
    int64_t m;
    int32_t segments, tiles;  // tiles of one segment
    int64_t total;            // units of all tiles
    int32_t parts;

    __device__ __forceinline__ int64_t first(int32_t part) const { return total * part / parts; }
    __device__ __forceinline__ Piece at(int64_t u, int64_t end) const
    {
        const int32_t f = (int32_t)(u / tiles);
        int lo = 0, hi = segments;  // last g with start[g] <= f
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (start[mid] <= f) lo = mid;
            else hi = mid;
        }
        Piece p;
        p.g = lo;
        p.units = start[lo + 1] - start[lo];
        const int64_t in = u - (int64_t)start[lo] * tiles;
        p.tile = (int32_t)(in / p.units);
        p.k0 = (int32_t)(in - (int64_t)p.tile * p.units);
        const int64_t left = end - u;
        p.k1 = p.units - p.k0 <= left ? p.units : p.k0 + (int32_t)left;
        segment_bounds(seg, lo, m, nullptr, p.lo, p.hi);
        return p;
    }
};

// Fills s_start [segments + 1]; every thread of the block calls it.
__device__ __forceinline__ void unit_starts(const int32_t* seg, int segments, int64_t m, int32_t* s_start,
                                            int32_t* status, int tid, int threads)
{
    __shared__ int32_t s_warp[32];
    const int lane = tid & 31, warp = tid >> 5;
    int32_t carry = 0;
    for (int g0 = 0; g0 < segments; g0 += threads) {
        const int g = g0 + tid;
        int32_t units = 0;
        if (g < segments) {
            int64_t a, b;
            segment_bounds(seg, g, m, status, a, b);
            units = b > a ? (int32_t)((b - a + kUnit - 1) / kUnit) : 1;
        }
        int32_t inc = units;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int32_t u = __shfl_up_sync(FULL_MASK, inc, d);
            if (lane >= d) inc += u;
        }
        if (lane == 31) s_warp[warp] = inc;
        __syncthreads();
        int32_t base = carry;
        for (int w = 0; w < threads / 32; ++w) {
            if (w < warp) base += s_warp[w];
            carry += s_warp[w];
        }
        if (g < segments) s_start[g] = base + inc - units;
        __syncthreads();
    }
    if (tid == 0) s_start[segments] = carry;
    __syncthreads();
}

// The tile that starts in share c and ends in a later one: its parts are slot `slot` of c
// and the first slots of the `more` shares after it (0: there is none).
struct Join {
    int32_t g, tile, slot, more;
};

__device__ __forceinline__ Join join_plan(const Shares& sh, int c, int64_t u0, int64_t u1)
{
    Join j{0, 0, 0, 0};
    if (u0 == u1) return j;
    const Piece p = sh.at(u1 - 1, u1);
    const int64_t first = u1 - 1 - p.k0, end = first + p.units;
    if (first < u0 || end <= u1) return j;
    j.g = p.g;
    j.tile = p.tile;
    j.slot = first == u0 ? 0 : 1;
    while (c + 1 + j.more < sh.parts && sh.first(c + 1 + j.more) < end) ++j.more;
    return j;
}

template <typename T, int BN, bool GATHER>
__global__ void __launch_bounds__(GATHER ? kThreads + kGatherThreads : kThreads, 1)
k_grouped_wgrad_tc(GroupedWgradArgs a, float* __restrict__ part, Join* __restrict__ plan, uint64_t wait_ns,
                   const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_dy)
{
    using S = Shape<BN>;
    constexpr int kAll = GATHER ? kThreads + kGatherThreads : kThreads;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* staging = smem + (size_t)S::kStages * S::kStage;
    uint64_t* full = reinterpret_cast<uint64_t*>(staging + S::kStaging);
    uint64_t* empty = full + S::kStages;
    uint64_t* acc_full = empty + S::kStages;
    uint64_t* acc_empty = acc_full + 2;
    uint32_t* s_ctrl = reinterpret_cast<uint32_t*>(acc_empty + 2);
    int32_t* s_start = reinterpret_cast<int32_t*>(s_ctrl + 4);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            ptx::mbar_init(&full[s], GATHER ? kGatherThreads : 1);
            ptx::mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            ptx::mbar_init(&acc_full[b], 1);
            ptx::mbar_init(&acc_empty[b], 4);
        }
        ptx::mbar_init_fence();
        if (!GATHER) {
            ptx::prefetch_tmap(&map_x);
            ptx::prefetch_tmap(&map_dy);
        }
    }
    if (warp == 1) ptx::tmem_alloc_cg<1>(s_ctrl, S::kTmemCols);
    unit_starts(a.seg, a.segments, a.m, s_start, blockIdx.x == 0 ? a.status : nullptr, tid, kAll);
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = s_ctrl[0];
    const int cols = (a.cout + BN - 1) / BN, tiles = (a.cin + kTileM - 1) / kTileM * cols;
    const int64_t total = (int64_t)s_start[a.segments] * tiles;
    const int32_t parts = total < (int64_t)gridDim.x ? (int32_t)total : (int32_t)gridDim.x;
    const Shares sh{s_start, a.seg, a.m, a.segments, tiles, total, parts};
    const bool at_work = (int)blockIdx.x < parts;
    const int64_t u0 = at_work ? sh.first(blockIdx.x) : 0, u1 = at_work ? sh.first(blockIdx.x + 1) : 0;
    bool ok = true;
    if (tid == 0) plan[blockIdx.x] = join_plan(sh, blockIdx.x, u0, u1);

    if (warp == 0) {
        // ------------------------------------------------------ dense loads
        if (!GATHER && lane == 0) {
            uint32_t it = 0;
            for (int64_t u = u0; u < u1 && ok;) {
                const Piece p = sh.at(u, u1);
                u += p.k1 - p.k0;
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
        for (int64_t u = u0; u < u1 && ok;) {
            const Piece p = sh.at(u, u1);
            u += p.k1 - p.k0;
            if (p.lo == p.hi) continue;
            const uint32_t b = n & 1;
            if (n >= 2) ok = __all_sync(FULL_MASK, ptx::mbar_wait(&acc_empty[b], ((n >> 1) - 1) & 1, wait_ns));
            if (!ok) break;
            ptx::tc_fence_after();
            const uint32_t d = tmem + b * BN;
            for (int k = p.k0; k < p.k1; ++k, ++it) {
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
                if (lane == 0) {
                    if (GATHER) ptx::fence_proxy_async_smem();
                    ptx::tc_fence_after();
                    const uint32_t base = ptx::smem_u32(stage);
                    const uint64_t ad = ptx::desc_mn_sw128(base, kAtom), bd = ptx::desc_mn_sw128(base + S::kABytes, kAtom);
#pragma unroll
                    for (int q = 0; q < kUnit / 16; ++q)
                        ptx::mma_f16<1>(d, ad + (uint64_t)(q * (2048 >> 4)), bd + (uint64_t)(q * (2048 >> 4)), idesc,
                                        k != p.k0 || q != 0);
                    ptx::mma_commit(&empty[s]);
                }
                __syncwarp();
            }
            if (!ok) break;
            if (lane == 0) ptx::mma_commit(&acc_full[b]);
            ++n;
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
            for (int64_t u = u0; u < u1 && ok;) {
                const Piece p = sh.at(u, u1);
                u += p.k1 - p.k0;
                if (p.lo == p.hi) continue;
                const int c0 = p.tile / cols * kTileM + piece * 8, n0 = p.tile % cols * BN + piece * 8;
                // the rows of thread e's two reduction indices of unit k (-1: zeros)
                auto rows = [&](int k, int64_t (&xr)[2], int64_t (&yr)[2]) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const int64_t r = p.lo + (int64_t)k * kUnit + r0 + 32 * j;
                        xr[j] = yr[j] = -1;
                        if (k < p.k1 && r < p.hi) {
                            xr[j] = row_at(a.x_rows, r, a.n_x, a.status);
                            yr[j] = row_at(a.y_rows, r, a.n_y, a.status);
                            if (xr[j] < 0 || yr[j] < 0) xr[j] = yr[j] = -1;
                        }
                    }
                };
                int64_t xr[2], yr[2], xn[2], yn[2];
                rows(p.k0, xr, yr);
                for (int k = p.k0; k < p.k1; ++k, ++it) {
                    rows(k + 1, xn, yn);
                    const int s = it % S::kStages;
                    if (it >= S::kStages) ok = ptx::mbar_wait(&empty[s], ((it / S::kStages) - 1) & 1, wait_ns);
                    if (!ok) break;
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
                        xr[j] = xn[j];
                        yr[j] = yn[j];
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
        uint8_t* box = staging + (warp - 2) * (32 * 128);
        uint32_t n = 0;
        for (int64_t u = u0; u < u1 && ok;) {
            const Piece p = sh.at(u, u1);
            const bool at_start = u == u0;
            u += p.k1 - p.k0;
            const uint32_t b = n & 1;
            const bool some = p.lo != p.hi;
            if (some) {
                ok = __all_sync(FULL_MASK, ptx::mbar_wait(&acc_full[b], (n >> 1) & 1, wait_ns));
                if (!ok) break;
                ptx::tc_fence_after();
                ++n;
            }
            const int c0 = p.tile / cols * kTileM + quarter * 32, n0 = p.tile % cols * BN;
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
                dst = part + ((int64_t)blockIdx.x * 2 + (at_start ? 0 : 1)) * (kTileM * BN) + quarter * 32 * BN;
                pitch = BN;
                rows = 32;
                width = BN;
            }
            const int piece = lane & 7;
#pragma unroll 1
            for (int c = 0; c < BN / 32 && c * 32 < width; ++c) {
                uint32_t v[32];
                if (some) {
                    ptx::tmem_ld32(tmem + ((uint32_t)(quarter * 32) << 16) + b * BN + c * 32, v);
                    ptx::tmem_ld_wait();
                } else {
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = 0u;
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    *reinterpret_cast<uint4*>(box + lane * 128 + ((j ^ (lane & 7)) << 4)) =
                        make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int rr = j * 4 + (lane >> 3);
                    const uint4 w = *reinterpret_cast<const uint4*>(box + rr * 128 + ((piece ^ (rr & 7)) << 4));
                    if (rr < rows && c * 32 + piece * 4 < width)
                        *reinterpret_cast<uint4*>(dst + rr * pitch + c * 32 + piece * 4) = w;
                }
                __syncwarp();
            }
            if (some) {
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(&acc_empty[b]);
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
k_grouped_wgrad_join(GroupedWgradArgs a, const float* __restrict__ part, const Join* __restrict__ plan)
{
    const int c = blockIdx.x;
    const Join j = plan[c];
    if (j.more == 0) return;
    const int cols = (a.cout + BN - 1) / BN;
    const int r = blockIdx.y * kJoinRows + threadIdx.x / (BN / 4), n = threadIdx.x % (BN / 4) * 4;
    const int row = j.tile / cols * kTileM + r, col = j.tile % cols * BN + n;
    if (row >= a.cin || col >= a.cout) return;
    constexpr int64_t kSlot = kTileM * BN;
    const float* src = part + r * BN + n;
    float4 s = __ldcs(reinterpret_cast<const float4*>(src + ((int64_t)c * 2 + j.slot) * kSlot));
    src += (int64_t)(c + 1) * 2 * kSlot;
#pragma unroll 8
    for (int q = 0; q < j.more; ++q) {
        const float4 v = __ldcs(reinterpret_cast<const float4*>(src + q * 2 * kSlot));
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
    }
    *reinterpret_cast<float4*>(a.dw + ((int64_t)j.g * a.cin + row) * a.cout + col) = s;
}

template <typename T, int BN, bool GATHER>
spc_status launch(const GroupedWgradArgs& a, float* part, cudaStream_t st)
{
    using S = Shape<BN>;
    CUtensorMap mx, my;
    if (!tmap_2d(&mx, Fmt<T>::t, 2, a.x, (uint64_t)a.cin, (uint64_t)a.n_x, 64, kUnit, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !tmap_2d(&my, Fmt<T>::t, 2, a.dy, (uint64_t)a.cout, (uint64_t)a.n_y, 64, kUnit, CU_TENSOR_MAP_SWIZZLE_128B))
        return SPC_ERR_CUDA;
    auto* kernel = k_grouped_wgrad_tc<T, BN, GATHER>;
    const size_t smem = S::smem(a.segments);
    SPC_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem));
    const int parts = grouped_wgrad_parts();
    Join* plan = reinterpret_cast<Join*>(part + (int64_t)parts * 2 * kTileM * 256);
    kernel<<<parts, GATHER ? kThreads + kGatherThreads : kThreads, smem, st>>>(a, part, plan, wait_limit_ns(), mx, my);
    SPC_LAUNCH_CHECK();
    k_grouped_wgrad_join<BN><<<dim3(parts, kTileM / kJoinRows), kJoinRows * BN / 4, 0, st>>>(a, part, plan);
    SPC_LAUNCH_CHECK();
    return SPC_OK;
}

template <typename T, int BN>
spc_status pick(const GroupedWgradArgs& a, float* part, cudaStream_t st)
{
    return a.x_rows || a.y_rows ? launch<T, BN, true>(a, part, st) : launch<T, BN, false>(a, part, st);
}

}  // namespace

int grouped_wgrad_parts() { return sm_count(); }

// Two parts of a tile for each CTA.
size_t grouped_wgrad_tc_ws_bytes()
{
    return align_up((sizeof(float) * 2 * kTileM * 256 + sizeof(Join)) * (size_t)grouped_wgrad_parts(), 256);
}

bool grouped_wgrad_tc_supported(const GroupedWgradArgs& a, spc_dtype dt)
{
    return (dt == SPC_F16 || dt == SPC_BF16) && a.cin % 8 == 0 && a.cout % 8 == 0 && a.n_x > 0 && a.n_y > 0;
}

spc_status grouped_wgrad_tc(const GroupedWgradArgs& a, spc_dtype dt, void* ws, cudaStream_t st)
{
    float* part = static_cast<float*>(ws);
    if (dt == SPC_F16) return a.cout <= 128 ? pick<__half, 128>(a, part, st) : pick<__half, 256>(a, part, st);
    return a.cout <= 128 ? pick<__nv_bfloat16, 128>(a, part, st) : pick<__nv_bfloat16, 256>(a, part, st);
}

}  // namespace spc
