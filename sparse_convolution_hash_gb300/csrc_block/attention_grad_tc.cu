// attention_grad_tc.cu -- the gradients of attention over segments on the 5th-generation tensor cores: two kernels,
// each of which keeps 128 rows of one side and walks over the other side's rows 64 at a time.
//   dk, dv   keeps keys: S^T = K Q^T and dP^T = V dO^T, then dV += P^T dO and dK += dS^T Q;
//   dq       keeps queries: S = Q K^T and dP = dO V^T, then dQ += dS K;
// with P = exp(S - lse) and dS = P (dP - delta), written as 16 bits in the place of S and dP, a thread to a lane.
// Seven products where five would do, were dq summed across blocks; but then its bits would hang on their order.
//
// BUFS steps are in work at any time, each with 128 columns of tensor memory and four warps (eight for heads of more than
// 64, where a block has the SM to itself): while one's probabilities are taken, the others' products run.  Three where heads of up to 64
// channels leave the columns, two beyond; one where the walk is short, so that two blocks share an SM and one's first
// loads and last stores run beside the other's steps.  S and dP are issued by one warp and the sums by another, as a warp's waits
// queue up behind its own products (8,148 us with one of one lane, 6,731 with one, 5,984 with two; four gave 6,227).
//
// 32,768 rows in 2 samples, 8 heads of 128 bf16: 6.04 ms, 940 TFLOP/s of the five products that the formula needs and
// 1,316 of the seven that run, 67% of measured cuBLAS.  The kernel of dk and dv has shared memory at work 93% of the time: 59 for the
// products' operands (a product of 128 x 64 x 16 reads 6 KB, 48 cycles for 32 of arithmetic), 34 for the columns' lse and
// delta, which every thread reads.  That of dq waits for its own chain of S, dS and sums (operands 57%, tensor cores 51%).
//
// fp16: P is kept times 2^14, and each kept row's dS times a power of two for which the largest possible value on the block's walk
// stays below 2^14, so small probabilities and gradients keep their digits.  With |P| <= 1 and |dP| <= |do| |v| that value is
// |do| max|v| + |delta| for a row of dq, max|do| |v| + max|delta| for one of dk, the maxima over rows of the same segment and
// heads: what other segments and heads hold has no say (one factor for the whole call lost the digits of segments whose do was
// smaller than another's by 2^20).  The maxima cost a block some loads before its first step: 120,000 rows in 600 windows 357 us
// against 348 with the one factor, 32,768 rows in 2 samples, 8 heads of 128 6.02 ms against 5.94.
//
// Waits are bounded as in the forward kernel.
#include "attention_tc.cuh"

namespace spc {

namespace {

constexpr int kStep = 64;       // rows of the streamed side
// Steps up to which one buffer a block and two blocks an SM are faster than three buffers (8 heads of 64, 30,000 rows in
// samples of 1,000: 382 us against 414; of 2,000: 632 and 637; of 4,096: 1,257 against 1,220; of 8,192: 2,315 against 2,182).
constexpr int kShortWalk = 40;

template <int D, int BUFS>
struct Shape {
    static constexpr int kBoxes = D / 64;
    static constexpr int kKept = 128 * 128 * kBoxes;      // bytes of the 128 rows that a block keeps
    static constexpr int kHalf = kStep * 128 * kBoxes;    // bytes of a step's rows of one operand
    static constexpr int kStage = 2 * kHalf;
    static constexpr int kStages = BUFS == 3 ? 6 : 4;
    static constexpr int kHalves = BUFS == 2 ? 2 : 1;     // four warps for each 64 / kHalves columns of a buffer
    static constexpr int kThreads = 128 + 128 * BUFS * kHalves;
    static constexpr int kCols = BUFS == 1 ? 256 : 512;   // tensor memory
    static constexpr int kBars = 3 * kStages + 4 + 3 * BUFS;
    static_assert(BUFS * 128 + 2 * D <= kCols, "");
    // where the 16 rows q of P (and dS) lie: each half's in the place of its own scores, which the other half's warps do not wait for
    static __device__ constexpr int column(int q) { return kHalves == 2 ? (q >> 1) * 32 + (q & 1) * 8 : q * 8; }
    static constexpr size_t kSmem = 1024 + 2 * (size_t)kKept + (size_t)kStages * (kStage + 2 * kStep * 4) + 8 * kBars + 16;
};

// A lane's factors of P (2^up) and of dS beside P's, and what undoes them in the sums.
struct Scales {
    float up, ds, back_p, back_ds;
};

// most: no dP - delta of this lane is larger.
template <typename T>
__device__ __forceinline__ Scales scales(float most)
{
    if constexpr (!std::is_same<T, __half>::value) return Scales{0.f, 1.f, 1.f, 1.f};
    else {
        int e = 0;
        if (most > 0.f && most < 3e38f) frexpf(most, &e);
        e = min(max(e, -100), 100);
        return Scales{14.f, ldexpf(1.f, -e), 0x1p-14f, ldexpf(1.f, e - 14)};
    }
}

// W columns of probabilities and their gradients, as 16-bit pairs.
template <typename T, int W>
__device__ __forceinline__ void grad_of(const uint32_t (&s)[W], const uint32_t (&dp)[W], F2 c, const F2 (&minus_lse)[W / 2],
                                        const F2 (&minus_delta)[W / 2], F2 ds_scale, uint32_t (&p)[W / 2], uint32_t (&ds)[W / 2])
{
#pragma unroll
    for (int y = 0; y < W / 2; ++y) {
        F2 e = fma(F2{__uint_as_float(s[2 * y]), __uint_as_float(s[2 * y + 1])}, c, minus_lse[y]);
        e = F2{ptx::ex2(e.x), ptx::ex2(e.y)};
        F2 g = add(F2{__uint_as_float(dp[2 * y]), __uint_as_float(dp[2 * y + 1])}, minus_delta[y]);
        p[y] = pack2<T>(e.x, e.y);
        if constexpr (std::is_same<T, __half>::value) g = mul(g, ds_scale);
        g = mul(g, e);
        ds[y] = pack2<T>(g.x, g.y);
    }
}

// A row of `width` channels from tensor memory, 32 columns from x on in steps of `stride`, to T or fp32 parts.
template <typename T>
__device__ __forceinline__ void store_row(uint32_t at, int x0, int stride, int d, float mul, bool there, T* out, float* part)
{
#pragma unroll 1
    for (int x = x0; x < d; x += stride) {
        uint32_t v[32];
        __syncwarp();
        ptx::tmem_ld32(at + x, v);
        ptx::tmem_ld_wait();
        if (!there) continue;
        if (part) {
#pragma unroll
            for (int y = 0; y < 32; y += 4)
                if (x + y < d)
                    *reinterpret_cast<float4*>(part + x + y) = make_float4(__uint_as_float(v[y]) * mul, __uint_as_float(v[y + 1]) * mul,
                                                                           __uint_as_float(v[y + 2]) * mul, __uint_as_float(v[y + 3]) * mul);
        } else {
#pragma unroll
            for (int y = 0; y < 32; y += 8) {
                uint4 w;
                w.x = pack2<T>(__uint_as_float(v[y]) * mul, __uint_as_float(v[y + 1]) * mul);
                w.y = pack2<T>(__uint_as_float(v[y + 2]) * mul, __uint_as_float(v[y + 3]) * mul);
                w.z = pack2<T>(__uint_as_float(v[y + 4]) * mul, __uint_as_float(v[y + 5]) * mul);
                w.w = pack2<T>(__uint_as_float(v[y + 6]) * mul, __uint_as_float(v[y + 7]) * mul);
                if (x + y < d) *reinterpret_cast<uint4*>(out + x + y) = w;
            }
        }
    }
}

template <typename T>
__device__ __forceinline__ void store_zeros(int x0, int stride, int d, bool there, T* out, float* part)
{
    if (!there) return;
    for (int x = x0; x < d; x += stride)
        for (int y = x; y < min(x + 32, d); y += 8) {
            if (part) {
                *reinterpret_cast<float4*>(part + y) = make_float4(0.f, 0.f, 0.f, 0.f);
                *reinterpret_cast<float4*>(part + y + 4) = make_float4(0.f, 0.f, 0.f, 0.f);
            } else {
                *reinterpret_cast<uint4*>(out + y) = make_uint4(0u, 0u, 0u, 0u);
            }
        }
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}

// KEYS: the kernel of dk and dv (keeps keys, walks over the queries of every head that shares them), else of dq.
// grid: slots of 128 rows, heads of the kept side, splits
template <typename T, int D, int BUFS, bool KEYS>
__global__ void __launch_bounds__(Shape<D, BUFS>::kThreads, BUFS == 1 ? 2 : 1)
k_attn_grad_tc(AttnArgs a, uint64_t wait_ns, const __grid_constant__ CUtensorMap kept1, const __grid_constant__ CUtensorMap kept2,
               const __grid_constant__ CUtensorMap step1, const __grid_constant__ CUtensorMap step2)
{
    using S = Shape<D, BUFS>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* ring = smem + 2 * S::kKept;
    float* stats = reinterpret_cast<float*>(ring + (size_t)S::kStages * S::kStage);  // [stages][2][kStep]: -lse log2 e, -delta
    uint64_t* full = reinterpret_cast<uint64_t*>(stats + S::kStages * 2 * kStep);
    uint64_t* empty = full + S::kStages;
    uint64_t* ready = empty + S::kStages;
    uint64_t* kept_full = ready + S::kStages;
    uint64_t* drain = kept_full + 1;   // of the two warps that issue
    uint64_t* s_full = drain + 2;          // [buffer]: S and dP of a step
    uint64_t* p_full = s_full + BUFS;      // [buffer]: P and dS
    uint64_t* sum_full = p_full + BUFS;    // [buffer]: the sums with them
    uint64_t* o_full = sum_full + BUFS;    // all sums
    uint32_t* s_ctrl = reinterpret_cast<uint32_t*>(o_full + 1);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    wait_for_kernel_before();
    const int32_t* seg = KEYS ? a.seg_k : a.seg_q;
    const int64_t rows = KEYS ? a.nk : a.nq;
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) attn_check(seg, a.segments, rows, a.status, tid, S::kThreads);
    AttnTile t;
    if (!attn_tile(seg, KEYS ? a.seg_q : a.seg_k, a.segments, rows, KEYS ? a.nq : a.nk, 128, blockIdx.x, t)) return;
    const int per = a.hq / a.hk;
    const int kept_head = blockIdx.y, splits = KEYS ? a.splits_kv : a.splits;
    // steps [from, to) of all: KEYS, those of every query head, one head after the other
    const int64_t steps_each = (t.hi - t.lo + kStep - 1) / kStep, all = steps_each * (KEYS ? per : 1);
    const int64_t from = all * blockIdx.z / splits, to = all * (blockIdx.z + 1) / splits;
    const int n = (int)(to - from);
    auto step_head = [&](int j) { return KEYS ? kept_head * per + (int)((from + j) / steps_each) : kept_head / per; };
    auto step_row = [&](int j) { return t.lo + (KEYS ? (from + j) % steps_each : from + j) * kStep; };

    if (tid == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            ptx::mbar_init(&full[s], 1);
            ptx::mbar_init(&empty[s], 1);
            ptx::mbar_init(&ready[s], 32);
        }
        ptx::mbar_init(kept_full, 1);
        ptx::mbar_init(&drain[0], 1);
        ptx::mbar_init(&drain[1], 1);
        for (int i = 0; i < BUFS; ++i) {
            ptx::mbar_init(&sum_full[i], 1);
            ptx::mbar_init(&s_full[i], 1);
            ptx::mbar_init(&p_full[i], 4 * S::kHalves);
        }
        ptx::mbar_init(o_full, 1);
        ptx::mbar_init_fence();
    }
    if (warp == 1) {
        ptx::tmem_alloc(s_ctrl, S::kCols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = s_ctrl[0], kept_base = ptx::smem_u32(smem), ring_base = ptx::smem_u32(ring);
    // tensor memory: step buffers of 128 columns (S, dP), then the sums: dv and dk, or dq
    const uint32_t sum1 = tmem + BUFS * 128, sum2 = sum1 + D;
    bool ok = true;
    if (warp == 0) {
        // ------------------------------------------------------------ loads
        if (n > 0) {
            if (attn_elect()) {
                ptx::mbar_arrive_expect_tx(kept_full, 2 * S::kKept);
#pragma unroll
                for (int b = 0; b < S::kBoxes; ++b) {
                    ptx::tma_load3d<1>(kept_base + b * 16384, &kept1, b * 64, kept_head, (int32_t)t.row, ptx::smem_u32(kept_full));
                    ptx::tma_load3d<1>(kept_base + S::kKept + b * 16384, &kept2, b * 64, kept_head, (int32_t)t.row, ptx::smem_u32(kept_full));
                }
            }
            __syncwarp();
            int it = 0, head = step_head(0), row = (int)step_row(0);
            for (; it < n; ++it) {
                const int s = it % S::kStages;
                if (it >= S::kStages) ok = attn_wait(&empty[s], (it / S::kStages - 1) & 1, wait_ns);
                if (!ok) break;
                if (attn_elect()) {
                    const uint32_t base = ring_base + (uint32_t)s * S::kStage, bar = ptx::smem_u32(&full[s]);
                    ptx::mbar_arrive_expect_tx(&full[s], S::kStage);
#pragma unroll
                    for (int b = 0; b < S::kBoxes; ++b) {
                        ptx::tma_load3d<1>(base + b * (kStep * 128), &step1, b * 64, head, row, bar);
                        ptx::tma_load3d<1>(base + S::kHalf + b * (kStep * 128), &step2, b * 64, head, row, bar);
                    }
                }
                __syncwarp();
                row += kStep;
                if (KEYS && row >= t.hi) {
                    row = (int)t.lo;
                    ++head;
                }
            }
            if (!ok && lane == 0) set_status(a.status, SPC_ERR_TIMEOUT);
            // what is in flight has to land before the block's shared memory goes
            ptx::mbar_wait(kept_full, 0, kAttnDrainNs);
            for (int j = it > S::kStages ? it - S::kStages : 0; j < it; ++j)
                ptx::mbar_wait(&full[j % S::kStages], (j / S::kStages) & 1, kAttnDrainNs);
        }
    } else if (warp == 1 || warp == 3) {
        // -------------------- MMAs: S and dP by one warp, the sums by another, as a warp's waits queue up behind its own
        if (n > 0) {
            const int steps = (a.d + 15) / 16;
            if (warp == 1) {
                const uint32_t idesc = ptx::idesc_make(AttnFmt<T>::v, 128, kStep);
                const uint64_t kept_desc = ptx::desc_k_sw128(kept_base), k_desc = ptx::desc_k_sw128(ring_base);
                ok = attn_wait(kept_full, 0, wait_ns);
                for (int j = 0; j < n && ok; ++j) {
                    const int s = j % S::kStages;
                    const uint32_t parity = (j / S::kStages) & 1;
                    ok = attn_wait(&full[s], parity, wait_ns) && (!KEYS || attn_wait(&ready[s], parity, wait_ns));
                    // in the place of P and dS, once the sums of step j - BUFS have them
                    const int b = j % BUFS;
                    if (ok && j >= BUFS) ok = attn_wait(&sum_full[b], (j / BUFS - 1) & 1, wait_ns);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    if (attn_elect()) {
                        const uint64_t rows = k_desc + s * (S::kStage >> 4);
                        const uint32_t d = tmem + b * 128;
                        attn_mma_ss<D / 16>(d, kept_desc, 16384, rows, kStep * 128, idesc, steps);
                        attn_mma_ss<D / 16>(d + 64, kept_desc + (S::kKept >> 4), 16384, rows + (S::kHalf >> 4), kStep * 128, idesc, steps);
                        ptx::mma_commit(&s_full[b]);
                    }
                    __syncwarp();
                }
            } else {
                const uint32_t idesc = ptx::idesc_make(AttnFmt<T>::v, 128, steps * 16) | 1u << 16;
                const uint64_t mn_desc = ptx::desc_mn_sw128(ring_base, kStep * 128);
                for (int j = 0; j < n && ok; ++j) {
                    const int s = j % S::kStages, b = j % BUFS;
                    const uint32_t parity = (j / S::kStages) & 1;
                    ok = attn_wait(&full[s], parity, wait_ns) && (!KEYS || attn_wait(&ready[s], parity, wait_ns)) &&
                         attn_wait(&p_full[b], (j / BUFS) & 1, wait_ns);
                    if (!ok) break;
                    ptx::tc_fence_after();
                    if (attn_elect()) {
                        const uint32_t p = tmem + b * 128;
                        const uint64_t d1 = mn_desc + s * (S::kStage >> 4), d2 = d1 + (S::kHalf >> 4);
                        if (KEYS) {
#pragma unroll
                            for (int q = 0; q < kStep / 16; ++q) ptx::mma_f16_ts(sum1, p + S::column(q), d2 + q * 128, idesc, q > 0 || j > 0);  // dV += P^T dO
                        }
#pragma unroll
                        for (int q = 0; q < kStep / 16; ++q)  // dK += dS^T Q, dQ += dS K
                            ptx::mma_f16_ts(KEYS ? sum2 : sum1, p + 64 + S::column(q), d1 + q * 128, idesc, q > 0 || j > 0);
                        ptx::mma_commit(&sum_full[b]);
                        ptx::mma_commit(&empty[s]);
                        if (j + 1 == n) ptx::mma_commit(o_full);
                    }
                    __syncwarp();
                }
            }
            if (!ok && lane == 0) set_status(a.status, SPC_ERR_TIMEOUT);
            uint64_t* mine = &drain[warp >> 1];
            if (attn_elect()) ptx::mma_commit(mine);
            __syncwarp();
            ptx::mbar_wait(mine, 0, kAttnDrainNs);
        }
    } else if (warp == 2) {
        // ------------------------------- the queries' log-sums and row sums, and rows past the segment's end
        if (KEYS) {
            int64_t row = n > 0 ? step_row(0) : 0;
            int head = n > 0 ? step_head(0) : 0;
            for (int it = 0; it < n; ++it) {
                const int s = it % S::kStages;
                if (it >= S::kStages) ok = attn_wait(&empty[s], (it / S::kStages - 1) & 1, wait_ns);
                if (!ok) break;
                const int64_t at = (int64_t)head * a.nq + row;
                const int valid = (int)min((int64_t)kStep, t.hi - row);
                float* to_s = stats + s * 2 * kStep;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int i = lane + 32 * x;
                    if (i < valid) {
                        cp_async4(ptx::smem_u32(to_s + i), a.lse2 + at + i);
                        cp_async4(ptx::smem_u32(to_s + kStep + i), a.delta + at + i);
                    }
                }
                if (valid == kStep) {
                    ptx::cp_async_arrive_noinc(&ready[s]);
                } else {
                    for (int i = valid + lane; i < kStep; i += 32) {
                        to_s[i] = -INFINITY;  // no probability
                        to_s[kStep + i] = 0.f;
                    }
                    ok = attn_wait(&full[s], (it / S::kStages) & 1, wait_ns);
                    if (!ok) break;
                    const uint32_t base = ring_base + (uint32_t)s * S::kStage;
                    attn_clear_rows<S::kBoxes>(base, kStep, valid, lane, 32);
                    attn_clear_rows<S::kBoxes>(base + S::kHalf, kStep, valid, lane, 32);
                    ptx::cp_async_wait_all();
                    ptx::mbar_arrive(&ready[s]);
                }
                row += kStep;
                if (row >= t.hi) {
                    row = t.lo;
                    ++head;
                }
            }
            if (!ok && lane == 0) set_status(a.status, SPC_ERR_TIMEOUT);
            ptx::cp_async_wait_all();
        }
    } else if (warp >= 4) {
        // ------------------------------------------- probabilities, their gradients, results
        const int b = (warp - 4) / (4 * S::kHalves), half = ((warp - 4) >> 2) % S::kHalves, quarter = warp & 3, r = quarter * 32 + lane;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const uint32_t s_at = tmem + lanes + b * 128;
        const float c = a.scale * kLog2e;
        const int64_t row = t.row + r;
        const bool there = row < t.end;
        float my_lse = -INFINITY, my_delta = 0.f;
        if (!KEYS && there) {
            my_lse = fetch(a.lse2 + (int64_t)kept_head * a.nq + row);
            my_delta = fetch(a.delta + (int64_t)kept_head * a.nq + row);
        }
        float most = 0.f;
        if constexpr (std::is_same<T, __half>::value) {
            const float mine = there ? fetch(KEYS ? a.norm_v + kept_head * a.nk + row : a.norm_do + kept_head * a.nq + row) : 0.f;
            // the largest norms (and, of queries, |delta|) of the rows on the walk
            constexpr int kWarps = 4 * BUFS * S::kHalves;
            __shared__ float tops[2][kWarps];
            float top = 0.f, top_delta = 0.f;
            auto take = [&](int head, int64_t begin, int64_t end) {
                const int64_t first = head * (KEYS ? a.nq : a.nk);
                const float* norms = (KEYS ? a.norm_do : a.norm_v) + first;
                const float* deltas = a.delta + first;
#pragma unroll 4
                for (int64_t at = begin + tid - 128; at < end; at += 32 * kWarps) {
                    top = fmaxf(top, fetch(norms + at));
                    if (KEYS) {
                        const float delta = fabsf(fetch(deltas + at));
                        top_delta = fmaxf(top_delta, delta < INFINITY ? delta : 0.f);
                    }
                }
            };
            if (splits == 1) {  // without the divisions (120,000 rows in 600 windows 366 us against 372)
                for (int h = 0; h < (KEYS ? per : 1); ++h) take(KEYS ? kept_head * per + h : kept_head / per, t.lo, t.hi);
            } else if (n > 0) {
                const int first = step_head(0), last = step_head(n - 1);
                const int64_t begin = step_row(0), end = min(t.hi, step_row(n - 1) + kStep);
                for (int h = first; h <= last; ++h) take(h, h == first ? begin : t.lo, h == last ? end : t.hi);
            }
            // non-negative numbers are ordered as their bits
            top = __uint_as_float(__reduce_max_sync(FULL_MASK, __float_as_uint(top)));
            top_delta = __uint_as_float(__reduce_max_sync(FULL_MASK, __float_as_uint(top_delta)));
            if (lane == 0) {
                tops[0][warp - 4] = top;
                tops[1][warp - 4] = top_delta;
            }
            ptx::bar_sync_named(1, 32 * kWarps);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                top = fmaxf(top, tops[0][w]);
                top_delta = fmaxf(top_delta, tops[1][w]);
            }
            most = fmaf(top, mine, KEYS ? top_delta : fabsf(my_delta));
        }
        const Scales sc = scales<T>(most);
        my_lse += sc.up;
        for (int j = b; j < n; j += BUFS) {
            const int s = j % S::kStages;
            ok = attn_wait(&s_full[b], (j / BUFS) & 1, wait_ns);
            if (KEYS && ok) ok = attn_wait(&ready[s], (j / S::kStages) & 1, wait_ns);
            if (!ok) break;
            ptx::tc_fence_after();
            const float* st = stats + s * 2 * kStep;
            const int64_t left = KEYS ? kStep : t.hi - step_row(j);
            // minus lse and minus delta of W columns from x on
            auto column_stats = [&](auto& ml, auto& md, int x) {
                constexpr int H = sizeof(ml) / sizeof(F2);
#pragma unroll
                for (int y = 0; y < H; y += 2) {
                    float4 l4 = make_float4(my_lse, my_lse, my_lse, my_lse), d4 = make_float4(my_delta, my_delta, my_delta, my_delta);
                    if (KEYS) {
                        l4 = *reinterpret_cast<const float4*>(st + x + 2 * y);
                        d4 = *reinterpret_cast<const float4*>(st + kStep + x + 2 * y);
                    }
                    ml[y] = F2{l4.x, l4.y};
                    ml[y + 1] = F2{l4.z, l4.w};
                    if constexpr (KEYS && std::is_same<T, __half>::value) {
                        ml[y] = add(ml[y], both(sc.up));
                        ml[y + 1] = add(ml[y + 1], both(sc.up));
                    }
                    md[y] = F2{d4.x, d4.y};
                    md[y + 1] = F2{d4.z, d4.w};
                }
            };
            // dS of keys past the segment's end is zero (their S and dP may be NaN)
            auto cut = [&](auto& ds, int x) {
                if (!KEYS && left < kStep) {
                    constexpr int H = sizeof(ds) / 4;
#pragma unroll
                    for (int y = 0; y < H; ++y)
                        ds[y] &= (x + 2 * y < left ? 0x0000ffffu : 0u) | (x + 2 * y + 1 < left ? 0xffff0000u : 0u);
                }
            };
            // P and dS go in the place of columns that have been read, half as many
            constexpr int kColumns = kStep / S::kHalves;
            const int x0 = half * kColumns;
            uint32_t sv[2][16], dp[2][16];
            ptx::tmem_ld16(s_at + x0, sv[0]);
            ptx::tmem_ld16(s_at + 64 + x0, dp[0]);
#pragma unroll
            for (int x = 0; x < kColumns; x += 16) {
                const int now = x >> 4 & 1;
                uint32_t p[8], ds[8];
                F2 ml[8], md[8];
                column_stats(ml, md, x0 + x);
                ptx::tmem_ld_wait();
                if (x + 16 < kColumns) {  // the next columns while these are worked on
                    ptx::tmem_ld16(s_at + x0 + x + 16, sv[now ^ 1]);
                    ptx::tmem_ld16(s_at + 64 + x0 + x + 16, dp[now ^ 1]);
                }
                grad_of<T, 16>(sv[now], dp[now], both(c), ml, md, both(sc.ds), p, ds);
                cut(ds, x0 + x);
                if (KEYS) ptx::tmem_st8(s_at + x0 + x / 2, p);
                ptx::tmem_st8(s_at + 64 + x0 + x / 2, ds);
            }
            ptx::tmem_st_wait();
            if (!KEYS && left < kStep) {
                ok = attn_wait(&full[s], (j / S::kStages) & 1, wait_ns);
                if (!ok) break;
                attn_clear_rows<S::kBoxes>(ring_base + (uint32_t)s * S::kStage, kStep, (int)left, half * 128 + r, 128 * S::kHalves);
            }
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&p_full[b]);
        }
        if (ok && n > 0) ok = attn_wait(o_full, 0, wait_ns);
        ptx::tc_fence_after();
        if (!ok && lane == 0) set_status(a.status, SPC_ERR_TIMEOUT);
        if (ok) {
            if (KEYS) {
                // the first four warps dv, the next ones dk
                const int64_t width = (int64_t)a.hk * a.d, off = row * width + (int64_t)kept_head * a.d, one = a.nk * width;
                for (int which = b; which < 2; which += BUFS == 1 ? 1 : 2) {
                    T* out = which == 0 ? static_cast<T*>(a.dv) + row * a.lddv + (int64_t)kept_head * a.d
                                        : static_cast<T*>(a.dk) + row * a.lddk + (int64_t)kept_head * a.d;
                    float* part = splits > 1 ? a.part_kv + ((which == 0 ? splits : 0) + blockIdx.z) * one + off : nullptr;
                    const int x0 = 32 * half, stride = 32 * S::kHalves;
                    if (n > 0) store_row<T>((which == 0 ? sum1 : sum2) + lanes, x0, stride, a.d, which == 0 ? sc.back_p : sc.back_ds * a.scale, there, out, part);
                    else store_zeros<T>(x0, stride, a.d, there, out, part);
                }
            } else if (b < 2) {
                T* out = static_cast<T*>(a.dq) + row * a.lddq + (int64_t)kept_head * a.d;
                float* part = splits > 1 ? a.part + ((blockIdx.z * a.nq + row) * a.hq + kept_head) * a.d : nullptr;
                const int x0 = 32 * (b * S::kHalves + half);
                constexpr int kStride = 32 * (BUFS == 1 ? 1 : 2) * S::kHalves;
                if (n > 0) store_row<T>(sum1 + lanes, x0, kStride, a.d, sc.back_ds * a.scale, there, out, part);
                else store_zeros<T>(x0, kStride, a.d, there, out, part);
            }
        }
    }
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, S::kCols);
    }
}

template <typename T, int D, int BUFS, bool KEYS>
spc_status launch(const AttnArgs& a, cudaStream_t st)
{
    using S = Shape<D, BUFS>;
    CUtensorMap q, g, k, v;
    const int box_q = KEYS ? kStep : 128, box_k = KEYS ? 128 : kStep;
    if (!attn_tmap<T>(&q, a.q, a.ldq, a.nq, a.hq, a.d, 1, box_q) || !attn_tmap<T>(&g, a.dout, a.lddo, a.nq, a.hq, a.d, 1, box_q) ||
        !attn_tmap<T>(&k, a.k, a.ldk, a.nk, a.hk, a.d, 1, box_k) || !attn_tmap<T>(&v, a.v, a.ldv, a.nk, a.hk, a.d, 1, box_k))
        return SPC_ERR_UNSUPPORTED;
    const int64_t slots = attn_slots(KEYS ? a.nk : a.nq, a.segments, 128);
    if (slots > INT32_MAX) return SPC_ERR_UNSUPPORTED;
    const spc_status s = allow_smem<k_attn_grad_tc<T, D, BUFS, KEYS>>();
    if (s != SPC_OK) return s;
    const dim3 grid((unsigned)slots, (unsigned)(KEYS ? a.hk : a.hq), (unsigned)(KEYS ? a.splits_kv : a.splits));
    if (KEYS) return attn_start_kernel<k_attn_grad_tc<T, D, BUFS, KEYS>>(grid, S::kThreads, S::kSmem, st, a, wait_limit_ns(), k, v, q, g);
    return attn_start_kernel<k_attn_grad_tc<T, D, BUFS, KEYS>>(grid, S::kThreads, S::kSmem, st, a, wait_limit_ns(), q, g, k, v);
}

template <typename T, bool KEYS>
spc_status pick(const AttnArgs& a, cudaStream_t st)
{
    if (a.d > 64) return launch<T, 128, 2, KEYS>(a, st);
    // steps of a block's walk, were all segments alike
    const int64_t steps = KEYS ? ceil_div(a.nq, (int64_t)a.segments * kStep) * (a.hq / a.hk) / a.splits_kv
                               : ceil_div(a.nk, (int64_t)a.segments * kStep) / a.splits;
    return steps <= kShortWalk ? launch<T, 64, 1, KEYS>(a, st) : launch<T, 64, 3, KEYS>(a, st);
}

template <typename T>
spc_status both_kernels(const AttnArgs& a, cudaStream_t st)
{
    const spc_status s = pick<T, true>(a, st);
    return s != SPC_OK ? s : pick<T, false>(a, st);
}

}  // namespace

spc_status attention_bwd_tc(const AttnArgs& a, spc_dtype dt, cudaStream_t st)
{
    return dt == SPC_F16 ? both_kernels<__half>(a, st) : both_kernels<__nv_bfloat16>(a, st);
}

}  // namespace spc
