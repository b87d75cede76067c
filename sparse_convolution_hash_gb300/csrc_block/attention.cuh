// attention.cuh -- what the attention kernels share: how a block finds its tile among the segments, how the work
// along the other axis is split, and their arguments.
//
// Queries and keys of segment s are the rows seg_q[s] .. seg_q[s + 1) - 1 and seg_k[s] .. seg_k[s + 1) - 1.  A tile
// is P rows of one segment.  No call knows the segments' sizes on the host, so tiles are numbered by slots:
// segment s has the slots from start(s) / P + s + 1 on, which are at least as many as its tiles and
// follow one another, n / P + segments + 2 in all; a slot behind a segment's last tile has no work.  The rows
// before the first segment and behind the last take part as two segments without keys.
#pragma once

#include "layers.cuh"

namespace spc {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

namespace ptx {

// 2^x, to about 2^-22 of itself; results below 2^-126 are 0.
__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace ptx

struct AttnArgs {
    const void* q;
    const void* k;
    const void* v;
    const int32_t* seg_q;
    const int32_t* seg_k;
    int64_t ldq, ldk, ldv;    // elements from row to row
    int64_t nq, nk;
    int32_t segments, hq, hk, d;
    float scale;
    // forward: o and lse are results; backward: arguments
    void* o;
    int64_t ldo;
    float* lse;               // [nq, hq]
    // backward
    const void* dout;
    int64_t lddo;
    void* dq;
    void* dk;
    void* dv;
    int64_t lddq, lddk, lddv;
    int32_t* status;
    // workspace, carved by attention_plan
    int32_t splits, splits_kv;
    float* part;              // [splits][nq][hq][d]: o (with part_lse) or dq
    float* part_lse;          // [splits][nq][hq]
    float* part_kv;           // [2][splits_kv][nk][hk][d]: dk, dv
    float* lse2;              // [hq][nq]: minus lse, to base 2 (-inf for a query without keys: no probability)
    float* delta;             // [hq][nq]: minus the sum of do o
    float* norm_do;           // fp16 on tensor cores: [hq][nq], [hk][nk]: norms of the rows of do and of v, 0 where not finite
    float* norm_v;
};

// What attn_tile's search numbers in 32 bits: a candidate and 31 steps of a 32nd of them.
constexpr int32_t kAttnMostSegments = 1 << 30;

inline int64_t attn_slots(int64_t n, int32_t segments, int32_t rows) { return n / rows + segments + 2; }

// A tile: rows [row, end) of its own axis (at most P), the segment's rows [lo, hi) of the other one.
struct AttnTile {
    int64_t row, end, lo, hi;
};

__device__ __forceinline__ int64_t attn_start(const int32_t* seg, int segments, int s, int64_t n)
{
    if (s < 0) return 0;
    if (s > segments) return n;
    const int64_t a = fetch(seg + s);
    return a < 0 ? 0 : (a > n ? n : a);
}

// Called by whole warps.  False where the slot has no work.
__device__ __forceinline__ bool attn_tile(const int32_t* seg, const int32_t* other, int segments, int64_t n, int64_t n_other,
                                          int P, int64_t slot, AttnTile& t)
{
    const int lane = threadIdx.x & 31;
    int lo = -1, count = segments + 2;  // candidates lo .. lo + count - 1; the first one's slots begin at or before `slot`
    while (count > 1) {
        const int step = (count + 31) / 32, s = lo + lane * step;
        const bool before = lane * step < count && attn_start(seg, segments, s, n) / P + s + 1 <= slot;
        const int last = max(__popc(__ballot_sync(FULL_MASK, before)) - 1, 0);
        lo += last * step;
        count = min(step, count - last * step);
    }
    const int64_t first = attn_start(seg, segments, lo, n), end = attn_start(seg, segments, lo + 1, n);
    t.row = first + (slot - (first / P + lo + 1)) * P;
    if (t.row < first || t.row >= end) return false;
    t.end = min(end, t.row + P);
    t.lo = t.hi = 0;
    if (lo >= 0 && lo < segments) {
        t.lo = attn_start(other, segments, lo, n_other);
        t.hi = max(t.lo, attn_start(other, segments, lo + 1, n_other));
    }
    return true;
}

// Offsets out of range or order are reported by one block's threads, whichever tiles they belong to.
__device__ __forceinline__ void attn_check(const int32_t* seg, int segments, int64_t n, int32_t* status, int tid, int threads)
{
    for (int s = tid; s < segments; s += threads) {
        const int64_t a = fetch(seg + s), b = fetch(seg + s + 1);
        if (a < 0 || b < a || b > n) set_status(status, SPC_ERR_ROW_INDEX);
    }
}

// The share of split z of Z, in tiles of `per` of the rows [lo, hi).
__device__ __forceinline__ void attn_share(int64_t lo, int64_t hi, int per, int z, int Z, int64_t& from, int64_t& to)
{
    const int64_t tiles = (hi - lo + per - 1) / per;
    from = lo + tiles * z / Z * per;
    to = min(hi, lo + tiles * (z + 1) / Z * per);
}

// ---------------------------------------------------------------- host side
// How the tensor-core forward kernel lays out queries: `heads` of the query heads that share a key head stand in
// one tile of 128 rows with `positions` positions, and a block has `tiles` such tiles.
struct AttnShape {
    int heads, positions, tiles;
};
AttnShape attn_shape(int64_t nq, int32_t segments, int32_t hq, int32_t hk, int32_t d);

// fp32 heads so narrow that a thread of the forward kernel keeps whole rows, and how many: four read keys and values half as often
// as two, two waste less of a block on short segments and give more blocks (8 heads of 16, us with four / two: 30,000 rows in
// segments of 150 148 / 106, of 300 179 / 148, of 500 193 / 214, of 1,000 361 / 409; 4 heads: 1,000 rows 22 / 16, 2,000 37 / 43).
constexpr int kAttnNarrow = 16;
int attn_rows_each(int64_t nq, int64_t nk, int32_t segments, int32_t hq);

// Kernels for 16-bit heads of a multiple of 8 channels, up to 128, on 16-byte boundaries.
bool attention_tc_supported(const AttnArgs& a, spc_dtype dt, bool backward);
size_t attention_ws_bytes(int64_t nq, int64_t nk, int32_t segments, int32_t hq, int32_t hk, int32_t d, spc_dtype dt, bool backward);
void attention_plan(AttnArgs& a, spc_dtype dt, void* ws, bool backward);
spc_status attention_fwd(const AttnArgs& a, spc_dtype dt, cudaStream_t st);
spc_status attention_bwd(const AttnArgs& a, spc_dtype dt, cudaStream_t st);

spc_status attention_fwd_simt(const AttnArgs& a, spc_dtype dt, cudaStream_t st);
spc_status attention_bwd_simt(const AttnArgs& a, spc_dtype dt, cudaStream_t st);
spc_status attention_fwd_tc(const AttnArgs& a, spc_dtype dt, cudaStream_t st);
spc_status attention_bwd_tc(const AttnArgs& a, spc_dtype dt, cudaStream_t st);

template <auto KERNEL, typename... A>
spc_status attn_start_kernel(dim3 grid, int block, size_t smem, cudaStream_t st, A... args)
{
    if (smem > 32 * 1024) {  // 48 KB with the static part need no leave
        const spc_status s = allow_smem<KERNEL>();
        if (s != SPC_OK) return s;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1] = {beside_the_kernel_before()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    SPC_CUDA_TRY(cudaLaunchKernelEx(&cfg, KERNEL, args...));
    return SPC_OK;
}

}  // namespace spc
