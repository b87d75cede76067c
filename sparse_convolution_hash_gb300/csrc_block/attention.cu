// attention.cu -- attention over segments: which kernels take a call, how it is split, and the small kernels around
// the large ones: the joins of split results and the backward pass' row sums.
#include "attention.cuh"
#include "pairs.cuh"

namespace spc {

namespace {

constexpr int kBlock = 256;

// Splits along the other axis: few tiles leave SMs idle, so each tile's walk is cut until there are `blocks` for
// every SM, in shares of at least `least` rows of an axis of n_other.  An axis without rows has nothing to split, or to join.
int splits_for(int64_t n, int32_t segments, int64_t heads, int64_t n_other, int rows, int least, int blocks)
{
    if (n == 0) return 1;
    const int64_t tiles = std::max<int64_t>(1, std::max<int64_t>(ceil_div(n, rows), std::min<int64_t>(n, segments))) * heads;
    const int64_t wanted = blocks * (int64_t)sm_count() / tiles;
    return (int)std::max<int64_t>(1, std::min<int64_t>(wanted, ceil_div(n_other, least)));
}

constexpr int kSimtRows = 64, kLeastShare = 256;

bool wide_enough(int32_t d, spc_dtype dt) { return dt != SPC_F32 && d % 8 == 0; }

struct Layout {
    int32_t splits, splits_kv;
    size_t part, part_lse, part_kv, lse2, delta, norm_do, norm_v, bytes;
};

Layout layout(int64_t nq, int64_t nk, int32_t segments, int32_t hq, int32_t hk, int32_t d, spc_dtype dt, bool backward)
{
    Layout l = {};
    const bool tc = wide_enough(d, dt);
    if (tc && !backward) {
        const AttnShape f = attn_shape(nq, segments, hq, hk, d);
        l.splits = splits_for(nq, segments, hq / f.heads, nk, f.positions * f.tiles, kLeastShare, f.tiles == 2 ? 1 : 2);
    } else if (!backward && dt == SPC_F32 && d <= kAttnNarrow) {
        l.splits = splits_for(nq, segments, hq, nk, 32 * attn_rows_each(nq, nk, segments, hq), kLeastShare, 2);
    } else {
        l.splits = splits_for(nq, segments, hq, nk, kSimtRows, kLeastShare, tc ? 2 : 4);
    }
    l.splits_kv = backward ? splits_for(nk, segments, hk, nq * (hq / hk), kSimtRows, kLeastShare, 2) : 1;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += align_up(bytes, 256);
        return here;
    };
    const size_t rows = (size_t)nq * hq;
    if (l.splits > 1) {
        l.part = take(rows * l.splits * d * 4);
        l.part_lse = take(backward ? 0 : rows * l.splits * 4);
    }
    if (backward) {
        if (l.splits_kv > 1) l.part_kv = take((size_t)nk * hk * d * 4 * 2 * l.splits_kv);
        l.lse2 = take(rows * 4);
        l.delta = take(rows * 4);
        if (tc && dt == SPC_F16) {
            l.norm_do = take(rows * 4);
            l.norm_v = take((size_t)nk * hk * 4);
        }
    }
    l.bytes = at;
    return l;
}

// o and lse from the splits': weights exp(lse_z - lse).  WARPS warps to a row and head; they take the splits in turn, each
// with a maximum and sum of its own, and join in order.  One where there are few splits, as there are many rows then;
// eight beyond (one alone waits for memory once for every split: 24 us for the 38 splits of 4 queries, 8 heads).
constexpr int kJoinWarps = 8, kFewSplits = 8;
template <typename T, int WARPS>
__global__ void __launch_bounds__(32 * kJoinWarps)
k_attn_join(AttnArgs a)
{
    __shared__ float box[kJoinWarps][4 * 32], tops[kJoinWarps], totals[kJoinWarps];
    wait_for_kernel_before();
    const int lane = threadIdx.x & 31, mine = threadIdx.x >> 5, warp = mine % WARPS, first = mine - warp;
    const int64_t i = (int64_t)blockIdx.x * (kJoinWarps / WARPS) + mine / WARPS, rows = a.nq * a.hq;
    if (WARPS == 1 && i >= rows) return;
    float most = -INFINITY;
    for (int z = warp + WARPS * lane; z < a.splits; z += 32 * WARPS) most = fmaxf(most, fetch(a.part_lse + z * rows + i));
#pragma unroll
    for (int o = 16; o; o >>= 1) most = fmaxf(most, __shfl_xor_sync(FULL_MASK, most, o));
    float total = 0.f, v[4] = {0.f, 0.f, 0.f, 0.f};
    // an infinite or NaN sum is one split's: its weight is 1, so that it reaches the result
#pragma unroll 4
    for (int z = warp; z < a.splits; z += WARPS) {
        const float l = fetch(a.part_lse + z * rows + i);
        const float* from = a.part + (z * rows + i) * a.d;
        float x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = lane + 32 * j < a.d ? fetch(from + lane + 32 * j) : 0.f;
        const bool there = l != -INFINITY;  // a split without keys has written no sums
        const float w = !there ? 0.f : l == most ? 1.f : expf(l - most);
        total += w;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = there ? fmaf(w, x[j], v[j]) : v[j];
    }
    const int64_t row = i / a.hq, head = i - row * a.hq;
    T* to = static_cast<T*>(a.o) + row * a.ldo + head * a.d;
    if constexpr (WARPS > 1) {
#pragma unroll
        for (int j = 0; j < 4; ++j) box[mine][32 * j + lane] = v[j];
        if (lane == 0) {
            tops[mine] = most;
            totals[mine] = total;
        }
        __syncthreads();
        if (warp > 0) return;
        most = -INFINITY;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) most = fmaxf(most, tops[first + w]);
        total = v[0] = v[1] = v[2] = v[3] = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            if (totals[first + w] == 0.f) continue;
            const float f = tops[first + w] == most ? 1.f : expf(tops[first + w] - most);
            total = fmaf(f, totals[first + w], total);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = fmaf(f, box[first + w][32 * j + lane], v[j]);
        }
    }
    const bool any = total > 0.f || total != total;
    const float inv = any ? 1.f / total : 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (lane + 32 * j < a.d) to[lane + 32 * j] = elem<T>::from_f32(v[j] * inv);
    if (lane == 0) a.lse[i] = any ? most + logf(total) : -INFINITY;
}

// Sums of the splits' gradients in order; rows of `width` values, at `ld` in the result.
template <typename T>
__global__ void __launch_bounds__(kBlock)
k_attn_sum(const float* part, int splits, int64_t rows, int width, T* to, int64_t ld)
{
    wait_for_kernel_before();
    const int64_t i = (int64_t)blockIdx.x * kBlock + threadIdx.x, all = rows * width;
    if (i >= all) return;
    float s = 0.f;
#pragma unroll 4
    for (int z = 0; z < splits; ++z) s += fetch(part + z * all + i);
    const int64_t row = i / width;
    to[row * ld + (i - row * width)] = elem<T>::from_f32(s);
}

// Rows of one head (blockIdx.y), LANES lanes to a row, four rows to a group of lanes so that their loads overlap.
// DELTA: minus the sum of do o over the head's channels, and minus lse to base 2.  NORM (fp16): the norm of the row of do, or
// (no DELTA) of v.
constexpr int kRowsEach = 4;
template <typename T, int LANES, bool DELTA, bool NORM>
__global__ void __launch_bounds__(kBlock)
k_attn_rows(AttnArgs a, bool whole)
{
    wait_for_kernel_before();
    constexpr int V = 16 / sizeof(T), kGroups = kBlock / LANES;
    const int lane = threadIdx.x % LANES, head = blockIdx.y;
    const int64_t n = DELTA ? a.nq : a.nk, ld = DELTA ? a.lddo : a.ldv, row0 = (int64_t)blockIdx.x * (kGroups * kRowsEach) + threadIdx.x / LANES;
    const T* g = static_cast<const T*>(DELTA ? a.dout : a.v) + (int64_t)head * a.d;
    const T* o = static_cast<const T*>(a.o) + (int64_t)head * a.d;
    float sum[kRowsEach], square[kRowsEach];
#pragma unroll
    for (int k = 0; k < kRowsEach; ++k) {
        const int64_t row = row0 + k * kGroups;
        sum[k] = square[k] = 0.f;
        if (row >= n) continue;
        if (whole) {
            for (int c = lane * V; c < a.d; c += LANES * V) {
                const Vec<T, V> x = *reinterpret_cast<const Vec<T, V>*>(g + row * ld + c);
                Vec<T, V> y;
                if (DELTA) y = *reinterpret_cast<const Vec<T, V>*>(o + row * a.ldo + c);
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float u = elem<T>::to_f32(x.e[j]);
                    if (DELTA) sum[k] = fmaf(elem<T>::to_f32(y.e[j]), u, sum[k]);
                    if (NORM) square[k] = fmaf(u, u, square[k]);
                }
            }
        } else {
            for (int c = lane; c < a.d; c += LANES) {
                const float u = elem<T>::to_f32(g[row * ld + c]);
                if (DELTA) sum[k] = fmaf(elem<T>::to_f32(o[row * a.ldo + c]), u, sum[k]);
                if (NORM) square[k] = fmaf(u, u, square[k]);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < kRowsEach; ++k) {
        const int64_t row = row0 + k * kGroups;
#pragma unroll
        for (int x = LANES / 2; x; x >>= 1) {
            if (DELTA) sum[k] += __shfl_xor_sync(FULL_MASK, sum[k], x);
            if (NORM) square[k] += __shfl_xor_sync(FULL_MASK, square[k], x);
        }
        // rows that are not finite have no say (their results are not finite either)
        if (NORM && row < n && lane == 0) (DELTA ? a.norm_do : a.norm_v)[head * n + row] = square[k] < INFINITY ? sqrtf(square[k]) : 0.f;
        if (DELTA && row < n && lane == 0) {
            const float lse = fetch(a.lse + row * a.hq + head);
            a.delta[head * a.nq + row] = -sum[k];
            a.lse2[head * a.nq + row] = lse == -INFINITY ? -INFINITY : -lse * kLog2e;
        }
    }
}

template <typename T>
spc_status join_fwd(const AttnArgs& a, cudaStream_t st)
{
    const int64_t rows = a.nq * a.hq;
    if (rows > INT32_MAX) return SPC_ERR_UNSUPPORTED;
    if (a.splits > kFewSplits) return attn_start_kernel<k_attn_join<T, kJoinWarps>>(dim3((unsigned)rows), 32 * kJoinWarps, 0, st, a);
    return attn_start_kernel<k_attn_join<T, 1>>(dim3((unsigned)ceil_div(rows, kJoinWarps)), 32 * kJoinWarps, 0, st, a);
}

template <typename T>
spc_status sum(const float* part, int splits, int64_t rows, int width, void* to, int64_t ld, cudaStream_t st)
{
    const int64_t blocks = ceil_div(rows * width, kBlock);
    if (blocks > INT32_MAX) return SPC_ERR_UNSUPPORTED;
    return attn_start_kernel<k_attn_sum<T>>(dim3((unsigned)blocks), kBlock, 0, st, part, splits, rows, width, static_cast<T*>(to), ld);
}

template <typename T>
spc_status join_bwd(const AttnArgs& a, cudaStream_t st)
{
    spc_status s = SPC_OK;
    if (a.splits > 1) s = sum<T>(a.part, a.splits, a.nq, a.hq * a.d, a.dq, a.lddq, st);
    if (s == SPC_OK && a.splits_kv > 1) {
        const int64_t all = a.nk * a.hk * a.d;
        s = sum<T>(a.part_kv, a.splits_kv, a.nk, a.hk * a.d, a.dk, a.lddk, st);
        if (s == SPC_OK) s = sum<T>(a.part_kv + all * a.splits_kv, a.splits_kv, a.nk, a.hk * a.d, a.dv, a.lddv, st);
    }
    return s;
}

template <typename T, bool DELTA, bool NORM>
spc_status rows_of(const AttnArgs& a, cudaStream_t st)
{
    constexpr int V = 16 / (int)sizeof(T);
    const int64_t n = DELTA ? a.nq : a.nk;
    if (n == 0) return SPC_OK;
    const bool whole = a.d % V == 0 && (DELTA ? a.lddo : a.ldv) % V == 0 && aligned16(DELTA ? a.dout : a.v) &&
                       (!DELTA || (a.ldo % V == 0 && aligned16(a.o)));
    const int64_t vectors = ceil_div(a.d, V);
    const int lanes = vectors <= 4 ? 4 : vectors <= 8 ? 8 : 16;
    const int64_t blocks = ceil_div(n, (int64_t)(kBlock / lanes) * kRowsEach);
    if (blocks > INT32_MAX) return SPC_ERR_UNSUPPORTED;
    const dim3 grid((unsigned)blocks, (unsigned)(DELTA ? a.hq : a.hk));
    switch (lanes) {
    case 4: return attn_start_kernel<k_attn_rows<T, 4, DELTA, NORM>>(grid, kBlock, 0, st, a, whole);
    case 8: return attn_start_kernel<k_attn_rows<T, 8, DELTA, NORM>>(grid, kBlock, 0, st, a, whole);
    default: return attn_start_kernel<k_attn_rows<T, 16, DELTA, NORM>>(grid, kBlock, 0, st, a, whole);
    }
}

template <typename T>
spc_status row_sums(const AttnArgs& a, bool norms, cudaStream_t st)
{
    if constexpr (std::is_same<T, __half>::value) {
        if (norms) {
            const spc_status s = rows_of<T, false, true>(a, st);
            return s != SPC_OK ? s : rows_of<T, true, true>(a, st);
        }
    }
    return rows_of<T, true, false>(a, st);
}

}  // namespace

// The query heads of a tile: as many of those that share a key head as divide them and leave a tile two positions.
// A block of one tile leaves room for a second block on the SM, a block of two reads keys half as often.  One is faster
// for heads of up to 64 channels whatever the length (8 heads, 32,768 rows in samples of 200 to 32,768: 131 against 158 us
// at 200 rows, 606 against 642 at 8,192, 2,254 against 2,268 at 32,768), two for wider heads from some 1,500 rows
// a segment on (8 heads of 128: 222 against 237 us at 600, 179 and 179 at 1,500, 303 against 289 at 3,000,
// 736 against 674 at 8,192) where that many blocks still fill the SMs.
AttnShape attn_shape(int64_t nq, int32_t segments, int32_t hq, int32_t hk, int32_t d)
{
    AttnShape f;
    const int per = hq / hk;
    f.heads = 1;
    for (int g = 2; g <= std::min(per, 64); ++g)
        if (per % g == 0) f.heads = g;
    f.positions = 128 / f.heads;
    const int64_t blocks = ceil_div(nq, 2 * f.positions) * (hq / f.heads);
    f.tiles = d > 64 && nq / segments >= 12 * f.positions && blocks >= sm_count() ? 2 : 1;
    return f;
}

int attn_rows_each(int64_t nq, int64_t nk, int32_t segments, int32_t hq)
{
    const int64_t shares = ceil_div(nq, 128) * hq * ceil_div(nk, kLeastShare);
    return nq >= 450 * (int64_t)segments && shares >= 2 * (int64_t)sm_count() ? 4 : 2;
}

bool attention_tc_supported(const AttnArgs& a, spc_dtype dt, bool backward)
{
    const uintptr_t low = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v) |
                          reinterpret_cast<uintptr_t>(a.o);
    // TMA rows start on 16-byte boundaries; an empty tensor has no map
    if (!wide_enough(a.d, dt) || a.nq == 0 || a.nk == 0 || low % 16 || (a.ldq | a.ldk | a.ldv | a.ldo) % 8) return false;
    if (!backward) return true;
    const uintptr_t back = reinterpret_cast<uintptr_t>(a.dout) | reinterpret_cast<uintptr_t>(a.dq) | reinterpret_cast<uintptr_t>(a.dk) |
                           reinterpret_cast<uintptr_t>(a.dv);
    return back % 16 == 0 && (a.lddo | a.lddq | a.lddk | a.lddv) % 8 == 0;
}

size_t attention_ws_bytes(int64_t nq, int64_t nk, int32_t segments, int32_t hq, int32_t hk, int32_t d, spc_dtype dt, bool backward)
{
    return layout(nq, nk, segments, hq, hk, d, dt, backward).bytes;
}

void attention_plan(AttnArgs& a, spc_dtype dt, void* ws, bool backward)
{
    const Layout l = layout(a.nq, a.nk, a.segments, a.hq, a.hk, a.d, dt, backward);
    uint8_t* base = static_cast<uint8_t*>(ws);
    a.splits = l.splits;
    a.splits_kv = l.splits_kv;
    a.part = reinterpret_cast<float*>(base + l.part);
    a.part_lse = reinterpret_cast<float*>(base + l.part_lse);
    a.part_kv = reinterpret_cast<float*>(base + l.part_kv);
    a.lse2 = reinterpret_cast<float*>(base + l.lse2);
    a.delta = reinterpret_cast<float*>(base + l.delta);
    a.norm_do = reinterpret_cast<float*>(base + l.norm_do);
    a.norm_v = reinterpret_cast<float*>(base + l.norm_v);
}

spc_status attention_fwd(const AttnArgs& a, spc_dtype dt, cudaStream_t st)
{
    if (a.nq == 0) return SPC_OK;
    spc_status s = attention_tc_supported(a, dt, false) ? attention_fwd_tc(a, dt, st) : SPC_ERR_UNSUPPORTED;
    if (s == SPC_ERR_UNSUPPORTED) s = attention_fwd_simt(a, dt, st);  // strides that no tensor map holds, too
    if (s != SPC_OK || a.splits == 1) return s;
    switch (dt) {
    case SPC_F32: return join_fwd<float>(a, st);
    case SPC_F16: return join_fwd<__half>(a, st);
    default: return join_fwd<__nv_bfloat16>(a, st);
    }
}

spc_status attention_bwd(const AttnArgs& a, spc_dtype dt, cudaStream_t st)
{
    if (a.nq == 0 && a.nk == 0) return SPC_OK;
    const bool tc = attention_tc_supported(a, dt, true);
    spc_status s = dt == SPC_F32   ? row_sums<float>(a, tc, st)
                   : dt == SPC_F16 ? row_sums<__half>(a, tc, st)
                                   : row_sums<__nv_bfloat16>(a, tc, st);
    if (s != SPC_OK) return s;
    s = tc ? attention_bwd_tc(a, dt, st) : SPC_ERR_UNSUPPORTED;
    if (s == SPC_ERR_UNSUPPORTED) s = attention_bwd_simt(a, dt, st);
    if (s != SPC_OK) return s;
    switch (dt) {
    case SPC_F32: return join_bwd<float>(a, st);
    case SPC_F16: return join_bwd<__half>(a, st);
    default: return join_bwd<__nv_bfloat16>(a, st);
    }
}

}  // namespace spc
