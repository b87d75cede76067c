// grouped_simt.cu -- products grouped by segment on CUDA cores: fp32 in full fp32
// multiplies, and the 16-bit shapes that the tensor-core kernels do not take.
//
// A block computes TM positions x TN columns of one segment, 8 x 8 (4 x 4 in the small tile) per
// thread, 16 of the reduction at a time through two buffers in shared memory: the next
// chunk is on its way into registers while this one is multiplied, two columns per f32x2
// instruction.  Segment sizes are known on the device only, so the grid covers the most row
// tiles there can be (one partial tile per segment) and each block finds its segment in `seg`.
//
// 8,000 fp32 rows in 4 segments, 256 -> 1024: 144 us, 29 TFLOP/s.  The large tile's 130 registers leave one block of
// eight warps an SM, two a scheduler, and they wait for shared memory a third of the time: the FMA pipe is
// active 46%.  A segment of few rows pays for a whole 64-row tile (16 rows of 64 segments, 1024 -> 4096: 226 us, 77%
// of the shared-memory pipe).  A value's terms are added in one fp32 chain, or one per split of the rows.
#include "layers.cuh"
#include "pairs.cuh"

namespace spc {

namespace {

constexpr int kStep = 16, kBlock = 256;

// Row tile t of the positions: those of the segments in turn, between them the
// positions before the first and after the last (segment -1).  False past the last tile.
template <int kTile>
__device__ bool find_tile(const int32_t* seg, int segments, int64_t m, int64_t t, int32_t* status,
                          int& g, int64_t& lo, int64_t& hi)
{
    const int lane = threadIdx.x & 31;
    int64_t done = 0;
    for (int v0 = 0; v0 < segments + 2; v0 += 32) {
        const int v = v0 + lane;
        int64_t a = 0, b = 0;
        if (v == 0) {
            const int64_t f = __ldg(seg);
            b = f < 0 ? 0 : (f > m ? m : f);
        } else if (v <= segments) {
            segment_bounds(seg, v - 1, m, status, a, b);
        } else if (v == segments + 1) {
            const int64_t f = __ldg(seg + segments);
            a = f < 0 ? 0 : (f > m ? m : f);
            b = m;
        }
        const int64_t tiles = (b - a + kTile - 1) / kTile;
        int64_t inc = tiles;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int64_t u = __shfl_up_sync(FULL_MASK, inc, d);
            if (lane >= d) inc += u;
        }
        const unsigned hit = __ballot_sync(FULL_MASK, t < done + inc);
        if (hit) {
            const int src = __ffs(hit) - 1;
            const int64_t first = __shfl_sync(FULL_MASK, done + inc - tiles, src);
            a = __shfl_sync(FULL_MASK, a, src);
            b = __shfl_sync(FULL_MASK, b, src);
            const int w = v0 + src;
            g = w == 0 || w == segments + 1 ? -1 : w - 1;
            lo = a + (t - first) * kTile;
            hi = lo + kTile < b ? lo + kTile : b;
            return true;
        }
        done += __shfl_sync(FULL_MASK, inc, 31);
    }
    return false;
}

// The product of two chunks in shared memory: a thread's F x F values, rows ty F .. and columns
// tx F ..., in pairs of columns.
template <int F, int PITCH>
__device__ __forceinline__ void multiply(const float (*s_a)[PITCH], const float (*s_b)[PITCH], int ty, int tx, F2 (&acc)[F][F / 2])
{
#pragma unroll
    for (int k = 0; k < kStep; ++k) {
        float u[F], v[F];
#pragma unroll
        for (int i = 0; i < F; i += 4) {
            *reinterpret_cast<float4*>(u + i) = *reinterpret_cast<const float4*>(&s_a[k][ty * F + i]);
            *reinterpret_cast<float4*>(v + i) = *reinterpret_cast<const float4*>(&s_b[k][tx * F + i]);
        }
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int j = 0; j < F / 2; ++j) acc[i][j] = fma(both(u[i]), F2{v[2 * j], v[2 * j + 1]}, acc[i][j]);
    }
}

// Four neighbouring values of a row whose length is a multiple of four, as fp32.
template <typename T>
__device__ __forceinline__ float4 four_of(const T* p)
{
    Vec<T, 4> v = *reinterpret_cast<const Vec<T, 4>*>(p);
    F2 f[2];
    unpack<T, 4>(v, f);
    return make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
}

// One of the 16 x 16 threads' F x F corner of a TILE x TILE tile, TILE = 16 F.  L: values that a thread
// loads at once, 4 where every row's length is a multiple of that, else 1.
template <typename T, int F, int L>
__global__ void __launch_bounds__(kBlock) k_grouped_simt(GroupedArgs a)
{
    constexpr int TILE = 16 * F, PITCH = TILE + 4, LOADS = TILE * kStep / kBlock;
    __shared__ __align__(16) float s_a[2][kStep][PITCH], s_b[2][kStep][PITCH];
    __shared__ int32_t s_row[TILE];
    int g;
    int64_t lo, hi;
    if (!find_tile<TILE>(a.seg, a.segments, a.m, blockIdx.x, a.status, g, lo, hi)) return;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const int n0 = blockIdx.y * TILE;
    if (tid < TILE) s_row[tid] = lo + tid < hi ? (int32_t)row_at(a.in_rows, lo + tid, a.in_n, a.status) : -1;
    __syncthreads();
    const T* in = static_cast<const T*>(a.in);
    const T* w = static_cast<const T*>(a.w) + (int64_t)(g < 0 ? 0 : g) * a.k * a.n;
    F2 acc[F][F / 2];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F / 2; ++j) acc[i][j] = both(0.f);
    // load e of a chunk: rows by reduction index (neighbouring lanes, neighbouring k), weights as they lie
    constexpr int N = LOADS / L;
    float ra[N][L], rb[N][L];
    auto fetch = [&](float (&v)[L], const T* p, bool there) {
        if constexpr (L == 4) {
            const float4 f = there ? four_of(p) : make_float4(0.f, 0.f, 0.f, 0.f);
            v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
        } else {
            v[0] = there ? elem<T>::to_f32(*p) : 0.f;
        }
    };
    auto load = [&](int k0) {
#pragma unroll
        for (int q = 0; q < N; ++q) {
            const int e = (q * kBlock + tid) * L, r = e / kStep, k = k0 + e % kStep;
            const int32_t row = s_row[r];
            fetch(ra[q], in + (int64_t)row * a.k + k, row >= 0 && k < a.k);
            if (a.w_transposed) {
                fetch(rb[q], w + (int64_t)(n0 + r) * a.k + k, n0 + r < a.n && k < a.k);
            } else {
                const int j = e % TILE, kk = k0 + e / TILE;
                fetch(rb[q], w + (int64_t)kk * a.n + n0 + j, n0 + j < a.n && kk < a.k);
            }
        }
    };
    auto store = [&](int b) {
#pragma unroll
        for (int q = 0; q < N; ++q) {
            const int e = (q * kBlock + tid) * L;
#pragma unroll
            for (int l = 0; l < L; ++l) {
                s_a[b][e % kStep + l][e / kStep] = ra[q][l];
                if (a.w_transposed) s_b[b][e % kStep + l][e / kStep] = rb[q][l];
                else s_b[b][e / TILE][e % TILE + l] = rb[q][l];
            }
        }
    };
    const int chunks = g < 0 ? 0 : (a.k + kStep - 1) / kStep;
    if (chunks) {
        load(0);
        store(0);
        __syncthreads();
    }
    for (int c = 0; c < chunks; ++c) {
        if (c + 1 < chunks) load((c + 1) * kStep);
        multiply<F, PITCH>(s_a[c & 1], s_b[c & 1], ty, tx, acc);
        if (c + 1 < chunks) store((c + 1) & 1);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < F; ++i) {
        const int64_t r = lo + ty * F + i;
        if (r >= hi) break;
        const int64_t row = row_at(a.out_rows, r, a.m, a.status);
        if (row < 0) continue;
        T* out = static_cast<T*>(a.out) + row * a.n;
#pragma unroll
        for (int j = 0; j < F; ++j) {
            const int n = n0 + tx * F + j;
            if (n < a.n) out[n] = elem<T>::from_f32(j % 2 ? acc[i][j / 2].y : acc[i][j / 2].x);
        }
    }
}

// One split of a segment's rows; with more than one split the sums go to part [splits][segments][cin][cout].
template <typename T, int F, int L>
__global__ void __launch_bounds__(kBlock) k_grouped_wgrad_simt(GroupedWgradArgs a, int splits, float* part)
{
    constexpr int TILE = 16 * F, PITCH = TILE + 4, LOADS = TILE * kStep / kBlock;
    __shared__ __align__(16) float s_a[2][kStep][PITCH], s_b[2][kStep][PITCH];
    const int g = blockIdx.z / splits, split = blockIdx.z % splits, c0 = blockIdx.y * TILE, n0 = blockIdx.x * TILE;
    int64_t lo, hi;
    segment_bounds(a.seg, g, a.m, a.status, lo, hi);
    const int64_t len = ((hi - lo + splits - 1) / splits + kStep - 1) / kStep * kStep;
    lo = lo + split * len < hi ? lo + split * len : hi;
    hi = lo + len < hi ? lo + len : hi;
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
    const T* x = static_cast<const T*>(a.x);
    const T* dy = static_cast<const T*>(a.dy);
    F2 acc[F][F / 2];
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F / 2; ++j) acc[i][j] = both(0.f);
    constexpr int N = LOADS / L;
    float ra[N][L], rb[N][L];
    auto fetch = [&](float (&v)[L], const T* p, bool there) {
        if constexpr (L == 4) {
            const float4 f = there ? four_of(p) : make_float4(0.f, 0.f, 0.f, 0.f);
            v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
        } else {
            v[0] = there ? elem<T>::to_f32(*p) : 0.f;
        }
    };
    auto load = [&](int64_t r0) {
#pragma unroll
        for (int q = 0; q < N; ++q) {
            const int e = (q * kBlock + tid) * L, j = e % TILE;
            const int64_t r = r0 + e / TILE;
            const int64_t xr = r < hi ? row_at(a.x_rows, r, a.n_x, a.status) : -1;
            const int64_t yr = r < hi ? row_at(a.y_rows, r, a.n_y, a.status) : -1;
            const bool there = xr >= 0 && yr >= 0;
            fetch(ra[q], x + xr * a.cin + c0 + j, there && c0 + j < a.cin);
            fetch(rb[q], dy + yr * a.cout + n0 + j, there && n0 + j < a.cout);
        }
    };
    auto store = [&](int b) {
#pragma unroll
        for (int q = 0; q < N; ++q) {
            const int e = (q * kBlock + tid) * L;
#pragma unroll
            for (int l = 0; l < L; ++l) {
                s_a[b][e / TILE][e % TILE + l] = ra[q][l];
                s_b[b][e / TILE][e % TILE + l] = rb[q][l];
            }
        }
    };
    const int64_t chunks = (hi - lo + kStep - 1) / kStep;
    if (chunks) {
        load(lo);
        store(0);
        __syncthreads();
    }
    for (int64_t c = 0; c < chunks; ++c) {
        if (c + 1 < chunks) load(lo + (c + 1) * kStep);
        multiply<F, PITCH>(s_a[c & 1], s_b[c & 1], ty, tx, acc);
        if (c + 1 < chunks) store((c + 1) & 1);
        __syncthreads();
    }
    float* to = splits > 1 ? part + (int64_t)split * a.segments * a.cin * a.cout : a.dw;
#pragma unroll
    for (int i = 0; i < F; ++i)
#pragma unroll
        for (int j = 0; j < F; ++j) {
            const int c = c0 + ty * F + i, n = n0 + tx * F + j;
            if (c < a.cin && n < a.cout) to[((int64_t)g * a.cin + c) * a.cout + n] = j % 2 ? acc[i][j / 2].y : acc[i][j / 2].x;
        }
}

// dW as the sum of the splits, in their order.
__global__ void __launch_bounds__(kBlock) k_grouped_wgrad_sum(const float* __restrict__ part, int64_t values, int splits, float* __restrict__ dw)
{
    const int64_t i = (int64_t)blockIdx.x * kBlock + threadIdx.x;
    if (i >= values) return;
    float s = 0.f;
#pragma unroll 8
    for (int q = 0; q < splits; ++q) s += part[q * values + i];
    dw[i] = s;
}

template <typename T, int F, int L>
spc_status run(const GroupedArgs& a, cudaStream_t st)
{
    const int64_t tiles = a.m / (16 * F) + a.segments + 2, cols = ceil_div(a.n, 16 * F);
    if (cols > 65535) return SPC_ERR_UNSUPPORTED;
    k_grouped_simt<T, F, L><<<dim3((unsigned)tiles, (unsigned)cols), kBlock, 0, st>>>(a);
    SPC_LAUNCH_CHECK();
    return SPC_OK;
}

template <typename T, int F, int L>
spc_status run_wgrad(const GroupedWgradArgs& a, int splits, float* part, cudaStream_t st)
{
    const int64_t rows = ceil_div(a.cin, 16 * F);
    if (rows > 65535) return SPC_ERR_UNSUPPORTED;
    k_grouped_wgrad_simt<T, F, L><<<dim3((unsigned)ceil_div(a.cout, 16 * F), (unsigned)rows, (unsigned)(a.segments * splits)),
                                    kBlock, 0, st>>>(a, splits, part);
    SPC_LAUNCH_CHECK();
    if (splits == 1) return SPC_OK;
    const int64_t values = (int64_t)a.segments * a.cin * a.cout;
    k_grouped_wgrad_sum<<<(unsigned)ceil_div(values, kBlock), kBlock, 0, st>>>(part, values, splits, a.dw);
    SPC_LAUNCH_CHECK();
    return SPC_OK;
}

// 128 x 128 tiles once there are two for each SM, else 64 x 64 ones.
bool large(int64_t tiles) { return tiles >= 2 * (int64_t)sm_count(); }

bool large_wgrad(int32_t segments, int32_t cin, int32_t cout)
{
    return large(ceil_div(cin, 128) * ceil_div(cout, 128) * segments);
}

// Rows are split until there are about three blocks for each SM, of at least 128 rows of an even segment
// (fp32, 2 segments of 16,000 rows, 512 x 128: 113 us against 992 unsplit).
int splits_of(int32_t segments, int64_t m, int32_t cin, int32_t cout)
{
    if (large_wgrad(segments, cin, cout)) return 1;
    const int64_t blocks = ceil_div(cin, 64) * ceil_div(cout, 64) * segments;
    const int64_t most = std::min<int64_t>(64, std::min<int64_t>(m / segments / 128, 65535 / segments));
    return (int)std::max<int64_t>(1, std::min(most, 3 * (int64_t)sm_count() / blocks));
}

template <typename T>
spc_status run(const GroupedArgs& a, cudaStream_t st)
{
    const bool big = large(ceil_div(a.n, 128) * ceil_div(a.m, 128));
    if (a.n % 4 == 0 && a.k % 4 == 0) return big ? run<T, 8, 4>(a, st) : run<T, 4, 4>(a, st);
    return big ? run<T, 8, 1>(a, st) : run<T, 4, 1>(a, st);
}

template <typename T>
spc_status run_wgrad(const GroupedWgradArgs& a, float* part, cudaStream_t st)
{
    const bool big = large_wgrad(a.segments, a.cin, a.cout);
    const int splits = splits_of(a.segments, a.m, a.cin, a.cout);
    if (a.cin % 4 == 0 && a.cout % 4 == 0)
        return big ? run_wgrad<T, 8, 4>(a, splits, part, st) : run_wgrad<T, 4, 4>(a, splits, part, st);
    return big ? run_wgrad<T, 8, 1>(a, splits, part, st) : run_wgrad<T, 4, 1>(a, splits, part, st);
}

}  // namespace

spc_status grouped_simt(const GroupedArgs& a, spc_dtype dt, cudaStream_t st)
{
    switch (dt) {
    case SPC_F32: return run<float>(a, st);
    case SPC_F16: return run<__half>(a, st);
    default: return run<__nv_bfloat16>(a, st);
    }
}

size_t grouped_wgrad_simt_ws_bytes(int32_t segments, int64_t m, int32_t cin, int32_t cout)
{
    const int splits = splits_of(segments, m, cin, cout);
    return splits == 1 ? 0 : align_up(sizeof(float) * (size_t)splits * segments * cin * cout, 256);
}

spc_status grouped_wgrad_simt(const GroupedWgradArgs& a, spc_dtype dt, void* ws, cudaStream_t st)
{
    float* part = static_cast<float*>(ws);
    switch (dt) {
    case SPC_F32: return run_wgrad<float>(a, part, st);
    case SPC_F16: return run_wgrad<__half>(a, part, st);
    default: return run_wgrad<__nv_bfloat16>(a, part, st);
    }
}

}  // namespace spc
