// rope.cu -- rotary positions from voxel coordinates: pair i of a head's channels, (2 i, 2 i + 1), is turned by
// the cell's place on one of the three axes times the pair's step.
//
// A step is kept as a fraction of a turn in 64 bits, so the place times the step, modulo a turn, is one
// wrapping integer product: exact for every coordinate, where an angle in fp32 has lost its digits at a few
// thousand cells.  A thread takes the angles of one vector of channels of one row and turns that vector in all
// heads, several in flight: one sine and cosine for `heads` pairs, and memory is what bounds it.
#include <math.h>

#include "block.cuh"
#include "pairs.cuh"

namespace spc {

namespace {

constexpr int kBlock = 128;
constexpr int kMostPairs = 128;
constexpr int kAhead = 8;  // heads in flight a thread

struct Steps {
    uint64_t of[kMostPairs];
    int32_t end[3];  // pairs of z; of z and y; all
};

__device__ __forceinline__ void turn_of(const Steps& k, const int4& cell, int pair, bool back, float& s, float& c)
{
    const int32_t at = pair < k.end[0] ? cell.y : pair < k.end[1] ? cell.z : cell.w;
    const uint64_t phase = (uint64_t)(int64_t)at * k.of[pair];  // turns, 2^64 to one
    // its first 32 bits, rounded: off by 2^-33 of a turn, where the angle in fp32 is off by up to 2^-25
    sincospif((float)(int32_t)((phase + 0x80000000ull) >> 32) * 0x1p-31f, &s, &c);
    if (back) s = -s;
}

// A thread's row and its place among the row's `per_row`: a block takes whole rows, so that one division of small numbers
// does (12,345 rows of 3 heads of 40 fp32 4.4 us with one of 64 bits, 4.0 without), unless a row is more than a block.
__device__ __forceinline__ bool place_of(int64_t n, int per_row, int64_t& row, int& place)
{
    if (per_row <= kBlock) {
        const int rows = kBlock / per_row, mine = (int)threadIdx.x / per_row;
        row = (int64_t)blockIdx.x * rows + mine;
        place = (int)threadIdx.x - mine * per_row;
        return mine < rows && row < n;
    }
    const int64_t i = (int64_t)blockIdx.x * kBlock + threadIdx.x;
    row = i / per_row;
    place = (int)(i - row * per_row);
    return row < n;
}

// V channels to a vector (whole vectors of every head start on their boundary).
template <typename T, int V>
__global__ void __launch_bounds__(kBlock)
k_rope(const T* x, int64_t ldx, const int32_t* coords, int64_t n, int heads, int d, int heads_each,
       const __grid_constant__ Steps steps, bool back, T* y, int64_t ldy)
{
    using P = Vec<T, V>;
    wait_for_kernel_before();
    int64_t row;
    int place;
    if (!place_of(n, d / V, row, place)) return;
    const int c0 = place * V;
    const int h0 = blockIdx.y * heads_each, h1 = min(h0 + heads_each, heads);
    const int4 cell = *reinterpret_cast<const int4*>(coords + row * 4);
    const T* from = x + row * ldx + c0;
    T* to = y + row * ldy + c0;
    // fp32: the first heads are on their way while the angles are computed (125,559 rows of 3 heads of 128 77 us against 70); in 16 bits
    // the angles of twice as many channels want the registers (60,000 rows of 8 heads of 96 bf16 30.5 against 35.5)
    constexpr bool kLoadFirst = sizeof(T) == 4;
    P v[kAhead];
    auto load = [&](int h) {
#pragma unroll
        for (int q = 0; q < kAhead; ++q)
            if (h + q < h1) v[q] = *reinterpret_cast<const P*>(from + (int64_t)(h + q) * d);
    };
    if (kLoadFirst) load(h0);
    F2 cs[V / 2];
    bool turned[V / 2];
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
        turned[j] = c0 / 2 + j < steps.end[2];
        cs[j] = F2{1.f, 0.f};
        if (turned[j]) turn_of(steps, cell, c0 / 2 + j, back, cs[j].y, cs[j].x);
    }
    for (int h = h0; h < h1; h += kAhead) {
        if (!kLoadFirst || h > h0) load(h);
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            if (h + q >= h1) break;
            F2 f[V / 2];
            unpack<T, V>(v[q], f);
#pragma unroll
            for (int j = 0; j < V / 2; ++j) {
                const F2 a = f[j];
                if (turned[j]) f[j] = F2{a.x * cs[j].x - a.y * cs[j].y, a.x * cs[j].y + a.y * cs[j].x};
            }
            *reinterpret_cast<P*>(to + (int64_t)(h + q) * d) = pack<T, V>(f);
        }
    }
}

// Any number of channels, alignment and strides: a pair (or the odd last channel) of one head a thread at a time.
template <typename T>
__global__ void __launch_bounds__(kBlock)
k_rope_pairs(const T* x, int64_t ldx, const int32_t* coords, int64_t n, int heads, int d, int heads_each,
             const __grid_constant__ Steps steps, bool back, T* y, int64_t ldy)
{
    wait_for_kernel_before();
    int64_t row;
    int pair;
    if (!place_of(n, (d + 1) / 2, row, pair)) return;
    const int h0 = blockIdx.y * heads_each, h1 = min(h0 + heads_each, heads);
    const int4 cell = *reinterpret_cast<const int4*>(coords + row * 4);
    const bool turned = pair < steps.end[2], two = 2 * pair + 1 < d;
    float s = 0.f, c = 1.f;
    if (turned) turn_of(steps, cell, pair, back, s, c);
    for (int h = h0; h < h1; ++h) {
        const T* from = x + row * ldx + (int64_t)h * d + 2 * pair;
        T* to = y + row * ldy + (int64_t)h * d + 2 * pair;
        const float a = elem<T>::to_f32(from[0]), b = two ? elem<T>::to_f32(from[1]) : 0.f;
        to[0] = elem<T>::from_f32(turned ? a * c - b * s : a);
        if (two) to[1] = elem<T>::from_f32(turned ? a * s + b * c : b);
    }
}

template <typename T>
spc_status launch(const RopeArgs& a, const Steps& steps, cudaStream_t st)
{
    constexpr int V = 16 / (int)sizeof(T);
    const bool whole = a.d % V == 0 && a.ldx % V == 0 && a.ldy % V == 0 && aligned16(a.x) && aligned16(a.y);
    const int64_t per_row = whole ? a.d / V : (a.d + 1) / 2, threads = a.n * per_row;
    const int64_t blocks = per_row <= kBlock ? ceil_div(a.n, kBlock / per_row) : ceil_div(threads, kBlock);
    if (blocks > INT32_MAX) return SPC_ERR_UNSUPPORTED;
    // a thread takes all heads unless there are too few threads to fill the SMs
    int heads_each = a.heads;
    while (heads_each > 1 && threads * ceil_div(a.heads, heads_each) < (int64_t)sm_count() * 1024) heads_each = (heads_each + 1) / 2;
    while (ceil_div(a.heads, heads_each) > 65535) heads_each *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks, (unsigned)ceil_div(a.heads, heads_each));
    cfg.blockDim = dim3(kBlock);
    cfg.stream = st;
    cudaLaunchAttribute attr[1] = {beside_the_kernel_before()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    auto* kernel = whole ? k_rope<T, V> : k_rope_pairs<T>;
    SPC_CUDA_TRY(cudaLaunchKernelEx(&cfg, kernel, static_cast<const T*>(a.x), a.ldx, a.coords, a.n, a.heads, a.d, heads_each,
                                    steps, a.back != 0, static_cast<T*>(a.y), a.ldy));
    return SPC_OK;
}

}  // namespace

// step = base^(-j / p) / (2 pi) turns, j = 0 .. p - 1 of an axis' p pairs
void rope_steps(const int32_t* pairs, double base, uint64_t* steps)
{
    const long double turn = 6.283185307179586476925286766559005768L;
    for (int a = 0; a < 3; ++a)
        for (int j = 0; j < pairs[a]; ++j) {
            const long double t = expl(-logl((long double)base) * j / pairs[a]) / turn;
            *steps++ = (uint64_t)llrintl(t * 18446744073709551616.0L);
        }
}

spc_status rope(const RopeArgs& a, const int32_t* pairs, const uint64_t* steps, spc_dtype dt, cudaStream_t st)
{
    if (a.n == 0 || a.heads == 0) return SPC_OK;
    Steps k = {};
    k.end[0] = pairs[0];
    k.end[1] = pairs[0] + pairs[1];
    k.end[2] = pairs[0] + pairs[1] + pairs[2];
    for (int i = 0; i < k.end[2]; ++i) k.of[i] = steps[i];
    switch (dt) {
    case SPC_F32: return launch<float>(a, k, st);
    case SPC_F16: return launch<__half>(a, k, st);
    default: return launch<__nv_bfloat16>(a, k, st);
    }
}

}  // namespace spc
