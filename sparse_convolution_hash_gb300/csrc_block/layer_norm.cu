// layer_norm.cu -- y = gamma (x - mean) rstd + beta with the statistics of each row, and its gradients.
//
// A row is held in registers by a group of L threads (a part of a warp, a warp, or several warps), K vectors of V
// channels to a thread (neighbours read as 16 bytes, or, where rows do not start on such a boundary, in words of two
// channels, or one by one), so it is read once: the mean, then the sum of
// squares around it, then the result.  Where the mean is far from zero, what its rounding has left is
// taken off as well: the mean of the differences from it, which goes off the mean, the differences and, squared, the variance (without,
// rows of 1000.3 +- 0.01 were off by up to 0.016 and rows of one value by up to 0.17; with it for all rows 498,145 x 64 bf16 take 36 us against 28).
// In the backward pass a block keeps its channels for all of its rows,
// so the sums over the rows (dgamma, dbeta) also stay in registers; a block's groups join in shared memory and
// the blocks in a second, small kernel, always in the same order.
//
// Bound by memory: 16 operations stand against 4 to 8 bytes an element.  What has to be right is the number
// of bytes in flight, so a group works on R rows at once.
#include "block.cuh"
#include "pairs.cuh"

namespace spc {

namespace {

constexpr int kFwdBlock = 256, kWideFwdBlock = 512;
constexpr int kBwdBlock = 512;
constexpr int kLongBlock = 512;
constexpr int kJoinCols = 32, kJoinRows = 16;

__device__ __forceinline__ void let_next_kernel_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Sums of N values over the L threads of a group, in every thread.  Groups of more than a warp meet at a named
// barrier and pass their warps' sums through `box` (16 warps x N floats, double-buffered by `turn`).
template <int N>
__device__ __forceinline__ void group_sum(float (&v)[N], int L, float* box, int turn)
{
    for (int o = min(L, 32) >> 1; o; o >>= 1) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] += __shfl_xor_sync(FULL_MASK, v[j], o);
    }
    if (L > 32) {
        const int warp = threadIdx.x >> 5, warps = L >> 5, group = threadIdx.x / L;
        float* at = box + turn * (16 * N);
        if ((threadIdx.x & 31) == 0) {
#pragma unroll
            for (int j = 0; j < N; ++j) at[warp * N + j] = v[j];
        }
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(L) : "memory");
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = 0.f;
        for (int w = group * warps; w < (group + 1) * warps; ++w) {
#pragma unroll
            for (int j = 0; j < N; ++j) v[j] += at[w * N + j];
        }
    }
}

// Which channels a thread holds, in words of W (V, 2 or 1) neighbours: element j of its vector k.
template <int V, int W>
struct Place {
    int t, L, c;
    __device__ __forceinline__ int at(int k, int j) const { return ((k * (V / W) + j / W) * L + t) * W + j % W; }
    __device__ __forceinline__ bool in(int k, int j) const { return at(k, j) < c; }
};

// Zeros where the row has ended, or there is no row: they add nothing to any sum.  AGAIN: the row's first word where it has ended.
template <typename T, int V, int W, bool AGAIN = false>
__device__ __forceinline__ void load_row(const T* row, const Place<V, W>& w, int k, bool there, Vec<T, V>& v)
{
    if constexpr (W == V) {
        uint4 bits = make_uint4(0u, 0u, 0u, 0u);
        if (there && (AGAIN || w.in(k, 0))) bits = *reinterpret_cast<const uint4*>(row + (w.in(k, 0) ? w.at(k, 0) : 0));
        memcpy(&v, &bits, 16);
    } else {
        // as bits, which no instruction touches until the row's turn comes
        using Bits = std::conditional_t<sizeof(T) * W == 8, uint2, std::conditional_t<sizeof(T) * W == 4, uint32_t, uint16_t>>;
        Bits words[V / W];
#pragma unroll
        for (int q = 0; q < V / W; ++q) {
            words[q] = Bits{};
            if (there && (AGAIN || w.in(k, q * W))) words[q] = *reinterpret_cast<const Bits*>(row + (w.in(k, q * W) ? w.at(k, q * W) : 0));
        }
        memcpy(&v, words, 16);
    }
}

template <typename T, int V, int W>
__device__ __forceinline__ void store_row(T* row, const Place<V, W>& w, int k, const F2 (&f)[V / 2])
{
    const Vec<T, V> v = pack<T, V>(f);
#pragma unroll
    for (int j = 0; j < V; j += W) {
        Vec<T, W> word;
#pragma unroll
        for (int i = 0; i < W; ++i) word.e[i] = v.e[j + i];
        if (w.in(k, j)) *reinterpret_cast<Vec<T, W>*>(row + w.at(k, j)) = word;
    }
}

template <int V, int W>
__device__ __forceinline__ void load_affine(const float* p, float other, const Place<V, W>& w, int k, F2 (&f)[V / 2])
{
    if constexpr (W == V) {
#pragma unroll
        for (int j = 0; j < V; j += 4) {
            float4 v = make_float4(other, other, other, other);
            if (p && w.in(k, 0)) v = *reinterpret_cast<const float4*>(p + w.at(k, j));
            f[j / 2] = F2{v.x, v.y};
            f[j / 2 + 1] = F2{v.z, v.w};
        }
    } else if constexpr (W == 2) {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            float2 v = make_float2(other, other);
            if (p && w.in(k, 2 * j)) v = *reinterpret_cast<const float2*>(p + w.at(k, 2 * j));
            f[j] = F2{v.x, v.y};
        }
    } else {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            f[j].x = p && w.in(k, 2 * j) ? fetch(p + w.at(k, 2 * j)) : other;
            f[j].y = p && w.in(k, 2 * j + 1) ? fetch(p + w.at(k, 2 * j + 1)) : other;
        }
    }
}

// Whether a row's mean is so many spreads from zero that its rounding shows in the result: 16 in fp32, 256 in 16 bits (false where
// fp32 does not hold the squares, and for NaN).  fp32 rows of 1,000 are off by 2.4e-6 at most at 15 spreads without, by 7e-7 at 17 with what
// follows; but such rows take two to three times as long (498,145 x 64 bf16 71 us against 28).
template <typename T>
__device__ __forceinline__ bool far_from_zero(float mean, float var)
{
    return var < INFINITY && mean * mean > (sizeof(T) == 4 ? 0x1p8f : 0x1p16f) * var;
}

// A row that may be far from zero, from its start.  A call that reads the row again and gets nothing but addresses, so that it costs other
// rows next to nothing: with the differences kept, 32,768 x 1,024 bf16 took 44 us against 30, and inline 498,145 x 64 bf16 34 against 28.
// Sums have the kernel's order, so a row that turns out to be near zero gets the bits that it has among others of its kind.
template <typename T, int V, int K, int W>
__device__ __noinline__ void far_row(const T* x, T* y, const float* gamma, const float* beta, float* to_mean, float* to_rstd, int c, float eps,
                                     int L, bool there, float* box)
{
    constexpr int H = V / 2;
    const Place<V, W> w{(int)threadIdx.x & (L - 1), L, c};
    const float inv = 1.f / (float)c;
    auto differences = [&](int k, float mean, F2 (&d)[H]) {
        Vec<T, V> v;
        load_row<T, V, W>(x, w, k, there, v);
        unpack<T, V>(v, d);
#pragma unroll
        for (int j = 0; j < H; ++j) {
            d[j] = add(d[j], both(-mean));
            if (!w.in(k, 2 * j)) d[j].x = 0.f;
            if (!w.in(k, 2 * j + 1)) d[j].y = 0.f;
        }
    };
    float mean = 0.f, left = 0.f, var = 0.f;
#pragma unroll 1
    for (int turn = 0; turn < 3; ++turn) {  // the mean, the mean square around it, the mean of the differences
        F2 s{0.f, 0.f};
#pragma unroll 1
        for (int k = 0; k < K; ++k) {
            F2 d[H];
            differences(k, mean, d);
#pragma unroll
            for (int j = 0; j < H; ++j) s = turn == 1 ? fma(d[j], d[j], s) : add(s, d[j]);
        }
        float sum[1] = {s.x + s.y};
        group_sum<1>(sum, L, box, turn & 1);
        const float got = __fmul_rn(sum[0], inv);
        (turn == 0 ? mean : turn == 1 ? var : left) = got;
    }
    if (!there) return;
    if (far_from_zero<T>(mean, var)) var = fmaxf(var - left * left, 0.f);
    else left = 0.f;
    const float rstd = 1.f / sqrtf(var + eps);
#pragma unroll 1
    for (int k = 0; k < K; ++k) {
        F2 d[H], ga[H], be[H];
        differences(k, mean, d);
        load_affine<V, W>(gamma, 1.f, w, k, ga);
        load_affine<V, W>(beta, 0.f, w, k, be);
#pragma unroll
        for (int j = 0; j < H; ++j) d[j] = fma(mul(add(d[j], both(-left)), both(rstd)), ga[j], be[j]);
        store_row<T, V, W>(y, w, k, d);
    }
    if (w.t == 0) {
        *to_mean = mean + left;
        *to_rstd = rstd;
    }
}

// Blocks that share an SM: the call above must not cost the kernel any.
template <int V, int K, int BLOCK, int W>
constexpr int kFwdBlocks = V == 8 ? (K == 4 ? (W == V ? 1024 : 768) / BLOCK : 3) : 1024 / BLOCK;

// R rows of a group at a time.
template <typename T, int V, int K, int R, int BLOCK, int W>
__global__ void __launch_bounds__(BLOCK, kFwdBlocks<V, K, BLOCK, W>)
k_layer_norm(LayerNormArgs a, int L)
{
    constexpr int H = V / 2;
    __shared__ float box[2 * 16 * R];
    wait_for_kernel_before();
    let_next_kernel_start();
    const Place<V, W> w{(int)threadIdx.x & (L - 1), L, a.c};
    const int groups = BLOCK / L;
    const int64_t row0 = ((int64_t)blockIdx.x * groups + threadIdx.x / L) * R;
    const T* x = static_cast<const T*>(a.x);
    Vec<T, V> raw[R][K];
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
        for (int k = 0; k < K; ++k)
            load_row<T, V, W>(x + (row0 + r) * a.c, w, k, row0 + r < a.n, raw[r][k]);
    }
    F2 f[R][K][H];
    float sum[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        F2 s{0.f, 0.f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
            unpack<T, V>(raw[r][k], f[r][k]);
#pragma unroll
            for (int j = 0; j < H; ++j) s = add(s, f[r][k][j]);
        }
        sum[r] = s.x + s.y;
    }
    group_sum<R>(sum, L, box, 0);
    const float inv = 1.f / (float)a.c;
    float mean[R], sq[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        mean[r] = __fmul_rn(sum[r], inv);
        F2 s{0.f, 0.f};
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int j = 0; j < H; ++j) {
                f[r][k][j] = add(f[r][k][j], both(-mean[r]));
                F2 d = f[r][k][j];
                if (!w.in(k, 2 * j)) d.x = 0.f;
                if (!w.in(k, 2 * j + 1)) d.y = 0.f;
                s = fma(d, d, s);
            }
        }
        sq[r] = s.x + s.y;
    }
    group_sum<R>(sq, L, box, 1);
    bool far = false;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        sq[r] = __fmul_rn(sq[r], inv);  // not one with the sum with eps
        far |= far_from_zero<T>(mean[r], sq[r]);
    }
    if (__any_sync(FULL_MASK, far)) {  // the warps of a row hold the same numbers
        for (int64_t row = row0; row < row0 + R; ++row)
            far_row<T, V, K, W>(x + row * a.c, static_cast<T*>(a.out) + row * a.c, a.gamma, a.beta, a.mean + row, a.rstd + row, a.c, a.eps, L,
                                row < a.n, box);
        return;
    }
    T* y = static_cast<T*>(a.out);
    float rstd[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
        rstd[r] = 1.f / sqrtf(sq[r] + a.eps);
        if (w.t == 0 && row0 + r < a.n) {
            a.mean[row0 + r] = mean[r];
            a.rstd[row0 + r] = rstd[r];
        }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) {
        F2 ga[H], be[H];
        load_affine<V, W>(a.gamma, 1.f, w, k, ga);
        load_affine<V, W>(a.beta, 0.f, w, k, be);
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (row0 + r >= a.n) break;
#pragma unroll
            for (int j = 0; j < H; ++j) f[r][k][j] = fma(mul(f[r][k][j], both(rstd[r])), ga[j], be[j]);
            store_row<T, V, W>(y + (row0 + r) * a.c, w, k, f[r][k]);
        }
    }
}

// Persistent: a group takes R rows, the next R rows are read while these are worked on.
// part [blocks][2][c]: each block's sums of dy xh and of dy.
template <typename T, int V, int K, int R, int W>
__global__ void __launch_bounds__(kBwdBlock, 1)
k_layer_norm_grad(LayerNormArgs a, int L, float* part)
{
    constexpr int H = V / 2;
    // Past a row's end xh of x = 0 is infinite where mean rstd is, and dy's zeros do not silence that.  The row's first word stands
    // there instead, or, in long rows of single words, where those loads cost up to 15%, such a row's sum is taken again.
    constexpr bool kAgain = W == V || K == 1;
    extern __shared__ float joint[];  // [units][2][c]
    __shared__ float box[2 * 16 * 2 * R];
    wait_for_kernel_before();
    let_next_kernel_start();
    const Place<V, W> w{(int)threadIdx.x & (L - 1), L, a.c};
    const int groups = kBwdBlock / L;
    const T* x = static_cast<const T*>(a.x);
    const T* dy = static_cast<const T*>(a.dy);
    T* dx = static_cast<T*>(a.out);
    const float inv = 1.f / (float)a.c;
    F2 ga[K][H], dg[K][H], db[K][H];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        load_affine<V, W>(a.gamma, 1.f, w, k, ga[k]);
#pragma unroll
        for (int j = 0; j < H; ++j) dg[k][j] = db[k][j] = F2{0.f, 0.f};
    }
    Vec<T, V> xr[R][K], dr[R][K];
    float mr[R], sr[R];
    auto load = [&](int64_t row0) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool there = row0 + r < a.n;
            mr[r] = there ? fetch(a.mean + row0 + r) : 0.f;
            sr[r] = there ? fetch(a.rstd + row0 + r) : 0.f;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                load_row<T, V, W, kAgain>(x + (row0 + r) * a.c, w, k, there, xr[r][k]);
                load_row<T, V, W>(dy + (row0 + r) * a.c, w, k, there, dr[r][k]);
            }
        }
    };
    const int64_t step = (int64_t)gridDim.x * groups * R;
    // every group of a block makes the same number of turns, so that groups which share a warp's shuffles stay together
    const int64_t first = (int64_t)blockIdx.x * groups * R;
    const int64_t mine = (threadIdx.x / L) * R;
    int turn = 0;
    if (first < a.n) load(first + mine);
    for (int64_t base = first; base < a.n; base += step) {
        const int64_t row0 = base + mine;
        F2 xh[R][K][H], u[R][K][H];
        float s[2 * R], rs[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            F2 p{0.f, 0.f}, q{0.f, 0.f};
#pragma unroll
            for (int k = 0; k < K; ++k) {
                F2 g[H];
                unpack<T, V>(xr[r][k], xh[r][k]);
                unpack<T, V>(dr[r][k], g);
#pragma unroll
                for (int j = 0; j < H; ++j) {
                    // past the row's end dy is 0, and so is everything that this thread adds
                    xh[r][k][j] = mul(add(xh[r][k][j], both(-mr[r])), both(sr[r]));
                    dg[k][j] = fma(g[j], xh[r][k][j], dg[k][j]);
                    db[k][j] = add(db[k][j], g[j]);
                    u[r][k][j] = mul(g[j], ga[k][j]);
                    p = add(p, u[r][k][j]);
                    q = fma(u[r][k][j], xh[r][k][j], q);
                }
            }
            s[2 * r] = p.x + p.y;
            s[2 * r + 1] = q.x + q.y;
            if (!kAgain && fabsf(mr[r] * sr[r]) == INFINITY) {
                s[2 * r + 1] = 0.f;
#pragma unroll
                for (int k = 0; k < K; ++k) {
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const F2 v = u[r][k][j / 2], h = xh[r][k][j / 2];
                        if (w.in(k, j)) s[2 * r + 1] = j & 1 ? fmaf(v.y, h.y, s[2 * r + 1]) : fmaf(v.x, h.x, s[2 * r + 1]);
                    }
                }
            }
            rs[r] = sr[r];
        }
        if (base + step < a.n) load(base + step + mine);
        group_sum<2 * R>(s, L, box, turn);
        turn ^= 1;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            if (row0 + r >= a.n) break;
            const F2 am = both(-s[2 * r] * inv), bm = both(-s[2 * r + 1] * inv);
#pragma unroll
            for (int k = 0; k < K; ++k) {
#pragma unroll
                for (int j = 0; j < H; ++j) u[r][k][j] = mul(add(fma(xh[r][k][j], bm, u[r][k][j]), am), both(rs[r]));
                store_row<T, V, W>(dx + (row0 + r) * a.c, w, k, u[r][k]);
            }
        }
    }
    // groups that share a warp first, then the units (warps, or groups of several) of the block
    for (int o = L; o < 32; o <<= 1) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int j = 0; j < H; ++j) {
                dg[k][j].x += __shfl_xor_sync(FULL_MASK, dg[k][j].x, o);
                dg[k][j].y += __shfl_xor_sync(FULL_MASK, dg[k][j].y, o);
                db[k][j].x += __shfl_xor_sync(FULL_MASK, db[k][j].x, o);
                db[k][j].y += __shfl_xor_sync(FULL_MASK, db[k][j].y, o);
            }
        }
    }
    const int width = max(L, 32), units = kBwdBlock / width, unit = threadIdx.x / width;
    if ((threadIdx.x & (width - 1)) < L) {
        float* at = joint + (int64_t)unit * 2 * a.c;
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (w.in(k, j)) {
                    at[w.at(k, j)] = j & 1 ? dg[k][j / 2].y : dg[k][j / 2].x;
                    at[a.c + w.at(k, j)] = j & 1 ? db[k][j / 2].y : db[k][j / 2].x;
                }
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.c; i += kBwdBlock) {
        float s = 0.f;
        for (int u = 0; u < units; ++u) s += joint[(int64_t)u * 2 * a.c + i];
        part[(int64_t)blockIdx.x * 2 * a.c + i] = s;
    }
}

// dgamma and dbeta: the blocks' sums, each thread a sixteenth of them, then those in order.
__global__ void __launch_bounds__(kJoinCols * kJoinRows)
k_layer_norm_join(const float* part, int blocks, int c, float* dgamma, float* dbeta)
{
    __shared__ float box[kJoinRows][kJoinCols + 1];
    wait_for_kernel_before();
    const int col = blockIdx.x * kJoinCols + threadIdx.x % kJoinCols, row = threadIdx.x / kJoinCols;
    float s = 0.f;
    if (col < 2 * c)
        for (int b = row; b < blocks; b += kJoinRows) s += fetch(part + (int64_t)b * 2 * c + col);
    box[row][threadIdx.x % kJoinCols] = s;
    __syncthreads();
    if (row == 0 && col < 2 * c) {
        s = 0.f;
#pragma unroll
        for (int r = 0; r < kJoinRows; ++r) s += box[r][threadIdx.x];
        float* out = col < c ? dgamma : dbeta;
        if (out) out[col < c ? col : col - c] = s;
    }
}

// ------------------------------------------------------------- rows that registers do not hold
__device__ __forceinline__ float block_sum(float v, float* box)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(FULL_MASK, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) box[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < kLongBlock / 32; ++w) v += box[w];
    return v;
}

// A block to a row, which it reads three times.
template <typename T>
__global__ void __launch_bounds__(kLongBlock)
k_layer_norm_long(LayerNormArgs a)
{
    __shared__ float box[kLongBlock / 32];
    wait_for_kernel_before();
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + row * a.c;
    T* y = static_cast<T*>(a.out) + row * a.c;
    float s = 0.f;
    for (int i = threadIdx.x; i < a.c; i += kLongBlock) s += elem<T>::to_f32(x[i]);
    float mean = block_sum(s, box) / (float)a.c, left = 0.f;
    s = 0.f;
    float t = 0.f;
    for (int i = threadIdx.x; i < a.c; i += kLongBlock) {
        const float d = elem<T>::to_f32(x[i]) - mean;
        t += d;
        s = fmaf(d, d, s);
    }
    float var = block_sum(s, box) / (float)a.c;
    if (far_from_zero<T>(mean, var)) {
        left = block_sum(t, box) / (float)a.c;
        var = fmaxf(var - left * left, 0.f);
    }
    const float rstd = 1.f / sqrtf(var + a.eps);
    for (int i = threadIdx.x; i < a.c; i += kLongBlock) {
        const float z = (elem<T>::to_f32(x[i]) - mean - left) * rstd * (a.gamma ? fetch(a.gamma + i) : 1.f);
        y[i] = elem<T>::from_f32(z + (a.beta ? fetch(a.beta + i) : 0.f));
    }
    mean += left;
    if (threadIdx.x == 0) {
        a.mean[row] = mean;
        a.rstd[row] = rstd;
    }
}

// Sums over a share of the rows, a thread to a channel (before dx, which may take dy's or x's place).
template <typename T>
__global__ void __launch_bounds__(kLongBlock)
k_layer_norm_long_sums(LayerNormArgs a, float* part)
{
    wait_for_kernel_before();
    const int64_t c = (int64_t)blockIdx.x * kLongBlock + threadIdx.x;
    if (c >= a.c) return;
    const int64_t share = (a.n + gridDim.y - 1) / gridDim.y, lo = share * blockIdx.y, hi = min(lo + share, a.n);
    float g = 0.f, b = 0.f;
    for (int64_t r = lo; r < hi; ++r) {
        const float d = elem<T>::to_f32(static_cast<const T*>(a.dy)[r * a.c + c]);
        const float xh = (elem<T>::to_f32(static_cast<const T*>(a.x)[r * a.c + c]) - fetch(a.mean + r)) * fetch(a.rstd + r);
        g = fmaf(d, xh, g);
        b += d;
    }
    part[(int64_t)blockIdx.y * 2 * a.c + c] = g;
    part[(int64_t)blockIdx.y * 2 * a.c + a.c + c] = b;
}

template <typename T>
__global__ void __launch_bounds__(kLongBlock)
k_layer_norm_long_grad(LayerNormArgs a)
{
    __shared__ float box[kLongBlock / 32];
    wait_for_kernel_before();
    const int64_t row = blockIdx.x;
    const T* x = static_cast<const T*>(a.x) + row * a.c;
    const T* dy = static_cast<const T*>(a.dy) + row * a.c;
    T* dx = static_cast<T*>(a.out) + row * a.c;
    const float mean = fetch(a.mean + row), rstd = fetch(a.rstd + row);
    float p = 0.f, q = 0.f;
    for (int i = threadIdx.x; i < a.c; i += kLongBlock) {
        const float u = elem<T>::to_f32(dy[i]) * (a.gamma ? fetch(a.gamma + i) : 1.f);
        p += u;
        q = fmaf(u, (elem<T>::to_f32(x[i]) - mean) * rstd, q);
    }
    p = block_sum(p, box) / (float)a.c;
    q = block_sum(q, box) / (float)a.c;
    for (int i = threadIdx.x; i < a.c; i += kLongBlock) {
        const float u = elem<T>::to_f32(dy[i]) * (a.gamma ? fetch(a.gamma + i) : 1.f);
        const float xh = (elem<T>::to_f32(x[i]) - mean) * rstd;
        dx[i] = elem<T>::from_f32(rstd * (u - p - xh * q));
    }
}

// ---------------------------------------------------------------------- host
template <auto KERNEL, typename... A>
spc_status start(dim3 grid, int block, size_t smem, cudaStream_t st, A... args)
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

int pow2_at_least(int64_t v)
{
    int p = 1;
    while (p < v) p <<= 1;
    return p;
}

// Threads to a row: as many as hold it with K vectors each.
int lanes_for(int c, int per_thread) { return pow2_at_least(ceil_div(c, per_thread)); }

template <typename T, int V, int K, int R, int BLOCK, int W>
spc_status fwd(const LayerNormArgs& a, cudaStream_t st)
{
    const int L = lanes_for(a.c, V * K);
    const int64_t blocks = ceil_div(a.n, (int64_t)(BLOCK / L) * R);
    if (blocks > INT32_MAX) return SPC_ERR_UNSUPPORTED;
    return start<k_layer_norm<T, V, K, R, BLOCK, W>>(dim3((unsigned)blocks), BLOCK, 0, st, a, L);
}

// Rows that a warp holds with one vector a thread are taken four at once, with two vectors two at once; longer
// rows take four vectors a thread and as many warps as they need.
template <typename T, int W>
spc_status fwd_any(const LayerNormArgs& a, cudaStream_t st)
{
    constexpr int V = 16 / (int)sizeof(T);
    if (a.c <= 32 * V) return fwd<T, V, 1, 4, kFwdBlock, W>(a, st);
    if (a.c <= 64 * V) return fwd<T, V, 2, 2, kFwdBlock, W>(a, st);
    if (a.c <= 4 * V * kFwdBlock) return fwd<T, V, 4, 1, kFwdBlock, W>(a, st);
    if (a.c <= 4 * V * kWideFwdBlock) return fwd<T, V, 4, 1, kWideFwdBlock, W>(a, st);
    if (a.n > INT32_MAX) return SPC_ERR_UNSUPPORTED;
    return start<k_layer_norm_long<T>>(dim3((unsigned)a.n), kLongBlock, 0, st, a);
}

constexpr int kMostLongShares = 256, kBwdPer = 16;  // channels of a thread in the backward pass, at most

template <typename T, int V, int K, int R, int W>
spc_status bwd(const LayerNormArgs& a, float* part, int* blocks, cudaStream_t st)
{
    const int L = lanes_for(a.c, V * K), units = kBwdBlock / std::max(L, 32);
    *blocks = (int)std::min<int64_t>(sm_count(), ceil_div(a.n, (int64_t)(kBwdBlock / L) * R));
    return start<k_layer_norm_grad<T, V, K, R, W>>(dim3((unsigned)*blocks), kBwdBlock, (size_t)units * 2 * a.c * 4, st, a, L,
                                                       part);
}

template <typename T, int W>
spc_status bwd_any(const LayerNormArgs& a, float* part, cudaStream_t st)
{
    constexpr int V = 16 / (int)sizeof(T), K = kBwdPer / V;
    int blocks = 0;
    spc_status s = SPC_OK;
    if (a.n > 0) {
        // two rows at a time where a warp holds them, whole; addresses and bounds of single words take registers
        constexpr int kRows = W == V ? 2 : 1, kOneVector = V * (W == V ? 32 : kBwdBlock);
        if (a.c <= kOneVector) {
            s = bwd<T, V, 1, kRows, W>(a, part, &blocks, st);
        } else if (a.c <= kBwdPer * kBwdBlock) {
            s = bwd<T, V, K, 1, W>(a, part, &blocks, st);
        } else {
            if (a.n > INT32_MAX) return SPC_ERR_UNSUPPORTED;
            blocks = (int)std::min<int64_t>(kMostLongShares, a.n);
            s = start<k_layer_norm_long_sums<T>>(dim3((unsigned)ceil_div(a.c, kLongBlock), (unsigned)blocks), kLongBlock, 0, st,
                                                 a, part);
            if (s == SPC_OK) s = start<k_layer_norm_long_grad<T>>(dim3((unsigned)a.n), kLongBlock, 0, st, a);
        }
    }
    if (s != SPC_OK || (!a.dgamma && !a.dbeta)) return s;
    return start<k_layer_norm_join>(dim3((unsigned)ceil_div(2 * (int64_t)a.c, kJoinCols)), kJoinCols * kJoinRows, 0, st,
                                    (const float*)part, blocks, (int)a.c, a.dgamma, a.dbeta);
}

template <typename T>
spc_status any(const LayerNormArgs& a, float* part, bool backward, cudaStream_t st)
{
    // words of 16 bytes where rows and tensors start on such a boundary, else of two channels (40,000 rows of 334 bf16: 20 us forward, 30
    // backward, of 333 one by one 30 and 42, of 336 whole 16 and 20)
    constexpr int V = 16 / (int)sizeof(T);
    const uintptr_t low = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.out) | reinterpret_cast<uintptr_t>(a.dy) |
                          (uintptr_t)(a.c * (int64_t)sizeof(T));
    const uintptr_t affine = reinterpret_cast<uintptr_t>(a.gamma) | reinterpret_cast<uintptr_t>(a.beta);
    if ((low | affine) % 16 == 0) return backward ? bwd_any<T, V>(a, part, st) : fwd_any<T, V>(a, st);
    if (low % (2 * sizeof(T)) == 0 && affine % 8 == 0) return backward ? bwd_any<T, 2>(a, part, st) : fwd_any<T, 2>(a, st);
    return backward ? bwd_any<T, 1>(a, part, st) : fwd_any<T, 1>(a, st);
}

}  // namespace

size_t layer_norm_ws_bytes(int64_t n, int32_t c)
{
    const int64_t most = c <= kBwdPer * kBwdBlock ? sm_count() : kMostLongShares;
    return align_up((size_t)std::min<int64_t>(most, std::max<int64_t>(n, 1)) * 2 * c * 4, 256);
}

spc_status layer_norm(const LayerNormArgs& a, spc_dtype dt, void* ws, bool backward, cudaStream_t st)
{
    if (!backward && a.n == 0) return SPC_OK;
    float* part = static_cast<float*>(ws);
    switch (dt) {
    case SPC_F32: return any<float>(a, part, backward, st);
    case SPC_F16: return any<__half>(a, part, backward, st);
    default: return any<__nv_bfloat16>(a, part, backward, st);
    }
}

}  // namespace spc
