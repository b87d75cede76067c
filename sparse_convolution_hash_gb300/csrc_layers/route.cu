// route.cu -- the experts of each token and their weights, and the gradient by the logits.
//
// A row of logits lies in the registers of L lanes (4 to 32), eight neighbouring experts to a lane and chunk.
// The best is taken k times: each lane's own best, then the best of the lanes by shuffles, ties to the lowest
// expert.  Without a bias and groups the logits themselves are compared, which is exact.  With them the scores
// decide, p + bias, and fp32 is not enough for the last digit: the row's choice is made in fp32, and where two
// neighbours of the result lie closer than fp32's error (about one row in a hundred or fewer), made again in
// 64 bits.  The choice is therefore that of the formula in 64 bits, whatever the order of the sums.
//
// Bound by instructions: a row of 64 experts in 16 bits is 128 bytes.
#include <math.h>

#include "layers.cuh"
#include "pairs.cuh"

namespace spc {

namespace {

constexpr int kBlock = 128;
constexpr int kPer = 8;  // experts of a lane's chunk
constexpr int kNone = INT32_MAX;

__device__ __forceinline__ float exp_of(float x) { return expf(x); }
__device__ __forceinline__ double exp_of(double x) { return exp(x); }

template <typename S>
__device__ __forceinline__ S lanes_sum(S v, int L)
{
    for (int o = L >> 1; o; o >>= 1) v += __shfl_xor_sync(FULL_MASK, v, o);
    return v;
}
template <typename S>
__device__ __forceinline__ S lanes_max(S v, int L)
{
    for (int o = L >> 1; o; o >>= 1) v = max(v, __shfl_xor_sync(FULL_MASK, v, o));
    return v;
}

// Logits of a row, -inf where there is no expert, and for one that is not available (-inf, NaN); +inf counts as
// the largest finite number, so that differences exist.
template <typename T, int C>
__device__ __forceinline__ void load_logits(const T* row, int experts, int lane, int L, bool whole, float (&l)[C][kPer])
{
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e0 = (c * L + lane) * kPer;
        if (whole && e0 < experts) {
            constexpr int V = 16 / sizeof(T);
#pragma unroll
            for (int q = 0; q < kPer / V; ++q) {
                const Vec<T, V> v = *reinterpret_cast<const Vec<T, V>*>(row + e0 + q * V);
#pragma unroll
                for (int j = 0; j < V; ++j) l[c][q * V + j] = elem<T>::to_f32(v.e[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kPer; ++j) l[c][j] = e0 + j < experts ? elem<T>::to_f32(fetch(row + e0 + j)) : -INFINITY;
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) l[c][j] = l[c][j] > -INFINITY ? fminf(l[c][j], 3.402823466e38f) : -INFINITY;
    }
}

// Sum over the row of exp(l - most), `most` its largest logit (-inf: no expert is available).
template <typename S, int C>
__device__ __forceinline__ S exp_sum(const float (&l)[C][kPer], float most, int L)
{
    S s = 0;
#pragma unroll
    for (int c = 0; c < C; ++c) {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (l[c][j] > -INFINITY) s += exp_of((S)l[c][j] - (S)most);
    }
    return lanes_sum(s, L);
}

template <typename S>
__device__ __forceinline__ S score_of(float l, bool sigmoid, float most, S sum)
{
    return sigmoid ? (S)1 / ((S)1 + exp_of(-(S)l)) : exp_of((S)l - (S)most) / sum;
}

struct RouteShared {
    int32_t* expert;   // [rows][k] of this warp
    float* logit;      // [rows][k]
    double* c;         // [rows][experts], groups only
    double* best;      // [rows][groups]
};

// The row's k best, written to sh.expert and sh.logit by its lane 0.  S: the type that scores are compared in
// (BY_LOGIT: the logits, exactly).  Returns whether two neighbours, or the border of the kept groups, lie
// within the error of S.
template <typename S, bool BY_LOGIT, int C>
__device__ __forceinline__ bool choose(const RouteArgs& a, const float (&l)[C][kPer], int lane, int L, int sub, const RouteShared& sh)
{
    const S kLow = -INFINITY;
    const S rel = a.score == SPC_SCORE_SIGMOID ? (S)0x1p-20 : (S)0x1p-16;
    bool near = false;
    S c[C][kPer];
    if constexpr (BY_LOGIT) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) c[i][j] = l[i][j];
        }
    } else {
        const bool sigmoid = a.score == SPC_SCORE_SIGMOID;
        float most = -INFINITY;
#pragma unroll
        for (int i = 0; i < C; ++i) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) most = fmaxf(most, l[i][j]);
        }
        most = lanes_max(most, L);
        const S sum = sigmoid ? (S)1 : exp_sum<S>(l, most, L);
#pragma unroll
        for (int i = 0; i < C; ++i) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int e = (i * L + lane) * kPer + j;
                c[i][j] = l[i][j] > -INFINITY ? score_of<S>(l[i][j], sigmoid, most, sum) + (a.bias ? (S)fetch(a.bias + e) : (S)0) : kLow;
            }
        }
        if (a.groups > 1) {
            // a group's score: the sum of its two best (its only one's, where it has one)
            double* row = sh.c + (int64_t)sub * a.experts;
            double* best = sh.best + (int64_t)sub * a.groups;
            const int size = a.experts / a.groups;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < C; ++i) {
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    const int e = (i * L + lane) * kPer + j;
                    if (e < a.experts) row[e] = (double)c[i][j];
                }
            }
            __syncwarp();
            for (int g = lane; g < a.groups; g += L) {
                S first = kLow, second = kLow;
                for (int e = g * size; e < (g + 1) * size; ++e) {
                    const S v = (S)row[e];
                    if (v > first) {
                        second = first;
                        first = v;
                    } else if (v > second) {
                        second = v;
                    }
                }
                best[g] = (double)(second > kLow ? first + second : first);
            }
            __syncwarp();
            S least_kept = INFINITY, best_left = kLow;
            uint32_t kept_mask = 0;  // of this lane's groups, the first 32 (1,024 groups on 32 lanes)
            for (int g = lane, q = 0; g < a.groups; g += L, ++q) {
                const S mine = (S)best[g];
                int better = 0;
                for (int o = 0; o < a.groups; ++o) {
                    const S other = (S)best[o];
                    better += other > mine || (other == mine && o < g);
                }
                const bool keep = better < a.top_groups && mine > kLow;
                if (keep) least_kept = min(least_kept, mine);
                else best_left = max(best_left, mine);
                if (keep) kept_mask |= 1u << q;
            }
            least_kept = -lanes_max(-least_kept, L);
            best_left = lanes_max(best_left, L);
            if (best_left > kLow && least_kept < INFINITY)
                near = least_kept - best_left <= 2 * rel + (S)0x1p-21 * (fabs(least_kept) + fabs(best_left));
            __syncwarp();
            for (int g = lane, q = 0; g < a.groups; g += L, ++q) best[g] = kept_mask >> q & 1 ? 1.0 : 0.0;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < C; ++i) {
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                    const int e = (i * L + lane) * kPer + j;
                    if (e < a.experts && best[e / size] == 0.0) c[i][j] = kLow;
                }
            }
        }
    }
    S before = 0;
    float before_l = 0.f;
    int before_e = -1;
    // one round more than asked for shows the gap to the first that is left out
    const int rounds = BY_LOGIT ? a.top_k : a.top_k + 1;
    for (int r = 0; r < rounds; ++r) {
        S mine = kLow;
        int e_mine = kNone;
        float l_mine = 0.f;
#pragma unroll
        for (int i = 0; i < C; ++i) {
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if (c[i][j] > mine) {
                    mine = c[i][j];
                    e_mine = (i * L + lane) * kPer + j;
                    l_mine = l[i][j];
                }
        }
        S top = mine;
        int e_top = e_mine;
        float l_top = l_mine;
        for (int o = L >> 1; o; o >>= 1) {
            const S v = __shfl_xor_sync(FULL_MASK, top, o);
            const int e = __shfl_xor_sync(FULL_MASK, e_top, o);
            const float z = __shfl_xor_sync(FULL_MASK, l_top, o);
            if (v > top || (v == top && e < e_top)) {
                top = v;
                e_top = e;
                l_top = z;
            }
        }
        const bool found = e_top != kNone;
        if (!BY_LOGIT && r > 0 && found && before_e >= 0) {
            const float b0 = a.bias ? fetch(a.bias + before_e) : 0.f, b1 = a.bias ? fetch(a.bias + e_top) : 0.f;
            const S p0 = before - (S)b0, p1 = top - (S)b1;
            if (!(before_l == l_top && b0 == b1))
                near |= before - top <= rel * max(fabs(p0), fabs(p1)) + (S)0x1p-22 * (fabs(before) + fabs(top) + fabs((S)b0) + fabs((S)b1));
        }
        before = top;
        before_l = l_top;
        before_e = found ? e_top : -1;
        if (r < a.top_k && lane == 0) {
            sh.expert[sub * a.top_k + r] = found ? e_top : -1;
            sh.logit[sub * a.top_k + r] = l_top;
        }
        if (e_mine == e_top) {
#pragma unroll
            for (int i = 0; i < C; ++i) {
#pragma unroll
                for (int j = 0; j < kPer; ++j)
                    if ((i * L + lane) * kPer + j == e_top) c[i][j] = kLow;
            }
        }
    }
    return near;
}

template <typename T, int C>
__global__ void __launch_bounds__(kBlock)
k_route(RouteArgs a, int L, bool whole)
{
    extern __shared__ double room[];
    wait_for_kernel_before();
    const int lane = threadIdx.x & (L - 1), sub = (threadIdx.x & 31) / L, rows = 32 / L, warp = threadIdx.x >> 5;
    const int64_t row = ((int64_t)blockIdx.x * (kBlock / 32) + warp) * rows + sub, at = min(row, a.n - 1);
    RouteShared sh;
    const int grouped = a.groups > 1 ? rows * (a.experts + a.groups) : 0;
    double* mine = room + warp * grouped;
    sh.c = mine;
    sh.best = mine + (grouped ? rows * a.experts : 0);
    sh.logit = reinterpret_cast<float*>(room + (kBlock / 32) * grouped) + warp * 2 * rows * a.top_k;
    sh.expert = reinterpret_cast<int32_t*>(sh.logit + rows * a.top_k);
    float l[C][kPer];
    load_logits<T, C>(static_cast<const T*>(a.logits) + at * a.experts, a.experts, lane, L, whole, l);
    if (!a.bias && a.groups == 1) {
        choose<float, true, C>(a, l, lane, L, sub, sh);
    } else {
        const bool near = choose<float, false, C>(a, l, lane, L, sub, sh);
        if (__any_sync(FULL_MASK, near)) {
            __syncwarp();
            choose<double, false, C>(a, l, lane, L, sub, sh);
        }
    }
    float most = -INFINITY, sum = 1.f;
    const bool sigmoid = a.score == SPC_SCORE_SIGMOID;
    if (!sigmoid && !a.renorm) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) most = fmaxf(most, l[c][j]);
        }
        most = lanes_max(most, L);
        sum = exp_sum<float>(l, most, L);
    }
    __syncwarp();
    if (row >= a.n) return;
    const int32_t* expert = sh.expert + sub * a.top_k;
    const float* logit = sh.logit + sub * a.top_k;
    float total = 1.f;
    bool tiny = false;
    if (a.renorm) {
        total = 0.f;
        if (!sigmoid) {
            for (int r = 0; r < a.top_k; ++r)
                if (expert[r] >= 0) most = fmaxf(most, logit[r]);
        }
        for (int r = 0; r < a.top_k; ++r)
            if (expert[r] >= 0) total += score_of<float>(logit[r], sigmoid, most, 1.f);
        // scores that fp32 does not hold: sigmoid(l) is exp(l) there, to the last bit
        tiny = sigmoid && total < 1e-30f;
        if (tiny) {
            for (int r = 0; r < a.top_k; ++r)
                if (expert[r] >= 0) most = fmaxf(most, logit[r]);
            total = 0.f;
            for (int r = 0; r < a.top_k; ++r)
                if (expert[r] >= 0) total += expf(logit[r] - most);
        }
    }
    for (int r = lane; r < a.top_k; r += L) {
        float g = 0.f;
        if (expert[r] >= 0) {
            g = score_of<float>(logit[r], sigmoid && !tiny, most, sum);
            if (a.renorm) g = g / total;
        }
        a.expert[row * a.top_k + r] = expert[r];
        a.gate[row * a.top_k + r] = g * a.scale;
    }
}

// With s the scale, G the chosen experts and p the scores:
//   softmax  dl_e = p_e ([e in G] s dg_e - sum_G s dg p),           sigmoid  dl_e = [e in G] s dg_e p_e (1 - p_e)
// and with weights g = p / sum_G p:  dl_e = [e in G] s g_e (dg_e - sum_G g dg), times (1 - p_e) for sigmoid.
template <typename T, int C>
__global__ void __launch_bounds__(kBlock)
k_route_grad(RouteGradArgs a, int L, bool whole)
{
    wait_for_kernel_before();
    const int lane = threadIdx.x & (L - 1), sub = (threadIdx.x & 31) / L, rows = 32 / L, warp = threadIdx.x >> 5;
    const int64_t row = ((int64_t)blockIdx.x * (kBlock / 32) + warp) * rows + sub, at = min(row, a.n - 1);
    const T* logits = static_cast<const T*>(a.logits) + at * a.experts;
    const int32_t* expert = a.expert + at * a.top_k;
    const float* dgate = a.dgate + at * a.top_k;
    const bool sigmoid = a.score == SPC_SCORE_SIGMOID;
    float dl[C][kPer];
    float most = -INFINITY, sum = 1.f;
    if (!sigmoid && !a.renorm) {
        load_logits<T, C>(logits, a.experts, lane, L, whole, dl);
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) most = fmaxf(most, dl[c][j]);
        }
        most = lanes_max(most, L);
        sum = exp_sum<float>(dl, most, L);
    }
    // logit of the r-th chosen expert, -inf where there is none
    auto chosen = [&](int r, int& e) {
        e = fetch(expert + r);
        if (e < 0 || e >= a.experts) {
            if (e != -1) set_status(a.status, SPC_ERR_ROW_INDEX);
            e = -1;
            return -INFINITY;
        }
        const float l = elem<T>::to_f32(fetch(logits + e));
        if (!(l > -INFINITY)) e = -1;
        return l > -INFINITY ? fminf(l, 3.402823466e38f) : -INFINITY;
    };
    int e;
    float total = 1.f, dot = 0.f;
    bool tiny = false;
    if (a.renorm) {
        float largest = -INFINITY;
        total = 0.f;
        for (int r = 0; r < a.top_k; ++r) largest = fmaxf(largest, chosen(r, e));
        most = largest;
        for (int r = 0; r < a.top_k; ++r) {
            const float l = chosen(r, e);
            if (e >= 0) total += score_of<float>(l, sigmoid, most, 1.f);
        }
        tiny = sigmoid && total < 1e-30f;
        if (tiny) {
            total = 0.f;
            for (int r = 0; r < a.top_k; ++r) {
                const float l = chosen(r, e);
                if (e >= 0) total += expf(l - most);
            }
        }
    }
    if (a.renorm || !sigmoid) {
        for (int r = 0; r < a.top_k; ++r) {
            const float l = chosen(r, e);
            if (e >= 0) dot += score_of<float>(l, sigmoid && !tiny, most, sum) / total * fetch(dgate + r);
        }
    }
    if (!sigmoid && !a.renorm) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                dl[c][j] = dl[c][j] > -INFINITY ? -a.scale * dot * score_of<float>(dl[c][j], false, most, sum) : 0.f;
        }
    } else {
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int j = 0; j < kPer; ++j) dl[c][j] = 0.f;
        }
    }
    for (int r = 0; r < a.top_k; ++r) {
        const float l = chosen(r, e);
        if (e < 0 || (e / kPer) % L != lane) continue;
        float g = score_of<float>(l, sigmoid && !tiny, most, sum) / total;
        if (sigmoid) g *= 1.f / (1.f + expf(l));
        const float d = a.scale * g * (fetch(dgate + r) - (a.renorm ? dot : 0.f));
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if ((c * L + lane) * kPer + j == e) dl[c][j] += d;
        }
    }
    if (row >= a.n) return;
    T* out = static_cast<T*>(a.dlogits) + row * a.experts;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int e0 = (c * L + lane) * kPer;
        if (whole) {
            if (e0 >= a.experts) continue;
            constexpr int V = 16 / sizeof(T);
#pragma unroll
            for (int q = 0; q < kPer / V; ++q) {
                Vec<T, V> v;
#pragma unroll
                for (int j = 0; j < V; ++j) v.e[j] = elem<T>::from_f32(dl[c][q * V + j]);
                *reinterpret_cast<Vec<T, V>*>(out + e0 + q * V) = v;
            }
        } else {
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if (e0 + j < a.experts) out[e0 + j] = elem<T>::from_f32(dl[c][j]);
        }
    }
}

// Lanes to a row: eight experts each, up to a warp; beyond 256 experts four chunks of eight.
int lanes_for(int experts) { return experts <= 32 ? 4 : experts <= 64 ? 8 : experts <= 128 ? 16 : 32; }

template <auto KERNEL, typename A>
spc_status start(const A& a, size_t smem, bool whole, cudaStream_t st)
{
    const int L = lanes_for(a.experts);
    const int64_t blocks = ceil_div(a.n, (int64_t)(kBlock / 32) * (32 / L));
    if (blocks > INT32_MAX) return SPC_ERR_UNSUPPORTED;
    if (smem > 32 * 1024) {  // 48 KB with the static part need no leave
        const spc_status s = allow_smem<KERNEL>();
        if (s != SPC_OK) return s;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3(kBlock);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1] = {beside_the_kernel_before()};
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    SPC_CUDA_TRY(cudaLaunchKernelEx(&cfg, KERNEL, a, L, whole));
    return SPC_OK;
}

template <typename T>
spc_status fwd(const RouteArgs& a, cudaStream_t st)
{
    const bool whole = a.experts % kPer == 0 && aligned16(a.logits);
    const int warps = kBlock / 32, rows = 32 / lanes_for(a.experts);
    const size_t smem = (size_t)warps * rows * ((a.groups > 1 ? 8 * (size_t)(a.experts + a.groups) : 0) + 8 * (size_t)a.top_k);
    return a.experts <= 256 ? start<k_route<T, 1>>(a, smem, whole, st) : start<k_route<T, 4>>(a, smem, whole, st);
}

template <typename T>
spc_status bwd(const RouteGradArgs& a, cudaStream_t st)
{
    const bool whole = a.experts % kPer == 0 && aligned16(a.logits) && aligned16(a.dlogits);
    return a.experts <= 256 ? start<k_route_grad<T, 1>>(a, 0, whole, st) : start<k_route_grad<T, 4>>(a, 0, whole, st);
}

}  // namespace

spc_status route(const RouteArgs& a, spc_dtype dt, cudaStream_t st)
{
    if (a.n == 0) return SPC_OK;
    switch (dt) {
    case SPC_F32: return fwd<float>(a, st);
    case SPC_F16: return fwd<__half>(a, st);
    default: return fwd<__nv_bfloat16>(a, st);
    }
}

spc_status route_grad(const RouteGradArgs& a, spc_dtype dt, cudaStream_t st)
{
    if (a.n == 0) return SPC_OK;
    switch (dt) {
    case SPC_F32: return bwd<float>(a, st);
    case SPC_F16: return bwd<__half>(a, st);
    default: return bwd<__nv_bfloat16>(a, st);
    }
}

}  // namespace spc
