// layers.cuh -- internal launch interfaces of the layers between convolutions,
// and what their kernels share: how positions, rows and segments are read.
// Argument validation happens in layers_api.cu before these are called.
#pragma once

#include <atomic>

#include "common.cuh"

namespace spc {

// ------------------------------------------------------------- row segments
size_t row_segments_ws_bytes(int64_t n, int32_t segments);
spc_status row_segments(const int32_t* ids, int64_t id_stride, int64_t n, int32_t segments,
                        int32_t* seg, int32_t* order, void* ws, cudaStream_t st);

// --------------------------------------------------------------- group norm
struct NormArgs {
    const void* x;
    const void* dy;         // backward only
    const float* gamma;     // or NULL
    const float* beta;      // or NULL
    const int32_t* seg;
    const int32_t* order;   // or NULL
    void* out;              // y, or dx
    float* mean;            // written by the forward pass, read by the backward one
    float* rstd;
    float* dgamma;          // backward only, or NULL
    float* dbeta;
    int32_t* status;
    int64_t n;
    int32_t segments, c, groups, act;
    float eps;
};
size_t group_norm_ws_bytes(int64_t n, int32_t c, int32_t segments, int32_t groups, spc_dtype dt);
spc_status group_norm(const NormArgs& a, spc_dtype dt, void* ws, bool backward, cudaStream_t st);
spc_status group_norm_f32(const NormArgs& a, void* ws, bool backward, cudaStream_t st);
spc_status group_norm_f16(const NormArgs& a, void* ws, bool backward, cudaStream_t st);
spc_status group_norm_bf16(const NormArgs& a, void* ws, bool backward, cudaStream_t st);

// ------------------------------------------------------------------ dropout
spc_status dropout(const void* x, const void* residual, int64_t n, double p, const uint64_t* rng,
                   spc_dtype dt, void* y, cudaStream_t st);

// --------------------------------------------------------- grouped products
// out[out_rows(r)] = in[in_rows(r)] B[g], B[g] = w[g] ([k, n] row-major), or its
// transpose of a stored [n, k] when w_transposed.
struct GroupedArgs {
    const void* in;
    const void* w;
    const int32_t* seg;
    const int32_t* in_rows;   // or NULL
    const int32_t* out_rows;  // or NULL
    void* out;
    int32_t* status;
    int64_t in_n, m;
    int32_t segments, k, n, w_transposed;
};
// dw[g] = sum over g's positions of x[x_rows(r)]^T dy[y_rows(r)]
struct GroupedWgradArgs {
    const void* x;
    const void* dy;
    const int32_t* seg;
    const int32_t* x_rows;
    const int32_t* y_rows;
    float* dw;
    int32_t* status;
    int64_t n_x, n_y, m;
    int32_t segments, cin, cout;
};
spc_status grouped_simt(const GroupedArgs& a, spc_dtype dt, cudaStream_t st);
bool grouped_tc_supported(int32_t k, int32_t n, int64_t in_n, spc_dtype dt);
spc_status grouped_tc(const GroupedArgs& a, spc_dtype dt, cudaStream_t st);
size_t grouped_wgrad_tc_ws_bytes(int64_t m, int32_t cin, int32_t cout, bool listed);
bool grouped_wgrad_tc_supported(const GroupedWgradArgs& a, spc_dtype dt);
spc_status grouped_wgrad_tc(const GroupedWgradArgs& a, spc_dtype dt, void* ws, cudaStream_t st);
size_t grouped_wgrad_simt_ws_bytes(int32_t segments, int64_t m, int32_t cin, int32_t cout);
spc_status grouped_wgrad_simt(const GroupedWgradArgs& a, spc_dtype dt, void* ws, cudaStream_t st);

// Lets a kernel ask for as much dynamic shared memory as an SM has; set once per device, as every
// setting costs the host about as much as a launch.
constexpr int kMostSmem = 227 * 1024;
template <auto KERNEL>
spc_status allow_smem()
{
    static std::atomic<bool> done[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return SPC_ERR_CUDA;
    if (!done[dev].load(std::memory_order_relaxed)) {
        cudaFuncAttributes at;
        SPC_CUDA_TRY(cudaFuncGetAttributes(&at, KERNEL));
        SPC_CUDA_TRY(cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          kMostSmem - (int)at.sharedSizeBytes));
        done[dev].store(true, std::memory_order_relaxed);
    }
    return SPC_OK;
}

// Launch attribute of a kernel that may be set up while the one before it in the stream ends; it touches no
// memory of others before wait_for_kernel_before() (grouped forward, 2,048 rows in 8 segments, 512 x 512 bf16,
// repeated: 7.4 us against 7.9; 2,000 x 16 fp32 group norm 8.8 against 9.1).
inline cudaLaunchAttribute beside_the_kernel_before()
{
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    return at;
}
__device__ __forceinline__ void wait_for_kernel_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Such kernels read what others wrote by ordinary loads: one through the read-only path might be
// moved ahead of the wait.
template <typename T>
__device__ __forceinline__ T fetch(const T* p) { return *p; }

// ------------------------------------------------------------ device helpers
// Segment s as positions [lo, hi) inside [0, n): offsets out of range or out of
// order are reported and read as an empty (or cut) segment.
__device__ __forceinline__ void segment_bounds(const int32_t* seg, int s, int64_t n, int32_t* status,
                                               int64_t& lo, int64_t& hi)
{
    const int64_t a = fetch(seg + s), b = fetch(seg + s + 1);
    lo = a < 0 ? 0 : (a > n ? n : a);
    hi = b < lo ? lo : (b > n ? n : b);
    if (lo != a || hi != b) set_status(status, SPC_ERR_ROW_INDEX);
}

// The segment that holds position r: the last s with seg[s] <= r, -1 before the
// first, `segments` from seg[segments] on.
__device__ __forceinline__ int segment_of(const int32_t* seg, int segments, int64_t r)
{
    int lo = 0, hi = segments + 1;  // first index with seg[index] > r
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (fetch(seg + mid) > r) hi = mid;
        else lo = mid + 1;
    }
    return lo - 1;
}

// The row at position r, or -1 (reported) when the list names one out of [0, rows).
__device__ __forceinline__ int64_t row_at(const int32_t* list, int64_t r, int64_t rows, int32_t* status)
{
    if (!list) return r;
    const int32_t i = fetch(list + r);
    if (i < 0 || i >= rows) {
        set_status(status, SPC_ERR_ROW_INDEX);
        return -1;
    }
    return i;
}

}  // namespace spc
