// layers_api.cu -- the extern "C" entry points of the layers between
// convolutions (row segments, group norm, dropout, grouped products).
//
// As in the rest of the library each entry point checks its arguments on the
// host, returning an error before anything is enqueued, and enqueues its kernels
// on the caller's stream; nothing allocates or synchronises.
#include <math.h>

#include "layers.cuh"

using namespace spc;

namespace {

bool dtype_ok(spc_dtype dt) { return dt == SPC_F32 || dt == SPC_F16 || dt == SPC_BF16; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }
bool elem_aligned(const void* p, spc_dtype dt)
{
    return (reinterpret_cast<uintptr_t>(p) & (dt == SPC_F32 ? 3u : 1u)) == 0;
}
bool segments_ok(int32_t s) { return s >= 1 && s <= SPC_MAX_SEGMENTS; }

// What both passes of group norm ask of their arguments.
spc_status check_norm(const NormArgs& a, spc_dtype dt, const void* ws, size_t ws_bytes)
{
    if (!dtype_ok(dt) || a.n < 0 || a.c < 1 || a.groups < 1 || !segments_ok(a.segments))
        return SPC_ERR_INVALID_ARG;
    if (a.c % a.groups != 0) return SPC_ERR_INVALID_ARG;
    if (a.act != SPC_ACT_NONE && a.act != SPC_ACT_RELU && a.act != SPC_ACT_SILU)
        return SPC_ERR_INVALID_ARG;
    if (!a.seg || !a.mean || !a.rstd || !aligned4(a.seg) || !aligned4(a.mean) || !aligned4(a.rstd))
        return SPC_ERR_INVALID_ARG;
    if (!aligned4(a.gamma) || !aligned4(a.beta) || !aligned4(a.order)) return SPC_ERR_INVALID_ARG;
    if (a.n > 0 && (!a.x || !a.out || !elem_aligned(a.x, dt) || !elem_aligned(a.out, dt)))
        return SPC_ERR_INVALID_ARG;
    if (a.n > INT32_MAX - 1) return SPC_ERR_UNSUPPORTED;
    if (!ws || !aligned256(ws) || ws_bytes < group_norm_ws_bytes(a.n, a.c, a.segments, a.groups, dt))
        return SPC_ERR_WORKSPACE;
    return SPC_OK;
}

spc_status check_dropout(const void* x, int64_t n, double p, const uint64_t* rng, spc_dtype dt,
                         const void* y)
{
    if (!dtype_ok(dt) || n < 0 || !(p >= 0.0 && p <= 1.0)) return SPC_ERR_INVALID_ARG;
    if (!rng || (reinterpret_cast<uintptr_t>(rng) & 7u)) return SPC_ERR_INVALID_ARG;
    if (n > 0 && (!x || !y || !elem_aligned(x, dt) || !elem_aligned(y, dt))) return SPC_ERR_INVALID_ARG;
    return SPC_OK;
}

// The boundary that a grouped product's tensors start on: what its kernel moves at once.  Tensor cores: 16
// bytes; CUDA cores: four elements where every row is a multiple of that, else one.
size_t grouped_boundary(int32_t cin, int32_t cout, spc_dtype dt)
{
    const size_t e = dt == SPC_F32 ? 4 : 2;
    if (dt != SPC_F32 && cin % 8 == 0 && cout % 8 == 0) return 16;
    return cin % 4 == 0 && cout % 4 == 0 ? 4 * e : e;
}

// What the three grouped products ask of their arguments; `rows` of each operand
// must reach m when its row list is absent.
spc_status check_grouped(const void* a, const void* b, const void* out, const int32_t* seg,
                         const int32_t* a_rows, const int32_t* b_rows, int32_t segments,
                         int64_t n_a, int64_t n_b, int64_t m, int32_t cin, int32_t cout,
                         spc_dtype dt)
{
    if (!dtype_ok(dt) || !segments_ok(segments) || m < 0 || n_a < 0 || n_b < 0 || cin < 1 || cout < 1)
        return SPC_ERR_INVALID_ARG;
    if (!seg || !aligned4(seg) || !aligned4(a_rows) || !aligned4(b_rows)) return SPC_ERR_INVALID_ARG;
    if ((!a_rows && n_a < m) || (!b_rows && n_b < m)) return SPC_ERR_INVALID_ARG;
    const uintptr_t low = reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) | reinterpret_cast<uintptr_t>(out);
    if (low % grouped_boundary(cin, cout, dt) != 0) return SPC_ERR_INVALID_ARG;
    if (m > INT32_MAX - 1 || n_a > INT32_MAX - 1 || n_b > INT32_MAX - 1) return SPC_ERR_UNSUPPORTED;
    return SPC_OK;
}

// Tensor cores for 16-bit rows that TMA can load, else CUDA cores.
spc_status grouped_product(const GroupedArgs& a, spc_dtype dt, cudaStream_t st)
{
    if (grouped_tc_supported(a.k, a.n, a.in_n, dt)) {
        const spc_status s = grouped_tc(a, dt, st);
        if (s != SPC_ERR_UNSUPPORTED) return s;
    }
    return grouped_simt(a, dt, st);
}

}  // namespace

extern "C" {

size_t spc_row_segments_workspace_size(int64_t n, int32_t segments)
{
    return n < 0 || !segments_ok(segments) ? 0 : row_segments_ws_bytes(n, segments);
}

spc_status spc_row_segments(const int32_t* ids, int64_t id_stride, int64_t n, int32_t segments,
                            int32_t* seg, int32_t* order, void* ws, size_t ws_bytes, void* stream)
{
    if (n < 0 || !segments_ok(segments) || id_stride < 1 || !seg) return SPC_ERR_INVALID_ARG;
    if (n > 0 && !ids) return SPC_ERR_INVALID_ARG;
    if (!aligned4(ids) || !aligned4(seg) || !aligned4(order)) return SPC_ERR_INVALID_ARG;
    if (n > INT32_MAX - 1 || (n > 0 && id_stride > INT64_MAX / 8 / n)) return SPC_ERR_UNSUPPORTED;
    if (!ws || !aligned4(ws) || ws_bytes < row_segments_ws_bytes(n, segments)) return SPC_ERR_WORKSPACE;
    return row_segments(ids, id_stride, n, segments, seg, order, ws, static_cast<cudaStream_t>(stream));
}

size_t spc_group_norm_workspace_size(int64_t n, int32_t c, int32_t segments, int32_t groups,
                                     spc_dtype dt)
{
    if (n < 0 || c < 1 || groups < 1 || c % groups != 0 || !segments_ok(segments) || !dtype_ok(dt)) return 0;
    return group_norm_ws_bytes(n, c, segments, groups, dt);
}

spc_status spc_group_norm_fwd(const void* x, const float* gamma, const float* beta,
                              const int32_t* seg, const int32_t* order, int32_t segments, int64_t n,
                              int32_t c, int32_t groups, float eps, spc_activation act, spc_dtype dt,
                              void* y, float* mean, float* rstd, int32_t* status, void* ws,
                              size_t ws_bytes, void* stream)
{
    const NormArgs a{x, nullptr, gamma, beta, seg, order, y, mean, rstd, nullptr, nullptr, status,
                     n, segments, c, groups, (int32_t)act, eps};
    if (!(eps > 0.f) || isinf(eps)) return SPC_ERR_INVALID_ARG;
    const spc_status s = check_norm(a, dt, ws, ws_bytes);
    if (s != SPC_OK) return s;
    return group_norm(a, dt, ws, false, static_cast<cudaStream_t>(stream));
}

spc_status spc_group_norm_bwd(const void* dy, const void* x, const float* gamma, const float* beta,
                              const float* mean, const float* rstd, const int32_t* seg,
                              const int32_t* order, int32_t segments, int64_t n, int32_t c,
                              int32_t groups, spc_activation act, spc_dtype dt, void* dx,
                              float* dgamma, float* dbeta, int32_t* status, void* ws,
                              size_t ws_bytes, void* stream)
{
    const NormArgs a{x, dy, gamma, beta, seg, order, dx, const_cast<float*>(mean),
                     const_cast<float*>(rstd), dgamma, dbeta, status, n, segments, c, groups,
                     (int32_t)act, 0.f};
    const spc_status s = check_norm(a, dt, ws, ws_bytes);
    if (s != SPC_OK) return s;
    if (n > 0 && (!dy || !elem_aligned(dy, dt))) return SPC_ERR_INVALID_ARG;
    if (!aligned4(dgamma) || !aligned4(dbeta)) return SPC_ERR_INVALID_ARG;
    return group_norm(a, dt, ws, true, static_cast<cudaStream_t>(stream));
}

spc_status spc_dropout_fwd(const void* x, const void* residual, int64_t n, double p,
                           const uint64_t* rng, spc_dtype dt, void* y, void* stream)
{
    const spc_status s = check_dropout(x, n, p, rng, dt, y);
    if (s != SPC_OK) return s;
    if (residual && !elem_aligned(residual, dt)) return SPC_ERR_INVALID_ARG;
    return dropout(x, residual, n, p, rng, dt, y, static_cast<cudaStream_t>(stream));
}

spc_status spc_dropout_bwd(const void* dy, int64_t n, double p, const uint64_t* rng, spc_dtype dt,
                           void* dx, void* stream)
{
    const spc_status s = check_dropout(dy, n, p, rng, dt, dx);
    if (s != SPC_OK) return s;
    return dropout(dy, nullptr, n, p, rng, dt, dx, static_cast<cudaStream_t>(stream));
}

size_t spc_grouped_workspace_size(int32_t segments, int64_t m, int32_t cin, int32_t cout, spc_dtype dt,
                                  int32_t listed)
{
    if (!segments_ok(segments) || m < 0 || cin < 1 || cout < 1 || !dtype_ok(dt)) return 0;
    // the gradient by the weights keeps parts of sums there (on tensor cores parts of tiles, and listed
    // rows in order)
    const size_t simt = grouped_wgrad_simt_ws_bytes(segments, m, cin, cout);
    if (dt == SPC_F32 || cin % 8 || cout % 8) return simt;
    return std::max(simt, grouped_wgrad_tc_ws_bytes(m, cin, cout, listed != 0));
}

spc_status spc_grouped_fwd(const void* x, const void* w, const int32_t* seg, const int32_t* x_rows,
                           const int32_t* y_rows, int32_t segments, int64_t n_x, int64_t m,
                           int32_t cin, int32_t cout, spc_dtype dt, void* y, int32_t* status,
                           void* ws, size_t ws_bytes, void* stream)
{
    const spc_status s = check_grouped(x, w, y, seg, x_rows, y_rows, segments, n_x, m, m, cin, cout, dt);
    (void)ws;
    (void)ws_bytes;
    if (s != SPC_OK) return s;
    if (m == 0) return SPC_OK;
    if (!w || !y || (n_x > 0 && !x)) return SPC_ERR_INVALID_ARG;
    const GroupedArgs a{x, w, seg, x_rows, y_rows, y, status, n_x, m, segments, cin, cout, 0};
    return grouped_product(a, dt, static_cast<cudaStream_t>(stream));
}

spc_status spc_grouped_dgrad(const void* dy, const void* w, const int32_t* seg,
                             const int32_t* x_rows, const int32_t* y_rows, int32_t segments,
                             int64_t n_y, int64_t m, int32_t cin, int32_t cout, spc_dtype dt,
                             void* dx, int32_t* status, void* ws, size_t ws_bytes, void* stream)
{
    const spc_status s = check_grouped(dy, w, dx, seg, x_rows, y_rows, segments, m, n_y, m, cin, cout, dt);
    (void)ws;
    (void)ws_bytes;
    if (s != SPC_OK) return s;
    if (m == 0) return SPC_OK;
    if (!w || !dx || (n_y > 0 && !dy)) return SPC_ERR_INVALID_ARG;
    // W[g] as stored is [cin, cout]: the [n, k] of the product dy W[g]^T
    const GroupedArgs a{dy, w, seg, y_rows, x_rows, dx, status, n_y, m, segments, cout, cin, 1};
    return grouped_product(a, dt, static_cast<cudaStream_t>(stream));
}

spc_status spc_grouped_wgrad(const void* x, const void* dy, const int32_t* seg,
                             const int32_t* x_rows, const int32_t* y_rows, int32_t segments,
                             int64_t n_x, int64_t n_y, int64_t m, int32_t cin, int32_t cout,
                             spc_dtype dt, float* dw, int32_t* status, void* ws, size_t ws_bytes,
                             void* stream)
{
    const spc_status s = check_grouped(x, dy, dw, seg, x_rows, y_rows, segments, n_x, n_y, m, cin, cout, dt);
    if (s != SPC_OK) return s;
    if (!dw || !aligned4(dw) || (n_x > 0 && !x) || (n_y > 0 && !dy)) return SPC_ERR_INVALID_ARG;
    const size_t need = spc_grouped_workspace_size(segments, m, cin, cout, dt, x_rows || y_rows);
    if (need && (!ws || !aligned256(ws) || ws_bytes < need)) return SPC_ERR_WORKSPACE;
    const GroupedWgradArgs a{x, dy, seg, x_rows, y_rows, dw, status, n_x, n_y, m, segments, cin, cout};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return grouped_wgrad_tc_supported(a, dt) ? grouped_wgrad_tc(a, dt, ws, st) : grouped_wgrad_simt(a, dt, ws, st);
}

}  // extern "C"
