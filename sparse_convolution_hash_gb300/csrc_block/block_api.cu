// block_api.cu -- the extern "C" entry points of a transformer block's layers (layer norm, rotary positions,
// routing to experts, attention).
//
// As in the rest of the library each entry point checks its arguments on the
// host, returning an error before anything is enqueued, and enqueues its kernels
// on the caller's stream; nothing allocates or synchronises.
#include <math.h>

#include "attention.cuh"
#include "block.cuh"

using namespace spc;

namespace {

bool dtype_ok(spc_dtype dt) { return dt == SPC_F32 || dt == SPC_F16 || dt == SPC_BF16; }
bool on(const void* p, uintptr_t boundary) { return reinterpret_cast<uintptr_t>(p) % boundary == 0; }
uintptr_t bytes_of(spc_dtype dt) { return dt == SPC_F32 ? 4 : 2; }

// A tensor that n rows are read from or written to: there, and on an element's boundary.
bool rows_ok(const void* p, int64_t n, spc_dtype dt) { return on(p, bytes_of(dt)) && (n == 0 || p); }
bool floats_ok(const float* p, int64_t n) { return on(p, 4) && (n == 0 || p); }

// Rows of `width` elements, ld apart, whose last element has an address.
bool stride_ok(int64_t ld, int64_t width, int64_t n) { return ld >= width && (n < 2 || ld <= (INT64_MAX / 8 - width) / n); }

spc_status check_layer_norm(const LayerNormArgs& a, spc_dtype dt)
{
    if (!dtype_ok(dt) || a.n < 0 || a.c < 1 || a.c > INT32_MAX / 4) return SPC_ERR_INVALID_ARG;
    if (!on(a.gamma, 4) || !on(a.beta, 4)) return SPC_ERR_INVALID_ARG;
    if (!rows_ok(a.x, a.n, dt) || !rows_ok(a.out, a.n, dt) || !floats_ok(a.mean, a.n) || !floats_ok(a.rstd, a.n))
        return SPC_ERR_INVALID_ARG;
    return a.n > INT64_MAX / 8 / a.c ? SPC_ERR_UNSUPPORTED : SPC_OK;
}

spc_status check_rope(const RopeArgs& a, const int32_t* pairs, const uint64_t* steps, spc_dtype dt)
{
    if (!dtype_ok(dt) || !pairs || a.n < 0 || a.heads < 0 || a.d < 1) return SPC_ERR_INVALID_ARG;
    int64_t all = 0;
    for (int i = 0; i < 3; ++i) {
        if (pairs[i] < 0) return SPC_ERR_INVALID_ARG;
        all += pairs[i];
    }
    if (2 * all > a.d || (all > 0 && !steps)) return SPC_ERR_INVALID_ARG;
    if (all > 128 || a.heads > INT32_MAX / 4 || a.d > INT32_MAX / 4) return SPC_ERR_UNSUPPORTED;
    const int64_t width = (int64_t)a.heads * a.d;
    if (!stride_ok(a.ldx, width, a.n) || !stride_ok(a.ldy, width, a.n)) return SPC_ERR_INVALID_ARG;
    if (!rows_ok(a.x, a.n, dt) || !rows_ok(a.y, a.n, dt) || !on(a.coords, 16) || (a.n > 0 && !a.coords)) return SPC_ERR_INVALID_ARG;
    if (a.x == a.y && a.ldx != a.ldy && a.n > 1) return SPC_ERR_INVALID_ARG;
    return SPC_OK;
}

spc_status check_route(const void* logits, int64_t n, int32_t experts, int32_t top_k, int32_t score, float scale, spc_dtype dt)
{
    if (!dtype_ok(dt) || n < 0 || experts < 1 || top_k < 1 || top_k > experts) return SPC_ERR_INVALID_ARG;
    if (score != SPC_SCORE_SOFTMAX && score != SPC_SCORE_SIGMOID) return SPC_ERR_INVALID_ARG;
    if (!isfinite(scale) || !rows_ok(logits, n, dt)) return SPC_ERR_INVALID_ARG;
    return experts > SPC_MAX_SEGMENTS || top_k > SPC_MAX_TOP_K ? SPC_ERR_UNSUPPORTED : SPC_OK;
}

// Whether a result starts where an argument (or another result) does.
template <size_t N>
bool among(const void* result, const void* const (&others)[N])
{
    for (const void* p : others)
        if (result && result == p) return true;
    return false;
}

// Rows are 32-bit numbers, also those of a tile that begins before the last one.
bool attention_sizes_ok(int64_t nq, int64_t nk, int32_t segments, int32_t hq, int32_t d)
{
    return d <= 128 && hq <= 65535 && nq <= INT32_MAX - 128 && nk <= INT32_MAX - 128 && segments <= kAttnMostSegments;
}

spc_status check_attention(const AttnArgs& a, spc_dtype dt, bool backward)
{
    if (!dtype_ok(dt) || a.nq < 0 || a.nk < 0 || a.segments < 1 || a.hq < 1 || a.hk < 1 || a.d < 1) return SPC_ERR_INVALID_ARG;
    if (a.hq % a.hk != 0 || !(a.scale > 0.f) || isinf(a.scale)) return SPC_ERR_INVALID_ARG;
    if (!a.seg_q || !a.seg_k || !on(a.seg_q, 4) || !on(a.seg_k, 4)) return SPC_ERR_INVALID_ARG;
    const int64_t wq = (int64_t)a.hq * a.d, wk = (int64_t)a.hk * a.d;
    if (!stride_ok(a.ldq, wq, a.nq) || !stride_ok(a.ldk, wk, a.nk) || !stride_ok(a.ldv, wk, a.nk) || !stride_ok(a.ldo, wq, a.nq))
        return SPC_ERR_INVALID_ARG;
    if (!rows_ok(a.q, a.nq, dt) || !rows_ok(a.k, a.nk, dt) || !rows_ok(a.v, a.nk, dt) || !rows_ok(a.o, a.nq, dt) || !floats_ok(a.lse, a.nq))
        return SPC_ERR_INVALID_ARG;
    if (backward) {
        if (!stride_ok(a.lddo, wq, a.nq) || !stride_ok(a.lddq, wq, a.nq) || !stride_ok(a.lddk, wk, a.nk) || !stride_ok(a.lddv, wk, a.nk))
            return SPC_ERR_INVALID_ARG;
        if (!rows_ok(a.dout, a.nq, dt) || !rows_ok(a.dq, a.nq, dt) || !rows_ok(a.dk, a.nk, dt) || !rows_ok(a.dv, a.nk, dt))
            return SPC_ERR_INVALID_ARG;
    }
    if (!backward && among(a.o, {a.q, a.k, a.v})) return SPC_ERR_INVALID_ARG;
    if (backward && (among(a.dq, {a.q, a.k, a.v, a.o, a.dout, a.dk, a.dv}) || among(a.dk, {a.q, a.k, a.v, a.o, a.dout, a.dv}) ||
                     among(a.dv, {a.q, a.k, a.v, a.o, a.dout})))
        return SPC_ERR_INVALID_ARG;
    return attention_sizes_ok(a.nq, a.nk, a.segments, a.hq, a.d) ? SPC_OK : SPC_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" {

size_t spc_layer_norm_workspace_size(int64_t n, int32_t c)
{
    return n < 0 || c < 1 || c > INT32_MAX / 4 ? 0 : layer_norm_ws_bytes(n, c);
}

spc_status spc_layer_norm_fwd(const void* x, const float* gamma, const float* beta, int64_t n, int32_t c, float eps, spc_dtype dt,
                              void* y, float* mean, float* rstd, void* stream)
{
    const LayerNormArgs a{x, nullptr, gamma, beta, y, mean, rstd, nullptr, nullptr, n, c, eps};
    if (!(eps > 0.f) || isinf(eps)) return SPC_ERR_INVALID_ARG;
    const spc_status s = check_layer_norm(a, dt);
    return s != SPC_OK ? s : layer_norm(a, dt, nullptr, false, static_cast<cudaStream_t>(stream));
}

spc_status spc_layer_norm_bwd(const void* dy, const void* x, const float* gamma, const float* mean, const float* rstd, int64_t n,
                              int32_t c, spc_dtype dt, void* dx, float* dgamma, float* dbeta, void* ws, size_t ws_bytes,
                              void* stream)
{
    const LayerNormArgs a{x, dy, gamma, nullptr, dx, const_cast<float*>(mean), const_cast<float*>(rstd), dgamma, dbeta, n, c, 0.f};
    const spc_status s = check_layer_norm(a, dt);
    if (s != SPC_OK) return s;
    if (!rows_ok(dy, n, dt) || !on(dgamma, 4) || !on(dbeta, 4)) return SPC_ERR_INVALID_ARG;
    if (!ws || !on(ws, 256) || ws_bytes < layer_norm_ws_bytes(n, c)) return SPC_ERR_WORKSPACE;
    return layer_norm(a, dt, ws, true, static_cast<cudaStream_t>(stream));
}

spc_status spc_rope_steps(const int32_t pairs[3], double base, uint64_t* steps)
{
    // with base >= 1 no step is above a radian
    if (!pairs || pairs[0] < 0 || pairs[1] < 0 || pairs[2] < 0 || !(base >= 1.0) || isinf(base)) return SPC_ERR_INVALID_ARG;
    const int64_t all = (int64_t)pairs[0] + pairs[1] + pairs[2];
    if (all > 0 && !steps) return SPC_ERR_INVALID_ARG;
    if (all > 128) return SPC_ERR_UNSUPPORTED;
    rope_steps(pairs, base, steps);
    return SPC_OK;
}

spc_status spc_rope_fwd(const void* x, int64_t ldx, const int32_t* coords, const int32_t pairs[3], const uint64_t* steps, int64_t n,
                        int32_t heads, int32_t d, spc_dtype dt, void* y, int64_t ldy, void* stream)
{
    const RopeArgs a{x, ldx, coords, y, ldy, n, heads, d, 0};
    const spc_status s = check_rope(a, pairs, steps, dt);
    return s != SPC_OK ? s : rope(a, pairs, steps, dt, static_cast<cudaStream_t>(stream));
}

spc_status spc_rope_bwd(const void* dy, int64_t lddy, const int32_t* coords, const int32_t pairs[3], const uint64_t* steps, int64_t n,
                        int32_t heads, int32_t d, spc_dtype dt, void* dx, int64_t lddx, void* stream)
{
    const RopeArgs a{dy, lddy, coords, dx, lddx, n, heads, d, 1};
    const spc_status s = check_rope(a, pairs, steps, dt);
    return s != SPC_OK ? s : rope(a, pairs, steps, dt, static_cast<cudaStream_t>(stream));
}

spc_status spc_route_fwd(const void* logits, const float* bias, int64_t n, int32_t experts, int32_t top_k, spc_score score,
                         int32_t groups, int32_t top_groups, int32_t renorm, float scale, spc_dtype dt, int32_t* expert,
                         float* gate, void* stream)
{
    const RouteArgs a{logits, bias, expert, gate, n, experts, top_k, (int32_t)score, groups, top_groups, renorm, scale};
    const spc_status s = check_route(logits, n, experts, top_k, (int32_t)score, scale, dt);
    if (s == SPC_ERR_INVALID_ARG) return s;
    if (groups < 1 || experts % groups != 0 || top_groups < 1 || top_groups > groups || top_k > experts / groups * top_groups)
        return SPC_ERR_INVALID_ARG;
    if (!on(bias, 4) || !on(expert, 4) || (n > 0 && !expert) || !floats_ok(gate, n)) return SPC_ERR_INVALID_ARG;
    return s != SPC_OK ? s : route(a, dt, static_cast<cudaStream_t>(stream));
}

spc_status spc_route_bwd(const float* dgate, const void* logits, const int32_t* expert, int64_t n, int32_t experts, int32_t top_k,
                         spc_score score, int32_t renorm, float scale, spc_dtype dt, void* dlogits, int32_t* status, void* stream)
{
    const RouteGradArgs a{dgate, logits, expert, dlogits, status, n, experts, top_k, (int32_t)score, renorm, scale};
    const spc_status s = check_route(logits, n, experts, top_k, (int32_t)score, scale, dt);
    if (s == SPC_ERR_INVALID_ARG) return s;
    if (!floats_ok(dgate, n) || !on(expert, 4) || (n > 0 && !expert) || !rows_ok(dlogits, n, dt)) return SPC_ERR_INVALID_ARG;
    if (n > 0 && dlogits == logits) return SPC_ERR_INVALID_ARG;
    return s != SPC_OK ? s : route_grad(a, dt, static_cast<cudaStream_t>(stream));
}

size_t spc_attention_workspace_size(int64_t nq, int64_t nk, int32_t segments, int32_t hq, int32_t hk, int32_t d, spc_dtype dt,
                                    int32_t backward)
{
    if (nq < 0 || nk < 0 || segments < 1 || hq < 1 || hk < 1 || hq % hk != 0 || d < 1 || !dtype_ok(dt)) return 0;
    if (!attention_sizes_ok(nq, nk, segments, hq, d)) return 0;
    return attention_ws_bytes(nq, nk, segments, hq, hk, d, dt, backward != 0);
}

spc_status spc_attention_fwd(const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v, int64_t ldv,
                             const int32_t* seg_q, const int32_t* seg_k, int32_t segments, int64_t nq, int64_t nk, int32_t hq,
                             int32_t hk, int32_t d, float scale, spc_dtype dt, void* o, int64_t ldo, float* lse, int32_t* status,
                             void* ws, size_t ws_bytes, void* stream)
{
    AttnArgs a = {};
    a.q = q, a.k = k, a.v = v, a.seg_q = seg_q, a.seg_k = seg_k, a.ldq = ldq, a.ldk = ldk, a.ldv = ldv;
    a.nq = nq, a.nk = nk, a.segments = segments, a.hq = hq, a.hk = hk, a.d = d, a.scale = scale;
    a.o = o, a.ldo = ldo, a.lse = lse, a.status = status;
    const spc_status s = check_attention(a, dt, false);
    if (s != SPC_OK) return s;
    const size_t need = attention_ws_bytes(nq, nk, segments, hq, hk, d, dt, false);
    if (need && (!ws || !on(ws, 256) || ws_bytes < need)) return SPC_ERR_WORKSPACE;
    attention_plan(a, dt, ws, false);
    return attention_fwd(a, dt, static_cast<cudaStream_t>(stream));
}

spc_status spc_attention_bwd(const void* dout, int64_t lddo, const void* q, int64_t ldq, const void* k, int64_t ldk, const void* v,
                             int64_t ldv, const void* o, int64_t ldo, const float* lse, const int32_t* seg_q, const int32_t* seg_k,
                             int32_t segments, int64_t nq, int64_t nk, int32_t hq, int32_t hk, int32_t d, float scale, spc_dtype dt,
                             void* dq, int64_t lddq, void* dk, int64_t lddk, void* dv, int64_t lddv, int32_t* status, void* ws,
                             size_t ws_bytes, void* stream)
{
    AttnArgs a = {};
    a.q = q, a.k = k, a.v = v, a.seg_q = seg_q, a.seg_k = seg_k, a.ldq = ldq, a.ldk = ldk, a.ldv = ldv;
    a.nq = nq, a.nk = nk, a.segments = segments, a.hq = hq, a.hk = hk, a.d = d, a.scale = scale;
    a.o = const_cast<void*>(o), a.ldo = ldo, a.lse = const_cast<float*>(lse), a.status = status;
    a.dout = dout, a.lddo = lddo, a.dq = dq, a.lddq = lddq, a.dk = dk, a.lddk = lddk, a.dv = dv, a.lddv = lddv;
    const spc_status s = check_attention(a, dt, true);
    if (s != SPC_OK) return s;
    const size_t need = attention_ws_bytes(nq, nk, segments, hq, hk, d, dt, true);
    if (need && (!ws || !on(ws, 256) || ws_bytes < need)) return SPC_ERR_WORKSPACE;
    attention_plan(a, dt, ws, true);
    return attention_bwd(a, dt, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
