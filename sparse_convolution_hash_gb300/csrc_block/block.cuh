// block.cuh -- internal launch interfaces of a transformer block's layers: layer norm, rotary positions and
// routing to experts (attention.cuh: attention).  Argument validation happens in block_api.cu before these are called.
#pragma once

#include "layers.cuh"

namespace spc {

// --------------------------------------------------------------- layer norm
struct LayerNormArgs {
    const void* x;
    const void* dy;         // backward only
    const float* gamma;     // or NULL
    const float* beta;      // or NULL
    void* out;              // y, or dx
    float* mean;            // written by the forward pass, read by the backward one
    float* rstd;
    float* dgamma;          // backward only, or NULL
    float* dbeta;
    int64_t n;
    int32_t c;
    float eps;
};
size_t layer_norm_ws_bytes(int64_t n, int32_t c);
spc_status layer_norm(const LayerNormArgs& a, spc_dtype dt, void* ws, bool backward, cudaStream_t st);

// --------------------------------------------------------- rotary positions
struct RopeArgs {
    const void* x;
    int64_t ldx;
    const int32_t* coords;
    void* y;
    int64_t ldy;
    int64_t n;
    int32_t heads, d, back;
};
void rope_steps(const int32_t* pairs, double base, uint64_t* steps);
spc_status rope(const RopeArgs& a, const int32_t* pairs, const uint64_t* steps, spc_dtype dt, cudaStream_t st);

// ------------------------------------------------------- routing to experts
struct RouteArgs {
    const void* logits;
    const float* bias;      // or NULL
    int32_t* expert;
    float* gate;
    int64_t n;
    int32_t experts, top_k, score, groups, top_groups, renorm;
    float scale;
    int32_t lanes_log2;     // of a group, set by route()
};
struct RouteGradArgs {
    const float* dgate;
    const void* logits;
    const int32_t* expert;
    void* dlogits;
    int32_t* status;
    int64_t n;
    int32_t experts, top_k, score, renorm;
    float scale;
};
spc_status route(const RouteArgs& a, spc_dtype dt, cudaStream_t st);
spc_status route_grad(const RouteGradArgs& a, spc_dtype dt, cudaStream_t st);

}  // namespace spc
