// group_norm.cu -- group norm by element type, and its workspace.
#include "group_norm.cuh"

namespace spc {

size_t group_norm_ws_bytes(int64_t n, int32_t c, int32_t segments, int32_t groups, spc_dtype dt)
{
    (void)dt;
    // rows of more than kThreads vectors keep two sums per segment and channel instead
    const size_t wide = c > kThreads ? align_up(sizeof(float) * 2 * (size_t)c * (size_t)segments, 256) : 0;
    return std::max(carve(n, c, segments, groups, nullptr, nullptr), wide);
}

spc_status group_norm(const NormArgs& a, spc_dtype dt, void* ws, bool backward, cudaStream_t st)
{
    switch (dt) {
    case SPC_F32: return group_norm_f32(a, ws, backward, st);
    case SPC_F16: return group_norm_f16(a, ws, backward, st);
    default: return group_norm_bf16(a, ws, backward, st);
    }
}

}  // namespace spc
