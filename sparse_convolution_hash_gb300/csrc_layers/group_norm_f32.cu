// group_norm_f32.cu -- group norm of fp32 rows.
#include "group_norm.cuh"

namespace spc {

spc_status group_norm_f32(const NormArgs& a, void* ws, bool backward, cudaStream_t st)
{
    return norm_pass<float>(a, ws, backward, st);
}

}  // namespace spc
