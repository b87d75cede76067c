// group_norm_bf16.cu -- group norm of bf16 rows.
#include "group_norm.cuh"

namespace spc {

spc_status group_norm_bf16(const NormArgs& a, void* ws, bool backward, cudaStream_t st)
{
    return norm_pass<__nv_bfloat16>(a, ws, backward, st);
}

}  // namespace spc
