// group_norm_f16.cu -- group norm of fp16 rows.
#include "group_norm.cuh"

namespace spc {

spc_status group_norm_f16(const NormArgs& a, void* ws, bool backward, cudaStream_t st)
{
    return norm_pass<__half>(a, ws, backward, st);
}

}  // namespace spc
