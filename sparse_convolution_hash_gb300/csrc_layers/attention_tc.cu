#include "attention.cuh"
namespace spc {
bool attention_tc_supported(const AttnArgs&, spc_dtype, bool) { return false; }
spc_status attention_fwd_tc(const AttnArgs&, spc_dtype, cudaStream_t) { return SPC_ERR_UNSUPPORTED; }
spc_status attention_bwd_tc(const AttnArgs&, spc_dtype, cudaStream_t) { return SPC_ERR_UNSUPPORTED; }
}  // namespace spc
