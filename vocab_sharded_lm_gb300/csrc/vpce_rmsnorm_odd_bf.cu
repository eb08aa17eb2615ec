// Bf16 rows beside an fp32 residual stream off 16 bytes.
#include "vpce_rmsnorm_odd.cuh"

namespace vpce {
template cudaError_t rmsnorm_forward_odd<__nv_bfloat16, float>(const RmsNormParams&, GroupKind, int, cudaStream_t);
}  // namespace vpce
