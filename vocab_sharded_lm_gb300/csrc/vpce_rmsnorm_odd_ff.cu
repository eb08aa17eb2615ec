// Fp32 rows off 16 bytes.
#include "vpce_rmsnorm_odd.cuh"

namespace vpce {
template cudaError_t rmsnorm_forward_odd<float, float>(const RmsNormParams&, GroupKind, int, cudaStream_t);
}  // namespace vpce
