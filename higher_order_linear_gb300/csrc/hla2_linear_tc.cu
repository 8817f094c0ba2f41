#include "hla2_linear.cuh"
namespace hla2 {
bool lin_tc_supported(const LinWalk&, int) { return false; }
cudaError_t launch_lin_tc(const LinWalk&, bool, cudaStream_t) { return cudaErrorNotSupported; }
}  // namespace hla2
