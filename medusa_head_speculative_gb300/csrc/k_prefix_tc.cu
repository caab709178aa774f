#include "prefix.cuh"
namespace medusa {
bool prefix_tc_takes(int, int) { return false; }
cudaError_t launch_prefix_tc(const PxWork&, int, cudaStream_t) { return cudaErrorNotSupported; }
}  // namespace medusa
