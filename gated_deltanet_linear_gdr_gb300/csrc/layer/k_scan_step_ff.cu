// Selective scan of short rows, float32 tokens and step sizes.
#include "k_scan_step.cuh"

namespace gdr {

cudaError_t launch_scan_step_ff(const ScanParams &p, bool vec, cudaStream_t s) { return scan_step<float, float>(p, vec, s); }

}  // namespace gdr
