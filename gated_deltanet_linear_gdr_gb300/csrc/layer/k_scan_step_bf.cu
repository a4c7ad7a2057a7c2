// Selective scan of short rows, bfloat16 tokens, float32 step sizes.
#include "k_scan_step.cuh"

namespace gdr {

cudaError_t launch_scan_step_bf(const ScanParams &p, bool vec, cudaStream_t s) { return scan_step<uint16_t, float>(p, vec, s); }

}  // namespace gdr
