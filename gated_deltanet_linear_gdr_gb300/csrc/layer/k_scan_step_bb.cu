// Selective scan of short rows, bfloat16 tokens and step sizes.
#include "k_scan_step.cuh"

namespace gdr {

cudaError_t launch_scan_step_bb(const ScanParams &p, bool vec, cudaStream_t s) { return scan_step<uint16_t, uint16_t>(p, vec, s); }

}  // namespace gdr
