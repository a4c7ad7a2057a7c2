// Selective scan, bfloat16 tokens, float32 step sizes.
#include "k_scan.cuh"

namespace gdr {

cudaError_t launch_scan_bf(const ScanParams &p, bool vec, cudaStream_t s) { return scan_vec<uint16_t, float>(p, vec, s); }

}  // namespace gdr
