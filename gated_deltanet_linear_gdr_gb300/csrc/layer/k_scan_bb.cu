// Selective scan, bfloat16 tokens and step sizes.
#include "k_scan.cuh"

namespace gdr {

cudaError_t launch_scan_bb(const ScanParams &p, bool vec, cudaStream_t s) { return scan_vec<uint16_t, uint16_t>(p, vec, s); }

}  // namespace gdr
