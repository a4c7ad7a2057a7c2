// Selective scan, float32 tokens and pool.
#include "k_scan.cuh"

namespace gdr {

cudaError_t launch_scan_ff(const ScanParams &p, bool vec, cudaStream_t s) { return scan_vec<float, float>(p, vec, s); }

}  // namespace gdr
