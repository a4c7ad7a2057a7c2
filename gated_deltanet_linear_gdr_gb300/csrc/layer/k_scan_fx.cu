// Selective scan, float32 tokens over a bfloat16 pool.
#include "k_scan.cuh"

namespace gdr {

cudaError_t launch_scan_fx(const ScanParams &p, bool vec, cudaStream_t s) { return scan_vec<float, float, true>(p, vec, s); }

}  // namespace gdr
