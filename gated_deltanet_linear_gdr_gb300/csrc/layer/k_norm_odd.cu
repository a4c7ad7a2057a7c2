// Fused block norms on rows of odd width, base or strides: element by element,
// neighbouring threads on neighbouring elements.  Bound: load and store
// instructions, six to eight an element, 30 to 50% of the measured copy rate
// (4000 block boundaries of 8191 with a gate for each channel take 156 us in
// bfloat16 and 177 in float32; the aligned form 68 us for 8192 in bfloat16).
#include "k_norm.cuh"

namespace gdr {
namespace {

struct Single {
    // Wide rows: 1024 threads of 8 values take 126 us for 4000 rows of 6001, 512
    // threads of up to 32 took 187.
    template <class C> static cudaError_t rows(const NormParams &p, cudaStream_t s) {
        if (p.D <= 128) return go<C, 1, 4, 32>(p, s);
        if (p.D <= 512) return go<C, 1, 16, 32>(p, s);
        if (p.D <= 2048) return go<C, 1, 8, 256>(p, s);
        if (p.D <= 4096) return go<C, 1, 8, 512>(p, s);
        if (p.D <= 8192) return go<C, 1, 8, 1024>(p, s);
        return go<C, 1, 16, 1024>(p, s);
    }
};

}  // namespace

cudaError_t launch_norm_odd(const NormParams &p, cudaStream_t s) { return go_narrow<Single>(p, s); }

}  // namespace gdr
