// Fused block norms on rows of even width, base and strides that are not
// 16-byte vectors: two elements at a time.  Against one at a time, 9506 rows of
// 3194 (bfloat16, a gate for each channel) take 74 us for 130, 4000 rows of 6002 60
// for 124, 8000 rows of 1002 27 for 36; load and store instructions still
// bound them, at 35 to 60% of the measured copy rate.
#include "k_norm.cuh"

namespace gdr {
namespace {

struct Pairs {
    template <class C> static cudaError_t rows(const NormParams &p, cudaStream_t s) {
        if (p.D <= 128) return go<C, 2, 2, 32>(p, s);
        if (p.D <= 512) return go<C, 2, 8, 32>(p, s);
        if (p.D <= 2048) return go<C, 2, 4, 256>(p, s);
        if (p.D <= 4096) return go<C, 2, 8, 256>(p, s);
        if (p.D <= 8192) return go<C, 2, 8, 512>(p, s);
        return go<C, 2, 8, 1024>(p, s);
    }
};

}  // namespace

cudaError_t launch_norm_pairs(const NormParams &p, cudaStream_t s) { return go_narrow<Pairs>(p, s); }

}  // namespace gdr
