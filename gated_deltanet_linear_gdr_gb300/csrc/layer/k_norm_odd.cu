// Fused block norms on rows that are not 16-byte vectors (odd widths,
// strides or bases): element by element, neighbouring threads on neighbouring
// elements.
#include "k_norm.cuh"

namespace gdr {
namespace {

template <class C> cudaError_t go_odd(const NormParams &p, cudaStream_t s) {
    if (p.D <= 128) return go<C, 1, 4, 32>(p, s);
    if (p.D <= 512) return go<C, 1, 16, 32>(p, s);
    if (p.D <= 2048) return go<C, 1, 8, 256>(p, s);
    if (p.D <= 4096) return go<C, 1, 8, 512>(p, s);
    return go<C, 1, 32, 512>(p, s);
}

}  // namespace

cudaError_t launch_norm_odd(const NormParams &p, cudaStream_t s) {
    const bool bf_gate = p.gate && p.g_es && p.gate_bf16;
    if (p.x && p.x_bf16 && p.res && p.pre && p.out && p.out_bf16 && (bf_gate || !p.gate) && p.D > 256) {
        if (p.res_bf16) return p.gate ? go_odd<Cfg<1, 1, 1, 1, 1, -1, 1, 1>>(p, s) : go_odd<Cfg<1, 0, 0, 1, 1, -1, 1, 1>>(p, s);
        return p.gate ? go_odd<Cfg<1, 1, 1, 1, 0, -1, 1, 1>>(p, s) : go_odd<Cfg<1, 0, 0, 1, 0, -1, 1, 1>>(p, s);
    }
    return go_odd<Any>(p, s);
}

}  // namespace gdr
