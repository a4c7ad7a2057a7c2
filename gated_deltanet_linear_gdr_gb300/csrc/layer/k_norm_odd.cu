// Fused block norms on rows that are not 16-byte vectors (odd widths,
// strides or bases): element by element, neighbouring threads on neighbouring
// elements.  Bound: load and store instructions, a vector's eighth each (4000
// block boundaries of 8191 with a gate for each channel, bfloat16, take 156 us,
// 31% of the measured copy rate; in float32 177 us, 49%; the aligned form 68 us
// for 8192).
#include "k_norm.cuh"

namespace gdr {
namespace {

// Wide rows: 1024 threads of 8 values take 126 us for 4000 rows of 6001, 512
// threads of up to 32 took 187 (with everything read from the parameters 191
// and 455).
template <class C> cudaError_t go_odd(const NormParams &p, cudaStream_t s) {
    if (p.D <= 128) return go<C, 1, 4, 32>(p, s);
    if (p.D <= 512) return go<C, 1, 16, 32>(p, s);
    if (p.D <= 2048) return go<C, 1, 8, 256>(p, s);
    if (p.D <= 4096) return go<C, 1, 8, 512>(p, s);
    if (p.D <= 8192) return go<C, 1, 8, 1024>(p, s);
    return go<C, 1, 16, 1024>(p, s);
}

}  // namespace

cudaError_t launch_norm_odd(const NormParams &p, cudaStream_t s) {
    const bool elem_gate = p.gate && p.g_es, bf_gate = elem_gate && p.gate_bf16;
    if (p.x && p.x_bf16 && p.res && p.pre && p.out && p.out_bf16 && (bf_gate || !elem_gate) && p.D > 256) {
        if (p.res_bf16) return elem_gate ? go_odd<Cfg<1, 1, 1, 1, 1, -1, 1, 1>>(p, s) : go_odd<Cfg<1, 0, 0, 1, 1, -1, 1, 1>>(p, s);
        return elem_gate ? go_odd<Cfg<1, 1, 1, 1, 0, -1, 1, 1>>(p, s) : go_odd<Cfg<1, 0, 0, 1, 0, -1, 1, 1>>(p, s);
    }
    return go_odd<Any>(p, s);
}

}  // namespace gdr
