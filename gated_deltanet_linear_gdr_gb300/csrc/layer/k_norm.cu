// Fused block norms on rows that may be moved as 16-byte vectors, and the
// choice of kernel (the mathematics is in k_norm.cuh).
#include "k_norm.cuh"

namespace gdr {
namespace {

constexpr unsigned kManyRows = 152 * 128;  // 8 CTAs of 16 slices on every multiprocessor

// A slice of a warp takes a head's row, two of them where there are enough
// rows: 72 us against 80 for 507 thousand rows of 128 (four: 78).
template <class C> cudaError_t go_heads(const NormParams &p, cudaStream_t s) {
    if (p.rows >= kManyRows) {
        if (p.D <= 64) return go<C, 8, 1, 8, 2>(p, s);
        if (p.D <= 128) return go<C, 8, 1, 16, 2>(p, s);
        return go<C, 8, 1, 32, 2>(p, s);
    }
    if (p.D <= 64) return go<C, 8, 1, 8>(p, s);
    if (p.D <= 128) return go<C, 8, 1, 16>(p, s);
    return go<C, 8, 1, 32>(p, s);
}
// A CTA takes a wide row.  Few warps with several vectors each: 62 us at 256
// threads x 2 against 87 at 512 x 1 for 8192 rows of 4096.
template <class C> cudaError_t go_wide(const NormParams &p, cudaStream_t s) {
    if (p.D <= 256) return go<C, 8, 1, 32>(p, s);
    if (p.D <= 512) return go<C, 8, 2, 32>(p, s);
    if (p.D <= 1024) return go<C, 8, 2, 64>(p, s);
    if (p.D <= 2048) return go<C, 8, 2, 128>(p, s);
    if (p.D <= 4096) return go<C, 8, 2, 256>(p, s);
    if (p.D <= 8192) return go<C, 8, 2, 512>(p, s);
    return go<C, 8, 4, 512>(p, s);
}

// A block boundary whose gate, if it has one a channel, is of the block's type
// (8000 rows of 6000, all float32: 141 us; with everything read from the parameters 214).
template <int XB> cudaError_t go_boundary(const NormParams &p, cudaStream_t s) {
    const bool gate = p.gate && p.g_es;
    if (p.res_bf16) {
        if (gate) return p.post ? go_wide<Cfg<XB, 1, XB, 1, 1, 1, 1, 1>>(p, s) : go_wide<Cfg<XB, 1, XB, 1, 1, 0, 1, 1>>(p, s);
        return p.post ? go_wide<Cfg<XB, 0, 0, 1, 1, 1, 1, 1>>(p, s) : go_wide<Cfg<XB, 0, 0, 1, 1, 0, 1, 1>>(p, s);
    }
    if (gate) return p.post ? go_wide<Cfg<XB, 1, XB, 1, 0, 1, 1, 1>>(p, s) : go_wide<Cfg<XB, 1, XB, 1, 0, 0, 1, 1>>(p, s);
    return p.post ? go_wide<Cfg<XB, 0, 0, 1, 0, 1, 1, 1>>(p, s) : go_wide<Cfg<XB, 0, 0, 1, 0, 0, 1, 1>>(p, s);
}

}  // namespace

cudaError_t launch_norm(const NormParams &p, int vec, cudaStream_t s) {
    if (vec < 8) return vec == 2 ? launch_norm_pairs(p, s) : launch_norm_odd(p, s);
    if (p.x && !p.res && !p.res_out && p.gate && p.g_es && p.post && !p.pre && p.out && p.out_bf16 && p.D <= 256) {
        if (p.gate_bf16)
            return p.x_bf16 ? go_heads<Cfg<1, 1, 1, 0, 0, 1, 0, 1>>(p, s) : go_heads<Cfg<0, 1, 1, 0, 0, 1, 0, 1>>(p, s);
        return p.x_bf16 ? go_heads<Cfg<1, 1, 0, 0, 0, 1, 0, 1>>(p, s) : go_heads<Cfg<0, 1, 0, 0, 0, 1, 0, 1>>(p, s);
    }
    if (is_boundary(p)) return p.x_bf16 ? go_boundary<1>(p, s) : go_boundary<0>(p, s);
    return p.D <= 64 ? go<Any, 8, 1, 8>(p, s) : p.D <= 128 ? go<Any, 8, 1, 16>(p, s) : go_wide<Any>(p, s);
}

}  // namespace gdr
