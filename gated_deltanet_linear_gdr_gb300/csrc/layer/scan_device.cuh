// What the selective scan's kernels share: a state's decay, softplus and SiLU, and a row's facts.
#pragma once

#include "../gdr_device.cuh"
#include "layer_internal.h"

#include <type_traits>

namespace gdr {

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// A state's decay from d and its rate.  ex2.approx errs to one side by a fraction
// of an ulp, which a slow state adds up over its memory (1000 tokens: 3e-5); that
// is nothing beside bfloat16 tokens, and float32 tokens take expf, which does not.
// Rates are finite, so that tokens that are not there (d = 0) decay nothing; what an infinite one does to
// others stays the same.
template <typename TT> __device__ __forceinline__ float rate(float a) {
    const float r = sizeof(TT) == 2 ? a * kLog2e : a, most = 3.4028235e38f;
    return r > most ? most : r < -most ? -most : r;
}
template <typename TT> __device__ __forceinline__ float decay(float e) { return sizeof(TT) == 2 ? ex2(e) : expf(e); }

// A state's step from its decay and the token's own part.  EXACT (float32 tokens over a bfloat16 pool): product and sum are
// rounded one by one, as is every operation on the way to a state, so that all forms of a call, and plain
// float32 arithmetic, have the same states bit for bit.  Such a pool can make neighbours, 2^16 times as far apart, of states
// that differ in their last bit, and the next call starts from them.  A float32 pool does not, nor do bfloat16
// outputs show it: others take the fused form, half the instructions.
template <bool EXACT> __device__ __forceinline__ float advance(float power, float S, float own) {
    return EXACT ? __fadd_rn(__fmul_rn(power, S), own) : fmaf(power, S, own);
}
template <bool EXACT> __device__ __forceinline__ float2 advance(float2 power, float2 S, float2 own) {
    if (!EXACT) return __ffma2_rn(power, S, own);
    const float2 m = __fmul2_rn(power, S);  // added one by one: nvcc 13.0 makes one instruction of __fadd2_rn and this
    return make_float2(__fadd_rn(m.x, own.x), __fadd_rn(m.y, own.y));
}

// The readout's order, the same in every form, so that a row has the same bits in any call: groups of four states (up to
// 8 states: of two) by multiply-adds from 0; their sums by pairs (past 64 states by fours, as (0 + 1) + (2 + 3); float32
// tokens, 9 to 32 states: one by one); and those one after the other.  Warps have one group or two by the form, so bfloat16
// tokens need the pairs; for float32 they cost 1% (8 ragged rows x 4096 channels 654 us without).
__device__ constexpr int scan_group(int states_a_warp) { return states_a_warp < 4 ? 2 : 4; }

// log(1 + e^v) without cancellation: max(v, 0) + log1p(e^-|v|).  bfloat16 tokens: log1p(e) / e by its Chebyshev
// interpolation of degree 8 over [0, 1], off by 2^-22 at most.
template <typename TT> __device__ __forceinline__ float softplus(float v) {
    if (sizeof(TT) == 4) return __fadd_rn(fmaxf(v, 0.0f), log1pf(expf(-fabsf(v))));
    const float e = ex2(-kLog2e * fabsf(v));
    float q = 5.126102143e-03f;
    q = fmaf(q, e, -2.907406469e-02f);
    q = fmaf(q, e, 7.751608676e-02f);
    q = fmaf(q, e, -1.360224762e-01f);
    q = fmaf(q, e, 1.907688074e-01f);
    q = fmaf(q, e, -2.483539899e-01f);
    q = fmaf(q, e, 3.331812171e-01f);
    q = fmaf(q, e, -4.999944498e-01f);
    q = fmaf(q, e, 9.999999659e-01f);
    return fmaf(q, e, fmaxf(v, 0.0f));
}

__device__ __forceinline__ float silu(float z) { return z * rcp(1.0f + ex2(-kLog2e * z)); }

struct ScanUnit {
    int b;
    long long t0;     // the unit's first token
    int len;          // its tokens
    int slot;         // -1: output cleared, nothing else
    int kept;         // tokens of the unit after which the slot is written, 0: it is not
    long long piece;  // segment index over all rows (segmented calls)
    bool last;        // the row's last segment
};

// The row's facts; flags its problems where `leader`.  False: nothing to do.
__device__ __forceinline__ bool scan_row(const ScanParams &p, int b, bool leader, ScanUnit &u) {
    const int lo = p.offsets[b], hi = p.offsets[b + 1];
    u.b = b;
    u.slot = p.slot_idx[b];
    const int count = p.counts ? p.counts[b] : 0;
    if (lo < 0 || hi < lo || hi > p.T) {
        if (leader) flag(p.status, GDR_STATUS_BAD_OFFSETS);
        return false;
    }
    u.t0 = lo;
    u.len = hi - lo;
    u.kept = 0;
    u.piece = 0;
    u.last = true;
    if (u.len == 0) return false;
    unsigned problem = 0;
    if (p.max_len > 0 && u.len > p.max_len) problem = GDR_STATUS_ROW_TOO_LONG;
    else if (u.slot < -1 || u.slot >= p.max_slots) problem = GDR_STATUS_BAD_SLOT;
    if (problem) u.slot = -1;
    if (u.slot >= 0 && p.keep) {
        if (!p.counts) u.kept = u.len;
        else if (count < 0 || count > u.len) problem = GDR_STATUS_BAD_COUNT;
        else u.kept = count;
    }
    if (problem && leader) flag(p.status, problem);
    if (!p.out) {  // only states move: tokens that are not kept are not read
        u.len = u.slot >= 0 ? u.kept : 0;
        if (u.len == 0) return false;
    }
    return true;
}

// Tokens a segment in a call that is cut.  Rows lie on one another only where offsets decrease (a row that is flagged);
// their segments may then be more than the workspace has places for, and every row is one segment, however long.
__device__ __forceinline__ int scan_segment(const ScanParams &p) {
    bool ordered = true;
    for (int b = 0; b < p.batch; ++b) ordered &= p.offsets[b] <= p.offsets[b + 1];
    return ordered ? p.seg : 0x7fffffff;
}

}  // namespace gdr
