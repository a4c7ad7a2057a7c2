// Selective scan of single tokens: every state goes in and out once, with a
// handful of operations on it: HBM bound.  A warp is 4 * (32 / LK) channels of one
// row, dealt to its lanes as in k_scan.cuh; all of a lane's states and rates are
// asked for before anything else, and nothing goes through shared memory.
#include "scan_device.cuh"

namespace gdr {
namespace {

constexpr int kWarps = 4;

template <typename TT, typename DT, int KT, int LK, bool VEC>
__global__ void __launch_bounds__(32 * kWarps) k_scan_step(const __grid_constant__ ScanParams p, int tiles, unsigned units) {
    constexpr int W = 4 * (32 / LK), CH = 4;
    const int lane = threadIdx.x & 31;
    const unsigned unit = blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (unit >= units) return;
    const unsigned all = (unsigned)(p.nk * tiles), row = unit / all, tg = unit - row * all;
    const int g = (int)(tg / (unsigned)tiles), tile = (int)(tg - (unsigned)g * (unsigned)tiles);
    const int group = p.r * p.V, c0 = tile * W, width = min(W, group - c0);
    const int lk = lane % LK, cg = lane / LK;
    // this lane's four channels, and the one it finishes
    int chan[CH], chead[CH];
    bool on[CH];
#pragma unroll
    for (int e = 0; e < CH; ++e) {
        const int c = c0 + cg * 4 + e;
        on[e] = cg * 4 + e < width;
        chead[e] = on[e] ? g * p.r + c / p.V : 0;
        chan[e] = on[e] ? c % p.V : 0;
    }
    int mj = chan[0], mh = chead[0];
    bool mon = on[0];
#pragma unroll
    for (int e = 1; e < CH; ++e)
        if ((lk & 3) == e) {
            mj = chan[e];
            mh = chead[e];
            mon = on[e];
        }
    mon = mon && lk < 4;

    float A[KT][CH];
#pragma unroll
    for (int i = 0; i < KT; ++i) {
        const int k = lk * KT + i;
#pragma unroll
        for (int e = 0; e < CH; ++e) A[i][e] = 0.0f;
        if (k >= p.K) continue;
        if (VEC && p.a_vec) {
            if (on[0]) {
                Pack<float, 4> q;
                q.load(p.A + chead[0] * p.a_hs + k * p.a_ks + chan[0]);
#pragma unroll
                for (int e = 0; e < CH; ++e) A[i][e] = q.get(e);
            }
        } else {
#pragma unroll
            for (int e = 0; e < CH; ++e)
                if (on[e]) A[i][e] = p.A[chead[e] * p.a_hs + k * p.a_ks + chan[e] * p.a_vs];
        }
    }
    ScanUnit u;
    if (!scan_row(p, (int)row, tg == 0 && lane == 0, u)) return;
    TT *const out = static_cast<TT *>(p.out) + u.t0 * p.o_ts + (long long)mh * p.o_hs + mj;
    if (u.slot < 0) {
        if (mon) *out = TT(0);
        return;
    }
    float S[KT][CH];
    long long at[CH];
#pragma unroll
    for (int e = 0; e < CH; ++e) at[e] = (long long)u.slot * p.st_slot + (long long)chead[e] * p.st_head + chan[e];
#pragma unroll
    for (int i = 0; i < KT; ++i) {
        const int k = lk * KT + i;
#pragma unroll
        for (int e = 0; e < CH; ++e) S[i][e] = 0.0f;
        if (k >= p.K) continue;
        if constexpr (VEC) {
            if (!on[0]) continue;
            if (p.st_bf16) {
                Pack<uint16_t, 4> q;
                q.load(static_cast<const uint16_t *>(p.state) + at[0] + k * p.st_k);
#pragma unroll
                for (int e = 0; e < CH; ++e) S[i][e] = q.get(e);
            } else {
                Pack<float, 4> q;
                q.load(static_cast<const float *>(p.state) + at[0] + k * p.st_k);
#pragma unroll
                for (int e = 0; e < CH; ++e) S[i][e] = q.get(e);
            }
        } else {
#pragma unroll
            for (int e = 0; e < CH; ++e)
                if (on[e])
                    S[i][e] = p.st_bf16 ? to_f32(static_cast<const uint16_t *>(p.state)[at[e] + k * p.st_k])
                                        : static_cast<const float *>(p.state)[at[e] + k * p.st_k];
        }
    }
    // the token
    const TT *const xp = static_cast<const TT *>(p.x) + u.t0 * p.x_ts;
    const DT *const dp = static_cast<const DT *>(p.dt) + u.t0 * p.dt_ts;
    const TT *const bp = static_cast<const TT *>(p.B) + u.t0 * p.B_ts + (long long)g * p.B_hs;
    const TT *const cp = static_cast<const TT *>(p.C) + u.t0 * p.C_ts + (long long)g * p.C_hs;
    float d[CH], x[CH], B[KT], C[KT];
#pragma unroll
    for (int e = 0; e < CH; ++e) d[e] = x[e] = 0.0f;
    if (VEC && p.dt_es) {
        if (on[0]) {
            Pack<DT, 4> q;
            q.load(dp + (long long)chead[0] * p.dt_hs + chan[0]);
#pragma unroll
            for (int e = 0; e < CH; ++e) d[e] = q.get(e);
        }
    } else {
#pragma unroll
        for (int e = 0; e < CH; ++e)
            if (on[e]) d[e] = to_f32(dp[(long long)chead[e] * p.dt_hs + chan[e] * p.dt_es]);
    }
    if constexpr (VEC) {
        if (on[0]) {
            Pack<TT, 4> q;
            q.load(xp + (long long)chead[0] * p.x_hs + chan[0]);
#pragma unroll
            for (int e = 0; e < CH; ++e) x[e] = q.get(e);
        }
    } else {
#pragma unroll
        for (int e = 0; e < CH; ++e)
            if (on[e]) x[e] = to_f32(xp[(long long)chead[e] * p.x_hs + chan[e]]);
    }
    if (p.bias)
#pragma unroll
        for (int e = 0; e < CH; ++e)
            if (on[e]) d[e] += p.bias[chead[e] * p.b_hs + chan[e] * p.b_vs];
#pragma unroll
    for (int i = 0; i < KT; ++i) {
        const int k = lk * KT + i;
        B[i] = k < p.K ? to_f32(bp[k]) : 0.0f;
        C[i] = k < p.K && p.out ? to_f32(cp[k]) : 0.0f;
    }
    const float D = mon && p.D ? p.D[mh * p.d_hs + mj * p.d_vs] : 0.0f;
    const float mx = mon ? to_f32(xp[(long long)mh * p.x_hs + mj]) : 0.0f;
    const bool gated = mon && p.z;
    const float z = gated ? to_f32(static_cast<const TT *>(p.z)[u.t0 * p.z_ts + (long long)mh * p.z_hs + mj]) : 0.0f;

    float y[CH];
#pragma unroll
    for (int e = 0; e < CH; ++e) {
        const float de = p.softplus ? softplus<TT>(d[e]) : d[e], in = de * x[e];
        y[e] = 0.0f;
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            S[i][e] = fmaf(decay<TT>(de * rate<TT>(A[i][e])), S[i][e], in * B[i]);
            y[e] = fmaf(C[i], S[i][e], y[e]);
        }
    }
    if (u.kept > 0) {
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            const int k = lk * KT + i;
            if (k >= p.K) continue;
            if constexpr (VEC) {
                if (!on[0]) continue;
                if (p.st_bf16) {
                    Pack<uint16_t, 4> q;
#pragma unroll
                    for (int e = 0; e < CH; ++e) q.set(e, S[i][e]);
                    q.store(static_cast<uint16_t *>(p.state) + at[0] + k * p.st_k);
                } else {
                    Pack<float, 4> q;
#pragma unroll
                    for (int e = 0; e < CH; ++e) q.set(e, S[i][e]);
                    q.store(static_cast<float *>(p.state) + at[0] + k * p.st_k);
                }
            } else {
#pragma unroll
                for (int e = 0; e < CH; ++e) {
                    if (!on[e]) continue;
                    if (p.st_bf16) static_cast<uint16_t *>(p.state)[at[e] + k * p.st_k] = from_f32<uint16_t>(S[i][e]);
                    else static_cast<float *>(p.state)[at[e] + k * p.st_k] = S[i][e];
                }
            }
        }
    }
    float v = fmaf(D, mx, scan_readout<LK>(y, lk));
    if (gated) v *= silu(z);
    if (mon && p.out) *out = from_f32<TT>(v);
}

template <typename TT, typename DT, int KT, int LK> cudaError_t go(const ScanParams &p, bool vec, cudaStream_t s) {
    constexpr int W = 4 * (32 / LK);
    const long long tiles = ((long long)p.r * p.V + W - 1) / W, units = (long long)p.batch * p.nk * tiles;
    if (units >= 1ll << 31) return cudaErrorInvalidConfiguration;
    const unsigned blocks = (unsigned)((units + kWarps - 1) / kWarps);
    if (vec) k_scan_step<TT, DT, KT, LK, true><<<blocks, 32 * kWarps, 0, s>>>(p, (int)tiles, (unsigned)units);
    else k_scan_step<TT, DT, KT, LK, false><<<blocks, 32 * kWarps, 0, s>>>(p, (int)tiles, (unsigned)units);
    return cudaGetLastError();
}

// States a lane and lanes a channel, by K.
template <typename TT, typename DT> cudaError_t states(const ScanParams &p, bool vec, cudaStream_t s) {
    if (p.K <= 16) return go<TT, DT, 4, 4>(p, vec, s);
    if (p.K <= 32) return go<TT, DT, 8, 4>(p, vec, s);
    if (p.K <= 64) return go<TT, DT, 8, 8>(p, vec, s);
    return go<TT, DT, 8, 16>(p, vec, s);
}

}  // namespace

cudaError_t launch_scan_step(const ScanParams &p, bool tok_bf16, bool dt_bf16, bool vec, cudaStream_t s) {
    if (!tok_bf16) return states<float, float>(p, vec, s);
    return dt_bf16 ? states<uint16_t, uint16_t>(p, vec, s) : states<uint16_t, float>(p, vec, s);
}

}  // namespace gdr
