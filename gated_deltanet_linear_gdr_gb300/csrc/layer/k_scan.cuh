// Selective state space scan: every channel j keeps K states, and per token
//
//     d = softplus(dt + bias);  S_i <- exp(d A_i) S_i + (d x) B_i;  y = sum_i C_i S_i + D x
//
// in float32.  Each state has a decay of its own that follows the token, so there
// is no matrix product in it: 16 states cost a channel's token 16
// exponentials and 64 float32 operations (half as many instructions in pairs).
//
// A warp is a unit by itself: 4 * (32 / LK) channels of one row (or of one segment
// of it).  Lane (cg, lk) keeps states lk KT .. lk KT + KT - 1 of channels 4 cg .. 4 cg + 3 in
// registers for all of the unit's tokens, and their A.  Four channels by KT states
// a lane are what keeps shared memory out of the way: a token's d and d x are read
// for KT states each, its B and C for four channels each.
//
// Tokens go through in chunks of kChunk.  Lanes load a chunk as vectors along the
// channels, work out d and d x once a channel, and leave them with B and C in the
// warp's own piece of shared memory; the readout of a token is added up over lk by
// shuffles that leave every lane one channel, and goes back through shared
// memory, to be finished (D x, the gate) and stored as vectors.
#pragma once

#include "../gdr_device.cuh"
#include "layer_internal.h"

namespace gdr {

constexpr int kScanChunk = 16;
constexpr int kScanWarps = 4;  // a block's

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;

// log(1 + e^v) without cancellation: max(v, 0) + log1p(e^-|v|).
__device__ __forceinline__ float softplus(float v) { return fmaxf(v, 0.0f) + log1pf(__expf(-fabsf(v))); }

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

// Segment `piece` of all rows' segments, for calls of at most 32 rows: lane l counts row l's.
__device__ __forceinline__ bool scan_piece(const ScanParams &p, long long piece, bool leader, int lane, ScanUnit &u) {
    ScanUnit r;
    bool live = false;
    if (lane < p.batch) live = scan_row(p, lane, leader && piece == 0, r);
    int n = live ? pieces(r.len, p.seg) : 0, upto = n;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int o = __shfl_up_sync(kFull, upto, m);
        if (lane >= m) upto += o;
    }
    const unsigned behind = __ballot_sync(kFull, upto > piece);
    if (!behind) return false;
    const int b = __ffs(behind) - 1;
    const int s = (int)piece - __shfl_sync(kFull, upto - n, b);
    if (!scan_row(p, b, false, u)) return false;
    const long long from = (long long)s * p.seg;
    u.t0 += from;
    const long long left = u.len - from, kept = u.kept - from;
    u.last = left <= p.seg;
    u.len = (int)(left < p.seg ? left : p.seg);
    u.kept = kept <= 0 || kept > u.len ? 0 : (int)kept;
    u.piece = piece;
    return true;
}

// Where a warp's chunk lies in shared memory, in floats.
template <int KT, int LK> struct ScanShared {
    static constexpr int W = 4 * (32 / LK), KP = KT * LK;
    static constexpr int d = 0, x = d + kScanChunk * W, y = x + kScanChunk * W, B = y + kScanChunk * W,
                         C = B + kScanChunk * KP, bias = C + kScanChunk * KP, D = bias + W, size = D + W;
};

// FIRST: the pass over segments that only works out their own states, from zero,
// and the sums of their step sizes.
template <typename TT, typename DT, int KT, int LK, bool VEC, bool FIRST>
__global__ void __launch_bounds__(32 * kScanWarps) k_scan(const __grid_constant__ ScanParams p, int tiles, unsigned units) {
    using Sh = ScanShared<KT, LK>;
    constexpr int W = Sh::W, KP = Sh::KP, CH = 4;
    extern __shared__ __align__(16) float shared[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned unit = blockIdx.x * kScanWarps + warp;
    if (unit >= units) return;
    const unsigned all = (unsigned)(p.nk * tiles), row = unit / all, tg = unit - row * all;
    const int g = (int)(tg / (unsigned)tiles), tile = (int)(tg - (unsigned)g * (unsigned)tiles);
    ScanUnit u;
    if (p.seg) {
        if (!scan_piece(p, row, tg == 0 && !FIRST, lane, u)) return;
        if (FIRST && u.last) return;  // no segment starts from its state
    } else if (!scan_row(p, (int)row, tg == 0 && lane == 0, u)) {
        return;
    }
    const int group = p.r * p.V, c0 = tile * W;  // channels of the key head's value heads, this warp's first
    const int width = min(W, group - c0);
    float *const sh = shared + warp * Sh::size;

    // A channel of the group as (value head, channel).
    auto head = [&](int c, int &j) {
        const int h = c / p.V;
        j = c - h * p.V;
        return g * p.r + h;
    };

    // tokens by vectors: lane's piece of 8 channels, of token lane / PCS and every TPP-th behind it
    constexpr int PCS = W / 8, TPP = 32 / PCS;
    const int pc = lane % PCS, pt = lane / PCS;
    int pj = 0, ph = 0;
    bool pon = false;
    // tokens one by one: channel lane % W, of token lane / W and every (32 / W)-th behind it
    constexpr int TPS = 32 / W;
    const int sc = lane % W, stt = lane / W;
    if constexpr (VEC) {
        pon = pc * 8 < width;
        if (pon) ph = head(c0 + pc * 8, pj);
    } else {
        pon = sc < width;
        if (pon) ph = head(c0 + sc, pj);
    }

    if (u.slot < 0) {  // padding: zeros
        if constexpr (!FIRST) {
            TT *o = static_cast<TT *>(p.out) + u.t0 * p.o_ts + (long long)ph * p.o_hs + pj;
            if (pon) {
                if constexpr (VEC) {
                    for (int t = pt; t < u.len; t += TPP)
#pragma unroll
                        for (int i = 0; i < 8 * (int)sizeof(TT) / 16; ++i)
                            reinterpret_cast<uint4 *>(o + (long long)t * p.o_ts)[i] = make_uint4(0, 0, 0, 0);
                } else {
                    for (int t = stt; t < u.len; t += TPS) o[(long long)t * p.o_ts] = TT(0);
                }
            }
        }
        return;
    }

    // this lane's states and their rates, in pairs along K
    const int lk = lane % LK, cg = lane / LK;
    float2 S[CH][KT / 2], A[CH][KT / 2];
    long long st_at[CH];
    int chan[CH], chead[CH];
    bool on[CH];
#pragma unroll
    for (int e = 0; e < CH; ++e) {
        on[e] = cg * 4 + e < width;
        chead[e] = on[e] ? head(c0 + cg * 4 + e, chan[e]) : 0;
        if (!on[e]) chan[e] = 0;
        st_at[e] = (long long)u.slot * p.st_slot + (long long)chead[e] * p.st_head + chan[e];
    }
    // a state row's four channels, from the pool or from float32 segments' states
    auto get = [&](int k, float (&v)[CH]) {
#pragma unroll
        for (int e = 0; e < CH; ++e) v[e] = 0.0f;
        if (k >= p.K) return;
        if (p.seg) {
            const float *w = p.ws + (u.piece * p.nv + chead[0]) * (long long)p.K * p.V + (long long)k * p.V;
#pragma unroll
            for (int e = 0; e < CH; ++e)
                if (on[e]) v[e] = w[(long long)(chead[e] - chead[0]) * p.K * p.V + chan[e]];
        } else if (VEC) {
            if (!on[0]) return;
            if (p.st_bf16) {
                Pack<uint16_t, 4> q;
                q.load(static_cast<const uint16_t *>(p.state) + st_at[0] + k * p.st_k);
#pragma unroll
                for (int e = 0; e < CH; ++e) v[e] = q.get(e);
            } else {
                Pack<float, 4> q;
                q.load(static_cast<const float *>(p.state) + st_at[0] + k * p.st_k);
#pragma unroll
                for (int e = 0; e < CH; ++e) v[e] = q.get(e);
            }
        } else {
#pragma unroll
            for (int e = 0; e < CH; ++e)
                if (on[e])
                    v[e] = p.st_bf16 ? to_f32(static_cast<const uint16_t *>(p.state)[st_at[e] + k * p.st_k])
                                     : static_cast<const float *>(p.state)[st_at[e] + k * p.st_k];
        }
    };
#pragma unroll
    for (int i = 0; i < KT; ++i) {
        const int k = lk * KT + i;
        float v[CH], a[CH];
        if constexpr (FIRST) {
#pragma unroll
            for (int e = 0; e < CH; ++e) v[e] = 0.0f;
        } else {
            get(k, v);
        }
#pragma unroll
        for (int e = 0; e < CH; ++e) a[e] = 0.0f;
        if (k < p.K) {
            if (VEC && p.a_vec) {
                if (on[0]) {
                    const float4 q = *reinterpret_cast<const float4 *>(p.A + chead[0] * p.a_hs + k * p.a_ks + chan[0]);
                    a[0] = q.x;
                    a[1] = q.y;
                    a[2] = q.z;
                    a[3] = q.w;
                }
            } else {
#pragma unroll
                for (int e = 0; e < CH; ++e)
                    if (on[e]) a[e] = p.A[chead[e] * p.a_hs + k * p.a_ks + chan[e] * p.a_vs];
            }
        }
#pragma unroll
        for (int e = 0; e < CH; ++e) {
            (i & 1 ? S[e][i / 2].y : S[e][i / 2].x) = v[e];
            (i & 1 ? A[e][i / 2].y : A[e][i / 2].x) = a[e] * kLog2e;
        }
    }
    // the pool's new value
    auto put = [&]() {
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            const int k = lk * KT + i;
            if (k >= p.K) continue;
            float v[CH];
#pragma unroll
            for (int e = 0; e < CH; ++e) v[e] = i & 1 ? S[e][i / 2].y : S[e][i / 2].x;
            if constexpr (FIRST) {
                float *w = p.ws + (u.piece * p.nv + chead[0]) * (long long)p.K * p.V + (long long)k * p.V;
#pragma unroll
                for (int e = 0; e < CH; ++e)
                    if (on[e]) w[(long long)(chead[e] - chead[0]) * p.K * p.V + chan[e]] = v[e];
            } else if constexpr (VEC) {
                if (!on[0]) continue;
                if (p.st_bf16) {
                    Pack<uint16_t, 4> q;
#pragma unroll
                    for (int e = 0; e < CH; ++e) q.set(e, v[e]);
                    q.store(static_cast<uint16_t *>(p.state) + st_at[0] + k * p.st_k);
                } else {
                    Pack<float, 4> q;
#pragma unroll
                    for (int e = 0; e < CH; ++e) q.set(e, v[e]);
                    q.store(static_cast<float *>(p.state) + st_at[0] + k * p.st_k);
                }
            } else {
#pragma unroll
                for (int e = 0; e < CH; ++e) {
                    if (!on[e]) continue;
                    if (p.st_bf16) static_cast<uint16_t *>(p.state)[st_at[e] + k * p.st_k] = from_f32<uint16_t>(v[e]);
                    else static_cast<float *>(p.state)[st_at[e] + k * p.st_k] = v[e];
                }
            }
        }
    };

    for (int i = lane; i < W; i += 32) {
        int j = 0, h = 0;
        const bool in = i < width;
        if (in) h = head(c0 + i, j);
        sh[Sh::bias + i] = in && p.bias ? p.bias[h * p.b_hs + j * p.b_vs] : 0.0f;
        sh[Sh::D + i] = in && p.D ? p.D[h * p.d_hs + j * p.d_vs] : 0.0f;
    }
    for (int i = lane; i < kScanChunk * KP; i += 32) {  // states past K, and what no token writes
        sh[Sh::B + i] = 0.0f;
        sh[Sh::C + i] = 0.0f;
    }
    for (int i = lane; i < kScanChunk * W; i += 32) {
        sh[Sh::d + i] = 0.0f;
        sh[Sh::x + i] = 0.0f;
    }
    __syncwarp();

    const TT *const xp = static_cast<const TT *>(p.x) + u.t0 * p.x_ts + (long long)ph * p.x_hs + pj;
    const DT *const dp = static_cast<const DT *>(p.dt) + u.t0 * p.dt_ts + (long long)ph * p.dt_hs + pj * p.dt_es;
    const TT *const bp = static_cast<const TT *>(p.B) + u.t0 * p.B_ts + (long long)g * p.B_hs;
    const TT *const cp = static_cast<const TT *>(p.C) + u.t0 * p.C_ts + (long long)g * p.C_hs;
    const bool outputs = !FIRST && p.out;
    float2 dsum[CH / 2];
#pragma unroll
    for (int e = 0; e < CH / 2; ++e) dsum[e] = make_float2(0.0f, 0.0f);

    for (int base = 0; base < u.len; base += kScanChunk) {
        const int n = min(kScanChunk, u.len - base);
        // ---- stage a chunk
        if constexpr (VEC) {
            for (int t = pt; t < n; t += TPP) {
                if (!pon) continue;
                float d[8], x[8];
                if (p.dt_es) {
#pragma unroll
                    for (int i = 0; i < 8; i += 16 / (int)sizeof(DT)) {
                        Pack<DT, 16 / (int)sizeof(DT)> q;
                        q.load(dp + (long long)(base + t) * p.dt_ts + i);
#pragma unroll
                        for (int j = 0; j < 16 / (int)sizeof(DT); ++j) d[i + j] = q.get(j);
                    }
                } else {
                    const float v = to_f32(dp[(long long)(base + t) * p.dt_ts]);
#pragma unroll
                    for (int i = 0; i < 8; ++i) d[i] = v;
                }
#pragma unroll
                for (int i = 0; i < 8; i += 16 / (int)sizeof(TT)) {
                    Pack<TT, 16 / (int)sizeof(TT)> q;
                    q.load(xp + (long long)(base + t) * p.x_ts + i);
#pragma unroll
                    for (int j = 0; j < 16 / (int)sizeof(TT); ++j) x[i + j] = q.get(j);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    d[i] += sh[Sh::bias + pc * 8 + i];
                    if (p.softplus) d[i] = softplus(d[i]);
                    x[i] *= d[i];
                }
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    *reinterpret_cast<float4 *>(sh + Sh::d + t * W + pc * 8 + i) = make_float4(d[i], d[i + 1], d[i + 2], d[i + 3]);
                    *reinterpret_cast<float4 *>(sh + Sh::x + t * W + pc * 8 + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
                }
            }
        } else if (pon) {
            for (int t = stt; t < n; t += TPS) {
                float d = to_f32(dp[(long long)(base + t) * p.dt_ts]) + sh[Sh::bias + sc];
                if (p.softplus) d = softplus(d);
                sh[Sh::d + t * W + sc] = d;
                sh[Sh::x + t * W + sc] = d * to_f32(xp[(long long)(base + t) * p.x_ts]);
            }
        }
        for (int i = lane; i < n * p.K; i += 32) {
            const int t = i / p.K, k = i - t * p.K;
            sh[Sh::B + t * KP + k] = to_f32(bp[(long long)(base + t) * p.B_ts + k]);
            if (outputs) sh[Sh::C + t * KP + k] = to_f32(cp[(long long)(base + t) * p.C_ts + k]);
        }
        __syncwarp();
        // ---- its tokens, in two parts where the slot's state lies between them
        const int cut = u.kept - base;
        const bool inside = !FIRST && cut > 0 && cut <= n;
        int t = 0;
        for (int part = 0; part < 2; ++part) {
            const int end = part == 0 && inside ? cut : n;
            for (; t < end; ++t) {
                const float4 d4 = *reinterpret_cast<const float4 *>(sh + Sh::d + t * W + cg * 4);
                const float4 x4 = *reinterpret_cast<const float4 *>(sh + Sh::x + t * W + cg * 4);
                const float d[CH] = {d4.x, d4.y, d4.z, d4.w}, x[CH] = {x4.x, x4.y, x4.z, x4.w};
                float2 Bv[KT / 2], Cv[KT / 2];
#pragma unroll
                for (int i = 0; i < KT / 2; ++i) {
                    Bv[i] = *reinterpret_cast<const float2 *>(sh + Sh::B + t * KP + lk * KT + 2 * i);
                    Cv[i] = *reinterpret_cast<const float2 *>(sh + Sh::C + t * KP + lk * KT + 2 * i);
                }
                float y[CH];
#pragma unroll
                for (int e = 0; e < CH; ++e) {
                    float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll
                    for (int i = 0; i < KT / 2; ++i) {
                        float2 a = __fmul2_rn(make_float2(d[e], d[e]), A[e][i]);
                        a.x = ex2(a.x);
                        a.y = ex2(a.y);
                        S[e][i] = __ffma2_rn(a, S[e][i], __fmul2_rn(make_float2(x[e], x[e]), Bv[i]));
                        if (!FIRST) acc = __ffma2_rn(Cv[i], S[e][i], acc);
                    }
                    y[e] = acc.x + acc.y;
                }
                if constexpr (FIRST) {
                    dsum[0] = __fadd2_rn(dsum[0], make_float2(d[0], d[1]));
                    dsum[1] = __fadd2_rn(dsum[1], make_float2(d[2], d[3]));
                } else if (outputs) {
                    // over lk: two exchanges leave lane lk channel 4 cg + lk % 4, the rest add up
                    const bool up = lk & 2;
                    float a = up ? y[2] : y[0], b = up ? y[3] : y[1];
                    a += __shfl_xor_sync(kFull, up ? y[0] : y[2], 2);
                    b += __shfl_xor_sync(kFull, up ? y[1] : y[3], 2);
                    const bool odd = lk & 1;
                    float v = odd ? b : a;
                    v += __shfl_xor_sync(kFull, odd ? a : b, 1);
#pragma unroll
                    for (int m = 4; m < LK; m <<= 1) v += __shfl_xor_sync(kFull, v, m);
                    if (LK == 4 || lk < 4) sh[Sh::y + t * W + cg * 4 + (lk & 3)] = v;
                }
            }
            if (part == 0 && inside) put();
        }
        __syncwarp();
        // ---- finish and store its outputs
        if (outputs && pon) {
            const TT *const zp = static_cast<const TT *>(p.z) + (p.z ? u.t0 * p.z_ts + (long long)ph * p.z_hs + pj : 0);
            TT *const op = static_cast<TT *>(p.out) + u.t0 * p.o_ts + (long long)ph * p.o_hs + pj;
            if constexpr (VEC) {
                constexpr int C = 16 / (int)sizeof(TT);
                for (int tt = pt; tt < n; tt += TPP) {
#pragma unroll
                    for (int i = 0; i < 8; i += C) {
                        Pack<TT, C> x, z, o;
                        x.load(xp + (long long)(base + tt) * p.x_ts + i);
                        if (p.z) z.load(zp + (long long)(base + tt) * p.z_ts + i);
#pragma unroll
                        for (int j = 0; j < C; ++j) {
                            float y = fmaf(sh[Sh::D + pc * 8 + i + j], x.get(j), sh[Sh::y + tt * W + pc * 8 + i + j]);
                            if (p.z) {
                                const float zv = z.get(j);
                                y *= __fdividef(zv, 1.0f + __expf(-zv));
                            }
                            o.set(j, y);
                        }
                        o.store(op + (long long)(base + tt) * p.o_ts + i);
                    }
                }
            } else {
                for (int tt = stt; tt < n; tt += TPS) {
                    float y = fmaf(sh[Sh::D + sc], to_f32(xp[(long long)(base + tt) * p.x_ts]), sh[Sh::y + tt * W + sc]);
                    if (p.z) {
                        const float zv = to_f32(zp[(long long)(base + tt) * p.z_ts]);
                        y *= __fdividef(zv, 1.0f + __expf(-zv));
                    }
                    op[(long long)(base + tt) * p.o_ts] = from_f32<TT>(y);
                }
            }
        }
        __syncwarp();
    }
    if constexpr (FIRST) {
        put();
        if (lk == 0) {
            float *sum = p.ws + scan_pieces(p.T, p.seg, p.batch) * p.nv * p.K * p.V + u.piece * p.nv * p.V;
            const float d[CH] = {dsum[0].x, dsum[0].y, dsum[1].x, dsum[1].y};
#pragma unroll
            for (int e = 0; e < CH; ++e)
                if (on[e]) sum[(long long)chead[e] * p.V + chan[e]] = d[e];
        }
    }
}

template <typename TT, typename DT, int KT, int LK, bool VEC> cudaError_t scan_go(const ScanParams &p, cudaStream_t s) {
    using Sh = ScanShared<KT, LK>;
    constexpr int bytes = 4 * kScanWarps * Sh::size;
    static LaunchCache cache;
    LaunchInfo info;
    cudaError_t e = launch_info(cache, &info, [](LaunchInfo &) {
        if (bytes <= 48 << 10) return cudaSuccess;
        const cudaError_t f = cudaFuncSetAttribute(k_scan<TT, DT, KT, LK, VEC, false>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (f != cudaSuccess) return f;
        return cudaFuncSetAttribute(k_scan<TT, DT, KT, LK, VEC, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    });
    if (e != cudaSuccess) return e;
    const long long tiles = ((long long)p.r * p.V + Sh::W - 1) / Sh::W;
    const long long rows = p.seg ? scan_pieces(p.T, p.seg, p.batch) : p.batch, units = rows * p.nk * tiles;
    if (units >= 1ll << 31) return cudaErrorInvalidConfiguration;
    const unsigned blocks = (unsigned)((units + kScanWarps - 1) / kScanWarps);
    if (p.seg) {
        k_scan<TT, DT, KT, LK, VEC, true><<<blocks, 32 * kScanWarps, bytes, s>>>(p, (int)tiles, (unsigned)units);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        if ((e = launch_scan_join(p, s)) != cudaSuccess) return e;
    }
    k_scan<TT, DT, KT, LK, VEC, false><<<blocks, 32 * kScanWarps, bytes, s>>>(p, (int)tiles, (unsigned)units);
    return cudaGetLastError();
}

// States a lane and lanes a channel, by K.
template <typename TT, typename DT, bool VEC> cudaError_t scan_states(const ScanParams &p, cudaStream_t s) {
    if (p.K <= 8) return scan_go<TT, DT, 2, 4, VEC>(p, s);
    if (p.K <= 16) return scan_go<TT, DT, 4, 4, VEC>(p, s);
    if (p.K <= 32) return scan_go<TT, DT, 8, 4, VEC>(p, s);
    if (p.K <= 64) return scan_go<TT, DT, 8, 8, VEC>(p, s);
    return scan_go<TT, DT, 8, 16, VEC>(p, s);
}
template <typename TT, typename DT> cudaError_t scan_vec(const ScanParams &p, bool vec, cudaStream_t s) {
    return vec ? scan_states<TT, DT, true>(p, s) : scan_states<TT, DT, false>(p, s);
}

}  // namespace gdr
