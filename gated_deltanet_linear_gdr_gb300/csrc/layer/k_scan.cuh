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

#include "scan_device.cuh"

namespace gdr {

constexpr int kScanChunk = 16;
constexpr int kScanWarps = 4;  // a block's

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

// A warp's piece of shared memory, in bytes: two stages of raw chunks, then the chunk in float32.
template <typename TT, typename DT, int KT, int LK> struct ScanShared {
    static constexpr int W = 4 * (32 / LK), KP = KT * LK, N = kScanChunk;
    static constexpr bool wide = sizeof(TT) == 4;  // raw B and C are used as they are
    static constexpr int x = 0, z = x + N * W * (int)sizeof(TT), dt = z + N * W * (int)sizeof(TT), B = dt + N * W * (int)sizeof(DT),
                         C = B + N * KP * (int)sizeof(TT), stage = C + N * KP * (int)sizeof(TT);
    static constexpr int fd = 2 * stage, fx = fd + 4 * N * W, fy = fx + 4 * N * W, fB = fy + 4 * N * W,
                         fC = fB + (wide ? 0 : 4 * N * KP), bias = fC + (wide ? 0 : 4 * N * KP), D = bias + 4 * W,
                         bytes = D + 4 * W;
};

// READ: with outputs.  Without them states move only: into the slots, or (first != 0)
// each segment's own state, from zero, and the sum of its step sizes into the workspace.
template <typename TT, typename DT, int KT, int LK, bool VEC, bool READ>
__global__ void __launch_bounds__(32 * kScanWarps) k_scan(const __grid_constant__ ScanParams p, int tiles, unsigned units, int first) {
    using Sh = ScanShared<TT, DT, KT, LK>;
    constexpr int W = Sh::W, KP = Sh::KP, CH = 4, N = kScanChunk;
    extern __shared__ __align__(16) unsigned char shared[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned unit = blockIdx.x * kScanWarps + warp;
    if (unit >= units) return;
    const unsigned all = (unsigned)(p.nk * tiles), row = unit / all, tg = unit - row * all;
    const int g = (int)(tg / (unsigned)tiles), tile = (int)(tg - (unsigned)g * (unsigned)tiles);
    ScanUnit u;
    if (p.seg) {
        if (!scan_piece(p, row, tg == 0 && !first, lane, u)) return;
        if (first && u.last) return;  // no segment starts from its state
    } else if (!scan_row(p, (int)row, tg == 0 && lane == 0, u)) {
        return;
    }
    const int group = p.r * p.V, c0 = tile * W;  // channels of the key head's value heads, this warp's first
    const int width = min(W, group - c0);
    unsigned char *const sh = shared + warp * Sh::bytes;
    float *const fd = reinterpret_cast<float *>(sh + Sh::fd), *const fx = reinterpret_cast<float *>(sh + Sh::fx);
    float *const fy = reinterpret_cast<float *>(sh + Sh::fy);
    float *const fbias = reinterpret_cast<float *>(sh + Sh::bias), *const fD = reinterpret_cast<float *>(sh + Sh::D);

    // A channel of the group as (value head, channel).
    auto head = [&](int c, int &j) {
        const int h = c / p.V;
        j = c - h * p.V;
        return g * p.r + h;
    };

    // A lane's part in moving tokens: vectors of 8 channels (piece pc of tokens pt, pt + TPP, ...), or
    // one channel (sc of tokens ps, ps + TPS, ...) where rows are not such vectors.
    constexpr int PCS = W / 8, TPP = 32 / PCS, TPS = 32 / W;
    const int pc = lane % PCS, pt = lane / PCS, sc = lane % W, ps = lane / W;
    int mj = 0, mh = 0;
    const bool mon = (VEC ? pc * 8 : sc) < width;
    if (mon) mh = head(c0 + (VEC ? pc * 8 : sc), mj);

    if (u.slot < 0) {  // padding: zeros
        if (READ && mon) {
            TT *o = static_cast<TT *>(p.out) + u.t0 * p.o_ts + (long long)mh * p.o_hs + mj;
            if constexpr (VEC) {
                for (int t = pt; t < u.len; t += TPP)
#pragma unroll
                    for (int i = 0; i < 8 * (int)sizeof(TT) / 16; ++i)
                        reinterpret_cast<uint4 *>(o + (long long)t * p.o_ts)[i] = make_uint4(0, 0, 0, 0);
            } else {
                for (int t = ps; t < u.len; t += TPS) o[(long long)t * p.o_ts] = TT(0);
            }
        }
        return;
    }

    // ---- chunks on their way to shared memory
    const TT *const xp = static_cast<const TT *>(p.x) + u.t0 * p.x_ts + (long long)mh * p.x_hs + mj;
    const TT *const zp = READ && p.z ? static_cast<const TT *>(p.z) + u.t0 * p.z_ts + (long long)mh * p.z_hs + mj : nullptr;
    const DT *const dp = static_cast<const DT *>(p.dt) + u.t0 * p.dt_ts + (long long)mh * p.dt_hs + mj * p.dt_es;
    const TT *const bp = static_cast<const TT *>(p.B) + u.t0 * p.B_ts + (long long)g * p.B_hs;
    const TT *const cp = READ ? static_cast<const TT *>(p.C) + u.t0 * p.C_ts + (long long)g * p.C_hs : nullptr;

    auto rows = [&](auto *to, const auto *from, long long stride, int n, bool vec) {
        using T = std::remove_const_t<std::remove_pointer_t<decltype(from)>>;
        if (!mon) return;
        if constexpr (VEC) {
            if (vec) {
#pragma unroll
                for (int i = 0; i < (N + TPP - 1) / TPP; ++i) {
                    const int t = pt + i * TPP;
                    if (t < n)
#pragma unroll
                        for (int v = 0; v < 8; v += 16 / (int)sizeof(T))
                            cp_async16(to + t * W + pc * 8 + v, from + (long long)t * stride + v);
                }
            } else {  // one value for the head
                for (int t = pt; t < n; t += TPP) {
                    const T v = from[(long long)t * stride];
#pragma unroll
                    for (int i = 0; i < 8; ++i) to[t * W + pc * 8 + i] = v;
                }
            }
        } else if constexpr (sizeof(T) == 4) {
#pragma unroll 4
            for (int t = ps; t < n; t += TPS) cp_async4(to + t * W + sc, from + (long long)t * stride);
        } else {
            T v[N / TPS];
#pragma unroll
            for (int i = 0; i < N / TPS; ++i)
                if (ps + i * TPS < n) v[i] = from[(long long)(ps + i * TPS) * stride];
#pragma unroll
            for (int i = 0; i < N / TPS; ++i)
                if (ps + i * TPS < n) to[(ps + i * TPS) * W + sc] = v[i];
        }
    };
    const bool bc_vec = p.bc_vec && p.K == KP;
    auto states = [&](TT *to, const TT *from, long long stride, int n) {
        if (bc_vec) {
            constexpr int C = 16 / (int)sizeof(TT), VR = KP / C;
#pragma unroll
            for (int i = 0; i < (N * VR + 31) / 32; ++i) {
                const int t = (lane + 32 * i) / VR, v = (lane + 32 * i) % VR;
                if (t < n) cp_async16(to + t * KP + v * C, from + (long long)t * stride + v * C);
            }
        } else {
            for (int k = lane; k < p.K; k += 32) {
                if constexpr (sizeof(TT) == 4) {
#pragma unroll 4
                    for (int t = 0; t < n; ++t) cp_async4(to + t * KP + k, from + (long long)t * stride + k);
                } else {
                    TT v[N];
#pragma unroll
                    for (int t = 0; t < N; ++t)
                        if (t < n) v[t] = from[(long long)t * stride + k];
#pragma unroll
                    for (int t = 0; t < N; ++t)
                        if (t < n) to[t * KP + k] = v[t];
                }
            }
        }
    };
    auto fetch = [&](int base, int stage) {
        const int n = min(N, u.len - base);
        if (n > 0) {
            unsigned char *const to = sh + stage * Sh::stage;
            rows(reinterpret_cast<DT *>(to + Sh::dt), dp + (long long)base * p.dt_ts, p.dt_ts, n, p.dt_es != 0);
            rows(reinterpret_cast<TT *>(to + Sh::x), xp + (long long)base * p.x_ts, p.x_ts, n, true);
            states(reinterpret_cast<TT *>(to + Sh::B), bp + (long long)base * p.B_ts, p.B_ts, n);
            if (READ) {
                states(reinterpret_cast<TT *>(to + Sh::C), cp + (long long)base * p.C_ts, p.C_ts, n);
                if (zp) rows(reinterpret_cast<TT *>(to + Sh::z), zp + (long long)base * p.z_ts, p.z_ts, n, true);
            }
        }
        cp_async_commit();
    };
    for (int i = lane; i < 2 * Sh::stage / 16; i += 32) reinterpret_cast<uint4 *>(sh)[i] = make_uint4(0, 0, 0, 0);
    for (int i = lane; i < W; i += 32) {
        int j = 0, h = 0;
        const bool in = i < width;
        if (in) h = head(c0 + i, j);
        fbias[i] = in && p.bias ? p.bias[h * p.b_hs + j * p.b_vs] : 0.0f;
        fD[i] = in && p.D ? p.D[h * p.d_hs + j * p.d_vs] : 0.0f;
    }
    __syncwarp();
    fetch(0, 0);

    // ---- this lane's states and their rates, in pairs along K
    const int lk = lane % LK, cg = lane / LK;
    float2 S[CH][KT / 2], A[CH][KT / 2];
    long long st_at[CH];
    int chan[CH], chead[CH];
    bool on[CH];
#pragma unroll
    for (int e = 0; e < CH; ++e) {
        on[e] = cg * 4 + e < width;
        chan[e] = 0;
        chead[e] = on[e] ? head(c0 + cg * 4 + e, chan[e]) : 0;
        st_at[e] = (long long)u.slot * p.st_slot + (long long)chead[e] * p.st_head + chan[e];
    }
    // a segment's state in the workspace: [nv, K, V]
    auto segment = [&](int e, int k) {
        return p.ws + ((u.piece * p.nv + chead[e]) * p.K + k) * (long long)p.V + chan[e];
    };
#pragma unroll
    for (int i = 0; i < KT; ++i) {
        const int k = lk * KT + i;
        float v[CH], a[CH];
#pragma unroll
        for (int e = 0; e < CH; ++e) v[e] = a[e] = 0.0f;
        if (k < p.K) {
            if (first) {
            } else if (p.seg) {
#pragma unroll
                for (int e = 0; e < CH; ++e)
                    if (on[e]) v[e] = *segment(e, k);
            } else if constexpr (VEC) {
                if (on[0]) {
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
                }
            } else {
#pragma unroll
                for (int e = 0; e < CH; ++e)
                    if (on[e])
                        v[e] = p.st_bf16 ? to_f32(static_cast<const uint16_t *>(p.state)[st_at[e] + k * p.st_k])
                                         : static_cast<const float *>(p.state)[st_at[e] + k * p.st_k];
            }
            if (VEC && p.a_vec) {
                if (on[0]) {
                    Pack<float, 4> q;
                    q.load(p.A + chead[0] * p.a_hs + k * p.a_ks + chan[0]);
#pragma unroll
                    for (int e = 0; e < CH; ++e) a[e] = q.get(e);
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
            (i & 1 ? A[e][i / 2].y : A[e][i / 2].x) = rate<TT>(a[e]);
        }
    }
    // the states into their slot, or a segment's into the workspace
    auto put = [&]() {
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            const int k = lk * KT + i;
            if (k >= p.K) continue;
            float v[CH];
#pragma unroll
            for (int e = 0; e < CH; ++e) v[e] = i & 1 ? S[e][i / 2].y : S[e][i / 2].x;
            if (first) {
#pragma unroll
                for (int e = 0; e < CH; ++e)
                    if (on[e]) *segment(e, k) = v[e];
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

    float dsum[CH] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int base = 0, stage = 0; base < u.len; base += N, stage ^= 1) {
        const int n = min(N, u.len - base);
        fetch(base + N, stage ^ 1);
        cp_async_wait<1>();
        __syncwarp();
        unsigned char *const raw = sh + stage * Sh::stage;
        TT *const rx = reinterpret_cast<TT *>(raw + Sh::x);
        const TT *const rz = reinterpret_cast<const TT *>(raw + Sh::z);
        const DT *const rd = reinterpret_cast<const DT *>(raw + Sh::dt);
        // ---- d and d x, B and C in float32
#pragma unroll
        for (int i = 0; i < (N * PCS + 31) / 32; ++i) {
            const int t = pt + i * TPP, at = t * W + pc * 8;
            if (N * PCS % 32 && t >= N) continue;
#pragma unroll
            for (int v = 0; v < 8; v += 4) {
                Pack<DT, 4> dq;
                Pack<TT, 4> xq;
                dq.load(rd + at + v);
                xq.load(rx + at + v);
                const float4 b = *reinterpret_cast<const float4 *>(fbias + pc * 8 + v);
                float d[4] = {dq.get(0) + b.x, dq.get(1) + b.y, dq.get(2) + b.z, dq.get(3) + b.w}, x[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (p.softplus) d[j] = softplus<TT>(d[j]);
                    x[j] = d[j] * xq.get(j);
                }
                *reinterpret_cast<float4 *>(fd + at + v) = make_float4(d[0], d[1], d[2], d[3]);
                *reinterpret_cast<float4 *>(fx + at + v) = make_float4(x[0], x[1], x[2], x[3]);
            }
        }
        const float *fB = reinterpret_cast<const float *>(raw + Sh::B), *fC = reinterpret_cast<const float *>(raw + Sh::C);
        if constexpr (!Sh::wide) {
            float *const tB = reinterpret_cast<float *>(sh + Sh::fB), *const tC = reinterpret_cast<float *>(sh + Sh::fC);
#pragma unroll
            for (int i = 0; i < (N * KP / 4 + 31) / 32; ++i) {
                const int at = 4 * (lane + 32 * i);
                Pack<TT, 4> q;
                q.load(reinterpret_cast<const TT *>(raw + Sh::B) + at);
                *reinterpret_cast<float4 *>(tB + at) = make_float4(q.get(0), q.get(1), q.get(2), q.get(3));
                if (READ) {
                    q.load(reinterpret_cast<const TT *>(raw + Sh::C) + at);
                    *reinterpret_cast<float4 *>(tC + at) = make_float4(q.get(0), q.get(1), q.get(2), q.get(3));
                }
            }
            fB = tB;
            fC = tC;
        }
        __syncwarp();
        // ---- the tokens, in two parts where the slot's state lies between them
        struct Operands {
            float4 d, x;
            float2 B[KT / 2], C[KT / 2];
        };
        auto operands = [&](int t, Operands &o) {
            o.d = *reinterpret_cast<const float4 *>(fd + t * W + cg * 4);
            o.x = *reinterpret_cast<const float4 *>(fx + t * W + cg * 4);
#pragma unroll
            for (int i = 0; i < KT / 2; i += 2) {
                const float4 b = *reinterpret_cast<const float4 *>(fB + t * KP + lk * KT + 2 * i);
                o.B[i] = make_float2(b.x, b.y);
                o.B[i + 1] = make_float2(b.z, b.w);
                if (READ) {
                    const float4 c = *reinterpret_cast<const float4 *>(fC + t * KP + lk * KT + 2 * i);
                    o.C[i] = make_float2(c.x, c.y);
                    o.C[i + 1] = make_float2(c.z, c.w);
                }
            }
        };
        const int cut = u.kept - base;
        const bool inside = !first && cut > 0 && cut <= n;
        Operands now;
        operands(0, now);
        int t = 0;
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
            const int end = part == 0 && inside ? cut : n;
#pragma unroll 2
            for (; t < end; ++t) {
                Operands next;
                operands(t + 1 < N ? t + 1 : t, next);
                const float d[CH] = {now.d.x, now.d.y, now.d.z, now.d.w}, x[CH] = {now.x.x, now.x.y, now.x.z, now.x.w};
                float y[CH];
#pragma unroll
                for (int e = 0; e < CH; ++e) {
#pragma unroll
                    for (int i = 0; i < KT / 2; ++i) {
                        const float2 a = __fmul2_rn(make_float2(d[e], d[e]), A[e][i]);
                        const float2 in = __fmul2_rn(make_float2(x[e], x[e]), now.B[i]);
                        S[e][i].x = fmaf(decay<TT>(a.x), S[e][i].x, in.x);
                        S[e][i].y = fmaf(decay<TT>(a.y), S[e][i].y, in.y);
                        if (READ) {
                            y[e] = i == 0 ? now.C[i].x * S[e][i].x : fmaf(now.C[i].x, S[e][i].x, y[e]);
                            y[e] = fmaf(now.C[i].y, S[e][i].y, y[e]);
                        }
                    }
                    if (!READ) dsum[e] += d[e];
                }
                if (READ) {
                    const float v = scan_readout<LK>(y, lk);
                    if (LK == 4 || lk < 4) fy[t * W + cg * 4 + (lk & 3)] = v;
                }
                now = next;
            }
            if (part == 0 && inside) put();
        }
        __syncwarp();
        // ---- its outputs
        if constexpr (READ) {
#pragma unroll
            for (int i = 0; i < (N * PCS + 31) / 32; ++i) {
                const int t = pt + i * TPP, at = t * W + pc * 8;
                if (t >= n) continue;
                constexpr int C = 16 / (int)sizeof(TT);
#pragma unroll
                for (int v = 0; v < 8; v += C) {
                    Pack<TT, C> x, z, o;
                    x.load(rx + at + v);
                    if (zp) z.load(rz + at + v);
#pragma unroll
                    for (int j = 0; j < C; ++j) {
                        float y = fmaf(fD[pc * 8 + v + j], x.get(j), fy[at + v + j]);
                        if (zp) y *= silu(z.get(j));
                        o.set(j, y);
                    }
                    if constexpr (VEC) {
                        if (mon) o.store(static_cast<TT *>(p.out) + (u.t0 + base + t) * p.o_ts + (long long)mh * p.o_hs + mj + v);
                    } else {
                        o.store(rx + at + v);
                    }
                }
            }
            if constexpr (!VEC) {
                __syncwarp();
                if (mon) {
                    TT *const to = static_cast<TT *>(p.out) + (u.t0 + base) * p.o_ts + (long long)mh * p.o_hs + mj;
#pragma unroll 4
                    for (int t = ps; t < n; t += TPS) to[(long long)t * p.o_ts] = rx[t * W + sc];
                }
            }
        }
        __syncwarp();
    }
    if (first) {
        put();
        if (lk == 0) {
            float *sum = p.ws + scan_pieces(p.T, p.seg, p.batch) * p.nv * p.K * p.V + u.piece * p.nv * p.V;
#pragma unroll
            for (int e = 0; e < CH; ++e)
                if (on[e]) sum[(long long)chead[e] * p.V + chan[e]] = dsum[e];
        }
    }
}

template <typename TT, typename DT, int KT, int LK, bool VEC> cudaError_t scan_go(const ScanParams &p, cudaStream_t s) {
    using Sh = ScanShared<TT, DT, KT, LK>;
    constexpr int bytes = kScanWarps * Sh::bytes;
    static_assert(bytes <= 227 << 10, "a block's shared memory");
    static LaunchCache cache;
    LaunchInfo info;
    cudaError_t e = launch_info(cache, &info, [](LaunchInfo &) {
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
        k_scan<TT, DT, KT, LK, VEC, false><<<blocks, 32 * kScanWarps, bytes, s>>>(p, (int)tiles, (unsigned)units, 1);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
        if ((e = launch_scan_join(p, s)) != cudaSuccess) return e;
    }
    if (p.out) k_scan<TT, DT, KT, LK, VEC, true><<<blocks, 32 * kScanWarps, bytes, s>>>(p, (int)tiles, (unsigned)units, 0);
    else k_scan<TT, DT, KT, LK, VEC, false><<<blocks, 32 * kScanWarps, bytes, s>>>(p, (int)tiles, (unsigned)units, 0);
    return cudaGetLastError();
}

// States a lane and lanes a channel, by K.
template <typename TT, typename DT, bool VEC> cudaError_t scan_states(const ScanParams &p, cudaStream_t s) {
    if (p.K <= 16) return scan_go<TT, DT, 4, 4, VEC>(p, s);
    if (p.K <= 32) return scan_go<TT, DT, 8, 4, VEC>(p, s);
    if (p.K <= 64) return scan_go<TT, DT, 8, 8, VEC>(p, s);
    return scan_go<TT, DT, 8, 16, VEC>(p, s);
}
template <typename TT, typename DT> cudaError_t scan_vec(const ScanParams &p, bool vec, cudaStream_t s) {
    return vec ? scan_states<TT, DT, true>(p, s) : scan_states<TT, DT, false>(p, s);
}

}  // namespace gdr
