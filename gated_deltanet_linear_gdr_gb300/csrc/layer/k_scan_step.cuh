// Selective scan of single tokens and short rows (drafts): every state goes in and
// out once, with a handful of operations on it a token: HBM bound, or bound by the
// steps that follow one another.  A block is 128 channels of some rows.
// Its NW warps share the states, KT each, four channels a lane, so that a warp
// moves whole runs of 512 bytes.  What belongs to the channels (their places, the
// rates, the bias) is worked out once for all the block's rows; the next row's
// states are on their way while one is worked on.  The partial readouts meet in
// shared memory, and one thread finishes each channel.
//
// Measured, bfloat16 tokens, float32 pool, 16 states: 256 single tokens x 4096 channels 33 us a call with pools in
// turn (4.2 TB/s of states and tokens, 62% of the copy rate), 28 on the device alone, where half of the states come from L2;
// waits for memory are the largest stall.  With channels but not B and C in vectors (27 states) 85 us, against 225 with
// everything one by one.
#pragma once

#include "scan_device.cuh"

namespace gdr {
namespace {

constexpr int kStepTile = 128;  // a block's channels
constexpr int kStepRows = 32;   // a block's rows at most

// Four neighbouring values as they came, one vector (VEC) or one by one, taken apart only where
// they are used: a load that is on its way for long must not be waited for by what unpacks it.
template <typename T, bool VEC> struct Four;
template <> struct Four<uint16_t, true> {
    uint2 v;
    __device__ __forceinline__ void load(const uint16_t *p) { v = *reinterpret_cast<const uint2 *>(p); }
    __device__ __forceinline__ void load_first(const uint16_t *p) { v.x = *p; }
    __device__ __forceinline__ float get(int i) const {
        const unsigned w = i < 2 ? v.x : v.y;
        return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
    }
};
template <> struct Four<float, true> {
    float4 v;
    __device__ __forceinline__ void load(const float *p) { v = *reinterpret_cast<const float4 *>(p); }
    __device__ __forceinline__ void load_first(const float *p) { v.x = *p; }
    __device__ __forceinline__ float get(int i) const { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
};
template <typename T> struct Four<T, false> {
    T e[4];
    __device__ __forceinline__ float get(int i) const { return to_f32(e[i]); }
};
template <typename T, bool VEC>
__device__ __forceinline__ void gather4(const T *base, const long long (&at)[4], const bool (&on)[4], Four<T, VEC> &v) {
    if constexpr (VEC) {
        if (on[0]) v.load(base + at[0]);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (on[e]) v.e[e] = base[at[e]];
    }
}
template <bool VEC, typename T>
__device__ __forceinline__ void scatter4(T *base, const long long (&at)[4], const bool (&on)[4], const float (&v)[4]) {
    if constexpr (VEC) {
        if (on[0]) {
            Pack<T, 4> q;
#pragma unroll
            for (int e = 0; e < 4; ++e) q.set(e, v[e]);
            q.store(base + at[0]);
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (on[e]) base[at[e]] = from_f32<T>(v[e]);
    }
}

// A row as the block's setup leaves it: where its token's values and its states begin.
template <typename TT, typename DT, typename ST> struct StepRow {
    ST *state;
    const DT *dt;
    const TT *x, *z, *B, *C;
    TT *out;
    int len;   // tokens, 0: nothing to do
    int kept;  // tokens after which the states are kept, 0: they are not; -1: zeros only
};

// VEC: four channels are a vector everywhere (dt: that, or one value a head).  BC: so are four states of B
// and C, and K is a multiple of KT.  ONE: rows of one token.  PAIRS: up to 8 states, read out by groups of two.  Sixteen warps a multiprocessor, 128 registers each.
template <typename TT, typename DT, typename ST, int KT, int NW, bool VEC, bool BC, bool ONE, bool PAIRS>
__global__ void __launch_bounds__(32 * NW, 16 / NW)
    k_scan_step(const __grid_constant__ ScanParams p, int tiles, int rows) {
    __shared__ __align__(16) float part[2][NW][kStepTile];
    __shared__ StepRow<TT, DT, ST> info[kStepRows];
    constexpr bool AHEAD = BC && ONE && KT <= 4;  // there are registers for two rows' states
    constexpr bool EXACT = sizeof(TT) == 4 && sizeof(ST) == 2;
    constexpr int KV = KT / 4, G = PAIRS ? 2 : 4, Q = PAIRS || (sizeof(TT) == 4 && NW <= 8) ? 1 : 2;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned all = (unsigned)(p.nk * tiles), block = blockIdx.x / all, tg = blockIdx.x - block * all;
    const int g = (int)(tg / (unsigned)tiles), tile = (int)(tg - (unsigned)g * (unsigned)tiles);
    const int c0 = tile * kStepTile, width = min(kStepTile, p.r * p.V - c0);
    const int b0 = (int)block * rows, nrows = min(rows, p.batch - b0);
    if (tid < nrows) {
        ScanUnit u;
        StepRow<TT, DT, ST> r;
        r.len = 0;
        if (scan_row(p, b0 + tid, tg == 0, u)) {
            r.len = u.len;
            r.kept = u.slot < 0 ? -1 : u.kept;
            r.state = static_cast<ST *>(p.state) + (u.slot < 0 ? 0 : u.slot * p.st_slot);
            r.dt = static_cast<const DT *>(p.dt) + u.t0 * p.dt_ts;
            r.x = static_cast<const TT *>(p.x) + u.t0 * p.x_ts;
            r.z = static_cast<const TT *>(p.z) + (p.z ? u.t0 * p.z_ts : 0);
            r.B = static_cast<const TT *>(p.B) + u.t0 * p.B_ts + (long long)g * p.B_hs;
            r.C = static_cast<const TT *>(p.C) + (p.C ? u.t0 * p.C_ts + (long long)g * p.C_hs : 0);
            r.out = static_cast<TT *>(p.out) + (p.out ? u.t0 * p.o_ts : 0);
        }
        info[tid] = r;
    }
    // this lane's four channels, and the one this thread finishes
    const int have = min(KT, p.K - warp * KT);  // states that there are, 0 or less: none
    const long long k0 = (long long)warp * KT;
    long long st_at[4], x_at[4], d_at[4];
    bool on[4];
    float A[KT][4], bias[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        on[e] = lane * 4 + e < width;
        const int c = on[e] ? c0 + lane * 4 + e : 0, q = c / p.V, h = g * p.r + q, j = c - q * p.V;
        st_at[e] = k0 * p.st_k + h * p.st_head + j;
        x_at[e] = h * p.x_hs + j;
        d_at[e] = h * p.dt_hs + j * p.dt_es;
        bias[e] = p.bias && on[e] ? p.bias[h * p.b_hs + j * p.b_vs] : 0.0f;
        const float *const ap = p.A + k0 * p.a_ks + h * p.a_hs + j * p.a_vs;
#pragma unroll
        for (int i = 0; i < KT; ++i) A[i][e] = i < have && on[e] ? rate<TT>(ap[i * p.a_ks]) : 0.0f;
    }
    const bool mon = tid < width && p.out, gate = mon && p.z;
    const int mq = mon ? (c0 + tid) / p.V : 0, mh = g * p.r + mq, mj = mon ? c0 + tid - mq * p.V : 0;
    const long long mx_at = mh * p.x_hs + mj, mz_at = mh * p.z_hs + mj, mo_at = mh * p.o_hs + mj;
    const float D = mon && p.D ? p.D[mh * p.d_hs + mj * p.d_vs] : 0.0f;
    __syncthreads();

    struct Token {
        Four<DT, VEC> d;
        Four<TT, VEC> x;
        Four<TT, BC> B[KV], C[KV];
        TT mx, mz;
    };
    struct Row {
        Four<ST, VEC> S[KT];
        Token t;  // its first token
    };
    auto ask_token = [&](const StepRow<TT, DT, ST> &w, int t, Token &v) {
        if (have > 0) {
            if constexpr (VEC) {
                if (on[0]) {
                    const DT *const d = w.dt + t * p.dt_ts + d_at[0];
                    if (p.dt_es) v.d.load(d);
                    else v.d.load_first(d);  // the head's only one
                }
            } else {
                gather4(w.dt + t * p.dt_ts, d_at, on, v.d);
            }
            gather4(w.x + t * p.x_ts, x_at, on, v.x);
            const TT *const b = w.B + t * p.B_ts + k0, *const c = w.C + t * p.C_ts + k0;
#pragma unroll
            for (int i = 0; i < KV; ++i) {
                if constexpr (BC) {
                    v.B[i].load(b + 4 * i);
                    if (p.out) v.C[i].load(c + 4 * i);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (4 * i + k < have) {
                            v.B[i].e[k] = b[4 * i + k];
                            if (p.out) v.C[i].e[k] = c[4 * i + k];
                        }
                }
            }
        }
        if (mon) v.mx = w.x[t * p.x_ts + mx_at];
        if (gate) v.mz = w.z[t * p.z_ts + mz_at];
    };
    auto ask = [&](int r, Row &v) {
        const StepRow<TT, DT, ST> &w = info[r];
        if (w.len == 0 || w.kept < 0) return;
#pragma unroll
        for (int i = 0; i < KT; ++i)
            if (i < have) gather4(w.state + i * p.st_k, st_at, on, v.S[i]);
        ask_token(w, 0, v.t);
    };
    int exchanges = 0;
    auto turn = [&](int r, const Row &v) {
        const StepRow<TT, DT, ST> &w = info[r];
        const int len = w.len;
        if (w.kept < 0) {
            if (mon)
                for (int t = 0; t < len; ++t) w.out[t * p.o_ts + mo_at] = TT(0);
            return;
        }
        float S[KT][4];
#pragma unroll
        for (int i = 0; i < KT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) S[i][e] = v.S[i].get(e);
        Token now = v.t;
#pragma unroll 1
        for (int t = 0; t < len; ++t) {
            Token next;
            if (!ONE && t + 1 < len) ask_token(w, t + 1, next);
            float y[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            [[maybe_unused]] float first[4];  // the first of a warp's two groups
            if (have > 0) {
                float d[4], in[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    d[e] = (VEC && !p.dt_es ? now.d.get(0) : now.d.get(e)) + bias[e];
                    if (p.softplus) d[e] = softplus<TT>(d[e]);
                    in[e] = __fmul_rn(d[e], now.x.get(e));
                }
#pragma unroll
                for (int i = 0; i < KT; ++i) {
                    if (!BC && i >= have) continue;
                    const float B = now.B[i / 4].get(i % 4), C = now.C[i / 4].get(i % 4);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        S[i][e] = advance<EXACT>(decay<TT>(__fmul_rn(d[e], A[i][e])), S[i][e], __fmul_rn(in[e], B));
                        if (G < KT && i == G) {
                            first[e] = y[e];
                            y[e] = 0.0f;
                        }
                        y[e] = fmaf(C, S[i][e], y[e]);  // of no meaning, and not used, where there are no outputs
                    }
                }
                if constexpr (G < KT) {
                    if (have > G) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) y[e] = first[e] + y[e];
                    }
                }
                if (t + 1 == w.kept) {
#pragma unroll
                    for (int i = 0; i < KT; ++i)
                        if (i < have) scatter4<VEC>(w.state + i * p.st_k, st_at, on, S[i]);
                }
            }
            if (p.out) {
                float (&q)[NW][kStepTile] = part[exchanges++ & 1];
                *reinterpret_cast<float4 *>(&q[warp][lane * 4]) = make_float4(y[0], y[1], y[2], y[3]);
                __syncthreads();
                if (mon) {
                    float o = 0.0f;
#pragma unroll
                    for (int i = 0; i < NW; i += Q) o += Q == 1 ? q[i][tid] : q[i][tid] + q[i + 1][tid];
                    o = fmaf(D, to_f32(now.mx), o);
                    if (gate) o *= silu(to_f32(now.mz));
                    w.out[t * p.o_ts + mo_at] = from_f32<TT>(o);
                }
            }
            if (ONE) break;
            now = next;
        }
    };
    if constexpr (AHEAD) {
        Row v[2];
        ask(0, v[0]);
        for (int r = 0; r < nrows; ++r) {
            if (r + 1 < nrows) ask(r + 1, v[1]);
            turn(r, v[0]);
            if (++r >= nrows) break;
            if (r + 1 < nrows) ask(r + 1, v[0]);
            turn(r, v[1]);
        }
    } else {
        Row v;
        for (int r = 0; r < nrows; ++r) {
            ask(r, v);
            turn(r, v);
        }
    }
}

template <typename TT, typename DT, typename ST, int KT, int NW, bool VEC, bool BC, bool ONE, bool PAIRS>
cudaError_t go(const ScanParams &p, cudaStream_t s) {
    const long long tiles = ((long long)p.r * p.V + kStepTile - 1) / kStepTile, heads = p.nk * tiles;
    // as many rows a block as leaves each multiprocessor its blocks once over
    const long long at_once = 152 * (16 / NW);
    long long rows = (p.batch * heads + at_once - 1) / at_once;
    if (rows > kStepRows) rows = kStepRows;
    const long long blocks = (p.batch + rows - 1) / rows * heads;
    if (blocks >= 1ll << 31) return cudaErrorInvalidConfiguration;
    k_scan_step<TT, DT, ST, KT, NW, VEC, BC, ONE, PAIRS><<<(unsigned)blocks, 32 * NW, 0, s>>>(p, (int)tiles, (int)rows);
    return cudaGetLastError();
}
template <typename TT, typename DT, typename ST, int KT, int NW, bool PAIRS = false>
cudaError_t step_form(const ScanParams &p, bool vec, cudaStream_t s) {
    if (!vec) return go<TT, DT, ST, KT, NW, false, false, false, PAIRS>(p, s);
    if (!p.bc_vec || p.K % KT != 0) return go<TT, DT, ST, KT, NW, true, false, false, PAIRS>(p, s);
    return p.max_len == 1 ? go<TT, DT, ST, KT, NW, true, true, true, PAIRS>(p, s) : go<TT, DT, ST, KT, NW, true, true, false, PAIRS>(p, s);
}
// States a warp has and warps, by K.  Four states a warp wherever they fit leave registers for the next row's.  Measured
// against four warps of 8, 16 and 32 states, 256 single tokens x 4096 channels, us: 32 states 59 / 78; x 2048 channels: 64 states
// 61 / 82, 128 states 118 / 371.
template <typename TT, typename DT, typename ST> cudaError_t step_states(const ScanParams &p, bool vec, cudaStream_t s) {
    if (p.K <= 8) return step_form<TT, DT, ST, 4, 4, true>(p, vec, s);
    if (p.K <= 16) return step_form<TT, DT, ST, 4, 4>(p, vec, s);
    if (p.K <= 32) return step_form<TT, DT, ST, 4, 8>(p, vec, s);
    if (p.K <= 64) return step_form<TT, DT, ST, 4, 16>(p, vec, s);
    return step_form<TT, DT, ST, 8, 16>(p, vec, s);
}
template <typename TT, typename DT> cudaError_t scan_step(const ScanParams &p, bool vec, cudaStream_t s) {
    return p.st_bf16 ? step_states<TT, DT, uint16_t>(p, vec, s) : step_states<TT, DT, float>(p, vec, s);
}

}  // namespace
}  // namespace gdr
