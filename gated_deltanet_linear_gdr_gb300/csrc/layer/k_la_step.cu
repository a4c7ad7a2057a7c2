// Decayed linear attention, recurrent form:
//
//     S <- lambda S + k v^T ;  o = scale S^T q     (per token, in float32)
//
// One CTA owns a (row, value head, tile of up to 128 columns) and keeps it in
// registers for all of the row's tokens: thread (rl, cg) holds state rows
// R rl .. R rl + R - 1 of 8 columns.  A state row's 16-byte vectors lie in
// neighbouring threads, so a warp moves whole 256-byte (bfloat16) or 512-byte
// (float32) runs; a token's q and k values of a thread are one vector.  The
// readout adds up over rl: per-thread partials go through shared memory, in a
// fixed order, so that results repeat bit for bit.
//
// A single token moves the state once in each direction and does 3 operations
// on an element: HBM bound.  What counts is bytes in flight: a thread asks for
// all of its state before anything else, and R is 8 rows of bfloat16 or 4 of
// float32 (32 registers of state), so that a multiprocessor holds three to four
// 32 or 64 KiB blocks at a time.  256 rows x 32 heads of 128 x 128, bfloat16: 85
// us, 91% of the measured copy rate.
#include "../gdr_device.cuh"
#include "layer_internal.h"

#include <type_traits>

namespace gdr {
namespace {

constexpr int kTok = 4;  // tokens whose partial outputs are joined behind one barrier

// N consecutive token values (N * sizeof(TT) is 8 bytes or a multiple of 16).
template <int N, typename TT>
__device__ __forceinline__ void loadn(const TT *p, bool vec, float (&x)[N]) {
    if (vec) {
        constexpr int C = N * (int)sizeof(TT) >= 16 ? 16 / (int)sizeof(TT) : N;
#pragma unroll
        for (int i = 0; i < N; i += C) {
            Pack<TT, C> w;
            w.load(p + i);
#pragma unroll
            for (int j = 0; j < C; ++j) x[i + j] = w.get(j);
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = to_f32(p[i]);
    }
}

// The same, kept in the tokens' own type: half the registers for bfloat16.
template <typename TT, int N> struct TokVec {
    static constexpr int C = N * (int)sizeof(TT) >= 16 ? 16 / (int)sizeof(TT) : N;
    Pack<TT, C> w[N / C];
    __device__ __forceinline__ void load(const TT *p, bool vec) {
#pragma unroll
        for (int i = 0; i < N / C; ++i) {
            if (vec) {
                w[i].load(p + i * C);
            } else {
#pragma unroll
                for (int j = 0; j < C; ++j) w[i].u.e[j] = p[i * C + j];
            }
        }
    }
    __device__ __forceinline__ float get(int i) const { return w[i / C].get(i % C); }
};

// In float32 from the start.
template <typename TT, int N> struct TokF32 {
    float x[N];
    __device__ __forceinline__ void load(const TT *p, bool vec) { loadn<N>(p, vec, x); }
    __device__ __forceinline__ float get(int i) const { return x[i]; }
};

// What every thread of a CTA knows about its unit.  false: nothing to do (the
// output of a skipped row has been cleared).
struct StepUnit {
    int h, tile, t0, len, slot, col0, W;
    float lam;
};
template <typename TT> __device__ __forceinline__ bool step_unit(const LaParams &p, StepUnit &u) {
    const int tid = threadIdx.x, nt = blockDim.x;
    const unsigned pos = blockIdx.x;
    u.tile = (int)(pos % (unsigned)p.tiles);
    const unsigned bh = pos / (unsigned)p.tiles;
    const int b = (int)(bh / (unsigned)p.nv);
    u.h = (int)(bh - (unsigned)b * (unsigned)p.nv);
    const int t0 = p.offsets[b], t1 = p.offsets[b + 1];
    const float d = p.decay[(long long)u.h * p.decay_s];
    u.slot = p.slot_idx[b];
    const bool leader = tid == 0 && u.h == 0 && u.tile == 0;
    u.col0 = u.tile * 128;
    u.W = min(128, p.V - u.col0);
    u.t0 = t0;
    u.len = t1 - t0;
    if (t0 < 0 || t1 < t0 || t1 > p.T) {
        if (leader) flag(p.status, GDR_STATUS_BAD_OFFSETS);
        return false;
    }
    if (t1 == t0) return false;
    const bool bad_decay = !(p.decay_is_log ? d <= 0.0f : (d >= 0.0f && d <= 1.0f));
    const bool too_long = p.max_len > 0 && t1 - t0 > p.max_len;
    if (u.slot < 0 || u.slot >= p.max_slots || bad_decay || too_long) {
        if (too_long) {
            if (leader) flag(p.status, GDR_STATUS_ROW_TOO_LONG);
        } else if (u.slot < -1 || u.slot >= p.max_slots) {
            if (leader) flag(p.status, GDR_STATUS_BAD_SLOT);
        } else if (u.slot >= 0 && tid == 0) {
            flag(p.status, GDR_STATUS_BAD_DECAY);
        }
        TT *out = static_cast<TT *>(p.out) + (long long)t0 * p.o_ts + (long long)u.h * p.o_hs + u.col0;
        clear_rows(out, p.o_ts, u.len, u.W, p.tok_vec, tid, nt);
        return false;
    }
    u.lam = p.decay_is_log ? expf(d) : d;
    return true;
}

// Single tokens.
template <typename ST, typename TT, int R>
__global__ void __launch_bounds__(2048 / R, sizeof(ST) == 2 ? 4 : 2) k_la_one(const __grid_constant__ LaParams p, int cg_n) {
    extern __shared__ float part[];  // [K / R, or half of it][8 * cg_n]
    constexpr int C = 16 / (int)sizeof(ST), NC = 8 / C;  // a thread's columns: NC vectors of C
    StepUnit u;
    if (!step_unit<TT>(p, u)) return;
    const int tid = threadIdx.x, rl_n = p.K / R, cg = tid % cg_n, rl = tid / cg_n, row_w = 8 * cg_n;
    int col[NC];
    bool on[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        col[i] = (i * cg_n + cg) * C;
        on[i] = rl < rl_n && col[i] < u.W;
    }
    ST *sp = static_cast<ST *>(p.state) + (long long)u.slot * p.st_slot + (long long)u.h * p.st_head +
             (long long)(rl * R) * p.st_k + u.col0;
    Pack<ST, C> s[R][NC];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < NC; ++i)
            if (on[i]) s[r][i].load(sp + r * p.st_k + col[i]);
    const int hk = u.h / p.r;
    float o[NC][C];
    std::conditional_t<sizeof(ST) == 2, TokVec<TT, R>, TokF32<TT, R>> q, k;
    if (rl < rl_n) {
        q.load(static_cast<const TT *>(p.q) + (long long)u.t0 * p.q_ts + (long long)hk * p.q_hs + rl * R, p.tok_vec);
        k.load(static_cast<const TT *>(p.k) + (long long)u.t0 * p.k_ts + (long long)hk * p.k_hs + rl * R, p.tok_vec);
        const TT *vp = static_cast<const TT *>(p.v) + (long long)u.t0 * p.v_ts + (long long)u.h * p.v_hs + u.col0;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            if (!on[i]) continue;
            float v[C];
            loadn<C>(vp + col[i], p.tok_vec, v);
#pragma unroll
            for (int j = 0; j < C; ++j) o[i][j] = 0.0f;
#pragma unroll
            for (int r = 0; r < R; ++r) {
#pragma unroll
                for (int j = 0; j < C; ++j) {
                    const float x = fmaf(k.get(r), v[j], u.lam * s[r][i].get(j));
                    o[i][j] = fmaf(q.get(r), x, o[i][j]);
                    s[r][i].set(j, x);
                }
                s[r][i].store(sp + r * p.st_k + col[i]);
            }
        }
    }
    // 16 threads across, the widest tile: the two row groups of a warp add up first
    const bool pair = cg_n == 16;
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < C; ++j) {
            if (pair) o[i][j] += __shfl_xor_sync(kFull, o[i][j], 16);
        }
    if (rl < rl_n && (!pair || (rl & 1) == 0))
#pragma unroll
        for (int i = 0; i < NC; ++i)
            if (on[i]) {
                float *to = part + (pair ? rl >> 1 : rl) * row_w + col[i];
#pragma unroll
                for (int j = 0; j < C; j += 4) *reinterpret_cast<float4 *>(to + j) = make_float4(o[i][j], o[i][j + 1], o[i][j + 2], o[i][j + 3]);
            }
    __syncthreads();
    TT *out = static_cast<TT *>(p.out) + (long long)u.t0 * p.o_ts + (long long)u.h * p.o_hs + u.col0;
    const int n = pair ? rl_n / 2 : rl_n;
    for (int c = tid; c < u.W; c += blockDim.x) {
        float x = 0.0f;
        for (int r = 0; r < n; ++r) x += part[r * row_w + c];
        out[c] = from_f32<TT>(x * p.scale);
    }
}

// Rows of any length; the next token's operands are asked for before the
// current one's results are handed over.  (R = 4, twice the warps at half the
// registers, measured 101 us against 85 for 64 rows of 5 tokens.)
template <typename ST, typename TT, int R>
__global__ void __launch_bounds__(2048 / R, 2) k_la_rows(const __grid_constant__ LaParams p, int cg_n) {
    extern __shared__ float part[];  // [kTok][K / R, or half of it][8 * cg_n]
    constexpr int C = 16 / (int)sizeof(ST), NC = 8 / C;  // a thread's columns: NC vectors of C
    StepUnit u;
    if (!step_unit<TT>(p, u)) return;
    const int tid = threadIdx.x, nt = blockDim.x, W = u.W;
    const int rl_n = p.K / R, cg = tid % cg_n, rl = tid / cg_n, row_w = 8 * cg_n;
    const bool mine = rl < rl_n, pair = cg_n == 16;
    const int n_part = pair ? rl_n / 2 : rl_n;
    int col[NC];
    bool on[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        col[i] = (i * cg_n + cg) * C;
        on[i] = mine && col[i] < W;
    }
    ST *sp = static_cast<ST *>(p.state) + (long long)u.slot * p.st_slot + (long long)u.h * p.st_head +
             (long long)(rl * R) * p.st_k + u.col0;
    Pack<ST, C> raw[R][NC];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < NC; ++i)
            if (on[i]) raw[r][i].load(sp + r * p.st_k + col[i]);

    const int hk = u.h / p.r;
    const TT *qp = static_cast<const TT *>(p.q) + (long long)u.t0 * p.q_ts + (long long)hk * p.q_hs + rl * R;
    const TT *kp = static_cast<const TT *>(p.k) + (long long)u.t0 * p.k_ts + (long long)hk * p.k_hs + rl * R;
    const TT *vp = static_cast<const TT *>(p.v) + (long long)u.t0 * p.v_ts + (long long)u.h * p.v_hs + u.col0;
    TT *out = static_cast<TT *>(p.out) + (long long)u.t0 * p.o_ts + (long long)u.h * p.o_hs + u.col0;
    float q[R], k[R], v[NC][C];
    auto fetch = [&]() {
        if (!mine) return;
        loadn<R>(qp, p.tok_vec, q);
        loadn<R>(kp, p.tok_vec, k);
#pragma unroll
        for (int i = 0; i < NC; ++i)
            if (on[i]) loadn<C>(vp + col[i], p.tok_vec, v[i]);
        qp += p.q_ts;
        kp += p.k_ts;
        vp += p.v_ts;
    };
    fetch();
    float s[R][NC][C];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < C; ++j) s[r][i][j] = on[i] ? raw[r][i].get(j) : 0.0f;

    const unsigned len = (unsigned)u.len;
    for (unsigned base = 0; base < len; base += kTok) {
        const int n = (int)min((unsigned)kTok, len - base);
        for (int t = 0; t < n; ++t) {
            float o[NC][C];
#pragma unroll
            for (int i = 0; i < NC; ++i)
#pragma unroll
                for (int j = 0; j < C; ++j) {
                    float acc = 0.0f;
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        s[r][i][j] = fmaf(k[r], v[i][j], u.lam * s[r][i][j]);
                        acc = fmaf(q[r], s[r][i][j], acc);
                    }
                    o[i][j] = acc;
                }
            if (base + t + 1 < len) fetch();
            if (pair) {
#pragma unroll
                for (int i = 0; i < NC; ++i)
#pragma unroll
                    for (int j = 0; j < C; ++j) o[i][j] += __shfl_xor_sync(kFull, o[i][j], 16);
            }
            if (mine && (!pair || (rl & 1) == 0))
#pragma unroll
                for (int i = 0; i < NC; ++i)
                    if (on[i]) {
                        float *to = part + (t * n_part + (pair ? rl >> 1 : rl)) * row_w + col[i];
#pragma unroll
                        for (int j = 0; j < C; j += 4)
                            *reinterpret_cast<float4 *>(to + j) = make_float4(o[i][j], o[i][j + 1], o[i][j + 2], o[i][j + 3]);
                    }
        }
        __syncthreads();
        for (int i = tid; i < n * W; i += nt) {
            const int t = i / W, c = i - t * W;
            float o = 0.0f;
            for (int r = 0; r < n_part; ++r) o += part[(t * n_part + r) * row_w + c];
            out[(long long)(base + t) * p.o_ts + c] = from_f32<TT>(o * p.scale);
        }
        __syncthreads();
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int i = 0; i < NC; ++i)
            if (on[i]) {
#pragma unroll
                for (int j = 0; j < C; ++j) raw[r][i].set(j, s[r][i][j]);
                raw[r][i].store(sp + r * p.st_k + col[i]);
            }
}

template <typename ST> constexpr int kOneRows = sizeof(ST) == 2 ? 8 : 4;

template <typename ST, typename TT> cudaError_t go(const LaParams &p, cudaStream_t s) {
    const int W = p.V < 128 ? p.V : 128, cg_n = W / 8;
    const unsigned blocks = (unsigned)p.batch * (unsigned)p.nv * (unsigned)p.tiles;
    if (p.max_len == 1) {
        constexpr int R = kOneRows<ST>;
        const int rl_n = p.K / R;
        k_la_one<ST, TT, R>
            <<<blocks, (cg_n * rl_n + 31) / 32 * 32, sizeof(float) * (cg_n == 16 ? rl_n / 2 : rl_n) * W, s>>>(p, cg_n);
    } else {
        const int rl_n = p.K / 8, n_part = cg_n == 16 ? rl_n / 2 : rl_n;
        k_la_rows<ST, TT, 8><<<blocks, (cg_n * rl_n + 31) / 32 * 32, sizeof(float) * kTok * n_part * W, s>>>(p, cg_n);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_la_step(const LaParams &p, bool tok_bf16, bool state_bf16, cudaStream_t s) {
    if (tok_bf16) return state_bf16 ? go<uint16_t, uint16_t>(p, s) : go<float, uint16_t>(p, s);
    return state_bf16 ? go<uint16_t, float>(p, s) : go<float, float>(p, s);
}

}  // namespace gdr
