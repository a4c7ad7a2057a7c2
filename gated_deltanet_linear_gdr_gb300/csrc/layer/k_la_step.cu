// Decayed linear attention, recurrent form:
//
//     S <- lambda S + k v^T ;  o = scale S^T q     (per token, in float32)
//
// One CTA owns a (row, value head, tile of up to 128 columns) and keeps it in
// registers for all of the row's tokens: thread (rl, cg) holds state rows
// 8 rl .. 8 rl + 7 of 8 columns.  A state row's 16-byte vectors lie in
// neighbouring threads, so a warp moves whole 256-byte (bfloat16) or 512-byte
// (float32) runs; a token's q and k values of a thread are one vector of 8.
// The readout adds up over rl: per-thread partials go through shared memory,
// in a fixed order, so that results repeat bit for bit.
//
// A single token moves the state once in each direction and does 3
// operations on an element: HBM bound.
#include "../gdr_device.cuh"
#include "layer_internal.h"

namespace gdr {
namespace {

constexpr int kTok = 4;  // tokens whose partial outputs are joined behind one barrier

// 8 consecutive token values.
template <typename TT>
__device__ __forceinline__ void load8(const TT *p, bool vec, float (&x)[8]) {
    if (vec) {
        constexpr int C = 16 / (int)sizeof(TT);
#pragma unroll
        for (int i = 0; i < 8; i += C) {
            Pack<TT, C> w;
            w.load(p + i);
#pragma unroll
            for (int j = 0; j < C; ++j) x[i + j] = w.get(j);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = to_f32(p[i]);
    }
}

template <typename ST, typename TT, bool ONE>
__global__ void __launch_bounds__(256) k_la_step(const __grid_constant__ LaParams p, int cg_n) {
    extern __shared__ float part[];  // [ONE ? 1 : kTok][rl_n][8 * cg_n]
    constexpr int C = 16 / (int)sizeof(ST), NC = 8 / C;  // a thread's columns: NC vectors of C
    const int tid = threadIdx.x, nt = blockDim.x;
    const unsigned u = blockIdx.x;
    const int tile = (int)(u % (unsigned)p.tiles);
    const unsigned bh = u / (unsigned)p.tiles;
    const int b = (int)(bh / (unsigned)p.nv), h = (int)(bh - (unsigned)b * (unsigned)p.nv);
    const int t0 = p.offsets[b], t1 = p.offsets[b + 1], slot = p.slot_idx[b];
    const bool leader = tid == 0 && h == 0 && tile == 0;
    const int col0 = tile * 128, W = min(128, p.V - col0);
    if (t0 < 0 || t1 < t0 || t1 > p.T) {
        if (leader) flag(p.status, GDR_STATUS_BAD_OFFSETS);
        return;
    }
    if (t1 == t0) return;
    TT *out = static_cast<TT *>(p.out) + (long long)t0 * p.o_ts + (long long)h * p.o_hs + col0;
    const float d = p.decay[(long long)h * p.decay_s];
    const bool bad_decay = !(p.decay_is_log ? d <= 0.0f : (d >= 0.0f && d <= 1.0f));
    const bool too_long = p.max_len > 0 && t1 - t0 > p.max_len;
    if (slot < 0 || slot >= p.max_slots || bad_decay || too_long) {
        if (too_long) {
            if (leader) flag(p.status, GDR_STATUS_ROW_TOO_LONG);
        } else if (slot < -1 || slot >= p.max_slots) {
            if (leader) flag(p.status, GDR_STATUS_BAD_SLOT);
        } else if (slot >= 0 && tid == 0) {
            flag(p.status, GDR_STATUS_BAD_DECAY);
        }
        for (int i = tid; i < (t1 - t0) * W; i += nt) out[(long long)(i / W) * p.o_ts + i % W] = from_f32<TT>(0.0f);
        return;
    }
    const float lam = p.decay_is_log ? expf(d) : d;
    const int rl_n = p.K / 8, cg = tid % cg_n, rl = tid / cg_n;
    const int row_w = 8 * cg_n;  // columns of a partial row

    // the state: issued first
    bool on[NC];
    int col[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
        col[i] = (i * cg_n + cg) * C;
        on[i] = rl < rl_n && col[i] < W;
    }
    ST *sp = static_cast<ST *>(p.state) + (long long)slot * p.st_slot + (long long)h * p.st_head +
             (long long)(rl * 8) * p.st_k + col0;
    Pack<ST, C> raw[8][NC];
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
        for (int i = 0; i < NC; ++i)
            if (on[i]) raw[r][i].load(sp + r * p.st_k + col[i]);

    const int hk = h / p.r;
    const TT *qp = static_cast<const TT *>(p.q) + (long long)t0 * p.q_ts + (long long)hk * p.q_hs + rl * 8;
    const TT *kp = static_cast<const TT *>(p.k) + (long long)t0 * p.k_ts + (long long)hk * p.k_hs + rl * 8;
    const TT *vp = static_cast<const TT *>(p.v) + (long long)t0 * p.v_ts + (long long)h * p.v_hs + col0;
    auto load_v = [&](const TT *v, float (&x)[NC][C]) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            if (!on[i]) continue;
            if (p.tok_vec) {
                constexpr int VB = C * (int)sizeof(TT) > 16 ? 16 / (int)sizeof(TT) : C;
#pragma unroll
                for (int j = 0; j < C; j += VB) {
                    Pack<TT, VB> w;
                    w.load(v + col[i] + j);
#pragma unroll
                    for (int e = 0; e < VB; ++e) x[i][j + e] = w.get(e);
                }
            } else {
#pragma unroll
                for (int j = 0; j < C; ++j) x[i][j] = to_f32(v[col[i] + j]);
            }
        }
    };
    float s[8][NC][C];
    // one token: s and this thread's partial readout
    auto step = [&](const float (&q)[8], const float (&k)[8], const float (&v)[NC][C], float (&o)[NC][C]) {
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < C; ++j) {
                float acc = 0.0f;
#pragma unroll
                for (int r = 0; r < 8; ++r) {
                    s[r][i][j] = fmaf(k[r], v[i][j], lam * s[r][i][j]);
                    acc = fmaf(q[r], s[r][i][j], acc);
                }
                o[i][j] = acc;
            }
    };
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
        for (int i = 0; i < NC; ++i)
#pragma unroll
            for (int j = 0; j < C; ++j) s[r][i][j] = on[i] ? raw[r][i].get(j) : 0.0f;

    const int L = t1 - t0;
    for (int base = 0; base < L; base += kTok) {
        const int n = ONE ? 1 : min(kTok, L - base);
#pragma unroll
        for (int t = 0; t < (ONE ? 1 : kTok); ++t) {
            if (t >= n) break;
            float q[8], k[8], v[NC][C], o[NC][C];
            if (rl < rl_n) {
                load8(qp, p.tok_vec, q);
                load8(kp, p.tok_vec, k);
                load_v(vp, v);
                step(q, k, v, o);
#pragma unroll
                for (int i = 0; i < NC; ++i)
                    if (on[i])
#pragma unroll
                        for (int j = 0; j < C; ++j) part[(t * rl_n + rl) * row_w + col[i] + j] = o[i][j];
            }
            qp += p.q_ts;
            kp += p.k_ts;
            vp += p.v_ts;
        }
        __syncthreads();
        for (int i = tid; i < n * W; i += nt) {
            const int t = i / W, c = i - t * W;
            float o = 0.0f;
            for (int r = 0; r < rl_n; ++r) o += part[(t * rl_n + r) * row_w + c];
            out[(long long)(base + t) * p.o_ts + c] = from_f32<TT>(o * p.scale);
        }
        if (!ONE) __syncthreads();
        if (ONE) break;
    }
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
        for (int i = 0; i < NC; ++i)
            if (on[i]) {
#pragma unroll
                for (int j = 0; j < C; ++j) raw[r][i].set(j, s[r][i][j]);
                raw[r][i].store(sp + r * p.st_k + col[i]);
            }
}

template <typename ST, typename TT> cudaError_t go(const LaParams &p, cudaStream_t s) {
    const int W = p.V < 128 ? p.V : 128, cg_n = W / 8, rl_n = p.K / 8;
    const int threads = (cg_n * rl_n + 31) / 32 * 32;
    const unsigned blocks = (unsigned)p.batch * (unsigned)p.nv * (unsigned)p.tiles;
    const bool one = p.max_len == 1;
    const size_t smem = sizeof(float) * (one ? 1 : kTok) * rl_n * W;
    if (one)
        k_la_step<ST, TT, true><<<blocks, threads, smem, s>>>(p, cg_n);
    else
        k_la_step<ST, TT, false><<<blocks, threads, smem, s>>>(p, cg_n);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_la_step(const LaParams &p, bool tok_bf16, bool state_bf16, cudaStream_t s) {
    if (tok_bf16) return state_bf16 ? go<uint16_t, uint16_t>(p, s) : go<float, uint16_t>(p, s);
    return state_bf16 ? go<uint16_t, float>(p, s) : go<float, float>(p, s);
}

}  // namespace gdr
