// Decayed linear attention for short rows (drafts, last pieces of prompts;
// bfloat16 tokens): the chunks of k_la_chunk.cu, 16 tokens each, in warp-level
// matrix instructions and registers.
//
//     O^T[:, i] = scale lambda^(i+1) (S0^T q_i)  +  V^T P~^T[:, i],
//     P~[i, j]  = scale lambda^(i-j) q_i . k_j for j <= i, else 0
//     S^T       = lambda^n S0^T + V~^T K,   V~[j] = lambda^(n-1-j) v_j
//
// A warp keeps its columns of S, transposed (value index = row), as float32
// accumulators.  Their layout is that of an A operand once rounded, and P's is
// that of a B operand, so that everything chains in registers; tokens and
// states pass through shared memory.  Operands made here go in as two bfloat16
// parts (V~ for a float32 pool as three), which keep 16 (24) bits: nothing is
// rounded to fewer but the results.
//
// Bound: HBM, a state in and out for a few tokens.  A CTA asks for its next
// chunk's tokens, and behind a row's last chunk for the next unit's state, before
// it computes the current one, two CTAs a multiprocessor.  1024 (row, head) pairs
// of 128 x 256 take 40 us here at 5 tokens, 42 at 16 and 70 at 32 (floor 21, 23
// and 27); the recurrent form of k_la_step.cu takes 30 + 11 a token, the roles of
// k_la_chunk.cu, which fill and drain for each unit, 87.  A warp keeps 32
// columns (16, twice the warps: 44 us).
#include "../gdr_device.cuh"
#include "layer_internal.h"

namespace gdr {
namespace {

constexpr int kT = 16;  // tokens a chunk

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void ldm4_t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(a)
                 : "memory");
}
__device__ __forceinline__ void stm4_t(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z),
                 "r"(w)
                 : "memory");
}
// 16 bytes, or zeros where there is nothing.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    const __nv_bfloat162 h2 = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h2);
}
__device__ __forceinline__ float low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
// The rounding of what the pair w leaves of (x, y).
__device__ __forceinline__ uint32_t rest(uint32_t w, float x, float y) { return pack(x - low(w), y - high(w)); }
__device__ __forceinline__ float power(float lg2, int n) { return n == 0 ? 1.0f : exp2f(lg2 * (float)n); }

// Shared memory of a CTA: two units' tokens and states, one unit's output.
// Rows are 16 bytes longer than their contents, so that the eight rows of a
// matrix start in different banks (and a float32 state's rows k, k + 2, k + 4,
// k + 6 eight apart).
template <typename ST, int KP, int VT, int MT> struct Lay {
    static constexpr int SK = KP * 2 + 16, SV = VT * 2 + 16, SS = VT * (int)sizeof(ST) + 16, SO = MT * 32 + 16;
    static constexpr int TOK = kT * (2 * SK + SV);  // Q | K | V
    static constexpr int STATE = KP * SS;
    static constexpr int WARPS = VT / (16 * MT), THREADS = 32 * WARPS;  // a warp for 16 MT columns
    static constexpr int OUT = WARPS * kT * SO;
    static constexpr int ALL = 2 * (TOK + STATE) + OUT;
};

struct ShortUnit {
    int h, col0, t0, len, slot;
    float lg2;
};

// MANY: rows of more than 16 tokens, a chunk after the other.  Compiled apart, for the one-chunk form has no register
// to spare (8 bytes spilled: 46 us for 40).
template <typename ST, int KP, int VT, int MT, bool MANY>
__global__ void __launch_bounds__(Lay<ST, KP, VT, MT>::THREADS, 2)
    k_la_small(const __grid_constant__ LaParams p, FastDiv per, FastDiv tiles) {
    using L = Lay<ST, KP, VT, MT>;
    constexpr int NT = L::THREADS, NK = KP / 8, CPS = 16 / (int)sizeof(ST);
    extern __shared__ __align__(16) unsigned char sm[];
    const uint32_t base = (uint32_t)__cvta_generic_to_shared(sm);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, c2 = 2 * (lane & 3), r4 = lane >> 2;
    const unsigned units = (unsigned)p.batch * per.d;
    const uint32_t s_out = base + 2 * (L::TOK + L::STATE) + warp * (kT * L::SO);

    // a unit's facts; len 0 where there is nothing to compute (a skipped row's output is cleared)
    auto facts = [&](unsigned pos) {
        ShortUnit u{};
        if (pos >= units) return u;
        const int b = (int)per.div(pos);
        const unsigned ht = pos - (unsigned)b * per.d;
        u.h = (int)tiles.div(ht);
        u.col0 = (int)(ht - (unsigned)u.h * tiles.d) * VT;
        const int t0 = p.offsets[b], t1 = p.offsets[b + 1];
        const float d = p.decay[(long long)u.h * p.decay_s];
        u.slot = p.slot_idx[b];
        u.t0 = t0;
        const bool leader = tid == 0 && ht == 0;
        if (t0 < 0 || t1 < t0 || t1 > p.T) {
            if (leader) flag(p.status, GDR_STATUS_BAD_OFFSETS);
            return u;
        }
        const int len = t1 - t0;
        const bool bad_decay = !(p.decay_is_log ? d <= 0.0f : (d >= 0.0f && d <= 1.0f)), too_long = len > p.max_len;
        if (len > 0 && (u.slot < 0 || u.slot >= p.max_slots || bad_decay || too_long)) {
            if (too_long) {
                if (leader) flag(p.status, GDR_STATUS_ROW_TOO_LONG);
            } else if (u.slot < -1 || u.slot >= p.max_slots) {
                if (leader) flag(p.status, GDR_STATUS_BAD_SLOT);
            } else if (u.slot >= 0 && tid == 0) {
                flag(p.status, GDR_STATUS_BAD_DECAY);
            }
            uint16_t *out = static_cast<uint16_t *>(p.out) + (long long)t0 * p.o_ts + (long long)u.h * p.o_hs + u.col0;
            clear_rows(out, p.o_ts, len, min(VT, p.V - u.col0), true, tid, NT);
            return u;
        }
        u.len = len;
        u.lg2 = p.decay_is_log ? d * 1.44269504088896340736f : log2f(d);
        return u;
    };
    auto pool_of = [&](const ShortUnit &u) {
        return static_cast<ST *>(p.state) + (long long)u.slot * p.st_slot + (long long)u.h * p.st_head + u.col0;
    };
    // asks for a unit's state, and for 16 of its tokens; what lies past the row's end, the key channels or the columns
    // reads as zero
    auto ask_state = [&](const ShortUnit &u, int buf) {
        if (u.len > 0) {
            const int W = min(VT, p.V - u.col0);
            const ST *pool = pool_of(u);
            const uint32_t st = base + 2 * L::TOK + buf * L::STATE;
            for (int i = tid; i < KP * (VT / CPS); i += NT) {
                const int k = i / (VT / CPS), c = i % (VT / CPS);
                const bool there = k < p.K && c * CPS < W;
                copy16(st + k * L::SS + c * 16, there ? pool + (long long)k * p.st_k + c * CPS : pool, there);
            }
        }
    };
    auto ask_tokens = [&](const ShortUnit &u, int at, int buf) {
        const int n = u.len - at;
        if (n > 0) {
            const int W = min(VT, p.V - u.col0), hk = u.h / p.r;
            const long long t0 = u.t0 + at;
            const uint32_t to = base + buf * L::TOK;
            const uint16_t *qp = static_cast<const uint16_t *>(p.q) + t0 * p.q_ts + (long long)hk * p.q_hs;
            const uint16_t *kp = static_cast<const uint16_t *>(p.k) + t0 * p.k_ts + (long long)hk * p.k_hs;
            const uint16_t *vp = static_cast<const uint16_t *>(p.v) + t0 * p.v_ts + (long long)u.h * p.v_hs + u.col0;
            for (int i = tid; i < kT * (KP / 8); i += NT) {
                const int t = i / (KP / 8), c = i % (KP / 8);
                const bool there = t < n && c * 8 < p.K;
                copy16(to + t * L::SK + c * 16, there ? qp + (long long)t * p.q_ts + c * 8 : qp, there);
                copy16(to + (kT + t) * L::SK + c * 16, there ? kp + (long long)t * p.k_ts + c * 8 : kp, there);
            }
            for (int i = tid; i < kT * (VT / 8); i += NT) {
                const int t = i / (VT / 8), c = i % (VT / 8);
                const bool there = t < n && c * 8 < W;
                copy16(to + 2 * kT * L::SK + t * L::SV + c * 16, there ? vp + (long long)t * p.v_ts + c * 8 : vp, there);
            }
        }
    };

    // this lane's row of matrix l / 8 of a 16 x 16 block stored by rows: (l & 7) + 8 * (l / 8 & 1) rows, 8 * (l / 16) columns
    const int m_row = (lane & 7) + ((lane >> 3) & 1) * 8, m_col = lane >> 4;
    // and of its transpose: (l & 7) + 8 * (l / 16) rows, 8 * (l / 8 & 1) columns
    const int x_row = (lane & 7) + (lane >> 4) * 8, x_col = ((lane >> 3) & 1) * 8;
    unsigned pos = blockIdx.x;
    ShortUnit u = facts(pos);
    ask_state(u, 0);
    ask_tokens(u, 0, 0);
    cp_async_commit();
    for (int buf = 0, tok = 0; pos < units; pos += gridDim.x, buf ^= 1) {
        // S^T: rows 16 mt + r4 (+ 8) of the warp's columns, key indices 8 n + c2, + 1
        float s[MT][NK][4];
        ShortUnit after;
        for (int at = 0;; at += kT, tok ^= 1) {
            const bool last = !MANY || u.len - at <= kT;
            const int tb = MANY ? tok : buf;
            if (last) {  // the other buffers were left behind a barrier ago
                after = facts(pos + gridDim.x);
                ask_state(after, buf ^ 1);
                ask_tokens(after, 0, tb ^ 1);
            } else {
                ask_tokens(u, at + kT, tb ^ 1);
            }
            cp_async_commit();
            cp_async_wait<1>();
            __syncthreads();
            if (u.len > 0) {
                const int n = MANY ? min(kT, u.len - at) : u.len, W = min(VT, p.V - u.col0), v0 = warp * 16 * MT;
                const uint32_t sq = base + tb * L::TOK, sk = sq + kT * L::SK, sv = sk + kT * L::SK;
                const uint32_t ss = base + 2 * L::TOK + buf * L::STATE;
                if (at == 0) {
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        if constexpr (sizeof(ST) == 2) {
#pragma unroll
                            for (int nk = 0; nk < NK; nk += 2) {
                                uint32_t r[4];  // blocks (keys 8 nk.., columns +0), (+0, +8), (keys 8 nk + 8.., +0), (.., +8)
                                ldm4_t(r, ss + (8 * nk + x_row) * L::SS + (v0 + mt * 16 + x_col) * 2);
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    s[mt][nk + (i >> 1)][(i & 1) * 2] = low(r[i]);
                                    s[mt][nk + (i >> 1)][(i & 1) * 2 + 1] = high(r[i]);
                                }
                            }
                        } else {
#pragma unroll
                            for (int nk = 0; nk < NK; ++nk)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    s[mt][nk][i] = *reinterpret_cast<const float *>(
                                        sm + 2 * L::TOK + buf * L::STATE + (8 * nk + c2 + (i & 1)) * L::SS +
                                        (v0 + mt * 16 + r4 + (i >> 1) * 8) * 4);
                        }
                    }
                }
                // P = Q K^T and S0^T Q^T
                float P[2][4] = {}, o[MT][2][4] = {};
#pragma unroll
                for (int ks = 0; ks < KP / 16; ++ks) {
                    uint32_t q[4], k[4];  // blocks (tokens +0, keys +0), (+8, +0), (+0, +8), (+8, +8)
                    ldm4(q, sq + m_row * L::SK + (ks * 16 + m_col * 8) * 2);
                    ldm4(k, sk + m_row * L::SK + (ks * 16 + m_col * 8) * 2);
                    mma(P[0], q, k[0], k[2]);
                    mma(P[1], q, k[1], k[3]);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const float(&x)[4] = s[mt][2 * ks], (&y)[4] = s[mt][2 * ks + 1];
                        const uint32_t a[4] = {pack(x[0], x[1]), pack(x[2], x[3]), pack(y[0], y[1]), pack(y[2], y[3])};
                        mma(o[mt][0], a, q[0], q[2]);
                        mma(o[mt][1], a, q[1], q[3]);
                        if (sizeof(ST) == 4 || (MANY && at > 0)) {  // a bfloat16 pool's state is exact as it comes
                            const uint32_t e[4] = {rest(a[0], x[0], x[1]), rest(a[1], x[2], x[3]), rest(a[2], y[0], y[1]),
                                                   rest(a[3], y[2], y[3])};
                            mma(o[mt][0], e, q[0], q[2]);
                            mma(o[mt][1], e, q[1], q[3]);
                        }
                    }
                }
                // P~ as B operand [j, i]: chosen where j <= i, whatever the other places hold
                uint32_t pb[2][2], pc[2][2];  // and what its rounding leaves
#pragma unroll
                for (int ih = 0; ih < 2; ++ih)
#pragma unroll
                    for (int jt = 0; jt < 2; ++jt) {
                        const int gap = r4 + 8 * ih - (8 * jt + c2);
                        const float x = gap < 0 ? 0.0f : P[jt][2 * ih] * (p.scale * power(u.lg2, gap));
                        const float y = gap < 1 ? 0.0f : P[jt][2 * ih + 1] * (p.scale * power(u.lg2, gap - 1));
                        pb[ih][jt] = pack(x, y);
                        pc[ih][jt] = rest(pb[ih][jt], x, y);
                    }
                const float lam_n = power(u.lg2, n);
                float f[2][2], wt[2][2];  // factors of outputs, and weights of values, of tokens 8 i + c2 + e
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int t = 8 * i + c2 + e;
                        f[i][e] = p.scale * power(u.lg2, t + 1);
                        wt[i][e] = n - 1 - t < 0 ? 0.0f : power(u.lg2, n - 1 - t);
                    }
                uint32_t va[MT][3][4];  // V~^T as A operand, its parts
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    uint32_t v[4];  // V^T: blocks (columns +0, tokens +0), (+8, +0), (+0, +8), (+8, +8)
                    ldm4_t(v, sv + x_row * L::SV + (v0 + mt * 16 + x_col) * 2);
#pragma unroll
                    for (int nt = 0; nt < 2; ++nt) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[mt][nt][i] *= f[nt][i & 1];
                        mma(o[mt][nt], v, pb[nt][0], pb[nt][1]);
                        mma(o[mt][nt], v, pc[nt][0], pc[nt][1]);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x = low(v[i]) * wt[i >> 1][0], y = high(v[i]) * wt[i >> 1][1];
                        va[mt][0][i] = pack(x, y);
                        const float x1 = x - low(va[mt][0][i]), y1 = y - high(va[mt][0][i]);
                        va[mt][1][i] = pack(x1, y1);
                        if constexpr (sizeof(ST) == 4) va[mt][2][i] = rest(va[mt][1][i], x1, y1);
                    }
                    // the output, turned: blocks (columns +0, tokens +0), (+8, +0), (+0, +8), (+8, +8)
                    stm4_t(s_out + x_row * L::SO + (mt * 16 + x_col) * 2, pack(o[mt][0][0], o[mt][0][1]), pack(o[mt][0][2], o[mt][0][3]),
                           pack(o[mt][1][0], o[mt][1][1]), pack(o[mt][1][2], o[mt][1][3]));
                }
                // S^T = lambda^n S^T + V~^T K
#pragma unroll
                for (int nk = 0; nk < NK; nk += 2) {
                    uint32_t k[4];  // blocks (tokens +0, keys 8 nk..), (+8, ..), (+0, keys 8 nk + 8..), (+8, ..)
                    ldm4_t(k, sk + m_row * L::SK + (nk + m_col) * 16);
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) s[mt][nk + e][i] *= lam_n;
#pragma unroll
                            for (int part = 0; part < (sizeof(ST) == 2 ? 2 : 3); ++part)
                                mma(s[mt][nk + e], va[mt][part], k[2 * e], k[2 * e + 1]);
                        }
                }
                if (last) {  // the state goes back through its place in shared memory (a warp's columns are its own)
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        if constexpr (sizeof(ST) == 2) {
#pragma unroll
                            for (int nk = 0; nk < NK; nk += 2)
                                stm4_t(ss + (8 * nk + x_row) * L::SS + (v0 + mt * 16 + x_col) * 2, pack(s[mt][nk][0], s[mt][nk][1]),
                                       pack(s[mt][nk][2], s[mt][nk][3]), pack(s[mt][nk + 1][0], s[mt][nk + 1][1]),
                                       pack(s[mt][nk + 1][2], s[mt][nk + 1][3]));
                        } else {
#pragma unroll
                            for (int nk = 0; nk < NK; ++nk)
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    *reinterpret_cast<float *>(sm + 2 * L::TOK + buf * L::STATE + (8 * nk + c2 + (i & 1)) * L::SS +
                                                               (v0 + mt * 16 + r4 + (i >> 1) * 8) * 4) = s[mt][nk][i];
                        }
                    }
                }
                __syncthreads();
                ST *pool = pool_of(u);
                for (int i = last ? tid : KP * (VT / CPS); i < KP * (VT / CPS); i += NT) {
                    const int k = i / (VT / CPS), c = i % (VT / CPS);
                    if (k < p.K && c * CPS < W)
                        *reinterpret_cast<uint4 *>(pool + (long long)k * p.st_k + c * CPS) =
                            *reinterpret_cast<const uint4 *>(sm + 2 * L::TOK + buf * L::STATE + k * L::SS + c * 16);
                }
                uint16_t *out = static_cast<uint16_t *>(p.out) + (long long)(u.t0 + at) * p.o_ts + (long long)u.h * p.o_hs + u.col0;
                for (int i = tid; i < n * (VT / 8); i += NT) {
                    const int t = i / (VT / 8), c = i % (VT / 8) * 8;
                    if (c < W)
                        *reinterpret_cast<uint4 *>(out + (long long)t * p.o_ts + c) = *reinterpret_cast<const uint4 *>(
                            sm + 2 * (L::TOK + L::STATE) + (c / (16 * MT)) * (kT * L::SO) + t * L::SO + c % (16 * MT) * 2);
                }
                __syncthreads();  // everyone is done with these buffers
            }
            if (last) break;
        }
        tok ^= 1;
        u = after;
    }
    cp_async_wait<0>();
}

template <typename ST, int KP, int VT, int MT, bool MANY> cudaError_t go_form(const LaParams &p, cudaStream_t s) {
    using L = Lay<ST, KP, VT, MT>;
    static LaunchCache cache;
    LaunchInfo li;
    const cudaError_t e = launch_info(cache, &li, [](LaunchInfo &l) {
        const cudaError_t r =
            cudaFuncSetAttribute(k_la_small<ST, KP, VT, MT, MANY>, cudaFuncAttributeMaxDynamicSharedMemorySize, L::ALL);
        return r != cudaSuccess ? r
                                : cudaOccupancyMaxActiveBlocksPerMultiprocessor(&l.occ, k_la_small<ST, KP, VT, MT, MANY>,
                                                                                L::THREADS, L::ALL);
    });
    if (e != cudaSuccess) return e;
    const unsigned tiles = (unsigned)(p.V + VT - 1) / VT, per = (unsigned)p.nv * tiles, units = (unsigned)p.batch * per;
    const unsigned most = (unsigned)li.sms * (unsigned)li.occ;
    k_la_small<ST, KP, VT, MT, MANY><<<units < most ? units : most, L::THREADS, L::ALL, s>>>(p, FastDiv(per), FastDiv(tiles));
    return cudaGetLastError();
}

template <typename ST, int KP, int VT, int MT> cudaError_t go(const LaParams &p, cudaStream_t s) {
    return p.max_len > kT ? go_form<ST, KP, VT, MT, true>(p, s) : go_form<ST, KP, VT, MT, false>(p, s);
}

}  // namespace

cudaError_t launch_la_small(const LaParams &p, bool state_bf16, cudaStream_t s) {
    const bool wide_k = p.K > 64;
    if (state_bf16) {
        if (p.V > 64) return wide_k ? go<uint16_t, 128, 128, 2>(p, s) : go<uint16_t, 64, 128, 2>(p, s);
        return wide_k ? go<uint16_t, 128, 64, 1>(p, s) : go<uint16_t, 64, 64, 1>(p, s);
    }
    return wide_k ? go<float, 128, 64, 1>(p, s) : go<float, 64, 64, 1>(p, s);
}

}  // namespace gdr
