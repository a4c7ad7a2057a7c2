// Norms around a block, fused with the block's gate, residual scale and
// residual add (gdr_block_norm): one pass over every operand.
//
//     N(x; w) = (x - m) / sqrt(mean((x - m)^2) + eps) * w
//     u = N(x; post) * act(g)   or   N(x * act(g); post)
//     h = residual + scale * u  ;  out = N(h; pre)
//
// A row of D values lives in the registers of TPR threads (a slice of a warp
// for head sizes, a whole CTA for model widths), so both norms of a block
// boundary and the mean of the centred form cost reductions and no second
// read.  Sums are float32; the centred form subtracts the mean before it
// squares.  Bound: HBM for large calls (an 8192 x 4096 block boundary with both
// norms and a gate moves 336 MB in 62 us, 80% of the measured copy rate; with a
// float32 residual stream 76 us, 91%; 507 thousand heads of 128 72 us, 79%),
// launch latency for small ones.
#pragma once

#include "../gdr_device.cuh"
#include "layer_internal.h"

namespace gdr {
namespace {

// VEC neighbouring elements as they lie in memory.
template <int VEC> struct Raw;
template <> struct Raw<8> {
    uint4 a, b;
    __device__ __forceinline__ void load(const void *base, long long at, bool bf16) {
        if (bf16) {
            a = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + at);
        } else {
            const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const float *>(base) + at);
            a = p[0];
            b = p[1];
        }
    }
    __device__ __forceinline__ void get(bool bf16, float (&x)[8]) const {
        if (bf16) {
            const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        } else {
            const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
        }
    }
};
template <> struct Raw<2> {
    uint2 a;
    __device__ __forceinline__ void load(const void *base, long long at, bool bf16) {
        if (bf16)
            a.x = *reinterpret_cast<const uint32_t *>(static_cast<const uint16_t *>(base) + at);
        else
            a = *reinterpret_cast<const uint2 *>(static_cast<const float *>(base) + at);
    }
    __device__ __forceinline__ void get(bool bf16, float (&x)[2]) const {
        x[0] = __uint_as_float(bf16 ? a.x << 16 : a.x);
        x[1] = __uint_as_float(bf16 ? a.x & 0xffff0000u : a.y);
    }
};
template <> struct Raw<1> {
    float a;
    __device__ __forceinline__ void load(const void *base, long long at, bool bf16) {
        a = bf16 ? to_f32(static_cast<const uint16_t *>(base)[at]) : static_cast<const float *>(base)[at];
    }
    __device__ __forceinline__ void get(bool, float (&x)[1]) const { x[0] = a; }
};

template <int VEC>
__device__ __forceinline__ void put(void *base, long long at, bool bf16, const float (&x)[VEC]) {
    if constexpr (VEC == 8) {
        if (bf16) {
            uint4 w;
            uint32_t *e = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const __nv_bfloat162 h2 = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
                e[i] = *reinterpret_cast<const uint32_t *>(&h2);
            }
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + at) = w;
        } else {
            float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(base) + at);
            p[0] = make_float4(x[0], x[1], x[2], x[3]);
            p[1] = make_float4(x[4], x[5], x[6], x[7]);
        }
    } else if constexpr (VEC == 2) {
        if (bf16) {
            const __nv_bfloat162 h2 = __floats2bfloat162_rn(x[0], x[1]);
            *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(base) + at) = *reinterpret_cast<const uint32_t *>(&h2);
        } else {
            *reinterpret_cast<float2 *>(static_cast<float *>(base) + at) = make_float2(x[0], x[1]);
        }
    } else {
        if (bf16)
            static_cast<uint16_t *>(base)[at] = from_f32<uint16_t>(x[0]);
        else
            static_cast<float *>(base)[at] = x[0];
    }
}

// exp(x) to 2^-22: what rounding x log2(e) loses, which an fma gives exactly, and
// log2(e)'s own next digits are put right behind the power of two.
__device__ __forceinline__ float exp_near(float x) {
    constexpr float kL = 1.44269502f, kRest = 1.92596299e-8f, kLn2 = 0.693147181f;  // log2(e) = kL + kRest
    const float t = x * kL, lost = fabsf(x) < 200.0f ? fmaf(x, kRest, fmaf(x, kL, -t)) : 0.0f;  // past that e^x is 0 or infinity
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(t));
    return y * fmaf(lost, kLn2, 1.0f);
}
// act(g): g, g / (1 + exp(-g)) or 1 / (1 + exp(-g)); exp(-g) may overflow to
// infinity, whose quotient is the right limit of 0; a quotient below 2^-126 is 0
// too.  FAST: where every output is rounded to bfloat16, the exponential is good to
// 2^-22 and |g| 2^-24, which otherwise would show (7 units of float32 at -80).
template <bool FAST> __device__ __forceinline__ float activate(float g, int act) {
    if (act == 0) return g;
    float s;
    if (FAST)
        s = __fdividef(1.0f, 1.0f + __expf(-g));
    else
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + exp_near(-g)));
    return act == 1 ? g * s : s;
}

// Sum over the row's TPR threads; every thread gets it.  `buf` is the
// reduction's own shared array, so that one barrier is enough.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float *buf) {
#pragma unroll
    for (int m = 1; m < (TPR < 32 ? TPR : 32); m <<= 1) v += __shfl_xor_sync(kFull, v, m);
    if constexpr (TPR > 32) {
        constexpr int W = TPR / 32;
        if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
        __syncthreads();
        v = buf[threadIdx.x & (W - 1)];
#pragma unroll
        for (int m = 1; m < W; m <<= 1) v += __shfl_xor_sync(kFull, v, m);
    }
    return v;
}

// What a kernel knows about its call when it is compiled: 0, 1, or -1 for
// what it reads from the parameters.  Bounds first: a vector of 8 elements
// takes about 250 instructions with everything read from the parameters, which
// at 128 values a row is twice what HBM allows; about 90 with it known.
// GATE: 1 a gate with a value for each channel, 0 none or one with a value for each row.
// RES: 0 neither a residual nor a residual_out.
template <int XB, int GATE, int GB, int RES, int RB, int POST, int PRE, int OB> struct Cfg {
    static constexpr int x = XB < 0 ? -1 : 1, x_bf16 = XB, gate = GATE == 1 ? 1 : -1, gate_elem = GATE, gate_bf16 = GB, res = RES,
                         res_bf16 = RB, post = POST, pre = PRE, out_bf16 = OB;
    static constexpr bool coarse = OB == 1 && (RES == 0 || RB == 1);  // no output in float32
};
using Any = Cfg<-1, -1, -1, -1, -1, -1, -1, -1>;
template <int F> __device__ __forceinline__ bool is(bool runtime) { return F < 0 ? runtime : F != 0; }

template <int VEC, int NV, int TPR>
__device__ __forceinline__ void norm_row(float (&u)[NV][VEC], int lane, const NormParams &p, const float *w, float *buf) {
    if (p.centered) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) m += u[i][j];  // elements past D are 0
        m = row_sum<TPR>(m, buf) * p.inv_d;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if ((i * TPR + lane) * VEC < p.D)
#pragma unroll
                for (int j = 0; j < VEC; ++j) u[i][j] -= m;
    }
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) ss = fmaf(u[i][j], u[i][j], ss);
    ss = row_sum<TPR>(ss, buf + 32);
    const float inv = 1.0f / sqrtf(fmaf(ss, p.inv_d, p.eps));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = (i * TPR + lane) * VEC;
#pragma unroll
        for (int j = 0; j < VEC; ++j) u[i][j] *= inv;
        if (w && e < p.D) {
            float wv[VEC];
            Raw<VEC> r;
            r.load(w, e, false);
            r.get(false, wv);
#pragma unroll
            for (int j = 0; j < VEC; ++j) u[i][j] *= wv[j];
        }
    }
}

// What a thread asks for of one row.
template <class C, int VEC, int NV, int TPR> struct Row {
    Raw<VEC> x[NV], g[NV], r[NV];
    float g0;
    long long t, h;

    // Asks for every operand of the row; nothing is used yet.
    __device__ __forceinline__ void load(const NormParams &p, unsigned row, int lane) {
        t = p.heads_div.div(row);
        h = row - (unsigned)t * p.heads_div.d;
        const long long xo = t * p.x_ts + h * p.x_hs, go = t * p.g_ts + h * p.g_hs, ro = t * p.r_ts + h * p.r_hs;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (i * TPR + lane) * VEC;
            if (e < p.D) {
                if (is<C::x>(p.x != nullptr)) x[i].load(p.x, xo + e, is<C::x_bf16>(p.x_bf16));
                if (is<C::gate>(p.gate != nullptr) && is<C::gate_elem>(p.g_es))
                    g[i].load(p.gate, go + e, is<C::gate_bf16>(p.gate_bf16));
                if (is<C::res>(p.res != nullptr)) r[i].load(p.res, ro + e, is<C::res_bf16>(p.res_bf16));
            }
        }
        if (is<C::gate>(p.gate != nullptr) && !is<C::gate_elem>(p.g_es)) {
            Raw<1> w;
            w.load(p.gate, go, p.gate_bf16);
            g0 = w.a;
        }
    }

    __device__ __forceinline__ void gate_by(const NormParams &p, float (&u)[NV][VEC], int lane) const {
        const float all = is<C::gate_elem>(p.g_es) ? 1.0f : activate<C::coarse>(g0, p.act);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if ((i * TPR + lane) * VEC >= p.D) continue;
            if (is<C::gate_elem>(p.g_es)) {
                float y[VEC];
                g[i].get(is<C::gate_bf16>(p.gate_bf16), y);
                if (p.act) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) y[j] = activate<C::coarse>(y[j], p.act);
                }
#pragma unroll
                for (int j = 0; j < VEC; ++j) u[i][j] *= y[j];
            } else {
#pragma unroll
                for (int j = 0; j < VEC; ++j) u[i][j] *= all;
            }
        }
    }

    __device__ __forceinline__ void finish(const NormParams &p, int lane, bool live, float (*buf)[32]) const {
        float u[NV][VEC];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (is<C::x>(p.x != nullptr) && (i * TPR + lane) * VEC < p.D) {
                x[i].get(is<C::x_bf16>(p.x_bf16), u[i]);
            } else {
#pragma unroll
                for (int j = 0; j < VEC; ++j) u[i][j] = 0.0f;
            }
        }
        const bool gated = is<C::gate>(p.gate != nullptr);
        if (gated && p.gate_first) gate_by(p, u, lane);
        if (is<C::post>(p.post)) norm_row<VEC, NV, TPR>(u, lane, p, p.post_w, buf[0]);
        if (gated && !p.gate_first) gate_by(p, u, lane);
        if (is<C::res>(p.res != nullptr)) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if ((i * TPR + lane) * VEC >= p.D) continue;
                float y[VEC];
                r[i].get(is<C::res_bf16>(p.res_bf16), y);
#pragma unroll
                for (int j = 0; j < VEC; ++j) u[i][j] = is<C::x>(p.x != nullptr) ? fmaf(p.scale, u[i][j], y[j]) : y[j];
            }
        }
        if (C::res != 0 && p.res_out && live) {  // h, with a residual or without
            const long long at = t * p.ro_ts + h * p.ro_hs;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int e = (i * TPR + lane) * VEC;
                if (e < p.D) put<VEC>(p.res_out, at + e, is<C::res_bf16>(p.res_bf16), u[i]);
            }
        }
        if (!p.out) return;
        if (is<C::pre>(p.pre)) norm_row<VEC, NV, TPR>(u, lane, p, p.pre_w, buf[2]);
        if (!live) return;
        const long long at = t * p.o_ts + h * p.o_hs;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (i * TPR + lane) * VEC;
            if (e < p.D) put<VEC>(p.out, at + e, is<C::out_bf16>(p.out_bf16), u[i]);
        }
    }
};

// With everything read from the parameters, 512 threads of two vectors would
// take 82 registers each, one CTA a multiprocessor (7682 rows of 6168, float32:
// 210 us; 193 with two).
template <class C, int VEC, int NV, int TPR, int NR>
__global__ void __launch_bounds__(TPR <= 32 ? 256 : TPR, TPR == 512 && VEC * NV <= 16 ? 2 : 1) k_norm(const __grid_constant__ NormParams p) {
    static_assert(NR == 1 || TPR <= 32, "several rows a slice of a warp, or one a CTA");
    __shared__ float buf[4][32];
    constexpr unsigned RPC = TPR <= 32 ? 256 / TPR : 1;  // slices a CTA
    const int lane = TPR <= 32 ? threadIdx.x % TPR : threadIdx.x;
    const unsigned rows = p.rows, row0 = blockIdx.x * (RPC * NR) + threadIdx.x / TPR;
    // a slice past the last row repeats it without writing: it still takes part in its warp's shuffles
    Row<C, VEC, NV, TPR> in[NR];
#pragma unroll
    for (int n = 0; n < NR; ++n) in[n].load(p, min(row0 + n * RPC, rows - 1), lane);
#pragma unroll
    for (int n = 0; n < NR; ++n) in[n].finish(p, lane, row0 + n * RPC < rows, buf);
}

template <class C, int VEC, int NV, int TPR, int NR = 1> cudaError_t go(const NormParams &p, cudaStream_t s) {
    constexpr unsigned RPC = (TPR <= 32 ? 256 / TPR : 1) * NR;
    k_norm<C, VEC, NV, TPR, NR><<<(p.rows + RPC - 1) / RPC, TPR <= 32 ? 256 : TPR, 0, s>>>(p);
    return cudaGetLastError();
}

// A block boundary as models have it: what the kernels know when compiled.
inline bool is_boundary(const NormParams &p) {
    return p.x && p.res && p.pre && p.out && p.out_bf16 && p.D > 256 && (!p.gate || !p.g_es || p.gate_bf16 == p.x_bf16);
}

// Which kernel a call of rows that are not 16-byte vectors gets.
template <class Width, int XB> cudaError_t go_narrow_boundary(const NormParams &p, cudaStream_t s) {
    if (p.gate && p.g_es)
        return p.res_bf16 ? Width::template rows<Cfg<XB, 1, XB, 1, 1, -1, 1, 1>>(p, s)
                          : Width::template rows<Cfg<XB, 1, XB, 1, 0, -1, 1, 1>>(p, s);
    return p.res_bf16 ? Width::template rows<Cfg<XB, 0, 0, 1, 1, -1, 1, 1>>(p, s)
                      : Width::template rows<Cfg<XB, 0, 0, 1, 0, -1, 1, 1>>(p, s);
}
template <class Width> cudaError_t go_narrow(const NormParams &p, cudaStream_t s) {
    if (is_boundary(p)) return p.x_bf16 ? go_narrow_boundary<Width, 1>(p, s) : go_narrow_boundary<Width, 0>(p, s);
    return Width::template rows<Any>(p, s);
}

}  // namespace
}  // namespace gdr
