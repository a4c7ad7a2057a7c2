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
// squares.  Bound: HBM for large calls, launch latency for small ones.
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
    } else {
        if (bf16)
            static_cast<uint16_t *>(base)[at] = from_f32<uint16_t>(x[0]);
        else
            static_cast<float *>(base)[at] = x[0];
    }
}

// act(g): g, g / (1 + exp(-g)) or 1 / (1 + exp(-g)); exp(-g) may overflow to
// infinity, whose quotient is the right limit of 0.
__device__ __forceinline__ float activate(float g, int act) {
    if (act == 0) return g;
    const float s = __fdividef(1.0f, 1.0f + __expf(-g));  // 0 where the quotient is below 2^-126
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
        if (e < p.D) {
            float wv[VEC];
            if (w) {
                Raw<VEC> r;
                r.load(w, e, false);
                r.get(false, wv);
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) u[i][j] = w ? u[i][j] * inv * wv[j] : u[i][j] * inv;
        }
    }
}

template <int VEC, int NV, int TPR>
__global__ void __launch_bounds__(TPR <= 32 ? 256 : TPR) k_norm(const __grid_constant__ NormParams p) {
    __shared__ float buf[4][32];
    constexpr int RPC = TPR <= 32 ? 256 / TPR : 1;  // rows per CTA
    const int lane = TPR <= 32 ? threadIdx.x % TPR : threadIdx.x;
    const long long rows = p.tokens * p.heads;
    long long row = (long long)blockIdx.x * RPC + threadIdx.x / TPR;
    const bool live = row < rows;  // a dead slice of a warp still takes part in the shuffles
    if (!live) row = rows - 1;
    const long long t = (unsigned)row / (unsigned)p.heads, h = row - t * p.heads;

    // every operand of the row is asked for before anything is computed
    Raw<VEC> xr[NV], gr[NV], rr[NV];
    float g0 = 1.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = (i * TPR + lane) * VEC;
        if (e < p.D) {
            if (p.x) xr[i].load(p.x, t * p.x_ts + h * p.x_hs + e, p.x_bf16);
            if (p.gate && p.g_es) gr[i].load(p.gate, t * p.g_ts + h * p.g_hs + e, p.gate_bf16);
            if (p.res) rr[i].load(p.res, t * p.r_ts + h * p.r_hs + e, p.res_bf16);
        }
    }
    if (p.gate && !p.g_es) {
        Raw<1> g;
        g.load(p.gate, t * p.g_ts + h * p.g_hs, p.gate_bf16);
        g0 = activate(g.a, p.act);
    }

    float u[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (p.x && (i * TPR + lane) * VEC < p.D) {
            xr[i].get(p.x_bf16, u[i]);
        } else {
#pragma unroll
            for (int j = 0; j < VEC; ++j) u[i][j] = 0.0f;
        }
    }
    auto gate = [&]() {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if ((i * TPR + lane) * VEC >= p.D) continue;
            float g[VEC];
            if (p.g_es) {
                gr[i].get(p.gate_bf16, g);
#pragma unroll
                for (int j = 0; j < VEC; ++j) g[j] = activate(g[j], p.act);
            } else {
#pragma unroll
                for (int j = 0; j < VEC; ++j) g[j] = g0;
            }
#pragma unroll
            for (int j = 0; j < VEC; ++j) u[i][j] *= g[j];
        }
    };
    if (p.gate && p.gate_first) gate();
    if (p.post) norm_row<VEC, NV, TPR>(u, lane, p, p.post_w, buf[0]);
    if (p.gate && !p.gate_first) gate();
    if (p.res) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if ((i * TPR + lane) * VEC >= p.D) continue;
            float r[VEC];
            rr[i].get(p.res_bf16, r);
#pragma unroll
            for (int j = 0; j < VEC; ++j) u[i][j] = p.x ? fmaf(p.scale, u[i][j], r[j]) : r[j];
        }
    }
    if (p.res_out && live) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int e = (i * TPR + lane) * VEC;
            if (e < p.D) put<VEC>(p.res_out, t * p.ro_ts + h * p.ro_hs + e, p.res_bf16, u[i]);
        }
    }
    if (!p.out) return;
    if (p.pre) norm_row<VEC, NV, TPR>(u, lane, p, p.pre_w, buf[2]);
    if (!live) return;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int e = (i * TPR + lane) * VEC;
        if (e < p.D) put<VEC>(p.out, t * p.o_ts + h * p.o_hs + e, p.out_bf16, u[i]);
    }
}

template <int VEC, int NV, int TPR> cudaError_t go(const NormParams &p, cudaStream_t s) {
    constexpr int RPC = TPR <= 32 ? 256 / TPR : 1;
    const long long rows = p.tokens * p.heads;
    k_norm<VEC, NV, TPR><<<(unsigned)((rows + RPC - 1) / RPC), TPR <= 32 ? 256 : TPR, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm(const NormParams &p, bool vec, cudaStream_t s) {
    if (vec) {
        if (p.D <= 64) return go<8, 1, 8>(p, s);
        if (p.D <= 128) return go<8, 1, 16>(p, s);
        if (p.D <= 256) return go<8, 1, 32>(p, s);
        if (p.D <= 512) return go<8, 2, 32>(p, s);
        if (p.D <= 1024) return go<8, 1, 128>(p, s);
        if (p.D <= 2048) return go<8, 1, 256>(p, s);
        if (p.D <= 4096) return go<8, 2, 256>(p, s);
        if (p.D <= 8192) return go<8, 2, 512>(p, s);
        return go<8, 4, 512>(p, s);
    }
    if (p.D <= 128) return go<1, 4, 32>(p, s);
    if (p.D <= 512) return go<1, 16, 32>(p, s);
    if (p.D <= 2048) return go<1, 8, 256>(p, s);
    if (p.D <= 4096) return go<1, 16, 256>(p, s);
    return go<1, 32, 512>(p, s);
}

}  // namespace gdr
