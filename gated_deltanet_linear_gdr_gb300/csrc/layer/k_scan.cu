// Selective scan: the choice of types, and the join of a cut row's segments.
#include "scan_device.cuh"

namespace gdr {
namespace {

// A cut row's segments, one after the other, a thread an element (head, state, channel):
// segment s starts from S, and S <- exp(A sum(d)) S + (its own state from zero).  Reads a
// segment's own state and leaves its start state in its place.
__global__ void __launch_bounds__(256) k_scan_join(const __grid_constant__ ScanParams p) {
    const long long per = (long long)p.nv * p.K * p.V, i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= per) return;
    const long long most = scan_pieces(p.T, p.seg, p.batch);
    const int seg = scan_segment(p);
    long long piece = 0;
    ScanUnit u;
    int n = 0;
    for (int b = 0; b <= (int)blockIdx.y; ++b) {
        piece += n;
        n = scan_row(p, b, false, u) ? pieces(u.len, seg) : 0;
    }
    if (n == 0 || u.slot < 0) return;
    const long long kv = (long long)p.K * p.V, kj = i % kv;
    const int h = (int)(i / kv), k = (int)(kj / p.V), v = (int)(kj - (long long)k * p.V);
    const float a = p.A[h * p.a_hs + k * p.a_ks + v * p.a_vs];
    const long long at = (long long)u.slot * p.st_slot + (long long)h * p.st_head + (long long)k * p.st_k + v;
    float S = p.st_bf16 ? to_f32(static_cast<const uint16_t *>(p.state)[at]) : static_cast<const float *>(p.state)[at];
    float *own = p.ws + piece * per + i;
    const float *sum = p.ws + most * per + piece * p.nv * p.V + (long long)h * p.V + v;
    // eight segments' values on their way at a time
    constexpr int kAhead = 8;
    for (int s = 0; s < n; s += kAhead) {
        float o[kAhead], d[kAhead];
#pragma unroll
        for (int q = 0; q < kAhead; ++q) {
            const bool some = s + q + 1 < n;  // nothing starts from the last one's state
            o[q] = some ? own[q * per] : 0.0f;
            d[q] = some ? sum[q * (long long)p.nv * p.V] : 0.0f;
        }
#pragma unroll
        for (int q = 0; q < kAhead; ++q)
            if (s + q < n) {
                own[q * per] = S;
                S = fmaf(expf(a * d[q]), S, o[q]);
            }
        own += kAhead * per;
        sum += kAhead * (long long)p.nv * p.V;
    }
}

}  // namespace

cudaError_t launch_scan_join(const ScanParams &p, cudaStream_t s) {
    const long long per = (long long)p.nv * p.K * p.V;
    k_scan_join<<<dim3((unsigned)((per + 255) / 256), (unsigned)p.batch), 256, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_scan(const ScanParams &p, bool tok_bf16, bool dt_bf16, bool vec, cudaStream_t s) {
    if (!tok_bf16) return p.st_bf16 ? launch_scan_fx(p, vec, s) : launch_scan_ff(p, vec, s);
    return dt_bf16 ? launch_scan_bb(p, vec, s) : launch_scan_bf(p, vec, s);
}

cudaError_t launch_scan_step(const ScanParams &p, bool tok_bf16, bool dt_bf16, bool vec, cudaStream_t s) {
    if (!tok_bf16) return launch_scan_step_ff(p, vec, s);
    return dt_bf16 ? launch_scan_step_bb(p, vec, s) : launch_scan_step_bf(p, vec, s);
}

}  // namespace gdr
