// Internal launch parameters of the layer operators around the recurrence:
// decayed linear attention and the fused block norms.  Host code (api_layer.cu)
// validates the public argument structs and lowers them into these.
#pragma once

#include "../gdr_internal.h"

namespace gdr {

// Error text and status word shared by every entry point (api.cu).
int api_fail(int code, const char *text);
int api_ok();
int api_status(unsigned **out);

// How many pieces of `size` make up n, which may be as large as an int gets: rows
// may have up to 2^31 - 1 tokens.
#ifdef __CUDACC__
__host__ __device__
#endif
constexpr int pieces(int n, int size) { return n <= 0 ? 0 : (n - 1) / size + 1; }

// One decayed linear attention call, after validation.  Strides in elements.
struct LaParams {
    int batch, nv, nk, r;  // r = nv / nk
    int K, V;
    int tiles;             // column tiles of up to 128 values a (row, head) is cut into
    int decay_is_log;
    long long T;
    long long max_len;     // the caller's bound on row lengths, or <= 0
    const void *q, *k, *v;
    long long q_ts, q_hs, k_ts, k_hs, v_ts, v_hs;
    const float *decay;
    long long decay_s;
    float scale;
    void *out;
    long long o_ts, o_hs;
    void *state;
    long long st_slot, st_head, st_k;
    long long max_slots;
    const int *slot_idx, *offsets;
    int tok_vec;           // q, k, v and out rows may be moved as 16-byte vectors
    unsigned *status;
};

// Recurrent form on the FP32 pipes: any alignment, any row length; what single
// tokens, float32 tokens and rows that are not 16-byte vectors run on.
cudaError_t launch_la_step(const LaParams &p, bool tok_bf16, bool state_bf16, cudaStream_t s);

// Chunked form in warp-level matrix instructions: bfloat16 tokens whose rows are
// 16-byte vectors; for short rows (max_len bounds them).
cudaError_t launch_la_small(const LaParams &p, bool state_bf16, cudaStream_t s);

// Chunked form on the tensor cores: bfloat16 tokens whose rows are 16-byte
// vectors.  seg > 0 cuts rows into segments of that many tokens (a multiple of
// 64; batch <= 32) whose start states are worked out first, in ws.  Launches
// nothing and leaves *used false where a layout cannot be described to TMA.
cudaError_t launch_la_chunk(const LaParams &p, bool state_bf16, int seg, void *ws, cudaStream_t s, bool *used);

// One fused norm call, after validation.
struct NormParams {
    unsigned rows;     // tokens * heads
    FastDiv heads_div;
    int D;
    int x_bf16, gate_bf16, res_bf16, out_bf16;
    int act, gate_first, post, pre, centered;
    float eps, scale, inv_d;
    const void *x;
    long long x_ts, x_hs;
    const void *gate;
    long long g_ts, g_hs, g_es;
    const void *res;
    long long r_ts, r_hs;
    void *res_out;
    long long ro_ts, ro_hs;
    void *out;
    long long o_ts, o_hs;
    const float *post_w, *pre_w;
};
// vec: every row, gate and weight may be moved as vectors of 8 elements (16 bytes), of 2, or of 1.
cudaError_t launch_norm(const NormParams &p, int vec, cudaStream_t s);
cudaError_t launch_norm_pairs(const NormParams &p, cudaStream_t s);
cudaError_t launch_norm_odd(const NormParams &p, cudaStream_t s);

// One short convolution call, after validation.  Strides in elements.
struct ConvOpParams {
    int batch, channels, silu;
    int run, tiles;    // a block's tokens where it takes a run of them; channel tiles
    int keep;          // slots are written
    int vec;           // token rows may be moved as vectors of four
    int w_vec;         // a channel's weights lie together, four of them as one vector
    int st_run;        // a slot's [channels, width-1] lie together, 16-byte aligned
    int st_bf16;
    long long T, max_len;
    const void *x;
    long long x_ts;
    const float *w;
    long long w_cs, w_ts;
    const float *bias;
    void *out;         // or null: only states move
    long long o_ts;
    void *state;
    long long s_slot, s_chan, s_tap;
    long long max_slots;
    const int *slot_idx, *offsets, *counts;
    unsigned *status;
};
cudaError_t launch_short_conv(ConvOpParams p, int width, bool tok_bf16, cudaStream_t s);

// One selective scan call, after validation.  Strides in elements.
struct ScanParams {
    int batch, nv, nk, r;  // r = nv / nk
    int K, V;
    int softplus, keep;
    int st_bf16;
    int bc_vec;        // B and C rows may be moved as vectors of four
    long long T, max_len;
    const void *x, *dt, *B, *C, *z;
    long long x_ts, x_hs, dt_ts, dt_hs, dt_es, B_ts, B_hs, C_ts, C_hs, z_ts, z_hs;
    const float *A, *D, *bias;
    long long a_hs, a_ks, a_vs, d_hs, d_vs, b_hs, b_vs;
    void *out;         // or null: only states move
    long long o_ts, o_hs;
    void *state;
    long long st_slot, st_head, st_k;
    long long max_slots;
    const int *slot_idx, *offsets, *counts;
    // rows cut into segments of `seg` tokens (0: whole): ws holds, for each of them,
    // its own state from zero, which becomes its start state, and the sum of its step sizes; float32 tokens over
    // a bfloat16 pool: its start state alone, left by one pass through the row
    int seg;
    float *ws;
    unsigned *status;
};
// Most segments a call can have: rows end inside segments.
#ifdef __CUDACC__
__host__ __device__
#endif
inline long long scan_pieces(long long T, int seg, int batch) { return T / seg + batch; }
// Short rows (max_len bounds them), and any.  vec: four channels may be moved as one
// vector everywhere.
cudaError_t launch_scan_step(const ScanParams &p, bool tok_bf16, bool dt_bf16, bool vec, cudaStream_t s);
cudaError_t launch_scan(const ScanParams &p, bool tok_bf16, bool dt_bf16, bool vec, cudaStream_t s);
cudaError_t launch_scan_bb(const ScanParams &p, bool vec, cudaStream_t s);  // bfloat16 tokens and step sizes
cudaError_t launch_scan_bf(const ScanParams &p, bool vec, cudaStream_t s);  // bfloat16 tokens, float32 step sizes
cudaError_t launch_scan_ff(const ScanParams &p, bool vec, cudaStream_t s);  // float32, float32 pool
cudaError_t launch_scan_fx(const ScanParams &p, bool vec, cudaStream_t s);  // float32, bfloat16 pool
cudaError_t launch_scan_join(const ScanParams &p, cudaStream_t s);
cudaError_t launch_scan_step_bb(const ScanParams &p, bool vec, cudaStream_t s);
cudaError_t launch_scan_step_bf(const ScanParams &p, bool vec, cudaStream_t s);
cudaError_t launch_scan_step_ff(const ScanParams &p, bool vec, cudaStream_t s);

// One verification of drafts, after validation.
struct AcceptParams {
    int batch, vocab, width;
    long long T;
    const void *target, *draft;
    long long t_ts, d_ts;
    const int *tokens, *offsets;
    const float *u, *row_u;
    int *out;
    long long o_ts;
    int *counts;
    unsigned *status;
};
cudaError_t launch_accept(const AcceptParams &p, bool bf16, cudaStream_t s);

#ifdef __CUDACC__
// A skipped row's output: zeros over rows x width elements (a multiple of 8 up to
// 128), by the whole CTA of at least 32 threads.  vec: rows are 16-byte vectors.
template <typename TT>
__device__ __forceinline__ void clear_rows(TT *out, long long row_stride, int rows, int width, bool vec, int tid, int threads) {
    const int across = width / 8, down = threads / across, c = tid % across * 8;
    if (tid >= across * down) return;
    for (unsigned t = (unsigned)(tid / across); t < (unsigned)rows; t += (unsigned)down) {
        TT *const to = out + (long long)t * row_stride + c;
        if (vec) {
            for (int j = 0; j < 8 * (int)sizeof(TT) / 16; ++j) reinterpret_cast<uint4 *>(to)[j] = make_uint4(0, 0, 0, 0);
        } else {
            for (int j = 0; j < 8; ++j) to[j] = TT(0);  // all bits zero in either type
        }
    }
}
#endif

}  // namespace gdr
