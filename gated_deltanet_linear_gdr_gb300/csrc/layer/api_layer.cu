// C ABI of the layer operators: argument checks, lowering and the choice of
// form.  As in api.cu, every check runs before anything is launched.
#include <cmath>
#include <cstdarg>
#include <cstdio>

#include "layer_internal.h"

namespace {

int fail(int code, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return gdr::api_fail(code, buf);
}

bool aligned(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool is_dtype(int d) { return d == GDR_F32 || d == GDR_BF16; }
int esize(int d) { return d == GDR_BF16 ? 2 : 4; }

// Whether rows at p, with these strides in elements, may be moved as 16-byte vectors.
bool vector_rows(const void *p, int dtype, int64_t ts, int64_t hs) {
    const int64_t es = esize(dtype);
    return aligned(p, 16) && (ts * es) % 16 == 0 && (hs * es) % 16 == 0;
}

int check_linattn_sizes(const gdr_linattn_args *a, const char *fn) {
    if (!a) return fail(GDR_ERR_INVALID_ARG, "%s: args is NULL", fn);
    if (a->batch < 0) return fail(GDR_ERR_INVALID_ARG, "%s: batch %d < 0", fn, a->batch);
    if (a->nv <= 0 || a->nk <= 0)
        return fail(GDR_ERR_INVALID_ARG, "%s: nv=%d, nk=%d must be positive", fn, a->nv, a->nk);
    if (a->nv % a->nk != 0)
        return fail(GDR_ERR_INVALID_ARG, "%s: nv=%d is not a multiple of nk=%d", fn, a->nv, a->nk);
    if (a->K < 16 || a->K > 128 || a->K % 16 || a->V < 16 || a->V > 256 || a->V % 16)
        return fail(GDR_ERR_UNSUPPORTED, "%s: K=%d must be a multiple of 16 up to 128, V=%d one up to 256", fn, a->K,
                    a->V);
    if (!is_dtype(a->token_dtype) || !is_dtype(a->state_dtype))
        return fail(GDR_ERR_UNSUPPORTED, "%s: token_dtype %d, state_dtype %d (GDR_F32 or GDR_BF16)", fn,
                    a->token_dtype, a->state_dtype);
    if (a->total_tokens < 0) return fail(GDR_ERR_INVALID_ARG, "%s: total_tokens < 0", fn);
    if (a->total_tokens >= (1ll << 31))
        return fail(GDR_ERR_UNSUPPORTED, "%s: total_tokens must be < 2^31", fn);
    if ((int64_t)a->batch * a->nv * 4 >= (1ll << 31))  // units: up to four column tiles a head
        return fail(GDR_ERR_UNSUPPORTED, "%s: batch * nv must be < 2^29", fn);
    return GDR_OK;
}

int check_linattn(const gdr_linattn_args *a, const char *fn) {
    int rc = check_linattn_sizes(a, fn);
    if (rc) return rc;
    if (a->batch == 0) return GDR_OK;
    if (!a->state || !a->slot_idx || !a->offsets || !a->decay)
        return fail(GDR_ERR_INVALID_ARG, "%s: state/slot_idx/offsets/decay is NULL", fn);
    if (a->decay_stride < 0) return fail(GDR_ERR_INVALID_ARG, "%s: decay_stride < 0", fn);
    if (a->max_slots <= 0) return fail(GDR_ERR_INVALID_ARG, "%s: max_slots %lld", fn, (long long)a->max_slots);
    if (a->state_vdim_stride != 1)
        return fail(GDR_ERR_UNSUPPORTED, "%s: state_vdim_stride must be 1 (got %lld)", fn,
                    (long long)a->state_vdim_stride);
    if (a->state_slot_stride <= 0 || a->state_head_stride <= 0 || a->state_kdim_stride <= 0)
        return fail(GDR_ERR_INVALID_ARG, "%s: state strides must be positive", fn);
    const int64_t es = esize(a->state_dtype);
    if (!aligned(a->state, 16) || (a->state_slot_stride * es) % 16 || (a->state_head_stride * es) % 16 ||
        (a->state_kdim_stride * es) % 16)
        return fail(GDR_ERR_UNSUPPORTED, "%s: state base and strides must be 16-byte aligned", fn);
    if (a->total_tokens > 0) {
        if (!a->q || !a->k || !a->v || !a->out) return fail(GDR_ERR_INVALID_ARG, "%s: q/k/v/out is NULL", fn);
        if (a->q_seq_stride < 0 || a->q_head_stride < 0 || a->k_seq_stride < 0 || a->k_head_stride < 0 ||
            a->v_seq_stride < 0 || a->v_head_stride < 0)
            return fail(GDR_ERR_INVALID_ARG, "%s: q/k/v strides must not be negative", fn);
        if (a->out_seq_stride <= 0 || a->out_head_stride <= 0)
            return fail(GDR_ERR_INVALID_ARG, "%s: output strides must be positive", fn);
        const uintptr_t e = esize(a->token_dtype);
        if (!aligned(a->q, e) || !aligned(a->k, e) || !aligned(a->v, e) || !aligned(a->out, e))
            return fail(GDR_ERR_UNSUPPORTED, "%s: q/k/v/out must be aligned to their elements", fn);
    }
    if (a->workspace_bytes < 0) return fail(GDR_ERR_INVALID_ARG, "%s: workspace_bytes < 0", fn);
    if (a->workspace && !aligned(a->workspace, 16))
        return fail(GDR_ERR_UNSUPPORTED, "%s: workspace must be 16-byte aligned", fn);
    return GDR_OK;
}

// Whether rows are short enough for k_la_small.cu, whose time grows with a row's
// 16-token pieces, where k_la_chunk.cu's for a unit hardly does.  Measured, 64 rows x
// 16 heads of K x V, us, small against chunk: 64 x 64 40 / 50 at 96 tokens, 50 / 48 at
// 128; 64 x 128 38 / 42 at 48, 46 / 42 at 64 (128 x 64: 38 / 48, 46 / 46); 128 x 128,
// bfloat16 pool, 42 / 48 at 32, 54 / 48 at 48; float32 pool 40 / 50 at 16, 58 / 52 at 32.
// Where all units run at once (two a multiprocessor) the longest row, by the caller's
// bound, decides; where they queue, its mean with the average: 52 rows of 1 to 64 x 21
// heads of 64 x 128 46 / 44, of 1 to 96 58 / 50, 8 rows of 1 to 128 x 16 of 64 x 64 19 / 15.
bool short_rows(const gdr_linattn_args *a) {
    const bool wide_k = a->K > 64, wide_v = a->V > 64;
    const int most = wide_k && wide_v ? (a->state_dtype == GDR_BF16 ? 32 : 16) : wide_k || wide_v ? 48 : 96;
    if (a->max_row_len <= 0 || a->batch <= 0) return false;
    const double units = (double)a->batch * a->nv * ((a->V + 127) / 128), longest = (double)a->max_row_len;
    const double mean = std::fmin((double)a->total_tokens / a->batch, longest);
    return (units > 2 * 152 ? 0.5 * (longest + mean) : longest) <= most;
}

bool takes_pieces(const gdr_linattn_args *a, bool tok_vec) {
    return a->token_dtype == GDR_BF16 && tok_vec && a->max_row_len > 1 && short_rows(a);
}

bool takes_chunks(const gdr_linattn_args *a, bool tok_vec) {
    return a->token_dtype == GDR_BF16 && tok_vec && a->total_tokens > 0 && a->max_row_len != 1 && !short_rows(a);
}

bool token_vectors(const gdr_linattn_args *a) {
    return vector_rows(a->q, a->token_dtype, a->q_seq_stride, a->q_head_stride) &&
           vector_rows(a->k, a->token_dtype, a->k_seq_stride, a->k_head_stride) &&
           vector_rows(a->v, a->token_dtype, a->v_seq_stride, a->v_head_stride) &&
           vector_rows(a->out, a->token_dtype, a->out_seq_stride, a->out_head_stride);
}

gdr::LaParams lower(const gdr_linattn_args *a, unsigned *status) {
    gdr::LaParams p{};
    p.batch = a->batch;
    p.nv = a->nv;
    p.nk = a->nk;
    p.r = a->nv / a->nk;
    p.K = a->K;
    p.V = a->V;
    p.tiles = (a->V + 127) / 128;
    p.decay_is_log = a->decay_is_log ? 1 : 0;
    p.T = a->total_tokens;
    p.max_len = a->max_row_len;
    p.q = a->q;
    p.q_ts = a->q_seq_stride;
    p.q_hs = a->q_head_stride;
    p.k = a->k;
    p.k_ts = a->k_seq_stride;
    p.k_hs = a->k_head_stride;
    p.v = a->v;
    p.v_ts = a->v_seq_stride;
    p.v_hs = a->v_head_stride;
    p.decay = a->decay;
    p.decay_s = a->decay_stride;
    p.scale = a->scale > 0.0f ? a->scale : (float)(1.0 / std::sqrt((double)a->K));
    p.out = a->out;
    p.o_ts = a->out_seq_stride;
    p.o_hs = a->out_head_stride;
    p.state = a->state;
    p.st_slot = a->state_slot_stride;
    p.st_head = a->state_head_stride;
    p.st_k = a->state_kdim_stride;
    p.max_slots = a->max_slots;
    p.slot_idx = a->slot_idx;
    p.offsets = a->offsets;
    p.tok_vec = token_vectors(a);
    p.status = status;
    return p;
}

// Tokens a segment for rows that are cut, or 0.  One CTA does a (row, head,
// column tile) from end to end, so a call lasts about as many chunks as its
// longest row has, or as the fullest SM gets, and three chunks' time to fill
// and drain a unit.  Cut rows spread evenly, and cost a pass over k and v for
// the segments' own states (with the slower clock and memory of a full GPU,
// 0.75 of a chunk's time a chunk), two more launches and the states' traffic
// (12 chunks' time).  Measured, cut against whole, K = V = 128, bfloat16 pool:
// 16383 tokens x 32 heads 183 us against 365, 4000 x 32 70 / 101, 2000 x 4 36 /
// 54; left whole by this rule: 1000 x 16 40 / 33, 2 rows of 2000 x 16 54 / 58,
// 8000 x 64 174 / 191.
int plan_segments(const gdr_linattn_args *a) {
    constexpr double kSms = 152.0, kChunk = 64.0, kStatePass = 0.75, kUnit = 3.0, kExtra = 12.0;
    if (a->batch < 1 || a->batch > 32) return 0;
    const double tiles = (a->V + 127) / 128, heads = a->nv * tiles, T = (double)a->total_tokens;
    const double mean = std::ceil(T / a->batch / kChunk);
    double longest = a->max_row_len > 0 ? std::ceil((double)a->max_row_len / kChunk) : mean;
    if (longest > std::ceil(T / kChunk)) longest = std::ceil(T / kChunk);
    const double waves = std::ceil(a->batch * heads / kSms);
    double best = std::fmax(longest + kUnit, waves * (mean + kUnit));
    int seg = 0;
    for (int n = 2; n <= 64; ++n) {
        const double chunks = std::ceil(longest / n);
        if (chunks < 4) break;
        // a row's last segment is half full on average
        const double units = std::ceil(T / (chunks * kChunk) + 0.5 * (a->batch - 1)) * heads;
        const double cost = std::ceil(units / kSms) * (chunks * (1 + kStatePass) + 2 * kUnit) + kExtra;
        if (cost < 0.9 * best) {
            best = cost / 0.9;
            seg = (int)(chunks * kChunk);
        }
    }
    return seg;
}

int64_t segments_bytes(const gdr_linattn_args *a, int seg) {
    return (a->total_tokens / seg + a->batch) * (int64_t)a->nv * a->K * a->V * 4;
}

int launched(cudaError_t e, const char *fn) {
    if (e != cudaSuccess) return fail(GDR_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
    return gdr::api_ok();
}

}  // namespace

extern "C" {

int64_t gdr_linattn_workspace_bytes(const gdr_linattn_args *a) {
    const int rc = check_linattn_sizes(a, "gdr_linattn_workspace_bytes");
    if (rc) return rc;
    const int seg = takes_chunks(a, token_vectors(a)) ? plan_segments(a) : 0;
    return seg ? segments_bytes(a, seg) : 0;
}

int gdr_linattn_fwd(const gdr_linattn_args *a, void *stream) {
    const char *fn = "gdr_linattn_fwd";
    int rc = check_linattn(a, fn);
    if (rc) return rc;
    if (a->batch == 0) return gdr::api_ok();
    unsigned *st = nullptr;
    if ((rc = gdr::api_status(&st))) return rc;
    const gdr::LaParams p = lower(a, st);
    if (takes_pieces(a, p.tok_vec))
        return launched(gdr::launch_la_small(p, a->state_dtype == GDR_BF16, static_cast<cudaStream_t>(stream)), fn);
    if (takes_chunks(a, p.tok_vec)) {
        int seg = plan_segments(a);
        if (seg && (!a->workspace || a->workspace_bytes < segments_bytes(a, seg))) seg = 0;
        bool used = false;
        const cudaError_t e = gdr::launch_la_chunk(p, a->state_dtype == GDR_BF16, seg, a->workspace,
                                                   static_cast<cudaStream_t>(stream), &used);
        if (used || e != cudaSuccess) return launched(e, fn);
    }
    return launched(gdr::launch_la_step(p, a->token_dtype == GDR_BF16, a->state_dtype == GDR_BF16,
                                        static_cast<cudaStream_t>(stream)),
                    fn);
}

int gdr_block_norm(const gdr_norm_args *a, void *stream) {
    const char *fn = "gdr_block_norm";
    if (!a) return fail(GDR_ERR_INVALID_ARG, "%s: args is NULL", fn);
    if (a->tokens < 0 || a->heads <= 0 || a->D <= 0)
        return fail(GDR_ERR_INVALID_ARG, "%s: tokens=%lld, heads=%d, D=%d", fn, (long long)a->tokens, a->heads, a->D);
    if (a->D > 16384) return fail(GDR_ERR_UNSUPPORTED, "%s: D=%d is over 16384", fn, a->D);
    if (a->tokens * a->heads >= (1ll << 31))
        return fail(GDR_ERR_UNSUPPORTED, "%s: tokens * heads must be < 2^31", fn);
    if (!is_dtype(a->x_dtype) || !is_dtype(a->gate_dtype) || !is_dtype(a->residual_dtype) || !is_dtype(a->out_dtype))
        return fail(GDR_ERR_UNSUPPORTED, "%s: dtypes must be GDR_F32 or GDR_BF16", fn);
    if (a->activation < 0 || a->activation > 2)
        return fail(GDR_ERR_INVALID_ARG, "%s: activation %d (0 none, 1 SiLU, 2 sigmoid)", fn, a->activation);
    if (!(a->eps >= 0.0f)) return fail(GDR_ERR_INVALID_ARG, "%s: eps must be >= 0", fn);
    if (a->tokens == 0) return gdr::api_ok();
    if (!a->x && !a->residual) return fail(GDR_ERR_INVALID_ARG, "%s: x and residual are both NULL", fn);
    if (!a->x && (a->gate || a->has_post_norm))
        return fail(GDR_ERR_INVALID_ARG, "%s: a gate or a post norm needs x", fn);
    if (a->gate_first && !(a->gate && a->has_post_norm))
        return fail(GDR_ERR_INVALID_ARG, "%s: gate_first needs a gate and a post norm", fn);
    if (!a->out && !a->residual_out) return fail(GDR_ERR_INVALID_ARG, "%s: out and residual_out are both NULL", fn);
    if (a->gate && a->gate_elem_stride != 0 && a->gate_elem_stride != 1)
        return fail(GDR_ERR_UNSUPPORTED, "%s: gate_elem_stride must be 0 or 1 (got %lld)", fn,
                    (long long)a->gate_elem_stride);
    if ((a->x && (a->x_seq_stride < 0 || a->x_head_stride < 0)) ||
        (a->gate && (a->gate_seq_stride < 0 || a->gate_head_stride < 0)) ||
        (a->residual && (a->residual_seq_stride < 0 || a->residual_head_stride < 0)))
        return fail(GDR_ERR_INVALID_ARG, "%s: input strides must not be negative", fn);
    const bool more_tokens = a->tokens > 1, more_heads = a->heads > 1;
    if ((a->out && ((more_tokens && a->out_seq_stride <= 0) || (more_heads && a->out_head_stride <= 0))) ||
        (a->residual_out &&
         ((more_tokens && a->residual_out_seq_stride <= 0) || (more_heads && a->residual_out_head_stride <= 0))))
        return fail(GDR_ERR_INVALID_ARG, "%s: output strides must be positive", fn);
    if (!aligned(a->x, esize(a->x_dtype)) || !aligned(a->gate, esize(a->gate_dtype)) ||
        !aligned(a->residual, esize(a->residual_dtype)) || !aligned(a->residual_out, esize(a->residual_dtype)) ||
        !aligned(a->out, esize(a->out_dtype)) || !aligned(a->post_weight, 4) || !aligned(a->pre_weight, 4))
        return fail(GDR_ERR_UNSUPPORTED, "%s: buffers must be aligned to their elements", fn);

    gdr::NormParams p{};
    p.rows = (unsigned)(a->tokens * a->heads);
    p.heads_div = gdr::FastDiv((unsigned)a->heads);
    p.D = a->D;
    p.x_bf16 = a->x_dtype == GDR_BF16;
    p.gate_bf16 = a->gate_dtype == GDR_BF16;
    p.res_bf16 = a->residual_dtype == GDR_BF16;
    p.out_bf16 = a->out_dtype == GDR_BF16;
    p.act = a->activation;
    p.gate_first = a->gate_first ? 1 : 0;
    p.post = a->has_post_norm ? 1 : 0;
    p.pre = a->has_pre_norm ? 1 : 0;
    p.centered = a->centered ? 1 : 0;
    p.eps = a->eps;
    p.scale = a->residual_scale;
    p.inv_d = 1.0f / (float)a->D;
    p.x = a->x;
    p.x_ts = a->x_seq_stride;
    p.x_hs = a->x_head_stride;
    p.gate = a->gate;
    p.g_ts = a->gate_seq_stride;
    p.g_hs = a->gate_head_stride;
    p.g_es = a->gate_elem_stride;
    p.res = a->residual;
    p.r_ts = a->residual_seq_stride;
    p.r_hs = a->residual_head_stride;
    p.res_out = a->residual_out;
    p.ro_ts = a->residual_out_seq_stride;
    p.ro_hs = a->residual_out_head_stride;
    p.out = a->out;
    p.o_ts = a->out_seq_stride;
    p.o_hs = a->out_head_stride;
    p.post_w = a->post_weight;
    p.pre_w = a->pre_weight;
    // whether everything may be moved as vectors of `width` elements
    const auto by = [&](int width) {
        const auto rows = [&](const void *base, int dtype, int64_t ts, int64_t hs) {
            const int es = esize(dtype);
            return !base || (aligned(base, width * es < 16 ? width * es : 16) && ts % width == 0 && hs % width == 0);
        };
        return a->D % width == 0 && rows(a->x, a->x_dtype, p.x_ts, p.x_hs) &&
               (p.g_es == 0 || rows(a->gate, a->gate_dtype, p.g_ts, p.g_hs)) &&
               rows(a->residual, a->residual_dtype, p.r_ts, p.r_hs) &&
               rows(a->residual_out, a->residual_dtype, p.ro_ts, p.ro_hs) && rows(a->out, a->out_dtype, p.o_ts, p.o_hs) &&
               rows(a->post_weight, GDR_F32, 0, 0) && rows(a->pre_weight, GDR_F32, 0, 0);
    };
    const int vec = by(8) ? 8 : by(2) ? 2 : 1;
    return launched(gdr::launch_norm(p, vec, static_cast<cudaStream_t>(stream)), fn);
}

}  // extern "C"
