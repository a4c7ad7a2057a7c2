// C ABI of the state space layer's operators (short convolution, selective scan)
// and of the verification of drafts: argument checks, lowering and the cut of
// long rows.  As in api.cu, every check runs before anything is launched.
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

int launched(cudaError_t e, const char *fn) {
    if (e != cudaSuccess) return fail(GDR_ERR_CUDA, "%s: launch failed: %s", fn, cudaGetErrorString(e));
    return gdr::api_ok();
}

bool aligned(const void *p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool is_dtype(int d) { return d == GDR_F32 || d == GDR_BF16; }
int64_t esize(int d) { return d == GDR_BF16 ? 2 : 4; }

// Whether rows at p, with these strides in elements, may be moved as `bytes`-byte vectors.
bool vector_rows(const void *p, int dtype, int64_t bytes, int64_t a, int64_t b = 0, int64_t c = 0) {
    const int64_t es = esize(dtype);
    return aligned(p, (uintptr_t)bytes) && (a * es) % bytes == 0 && (b * es) % bytes == 0 && (c * es) % bytes == 0;
}

int check_tokens(int64_t total, int32_t batch, const char *fn) {
    if (batch < 0) return fail(GDR_ERR_INVALID_ARG, "%s: batch %d < 0", fn, batch);
    if (batch > (1 << 27)) return fail(GDR_ERR_UNSUPPORTED, "%s: batch must be at most 2^27", fn);
    if (total < 0) return fail(GDR_ERR_INVALID_ARG, "%s: total_tokens < 0", fn);
    if (total >= (1ll << 31)) return fail(GDR_ERR_UNSUPPORTED, "%s: total_tokens must be < 2^31", fn);
    return GDR_OK;
}

// Whether two buffers of rows (`width` elements, `rows` of them, strides in elements) have
// bytes in common.  Rows of one stride may lie between one another's (parts of one
// projection); with different strides their whole ranges must be apart.
bool rows_overlap(const void *a, int64_t as, const void *b, int64_t bs, int64_t rows, int64_t width, int64_t es) {
    if (rows <= 0 || width <= 0) return false;
    const int64_t pa = (int64_t)reinterpret_cast<uintptr_t>(a), pb = (int64_t)reinterpret_cast<uintptr_t>(b);
    const int64_t ea = pa + ((rows - 1) * as + width) * es, eb = pb + ((rows - 1) * bs + width) * es;
    if (ea <= pb || eb <= pa) return false;
    if (rows == 1 || as != bs || as < width) return true;
    int64_t d = (pb - pa) % (as * es);
    if (d < 0) d += as * es;
    return d < width * es || d > (as - width) * es;
}

// A tensor of [tokens, heads] runs of bytes, strides in bytes.
struct Runs {
    int64_t at, tokens, token_stride, heads, head_stride, run;
};
Runs runs(const void *p, int dtype, int64_t tokens, int64_t ts, int64_t heads, int64_t hs, int64_t width) {
    const int64_t es = esize(dtype);
    if (ts == 0) tokens = 1;  // all of them the same run
    if (hs == 0) heads = 1;
    return {(int64_t)reinterpret_cast<uintptr_t>(p), tokens, ts * es, heads, hs * es, width * es};
}

// Whether two such tensors have bytes in common.  Exact where they are parts of one projection (tokens of one stride, and
// heads of one stride or apart within a token, or the other way round); else their whole ranges must be apart.
bool runs_overlap(const Runs &a, const Runs &b) {
    struct Level {
        int64_t n, stride;
    };
    const bool tokens_outside = a.token_stride * (a.tokens > 1) >= a.head_stride * (a.heads > 1);
    const Level ao = tokens_outside ? Level{a.tokens, a.token_stride} : Level{a.heads, a.head_stride};
    const Level ai = tokens_outside ? Level{a.heads, a.head_stride} : Level{a.tokens, a.token_stride};
    const Level bo = tokens_outside ? Level{b.tokens, b.token_stride} : Level{b.heads, b.head_stride};
    const Level bi = tokens_outside ? Level{b.heads, b.head_stride} : Level{b.tokens, b.token_stride};
    const auto length = [](const Level &l, int64_t each) { return (l.n - 1) * l.stride + each; };
    const auto apart = [](int64_t la, int64_t lb, int64_t d) { return d >= la || -d >= lb; };  // b begins d behind a
    const auto one_stride = [](const Level &x, const Level &y, int64_t lx, int64_t ly) {
        const int64_t stride = x.n > 1 ? x.stride : y.stride;
        return (x.n > 1 || y.n > 1) && (x.n == 1 || y.n == 1 || x.stride == y.stride) && lx <= stride && ly <= stride ? stride : 0;
    };
    // runs of two inner levels, the second's first one d behind the first's
    const auto inner = [&](int64_t d) {
        if (apart(length(ai, a.run), length(bi, b.run), d)) return false;
        const int64_t stride = one_stride(ai, bi, a.run, b.run);
        if (!stride) return true;
        const int64_t m = (d % stride + stride) % stride;
        return !apart(a.run, b.run, m) || !apart(a.run, b.run, m - stride);
    };
    const int64_t la = length(ai, a.run), lb = length(bi, b.run), d = b.at - a.at;
    if (apart(length(ao, la), length(bo, lb), d)) return false;
    if (ao.n == 1 && bo.n == 1) return inner(d);
    const int64_t stride = one_stride(ao, bo, la, lb);
    if (!stride) return true;
    const int64_t m = (d % stride + stride) % stride;
    return inner(m) || inner(m - stride);
}

int check_conv(const gdr_short_conv_args *a, const char *fn) {
    if (!a) return fail(GDR_ERR_INVALID_ARG, "%s: args is NULL", fn);
    int rc = check_tokens(a->total_tokens, a->batch, fn);
    if (rc) return rc;
    if (a->channels <= 0) return fail(GDR_ERR_INVALID_ARG, "%s: channels %d", fn, a->channels);
    if (a->channels > (1 << 28)) return fail(GDR_ERR_UNSUPPORTED, "%s: channels must be at most 2^28", fn);
    if (a->width < 1 || a->width > 4) return fail(GDR_ERR_UNSUPPORTED, "%s: width %d must be 1 to 4", fn, a->width);
    if (a->activation < 0 || a->activation > 1)
        return fail(GDR_ERR_INVALID_ARG, "%s: activation %d (0 none, 1 SiLU)", fn, a->activation);
    if (!is_dtype(a->token_dtype) || !is_dtype(a->state_dtype))
        return fail(GDR_ERR_UNSUPPORTED, "%s: dtypes must be GDR_F32 or GDR_BF16", fn);
    if (a->batch == 0) return GDR_OK;
    if (!a->slot_idx || !a->offsets || !a->weight)
        return fail(GDR_ERR_INVALID_ARG, "%s: slot_idx/offsets/weight is NULL", fn);
    if (a->max_slots <= 0) return fail(GDR_ERR_INVALID_ARG, "%s: max_slots %lld", fn, (long long)a->max_slots);
    if (a->weight_chan_stride < 0 || a->weight_tap_stride < 0)
        return fail(GDR_ERR_INVALID_ARG, "%s: weight strides must not be negative", fn);
    if (!aligned(a->weight, 4) || !aligned(a->bias, 4))
        return fail(GDR_ERR_UNSUPPORTED, "%s: weight and bias must be aligned to their elements", fn);
    if (a->counts && !a->keep_state) return fail(GDR_ERR_INVALID_ARG, "%s: counts without keep_state", fn);
    if (!a->out && !a->keep_state) return fail(GDR_ERR_INVALID_ARG, "%s: neither out nor keep_state", fn);
    if (a->width > 1) {
        if (!a->conv_state) return fail(GDR_ERR_INVALID_ARG, "%s: conv_state is NULL", fn);
        if (a->state_slot_stride <= 0 || a->state_chan_stride <= 0 || a->state_tap_stride <= 0)
            return fail(GDR_ERR_INVALID_ARG, "%s: state strides must be positive", fn);
        if (!aligned(a->conv_state, esize(a->state_dtype)))
            return fail(GDR_ERR_UNSUPPORTED, "%s: conv_state must be aligned to its elements", fn);
    }
    if (a->total_tokens > 0) {
        const int64_t es = esize(a->token_dtype);
        if (!a->x) return fail(GDR_ERR_INVALID_ARG, "%s: x is NULL", fn);
        if (a->x_seq_stride < 0) return fail(GDR_ERR_INVALID_ARG, "%s: x_seq_stride < 0", fn);
        if (!aligned(a->x, es) || !aligned(a->out, es))
            return fail(GDR_ERR_UNSUPPORTED, "%s: x and out must be aligned to their elements", fn);
        if (a->out) {
            if (a->total_tokens > 1 && a->out_seq_stride < a->channels)
                return fail(GDR_ERR_INVALID_ARG, "%s: out_seq_stride must be at least channels", fn);
            if (rows_overlap(a->x, a->x_seq_stride, a->out, a->out_seq_stride, a->total_tokens, a->channels, es))
                return fail(GDR_ERR_INVALID_ARG, "%s: out lies on x", fn);
        }
    }
    return GDR_OK;
}

int check_scan_sizes(const gdr_scan_args *a, const char *fn) {
    if (!a) return fail(GDR_ERR_INVALID_ARG, "%s: args is NULL", fn);
    int rc = check_tokens(a->total_tokens, a->batch, fn);
    if (rc) return rc;
    if (a->total_tokens > (1ll << 31) - 32)  // tokens are counted in whole chunks
        return fail(GDR_ERR_UNSUPPORTED, "%s: total_tokens must be at most 2^31 - 32", fn);
    if (a->nv <= 0 || a->nk <= 0)
        return fail(GDR_ERR_INVALID_ARG, "%s: nv=%d, nk=%d must be positive", fn, a->nv, a->nk);
    if (a->nv % a->nk != 0)
        return fail(GDR_ERR_INVALID_ARG, "%s: nv=%d is not a multiple of nk=%d", fn, a->nv, a->nk);
    if (a->K < 1 || a->K > 128 || a->V < 1)
        return fail(GDR_ERR_UNSUPPORTED, "%s: K=%d must be 1 to 128, V=%d at least 1", fn, a->K, a->V);
    if ((int64_t)a->nv * a->V > (1 << 24))
        return fail(GDR_ERR_UNSUPPORTED, "%s: nv * V must be at most 2^24", fn);
    if (!is_dtype(a->token_dtype) || !is_dtype(a->state_dtype) ||
        (a->dt_dtype != a->token_dtype && a->dt_dtype != GDR_F32))
        return fail(GDR_ERR_UNSUPPORTED,
                    "%s: token_dtype %d, dt_dtype %d, state_dtype %d (GDR_F32 or GDR_BF16; dt the tokens' or GDR_F32)", fn,
                    a->token_dtype, a->dt_dtype, a->state_dtype);
    return GDR_OK;
}

int check_scan(const gdr_scan_args *a, const char *fn) {
    int rc = check_scan_sizes(a, fn);
    if (rc) return rc;
    if (a->batch == 0) return GDR_OK;
    if (!a->state || !a->slot_idx || !a->offsets || !a->A)
        return fail(GDR_ERR_INVALID_ARG, "%s: state/slot_idx/offsets/A is NULL", fn);
    if (a->max_slots <= 0) return fail(GDR_ERR_INVALID_ARG, "%s: max_slots %lld", fn, (long long)a->max_slots);
    if (a->state_vdim_stride != 1 && a->V > 1)
        return fail(GDR_ERR_UNSUPPORTED, "%s: state_vdim_stride must be 1 (got %lld)", fn,
                    (long long)a->state_vdim_stride);
    if (a->state_slot_stride <= 0 || a->state_head_stride <= 0 || a->state_kdim_stride <= 0)
        return fail(GDR_ERR_INVALID_ARG, "%s: state strides must be positive", fn);
    if (a->A_head_stride < 0 || a->A_kdim_stride < 0 || a->A_vdim_stride < 0 || a->D_head_stride < 0 ||
        a->D_vdim_stride < 0 || a->dt_bias_head_stride < 0 || a->dt_bias_vdim_stride < 0)
        return fail(GDR_ERR_INVALID_ARG, "%s: A, D and dt_bias strides must not be negative", fn);
    if (!aligned(a->state, esize(a->state_dtype)) || !aligned(a->A, 4) || !aligned(a->D, 4) || !aligned(a->dt_bias, 4))
        return fail(GDR_ERR_UNSUPPORTED, "%s: state, A, D and dt_bias must be aligned to their elements", fn);
    if (a->counts && !a->keep_state) return fail(GDR_ERR_INVALID_ARG, "%s: counts without keep_state", fn);
    if (!a->out && !a->keep_state) return fail(GDR_ERR_INVALID_ARG, "%s: neither out nor keep_state", fn);
    if (a->total_tokens > 0) {
        if (!a->x || !a->dt || !a->B || (a->out && !a->C)) return fail(GDR_ERR_INVALID_ARG, "%s: x/dt/B/C is NULL", fn);
        if (a->x_seq_stride < 0 || a->x_head_stride < 0 || a->dt_seq_stride < 0 || a->dt_head_stride < 0 ||
            a->B_seq_stride < 0 || a->B_head_stride < 0 || a->C_seq_stride < 0 || a->C_head_stride < 0 ||
            a->z_seq_stride < 0 || a->z_head_stride < 0)
            return fail(GDR_ERR_INVALID_ARG, "%s: x/dt/B/C/z strides must not be negative", fn);
        if (a->dt_elem_stride != 0 && a->dt_elem_stride != 1)
            return fail(GDR_ERR_UNSUPPORTED, "%s: dt_elem_stride must be 0 or 1 (got %lld)", fn,
                        (long long)a->dt_elem_stride);
        if (a->out && ((a->total_tokens > 1 && a->out_seq_stride <= 0) || (a->nv > 1 && a->out_head_stride <= 0)))
            return fail(GDR_ERR_INVALID_ARG, "%s: output strides must be positive", fn);
        const uintptr_t e = esize(a->token_dtype);
        if (!aligned(a->x, e) || !aligned(a->B, e) || !aligned(a->C, e) || !aligned(a->z, e) || !aligned(a->out, e) ||
            !aligned(a->dt, esize(a->dt_dtype)))
            return fail(GDR_ERR_UNSUPPORTED, "%s: x/dt/B/C/z/out must be aligned to their elements", fn);
    }
    if (a->workspace_bytes < 0) return fail(GDR_ERR_INVALID_ARG, "%s: workspace_bytes < 0", fn);
    if (a->workspace && !aligned(a->workspace, 16))
        return fail(GDR_ERR_UNSUPPORTED, "%s: workspace must be 16-byte aligned", fn);
    if (a->out && a->total_tokens > 0) {
        const auto wide = [&](const void *p, int64_t ts, int64_t hs) {
            return runs(p, a->token_dtype, a->total_tokens, ts, a->nv, hs, a->V);
        };
        const Runs out = wide(a->out, a->out_seq_stride, a->out_head_stride);
        const auto lies_on = [&](const void *p, int64_t ts, int64_t hs) {  // x or z, but not their place itself
            const bool itself = p == a->out && (ts == a->out_seq_stride || a->total_tokens == 1) &&
                                (hs == a->out_head_stride || a->nv == 1);
            return p && !itself && runs_overlap(out, wide(p, ts, hs));
        };
        const char *on = nullptr;
        if (lies_on(a->x, a->x_seq_stride, a->x_head_stride)) on = "x";
        else if (lies_on(a->z, a->z_seq_stride, a->z_head_stride)) on = "z";
        else if (runs_overlap(out, runs(a->dt, a->dt_dtype, a->total_tokens, a->dt_seq_stride, a->nv, a->dt_head_stride,
                                        a->dt_elem_stride ? a->V : 1))) on = "dt";
        else if (runs_overlap(out, runs(a->B, a->token_dtype, a->total_tokens, a->B_seq_stride, a->nk, a->B_head_stride, a->K))) on = "B";
        else if (runs_overlap(out, runs(a->C, a->token_dtype, a->total_tokens, a->C_seq_stride, a->nk, a->C_head_stride, a->K))) on = "C";
        if (on) return fail(GDR_ERR_INVALID_ARG, "%s: out lies on %s", fn, on);
    }
    return GDR_OK;
}

// Rows up to here go token by token (k_scan_step.cuh), longer ones by chunks (k_scan.cuh).  Measured, 64 rows x 32
// heads of 128 channels, 16 states, a pass with outputs and one without, us, steps against chunks: rows of 2
// 30 / 100, of 8 62 / 107, of 12 88 / 125, of 16 113 / 127.
constexpr int kShortRow = 16;

// float32 tokens over a bfloat16 pool: what a call leaves is rounded so that a state's last bit counts (scan_device.cuh),
// and joined segments would have others than the row's own order of operations.  The states of a cut row go through it
// in its order, eight of them a block, and only the outputs are computed by segments.
bool scan_ordered(const gdr_scan_args *a) { return a->token_dtype == GDR_F32 && a->state_dtype == GDR_BF16; }

// Tokens a segment for rows that are cut, or 0.  A block does 64 channels of a row from end to end, so a call
// lasts as long as its longest row, or as the fullest multiprocessor; a token of a block that has its
// multiprocessor to itself takes 0.6 of the time of one that shares it with a second.  Cut rows spread evenly, and
// cost a pass for the segments' own states (0.65 of a token's time a token), 48 tokens' time a segment to
// begin and end and 250 tokens' for two more launches.  Measured, cut against whole, 16 states, us: 16383 tokens x 2048
// channels 285 (864 tokens a segment; 2048: 330, 304: 320) against 948, 2048 x 2048 53 (256) / 123, 4 rows of 1024 to 4096 x 512 62 / 238;
// left whole by this rule: 2 rows of 4096 x 4096 287 / 237.  Where states go through in order, a token of them takes
// a third of the time of a token of 16 states, less beside more states.  Measured, cut against whole, float32, us: 16383
// tokens x 2048 channels 1200 / 1679, 8192 x 1024 channels x 64 states 734 / 2232, 2500 x 64 channels 158 / 265.
int plan_scan(const gdr_scan_args *a) {
    const bool ordered = scan_ordered(a);
    if (ordered && !a->out) return 0;
    if (a->batch < 1 || a->batch > 32 || !a->total_tokens || (a->max_row_len >= 1 && a->max_row_len <= kShortRow)) return 0;
    const double tiles = a->nk * std::ceil((double)a->nv / a->nk * a->V / 64), T = (double)a->total_tokens;
    const double sms = 152.0, slots = a->K <= 32 ? 2 * sms : sms;
    double longest = a->max_row_len > 0 ? (double)a->max_row_len : std::ceil(T / a->batch);
    if (longest > T) longest = T;
    constexpr double kAlone = 0.6, kFirst = 0.65, kUnit = 48.0, kExtra = 250.0, kStates = 0.34;
    const auto share = [&](double blocks) { return blocks <= sms ? kAlone : 1.0; };
    double best = std::fmax(longest * share(a->batch * tiles), T * tiles / slots);
    const double parts = std::ceil(a->K / 8.0) * tiles;
    const double states = kStates / std::fmax(1.0, a->K / 32.0) * std::fmax(longest, T * parts / sms);
    int seg = 0;
    for (int n = 2; n <= 64; ++n) {
        const double len = std::ceil(longest / n / 8) * 8;
        if (len < 128) break;
        const double blocks = std::ceil(T / len + 0.5 * (a->batch - 1)) * tiles;
        const double main = std::ceil(blocks / slots) * (len + kUnit) * share(blocks);
        const double cost = ordered ? main + states + kExtra / 2 : main * (1 + kFirst) + kExtra;
        if (cost < 0.9 * best) {
            best = cost / 0.9;
            seg = (int)len;
        }
    }
    return seg;
}

int64_t scan_bytes(const gdr_scan_args *a, int seg) {
    return gdr::scan_pieces(a->total_tokens, seg, a->batch) * (int64_t)a->nv * a->V * (a->K + (scan_ordered(a) ? 0 : 1)) * 4;
}

}  // namespace

extern "C" {

int gdr_short_conv(const gdr_short_conv_args *a, void *stream) {
    const char *fn = "gdr_short_conv";
    int rc = check_conv(a, fn);
    if (rc) return rc;
    if (a->batch == 0 || a->total_tokens == 0) return gdr::api_ok();
    gdr::ConvOpParams p{};
    if ((rc = gdr::api_status(&p.status))) return rc;
    p.batch = a->batch;
    p.channels = a->channels;
    p.silu = a->activation;
    p.keep = a->keep_state && a->width > 1;
    p.st_bf16 = a->state_dtype == GDR_BF16;
    p.T = a->total_tokens;
    p.max_len = a->max_row_len;
    p.x = a->x;
    p.x_ts = a->x_seq_stride;
    p.w = a->weight;
    p.w_cs = a->weight_chan_stride;
    p.w_ts = a->weight_tap_stride;
    p.bias = a->bias;
    p.out = a->out;
    p.o_ts = a->out_seq_stride;
    p.state = a->conv_state;
    p.s_slot = a->state_slot_stride;
    p.s_chan = a->state_chan_stride;
    p.s_tap = a->state_tap_stride;
    p.max_slots = a->max_slots;
    p.slot_idx = a->slot_idx;
    p.offsets = a->offsets;
    p.counts = a->counts;
    const int64_t es = esize(a->token_dtype);
    p.vec = a->channels % 4 == 0 && vector_rows(a->x, a->token_dtype, 4 * es, a->x_seq_stride) &&
            (!a->out || vector_rows(a->out, a->token_dtype, 4 * es, a->out_seq_stride));
    p.w_vec = a->weight_tap_stride == 1 && vector_rows(a->weight, GDR_F32, 16, a->weight_chan_stride);
    p.st_run = a->width > 1 && (a->state_tap_stride == 1 || a->width == 2) && a->state_chan_stride == a->width - 1 &&
               vector_rows(a->conv_state, a->state_dtype, 16, a->state_slot_stride);
    return launched(gdr::launch_short_conv(p, a->width, a->token_dtype == GDR_BF16, static_cast<cudaStream_t>(stream)), fn);
}

int64_t gdr_selective_scan_workspace_bytes(const gdr_scan_args *a) {
    const int rc = check_scan_sizes(a, "gdr_selective_scan_workspace_bytes");
    if (rc) return rc;
    const int seg = plan_scan(a);
    return seg ? scan_bytes(a, seg) : 0;
}

int gdr_selective_scan(const gdr_scan_args *a, void *stream) {
    const char *fn = "gdr_selective_scan";
    int rc = check_scan(a, fn);
    if (rc) return rc;
    if (a->batch == 0 || a->total_tokens == 0) return gdr::api_ok();
    gdr::ScanParams p{};
    if ((rc = gdr::api_status(&p.status))) return rc;
    p.batch = a->batch;
    p.nv = a->nv;
    p.nk = a->nk;
    p.r = a->nv / a->nk;
    p.K = a->K;
    p.V = a->V;
    p.softplus = a->dt_softplus ? 1 : 0;
    p.keep = a->keep_state ? 1 : 0;
    p.st_bf16 = a->state_dtype == GDR_BF16;
    p.T = a->total_tokens;
    p.max_len = a->max_row_len;
    p.x = a->x;
    p.x_ts = a->x_seq_stride;
    p.x_hs = a->x_head_stride;
    p.dt = a->dt;
    p.dt_ts = a->dt_seq_stride;
    p.dt_hs = a->dt_head_stride;
    p.dt_es = a->dt_elem_stride;
    p.B = a->B;
    p.B_ts = a->B_seq_stride;
    p.B_hs = a->B_head_stride;
    p.C = a->C;
    p.C_ts = a->C_seq_stride;
    p.C_hs = a->C_head_stride;
    p.z = a->z;
    p.z_ts = a->z_seq_stride;
    p.z_hs = a->z_head_stride;
    p.A = a->A;
    p.a_hs = a->A_head_stride;
    p.a_ks = a->A_kdim_stride;
    p.a_vs = a->A_vdim_stride;
    p.D = a->D;
    p.d_hs = a->D_head_stride;
    p.d_vs = a->D_vdim_stride;
    p.bias = a->dt_bias;
    p.b_hs = a->dt_bias_head_stride;
    p.b_vs = a->dt_bias_vdim_stride;
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
    p.counts = a->counts;
    const bool tb = a->token_dtype == GDR_BF16;
    // vectors of four values
    const int64_t four = 4 * esize(a->token_dtype);
    const bool vec = a->V % 4 == 0 && vector_rows(a->x, a->token_dtype, four, p.x_ts, p.x_hs) &&
                     (p.dt_es == 0 || vector_rows(a->dt, a->dt_dtype, 4 * esize(a->dt_dtype), p.dt_ts, p.dt_hs)) &&
                     (!a->out || vector_rows(a->out, a->token_dtype, four, p.o_ts, p.o_hs)) &&
                     (!a->z || vector_rows(a->z, a->token_dtype, four, p.z_ts, p.z_hs)) &&
                     vector_rows(a->state, a->state_dtype, 4 * esize(a->state_dtype), p.st_slot, p.st_head, p.st_k);
    p.bc_vec = vector_rows(a->B, a->token_dtype, four, p.B_ts, p.B_hs) &&
               (!a->out || vector_rows(a->C, a->token_dtype, four, p.C_ts, p.C_hs));
    p.seg = plan_scan(a);
    if (p.seg && (!a->workspace || a->workspace_bytes < scan_bytes(a, p.seg))) p.seg = 0;
    p.ws = static_cast<float *>(a->workspace);
    const bool db = a->dt_dtype == GDR_BF16;
    if (a->max_row_len >= 1 && a->max_row_len <= kShortRow)
        return launched(gdr::launch_scan_step(p, tb, db, vec, static_cast<cudaStream_t>(stream)), fn);
    return launched(gdr::launch_scan(p, tb, db, vec, static_cast<cudaStream_t>(stream)), fn);
}

int gdr_accept_drafts(const gdr_accept_args *a, void *stream) {
    const char *fn = "gdr_accept_drafts";
    if (!a) return fail(GDR_ERR_INVALID_ARG, "%s: args is NULL", fn);
    int rc = check_tokens(a->total_tokens, a->batch, fn);
    if (rc) return rc;
    if (a->vocab <= 0 || a->max_row_len <= 0)
        return fail(GDR_ERR_INVALID_ARG, "%s: vocab=%d and max_row_len=%d must be positive", fn, a->vocab, a->max_row_len);
    if (a->vocab > (1 << 28)) return fail(GDR_ERR_UNSUPPORTED, "%s: vocab must be at most 2^28", fn);
    if (!is_dtype(a->prob_dtype)) return fail(GDR_ERR_UNSUPPORTED, "%s: prob_dtype must be GDR_F32 or GDR_BF16", fn);
    if (a->batch == 0) return gdr::api_ok();
    if (!a->offsets || !a->row_uniforms || !a->out_tokens || !a->counts)
        return fail(GDR_ERR_INVALID_ARG, "%s: offsets/row_uniforms/out_tokens/counts is NULL", fn);
    if (a->batch > 1 && a->out_seq_stride < a->max_row_len)
        return fail(GDR_ERR_INVALID_ARG, "%s: out_seq_stride must be at least max_row_len", fn);
    if (a->total_tokens > 0) {
        if (!a->target || !a->tokens || !a->uniforms)
            return fail(GDR_ERR_INVALID_ARG, "%s: target/tokens/uniforms is NULL", fn);
        if (a->target_seq_stride < 0 || (a->draft && a->draft_seq_stride < 0))
            return fail(GDR_ERR_INVALID_ARG, "%s: probability strides must not be negative", fn);
        if (!aligned(a->target, esize(a->prob_dtype)) || !aligned(a->draft, esize(a->prob_dtype)))
            return fail(GDR_ERR_UNSUPPORTED, "%s: target and draft must be aligned to their elements", fn);
    }
    gdr::AcceptParams p{};
    if ((rc = gdr::api_status(&p.status))) return rc;
    p.batch = a->batch;
    p.vocab = a->vocab;
    p.width = a->max_row_len;
    p.T = a->total_tokens;
    p.target = a->target;
    p.t_ts = a->target_seq_stride;
    p.draft = a->draft;
    p.d_ts = a->draft_seq_stride;
    p.tokens = a->tokens;
    p.offsets = a->offsets;
    p.u = a->uniforms;
    p.row_u = a->row_uniforms;
    p.out = a->out_tokens;
    p.o_ts = a->out_seq_stride;
    p.counts = a->counts;
    return launched(gdr::launch_accept(p, a->prob_dtype == GDR_BF16, static_cast<cudaStream_t>(stream)), fn);
}

}  // extern "C"
