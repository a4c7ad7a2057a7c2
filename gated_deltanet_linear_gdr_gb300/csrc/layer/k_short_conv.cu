// Short causal convolution over ragged rows, a few taps a channel:
//
//     y[j] = act(bias + sum_m w[m] xe[j + m]),  xe = (the slot's last inputs, the row's inputs)
//
// A thread owns VE neighbouring channels (four as a vector, or one where rows are
// not such vectors) and walks along tokens with the
// last width-1 inputs in registers, so that an input is read once and a result
// written once.  A few operations a byte: HBM bound; what counts is bytes in
// flight, so kAhead tokens are asked for before the first is used.
//
// Two ways to deal the work out.  A block takes whole rows where they are short
// (single tokens, drafts).  Otherwise it takes a run of tokens, whichever rows
// they are of, so that ragged rows fill the GPU evenly; what is read twice are the
// width-1 tokens before a run.  The tokens of a row that need its slot's old
// inputs (the first width-1) belong to the block that has the row's first
// token, past the end of its run where they lie there.  Its threads also write
// the slot, from the row's last inputs: nobody else touches it, so old inputs
// are not overwritten before they are used, in one launch.
//
// Measured, bfloat16 tokens x 8192 channels, float32 pool: 8 ragged rows, 17702 tokens, 103 us (5.7 TB/s, 84% of
// the copy rate); 256 single tokens 15 us (8.4 at the copy rate, though most of the states come from L2 there; the call itself
// takes the host 11).  200000 rows of 5 tokens x 512 channels, lengths not bounded, 1031 us (664 at the copy rate).
#include "scan_device.cuh"

namespace gdr {
namespace {

constexpr int kThreads = 128;
constexpr int kAhead = 8;      // tokens of a batch
// Rows up to here are taken whole, vectors of channels and others.  Measured, whole against runs, us: 256 rows x 8192 channels, one
// token 14.9 / 18.3, 5 tokens 26.7 / 31.6, 7 tokens 32.7 / 41.0, 8 tokens 34.4 / 30.7, 16 tokens 56 / 41; 1000 rows of 7 tokens x
// 4096 channels 54.9 / 69.0; 64 rows of 2 to 8 tokens x 2047 channels, two calls, 14.3 / 18.5.
constexpr int kShortRow = 7, kShortOddRow = 8;
constexpr int kRows = 16;  // by blocks of so many at most

struct ConvRow {
    long long lo, hi;  // its tokens
    int slot;          // -1: nothing to compute
    int kept;          // inputs after which the slot is written, 0: it is not
    bool inside;       // its tokens exist: its output may be written
    unsigned problem;  // GDR_STATUS_* bit
};

__device__ __forceinline__ ConvRow conv_row(const ConvOpParams &p, int b) {
    ConvRow r;
    r.lo = p.offsets[b];
    r.hi = p.offsets[b + 1];
    r.slot = p.slot_idx[b];
    const int count = p.counts ? p.counts[b] : 0;
    const long long len = r.hi - r.lo;
    r.inside = r.lo >= 0 && len >= 0 && r.hi <= p.T;
    r.kept = 0;
    r.problem = 0;
    if (!r.inside) r.problem = GDR_STATUS_BAD_OFFSETS;
    else if (len == 0) r.slot = -1;
    else if (p.max_len > 0 && len > p.max_len) r.problem = GDR_STATUS_ROW_TOO_LONG;
    else if (r.slot < -1 || r.slot >= p.max_slots) r.problem = GDR_STATUS_BAD_SLOT;
    if (r.problem) r.slot = -1;
    if (r.slot >= 0 && p.keep) {
        if (!p.counts) r.kept = (int)len;
        else if (count < 0 || count > len) r.problem = GDR_STATUS_BAD_COUNT;
        else r.kept = count;
    }
    return r;
}

// The same N values a thread keeps together in memory, moved as vectors.
template <typename ST, int N> struct Together {
    static constexpr int C = N * (int)sizeof(ST) % 16 == 0 ? 16 / (int)sizeof(ST) : 8 / (int)sizeof(ST);
    static_assert(N % C == 0, "whole vectors");
    __device__ static __forceinline__ void load(const ST *p, float (&v)[N]) {
#pragma unroll
        for (int i = 0; i < N; i += C) {
            Pack<ST, C> q;
            q.load(p + i);
#pragma unroll
            for (int j = 0; j < C; ++j) v[i + j] = q.get(j);
        }
    }
    __device__ static __forceinline__ void store(ST *p, const float (&v)[N]) {
#pragma unroll
        for (int i = 0; i < N; i += C) {
            Pack<ST, C> q;
#pragma unroll
            for (int j = 0; j < C; ++j) q.set(j, v[i + j]);
            q.store(p + i);
        }
    }
};

template <typename TT, int W, int VE> struct ConvThread {
    static constexpr int N = W > 1 ? W - 1 : 1;  // inputs a row remembers
    const ConvOpParams &p;
    const int c0;
    float w[W][VE], bias[VE];
    float win[N][VE];  // the last inputs, oldest first

    __device__ __forceinline__ ConvThread(const ConvOpParams &pp, int c) : p(pp), c0(c) {}

    __device__ __forceinline__ const TT *x(long long t) const { return static_cast<const TT *>(p.x) + t * p.x_ts + c0; }
    __device__ __forceinline__ TT *out(long long t) const { return static_cast<TT *>(p.out) + t * p.o_ts + c0; }

    __device__ __forceinline__ void weights() {
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            const float *wp = p.w + (long long)(c0 + e) * p.w_cs;
            if (W == 4 && p.w_vec) {
                const float4 q = *reinterpret_cast<const float4 *>(wp);
                w[0][e] = q.x;
                w[1 % W][e] = q.y;
                w[2 % W][e] = q.z;
                w[3 % W][e] = q.w;
            } else {
#pragma unroll
                for (int m = 0; m < W; ++m) w[m][e] = wp[m * p.w_ts];
            }
            bias[e] = p.bias ? p.bias[c0 + e] : 0.0f;
        }
    }

    // A slot's inputs of this thread's channels, channel by channel.
    template <typename ST> __device__ __forceinline__ void read(int slot, float (&v)[VE * N]) const {
        const ST *s = static_cast<const ST *>(p.state) + (long long)slot * p.s_slot + (long long)c0 * p.s_chan;
        if (VE > 1 && p.st_run) {
            if constexpr (VE > 1) Together<ST, VE * N>::load(s, v);
        } else {
#pragma unroll
            for (int i = 0; i < VE * N; ++i) v[i] = to_f32(s[(i / N) * p.s_chan + (i % N) * p.s_tap]);
        }
    }
    template <typename ST> __device__ __forceinline__ void write(int slot, const float (&v)[VE * N]) const {
        ST *s = static_cast<ST *>(p.state) + (long long)slot * p.s_slot + (long long)c0 * p.s_chan;
        if (VE > 1 && p.st_run) {
            if constexpr (VE > 1) Together<ST, VE * N>::store(s, v);
        } else {
#pragma unroll
            for (int i = 0; i < VE * N; ++i) s[(i / N) * p.s_chan + (i % N) * p.s_tap] = from_f32<ST>(v[i]);
        }
    }

    // A slot's inputs, and a row's first token.
    struct Start {
        float v[VE * N];
        Pack<TT, VE> x;
    };
    __device__ __forceinline__ void ask_start(Start &s, int slot, long long lo) const {
        if constexpr (W > 1) {
            if (p.st_bf16) read<uint16_t>(slot, s.v);
            else read<float>(slot, s.v);
        }
        s.x.load(x(lo));
    }
    // A row's beginning: the slot's inputs into the window, and the slot's new ones, which are
    // entries kept .. kept + W - 2 of (old inputs, the row's inputs).
    __device__ __forceinline__ void begin(const Start &s, int slot, long long lo, int kept) {
        if constexpr (W > 1) {
#pragma unroll
            for (int i = 0; i < VE * N; ++i) win[i % N][i / N] = s.v[i];
            if (kept <= 0) return;
            float v[VE * N];
#pragma unroll
            for (int m = 0; m < N; ++m) {
                const int i = kept + m;  // entry of (old inputs, the row's)
                Pack<TT, VE> in = s.x;
                if (i > N) in.load(x(lo + i - N));
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    float y = in.get(e);
#pragma unroll
                    for (int j = 1; j < N; ++j)
                        if (i == j) y = win[j][e];
                    v[e * N + m] = y;
                }
            }
            if (p.st_bf16) write<uint16_t>(slot, v);
            else write<float>(slot, v);
        }
    }
    // The window in front of token t, all of it in the row.
    __device__ __forceinline__ void enter(long long t) {
        if constexpr (W > 1) {
#pragma unroll
            for (int m = 0; m < N; ++m) {
                Pack<TT, VE> in;
                in.load(x(t - N + m));
#pragma unroll
                for (int e = 0; e < VE; ++e) win[m][e] = in.get(e);
            }
        }
    }

    __device__ __forceinline__ void token(const Pack<TT, VE> &in, TT *to) {
        Pack<TT, VE> o;
#pragma unroll
        for (int e = 0; e < VE; ++e) {
            const float v = in.get(e);
            float y = bias[e];
#pragma unroll
            for (int m = 0; m < W - 1; ++m) y = fmaf(w[m][e], win[m][e], y);
            y = fmaf(w[W - 1][e], v, y);
            o.set(e, p.silu ? silu(y) : y);
#pragma unroll
            for (int m = 0; m + 1 < N; ++m) win[m][e] = win[m + 1][e];
            win[N - 1][e] = v;
        }
        o.store(to);
    }

    __device__ __forceinline__ void ask(Pack<TT, VE> (&in)[kAhead], const TT *&from) const {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            in[i].load(from);
            from += p.x_ts;
        }
    }
    __device__ __forceinline__ void tokens(const Pack<TT, VE> (&in)[kAhead], TT *&to) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            token(in[i], to);
            to += p.o_ts;
        }
    }
    // Two batches of kAhead tokens in turn: one is on its way while the other is worked on.
    __device__ __forceinline__ void run(long long s, long long e) {
        const TT *from = x(s);
        TT *to = out(s);
        int n = (int)(e - s);
        Pack<TT, VE> a[kAhead], b[kAhead];
        if (n >= kAhead) {
            ask(a, from);
            for (;;) {
                n -= kAhead;
                if (n < kAhead) {
                    tokens(a, to);
                    break;
                }
                ask(b, from);
                tokens(a, to);
                n -= kAhead;
                if (n < kAhead) {
                    tokens(b, to);
                    break;
                }
                ask(a, from);
                tokens(b, to);
            }
        }
        for (; n > 0; --n) {
            Pack<TT, VE> in;
            in.load(from);
            token(in, to);
            from += p.x_ts;
            to += p.o_ts;
        }
    }
    // A short row behind its first token, four tokens at a time.
    __device__ __forceinline__ void short_run(const Pack<TT, VE> &first, long long s, int n) {
        const TT *from = x(s);
        TT *to = out(s);
        token(first, to);
        for (int t = 1; t < n; t += 4) {
            Pack<TT, VE> in[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (t + i < n) in[i].load(from + (t + i) * p.x_ts);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (t + i < n) token(in[i], to + (t + i) * p.o_ts);
        }
    }
    __device__ __forceinline__ void clear(long long s, long long e) {
        Pack<TT, VE> o;
#pragma unroll
        for (int i = 0; i < VE; ++i) o.u.e[i] = TT(0);
        for (; s < e; ++s) o.store(out(s));
    }
};

// ROWS: a block takes whole rows, `run` of them; else a run of tokens.
template <typename TT, int W, int VE, bool ROWS>
__global__ void __launch_bounds__(kThreads) k_short_conv(const __grid_constant__ ConvOpParams p) {
    const unsigned block = blockIdx.x / (unsigned)p.tiles, tile = blockIdx.x - block * (unsigned)p.tiles;
    const int tid = threadIdx.x, c0 = (int)(tile * kThreads + threadIdx.x) * VE;
    const bool on = c0 < p.channels;
    using Thread = ConvThread<TT, W, VE>;
    Thread th(p, c0);
    if constexpr (ROWS) {
        __shared__ ConvRow rows[kRows];
        const int b0 = (int)block * p.run, n = min(p.run, p.batch - b0);
        if (tid < n) {
            const ConvRow r = conv_row(p, b0 + tid);
            if (r.problem && tile == 0) flag(p.status, r.problem);
            rows[tid] = r;
        }
        if (on && p.out) th.weights();
        __syncthreads();
        if (!on) return;
        // two rows at a time, so that twice the bytes are on their way
        auto live = [&](int i) { return i < n && rows[i].slot >= 0 && (p.out || rows[i].kept > 0); };
        auto row = [&](int i, const typename Thread::Start &s) {
            if (i >= n) return;
            const ConvRow &r = rows[i];
            if (live(i)) {
                th.begin(s, r.slot, r.lo, r.kept);
                if (p.out) th.short_run(s.x, r.lo, (int)(r.hi - r.lo));
            } else if (p.out && r.inside) {
                th.clear(r.lo, r.hi);
            }
        };
        for (int i = 0; i < n; i += 2) {
            typename Thread::Start a, b;
            if (live(i)) th.ask_start(a, rows[i].slot, rows[i].lo);
            if (live(i + 1)) th.ask_start(b, rows[i + 1].slot, rows[i + 1].lo);
            row(i, a);
            row(i + 1, b);
        }
    } else {
        const long long t0 = (long long)block * p.run, t1 = t0 + p.run < p.T ? t0 + p.run : p.T;
        if (tile == 0) {  // the blocks look at every row between them
            const long long runs = (p.T + p.run - 1) / p.run;
            for (long long b = (long long)block * kThreads + tid; b < p.batch; b += runs * kThreads) {
                const unsigned problem = conv_row(p, (int)b).problem;
                if (problem) flag(p.status, problem);
            }
        }
        // the row of the first token: the last one that does not begin behind it.  Where offsets decrease that
        // finds nothing, and the block goes through all of the rows.
        __shared__ int before[kThreads / 32];
        int n = 0;
        bool ascend = true;
#pragma unroll 8
        for (int i = tid; i <= p.batch; i += kThreads) {
            const int o = p.offsets[i];
            n += o <= t0;
            ascend &= i == 0 || p.offsets[i - 1] <= o;
        }
        n = __reduce_add_sync(kFull, n);
        if (tid % 32 == 0) before[tid / 32] = n;
        ascend = __syncthreads_and(ascend);
        if (!on) return;
        th.weights();
        int b = -1;
#pragma unroll
        for (int i = 0; i < kThreads / 32; ++i) b += before[i];
        for (b = b < 0 || !ascend ? 0 : b; b < p.batch && (!ascend || p.offsets[b] < t1); ++b) {
            const ConvRow r = conv_row(p, b);
            if (r.lo >= t1) continue;
            const bool first = r.lo >= t0;  // the row begins in this run
            const long long head = r.lo + (W - 1);
            const long long s = first ? r.lo : (t0 > head ? t0 : head), end = first && head > t1 ? head : t1;
            const long long e = r.hi < end ? r.hi : end;
            if (!r.inside || s >= e) continue;
            if (r.slot < 0) {
                th.clear(s, e);
                continue;
            }
            if (first) {
                typename Thread::Start start;
                th.ask_start(start, r.slot, r.lo);
                th.begin(start, r.slot, r.lo, r.kept);
            } else {
                th.enter(s);
            }
            th.run(s, e);
        }
    }
}

template <typename TT, int W> cudaError_t go(ConvOpParams p, cudaStream_t s) {
    constexpr int VE = 4;
    const int wide = (p.vec ? VE : 1) * kThreads;
    p.tiles = (p.channels + wide - 1) / wide;
    // Rows' lengths as far as the caller bounds them: whole rows where none is longer than that, and where
    // only states move.
    const bool rows = !p.out || (p.max_len > 0 && p.max_len <= (p.vec ? kShortRow : kShortOddRow));
    long long blocks;
    if (rows) {
        // as many rows a block as leaves each multiprocessor eight blocks
        const long long each = ((long long)p.batch * p.tiles + 152 * 8 - 1) / (152 * 8);
        p.run = (int)(each < kRows ? each : kRows);
        blocks = ((long long)p.batch + p.run - 1) / p.run;
    } else {
        // runs of up to 64 tokens, shorter ones where they would leave multiprocessors without work
        p.run = 64;
        while (p.run > 8 && (p.T + p.run - 1) / p.run * p.tiles < 152 * 12) p.run /= 2;
        // Every block reads all offsets, kThreads at a time: a token for each of those steps at least.
        const int steps = p.batch / kThreads + 1;
        if (p.run < steps) p.run = steps;
        blocks = (p.T + p.run - 1) / p.run;
    }
    blocks *= p.tiles;
    if (blocks <= 0) return cudaSuccess;
    if (blocks >= (1ll << 31)) return cudaErrorInvalidConfiguration;
    const unsigned n = (unsigned)blocks;
    if (p.vec) {
        if (rows) k_short_conv<TT, W, VE, true><<<n, kThreads, 0, s>>>(p);
        else k_short_conv<TT, W, VE, false><<<n, kThreads, 0, s>>>(p);
    } else {
        if (rows) k_short_conv<TT, W, 1, true><<<n, kThreads, 0, s>>>(p);
        else k_short_conv<TT, W, 1, false><<<n, kThreads, 0, s>>>(p);
    }
    return cudaGetLastError();
}

template <typename TT> cudaError_t width(const ConvOpParams &p, int w, cudaStream_t s) {
    return w == 4 ? go<TT, 4>(p, s) : w == 3 ? go<TT, 3>(p, s) : w == 2 ? go<TT, 2>(p, s) : go<TT, 1>(p, s);
}

}  // namespace

cudaError_t launch_short_conv(ConvOpParams p, int w, bool tok_bf16, cudaStream_t s) {
    return tok_bf16 ? width<uint16_t>(p, w, s) : width<float>(p, w, s);
}

}  // namespace gdr
