// Selective state space scan: every channel j keeps K states, and per token
//
//     d = softplus(dt + bias);  S_i <- exp(d A_i) S_i + (d x) B_i;  y = sum_i C_i S_i + D x
//
// in float32.  Each state has a decay of its own that follows the token, so there is no
// matrix product in it: a state's step is an exponential and four float32 operations.
//
// A block has 64 channels of one row (or of one segment of it), and all of its tokens
// follow one another, so what counts beside the work itself is how long a token takes.
// Warps share it by kind.  NW warps run the recurrence, KT states each of all 64
// channels, two channels a lane: a token is two vectors of d and d x a lane, KT values of B and
// C that every lane reads alike, and nothing else.  Four helper warps do the rest, a
// chunk of 8 tokens ahead and behind: they copy raw chunks into a ring, make d and d x of
// them once a channel, add up the NW partial readouts, apply D and the gate and store.
// One barrier a chunk hands both sides' buffers over.
//
// Measured, bfloat16 tokens, 16 states, 8 ragged rows, 17702 tokens x 4096 channels: 372 us, where the bytes
// alone would take 86 and the exponentials 124.  No one unit is full (counters: shared memory 64% of its
// cycles, FMA 46%, exponentials 39%, an instruction issued in 63%); a token's chain of barriers and shared memory
// reads, and their instructions, bound it.
#pragma once

#include "scan_device.cuh"

namespace gdr {

constexpr int kScanChunk = 8;     // tokens
constexpr int kScanTile = 64;     // a block's channels
constexpr int kScanHelpers = 128; // threads beside the recurrence's own

// An asynchronous copy of 4, 8 or 16 bytes to shared memory.
template <int BYTES> __device__ __forceinline__ void cp_async(void *to, const void *from) {
    const unsigned at = (unsigned)__cvta_generic_to_shared(to);
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;\n" ::"r"(at), "l"(from), "n"(BYTES) : "memory");
}

// Segment `piece` of all rows' segments, for calls of at most 32 rows: lane l counts row l's.
template <bool EXACT> __device__ __forceinline__ bool scan_piece(const ScanParams &p, long long piece, bool leader, int lane, ScanUnit &u) {
    ScanUnit r;
    bool live = false;
    if (lane < p.batch) live = scan_row(p, lane, leader && piece == 0, r);
    // as scan_segment(), a row a lane
    const bool decreases = lane < p.batch && p.offsets[lane] > p.offsets[lane + 1];
    const int seg = __any_sync(kFull, decreases) ? 0x7fffffff : p.seg;
    int n = live ? pieces(r.len, seg) : 0, upto = n;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int o = __shfl_up_sync(kFull, upto, m);
        if (lane >= m) upto += o;
    }
    const unsigned behind = __ballot_sync(kFull, upto > piece);
    if (!behind) return false;
    const int b = __ffs(behind) - 1;
    const int s = (int)piece - __shfl_sync(kFull, upto - n, b);
    if (!scan_row(p, b, false, u)) return false;
    const long long from = (long long)s * seg;
    u.t0 += from;
    const long long left = u.len - from, kept = u.kept - from;
    u.last = left <= seg;
    u.len = (int)(left < seg ? left : seg);
    u.kept = kept <= 0 || kept > u.len || EXACT ? 0 : (int)kept;
    u.piece = piece;
    return true;
}

// The first segment of row b among all rows' segments.
__device__ __forceinline__ long long scan_first_piece(const ScanParams &p, int b, int seg, int lane) {
    ScanUnit r;
    int n = 0;
    if (lane < b && scan_row(p, lane, false, r)) n = pieces(r.len, seg);
    return (long long)__reduce_add_sync(kFull, (unsigned)n);
}

// The n-th longest of up to 32 rows: blocks run in their order, and what comes last should be short.
__device__ __forceinline__ unsigned scan_longest(const ScanParams &p, unsigned n, int lane) {
    const int len = lane < p.batch ? p.offsets[lane + 1] - p.offsets[lane] : 0;
    unsigned rank = 0;
    for (int j = 0; j < p.batch; ++j) {
        const int o = __shfl_sync(kFull, len, j);
        rank += o > len || (o == len && j < lane);
    }
    return (unsigned)__ffs(__ballot_sync(kFull, lane < p.batch && rank == n)) - 1;
}

// A block's shared memory, in bytes: a ring of raw chunks, then two chunks' operands in
// float32 and the readout's partial sums.
template <typename TT, typename DT, int KT, int NW> struct ScanShared {
    static constexpr int W = kScanTile, KP = KT * NW, N = kScanChunk, ring = 5;
    static constexpr int x = 0, z = x + N * W * (int)sizeof(TT), dt = z + N * W * (int)sizeof(TT), B = dt + N * W * (int)sizeof(DT),
                         C = B + N * KP * (int)sizeof(TT), stage = C + N * KP * (int)sizeof(TT);
    static constexpr int fd = ring * stage, fx = fd + 2 * 4 * N * W, fB = fx + 2 * 4 * N * W, fC = fB + 2 * 4 * N * KP,
                         fy = fC + 2 * 4 * N * KP, bytes = fy + 2 * 4 * NW * N * W;
};

// READ: with outputs.  Without them states move only: into the slots, or (kOwn) each segment's own state, from zero, and
// the sum of its step sizes into the workspace, or (kOrdered) into the slots and each segment's start state into the
// workspace, a block KP of the states: without a readout they have nothing to do with one another.
enum ScanPass { kMain, kOwn, kOrdered };
template <typename TT, typename DT, int KT, int NW, bool VEC, bool READ, bool EXACT>
__global__ void __launch_bounds__(32 * NW + kScanHelpers, KT * NW <= 16 ? 2 : KT * NW <= 32 ? 2 : 1)
    k_scan(const __grid_constant__ ScanParams p, int tiles, int pass) {
    using Sh = ScanShared<TT, DT, KT, NW>;
    constexpr int W = Sh::W, KP = Sh::KP, N = Sh::N, R = Sh::ring;
    extern __shared__ __align__(16) unsigned char shared[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const bool first = !READ && !EXACT && pass == kOwn, ordered = !READ && EXACT && pass == kOrdered;
    const unsigned parts = ordered ? (unsigned)(p.K + KP - 1) / KP : 1;  // blocks that share the states
    const unsigned all = (unsigned)(p.nk * tiles) * parts;
    unsigned row = blockIdx.x / all;
    const unsigned part = ordered ? (blockIdx.x - row * all) % parts : 0, tg = (blockIdx.x - row * all) / parts;
    const int kbase = (int)part * KP, K = p.K - kbase;  // this block's states
    const int g = (int)(tg / (unsigned)tiles), tile = (int)(tg - (unsigned)g * (unsigned)tiles);
    ScanUnit u;
    if ((!p.seg || ordered) && p.batch <= 32) row = scan_longest(p, row, lane);
    if (p.seg && !ordered) {
        if (!scan_piece<EXACT>(p, row, tg == 0 && warp == 0 && !first, lane, u)) return;
        if (first && u.last) return;  // no segment starts from its state
    } else if (!scan_row(p, (int)row, tg == 0 && tid == 0, u)) {
        return;
    }
    const int seg = ordered ? scan_segment(p) : 0;
    if (ordered) u.piece = scan_first_piece(p, (int)row, seg, lane);
    const int c0 = tile * W, width = min(W, p.r * p.V - c0);  // channels of the key head's value heads, this block's first
    // A channel of the block as (value head, channel).
    auto head = [&](int c, int &j) {
        const int h = (c0 + c) / p.V;
        j = c0 + c - h * p.V;
        return g * p.r + h;
    };
    const int chunks = (u.len - 1) / N + 1;
    auto floats = [&](int at) { return reinterpret_cast<float *>(shared + at); };

    if (warp < NW) {
        // ---- the recurrence: states warp KT ... of channels 2 lane and 2 lane + 1, and their rates
        if (u.slot < 0) return;
        float2 S[KT], A[KT];
        int ch[2], cj[2];
        bool on[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            on[e] = 2 * lane + e < width;
            cj[e] = 0;
            ch[e] = on[e] ? head(2 * lane + e, cj[e]) : 0;
        }
        const int have = min(KT, K - warp * KT);  // states that there are
        const long long k0 = kbase + warp * KT;
        const long long st0 = (long long)u.slot * p.st_slot + (long long)ch[0] * p.st_head + cj[0] + k0 * p.st_k;
        const long long st1 = (long long)u.slot * p.st_slot + (long long)ch[1] * p.st_head + cj[1] + k0 * p.st_k;
        long long ws0 = ((u.piece * p.nv + ch[0]) * p.K + k0) * p.V + cj[0];  // in the workspace, [nv, K, V] a segment
        long long ws1 = ((u.piece * p.nv + ch[1]) * p.K + k0) * p.V + cj[1];
#pragma unroll
        for (int i = 0; i < KT; ++i) {
            S[i] = A[i] = make_float2(0.0f, 0.0f);
            if (i >= have) continue;
            if (on[0]) A[i].x = rate<TT>(p.A[ch[0] * p.a_hs + cj[0] * p.a_vs + (k0 + i) * p.a_ks]);
            if (on[1]) A[i].y = rate<TT>(p.A[ch[1] * p.a_hs + cj[1] * p.a_vs + (k0 + i) * p.a_ks]);
            if (first) continue;
            if (p.seg && !ordered) {
                if (on[0]) S[i].x = p.ws[ws0 + (long long)i * p.V];
                if (on[1]) S[i].y = p.ws[ws1 + (long long)i * p.V];
            } else if (p.st_bf16) {
                const uint16_t *s = static_cast<const uint16_t *>(p.state);
                if (on[0]) S[i].x = to_f32(s[st0 + i * p.st_k]);
                if (on[1]) S[i].y = to_f32(s[st1 + i * p.st_k]);
            } else {
                const float *s = static_cast<const float *>(p.state);
                if (on[0]) S[i].x = s[st0 + i * p.st_k];
                if (on[1]) S[i].y = s[st1 + i * p.st_k];
            }
        }
        // the states into their slot, or a segment's into the workspace
        auto put = [&](bool ws) {
#pragma unroll
            for (int i = 0; i < KT; ++i) {
                if (i >= have) continue;
                if (ws) {
                    if (on[0]) p.ws[ws0 + (long long)i * p.V] = S[i].x;
                    if (on[1]) p.ws[ws1 + (long long)i * p.V] = S[i].y;
                } else if (p.st_bf16) {
                    uint16_t *s = static_cast<uint16_t *>(p.state);
                    if (on[0]) s[st0 + i * p.st_k] = from_f32<uint16_t>(S[i].x);
                    if (on[1]) s[st1 + i * p.st_k] = from_f32<uint16_t>(S[i].y);
                } else {
                    float *s = static_cast<float *>(p.state);
                    if (on[0]) s[st0 + i * p.st_k] = S[i].x;
                    if (on[1]) s[st1 + i * p.st_k] = S[i].y;
                }
            }
        };
        // one token: its d and d x, B and C from shared memory
        auto token = [&](const float *d, const float *x, const float *b, const float *q) {
            const float2 dv = *reinterpret_cast<const float2 *>(d), xv = *reinterpret_cast<const float2 *>(x);
            float Bv[KT], Cv[KT];
#pragma unroll
            for (int i = 0; i < KT; i += KT < 4 ? 2 : 4) {
                if constexpr (KT < 4) {
                    *reinterpret_cast<float2 *>(Bv + i) = *reinterpret_cast<const float2 *>(b + i);
                    if (READ) *reinterpret_cast<float2 *>(Cv + i) = *reinterpret_cast<const float2 *>(q + i);
                } else {
                    *reinterpret_cast<float4 *>(Bv + i) = *reinterpret_cast<const float4 *>(b + i);
                    if (READ) *reinterpret_cast<float4 *>(Cv + i) = *reinterpret_cast<const float4 *>(q + i);
                }
            }
            constexpr int G = scan_group(KT);
            float2 y[KT / G];
#pragma unroll
            for (int i = 0; i < KT; ++i) {
                const float2 e = __fmul2_rn(dv, A[i]);
                S[i] = advance<EXACT>(make_float2(decay<TT>(e.x), decay<TT>(e.y)), S[i], __fmul2_rn(xv, make_float2(Bv[i], Bv[i])));
                if (READ) y[i / G] = __ffma2_rn(make_float2(Cv[i], Cv[i]), S[i], i % G ? y[i / G] : make_float2(0.0f, 0.0f));
            }
            if constexpr (READ) {
#pragma unroll
                for (int m = 1; m < KT / G; m *= 2)
#pragma unroll
                    for (int i = 0; i < KT / G; i += 2 * m) y[i] = __fadd2_rn(y[i], y[i + m]);
            }
            return y[0];
        };
        auto chunk = [&](auto half, int n, int cut) {  // tokens from the chunk on, and those of them before the slot's state
            constexpr int H = decltype(half)::value;
            const float *const d = floats(Sh::fd) + H * N * W + 2 * lane, *const x = floats(Sh::fx) + H * N * W + 2 * lane;
            const float *const b = floats(Sh::fB) + H * N * KP + warp * KT, *const q = floats(Sh::fC) + H * N * KP + warp * KT;
            float *const y = floats(Sh::fy) + (H * NW + warp) * N * W + 2 * lane;
            const bool here = (unsigned)(cut - 1) < (unsigned)N;
            if (here && cut < n && cut < N) {  // the slot's state lies inside
#pragma unroll 1
                for (int t = 0; t < N; ++t) {
                    const float2 v = token(d + t * W, x + t * W, b + t * KP, q + t * KP);
                    if (READ) *reinterpret_cast<float2 *>(y + t * W) = v;
                    if (t + 1 == cut) put(false);
                }
                return;
            }
#pragma unroll
            for (int t0 = 0; t0 < N; t0 += 4) {  // tokens behind the row's end are d = 0, d x = 0
                float2 v[4];
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    v[t] = token(d + (t0 + t) * W, x + (t0 + t) * W, b + (t0 + t) * KP, q + (t0 + t) * KP);
                if (READ)
#pragma unroll
                    for (int t = 0; t < 4; ++t) *reinterpret_cast<float2 *>(y + (t0 + t) * W) = v[t];
            }
            if (here) put(false);  // behind the chunk, or behind the row's last token
        };
        __syncthreads();
        int n = u.len, cut = first ? 0 : u.kept;
        // segments begin where chunks do
        int until = 0;
        auto begins = [&]() {
            if (!ordered || until-- > 0) return;
            until = seg / N - 1;
            put(true);
            ws0 += (long long)p.nv * p.K * p.V;
            ws1 += (long long)p.nv * p.K * p.V;
        };
        for (int k = 0; k <= chunks; ++k) {
            if (k < chunks) {
                begins();
                chunk(std::integral_constant<int, 0>{}, n, cut);
            }
            __syncthreads();
            if (++k > chunks) break;
            if (k < chunks) {
                begins();
                chunk(std::integral_constant<int, 1>{}, n - N, cut - N);
            }
            __syncthreads();
            n -= 2 * N;
            cut -= 2 * N;
        }
        if (first) put(true);
        return;
    }

    // ---- the helpers.  A thread has four values of a chunk: four channels of a token where rows are
    // vectors, else one channel of four tokens; it copies them, makes d and d x of them, and finishes
    // their outputs, so that raw values need no barrier.
    const int id = tid - 32 * NW;
    const int mt = VEC ? id / (W / 4) : id / W * 4, mc = VEC ? id % (W / 4) * 4 : id % W;
    const bool mon = mc < width;
    int mj = 0, mh = 0;
    if (mon) mh = head(mc, mj);
    auto at = [&](int i) { return VEC ? mt * W + mc + i : (mt + i) * W + mc; };
    TT *const op = READ ? static_cast<TT *>(p.out) + (u.t0 + mt) * p.o_ts + (long long)mh * p.o_hs + mj : nullptr;
    if (u.slot < 0) {  // padding: zeros
        if (READ && mon)
            for (int base = 0; base < u.len; base += N)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (base + mt + (VEC ? 0 : i) < u.len) op[(base + (VEC ? 0 : i)) * p.o_ts + (VEC ? i : 0)] = TT(0);
        return;
    }
    const TT *const xp = static_cast<const TT *>(p.x) + (u.t0 + mt) * p.x_ts + (long long)mh * p.x_hs + mj;
    const TT *const zp = READ && p.z ? static_cast<const TT *>(p.z) + (u.t0 + mt) * p.z_ts + (long long)mh * p.z_hs + mj : nullptr;
    const DT *const dp = static_cast<const DT *>(p.dt) + (u.t0 + mt) * p.dt_ts + (long long)mh * p.dt_hs + mj * p.dt_es;
    const TT *const bp = static_cast<const TT *>(p.B) + u.t0 * p.B_ts + (long long)g * p.B_hs + kbase;
    const TT *const cp = READ ? static_cast<const TT *>(p.C) + u.t0 * p.C_ts + (long long)g * p.C_hs : nullptr;
    float bias[4], D[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = mj + (VEC ? i : 0);
        bias[i] = mon && p.bias ? p.bias[mh * p.b_hs + j * p.b_vs] : 0.0f;
        D[i] = READ && mon && p.D ? p.D[mh * p.d_hs + j * p.d_vs] : 0.0f;
    }
    constexpr int NB = (READ ? 2 : 1) * N * KP;  // values of B and C in a chunk
    const bool bc_vec = p.bc_vec && (ordered ? K >= KP : K == KP);
    // a thread's of them: NV vectors of four, or NT one by one
    constexpr int NV = (NB / 4 + kScanHelpers - 1) / kScanHelpers, NT = (NB + kScanHelpers - 1) / kScanHelpers;
    // Values that no asynchronous copy can move (2 bytes, not as vectors) wait here for a chunk's time.
    constexpr bool slow = sizeof(TT) == 2;
    TT wx[4], wz[4], wbc[slow ? NT : 1];
    DT wd[4];

    auto copy = [&](auto *to, const auto *from, long long stride, auto (&wait)[4], int n) {
        using T = std::remove_const_t<std::remove_pointer_t<decltype(from)>>;
        if constexpr (VEC) {
            if (n > 0) cp_async<4 * (int)sizeof(T)>(to, from);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < n) {
                    if constexpr (sizeof(T) == 4) cp_async<4>(to + i * W, from + i * stride);
                    else wait[i] = from[i * stride];
                }
        }
    };
    // Asks for the next chunk: pointers and counts move on by one.
    const TT *fx_at = xp, *fz_at = zp;
    const DT *fd_at = dp;
    const TT *fb_at[NV];
    if (bc_vec)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = 4 * (id + i * kScanHelpers), w = v % (N * KP);
            fb_at[i] = v < N * KP ? bp + w / KP * p.B_ts + w % KP : cp + w / KP * p.C_ts + w % KP;
        }
    const long long dx = N * p.x_ts, dz = N * p.z_ts, dd = N * p.dt_ts;
    long long ahead = 0;  // tokens asked for
    auto fetch = [&](int f_at) {
        const int n = (int)(u.len - ahead);
        if (n > 0) {
            unsigned char *const to = shared + f_at;
            const int mine = mon ? n - mt : 0;
            if (VEC && !p.dt_es) {
                if (mine > 0) wd[0] = *fd_at;
            } else {
                copy(reinterpret_cast<DT *>(to + Sh::dt) + at(0), fd_at, p.dt_ts, wd, mine);
            }
            copy(reinterpret_cast<TT *>(to + Sh::x) + at(0), fx_at, p.x_ts, wx, mine);
            if (READ && zp) copy(reinterpret_cast<TT *>(to + Sh::z) + at(0), fz_at, p.z_ts, wz, mine);
            if (bc_vec) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int v = 4 * (id + i * kScanHelpers);
                    if (v < NB && v % (N * KP) / KP < n) cp_async<4 * (int)sizeof(TT)>(reinterpret_cast<TT *>(to + Sh::B) + v, fb_at[i]);
                    fb_at[i] += N * (v < N * KP ? p.B_ts : p.C_ts);
                }
            } else {
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    const int v = id + i * kScanHelpers, w = v % (N * KP), s = w / KP;
                    if (v < NB && s < n && w % KP < K) {
                        const TT *from = v < N * KP ? bp + (long long)(ahead + s) * p.B_ts + w % KP : cp + (long long)(ahead + s) * p.C_ts + w % KP;
                        if constexpr (!slow) cp_async<4>(reinterpret_cast<TT *>(to + Sh::B) + v, from);
                        else wbc[i] = *from;
                    }
                }
            }
            fx_at += dx;
            fz_at += dz;
            fd_at += dd;
        }
        cp_async_commit();
        ahead += N;
    };
    // What waited, to its place.  The braces count: of such loops without them, the first ones discarded, nvcc 13.0
    // drops the last one too.
    auto land = [&](int f_at) {
        unsigned char *const to = shared + f_at;
        if constexpr (VEC) {
            if (!p.dt_es) {  // a head's only step size
                Pack<DT, 4> q;
#pragma unroll
                for (int i = 0; i < 4; ++i) q.u.e[i] = wd[0];
                q.store(reinterpret_cast<DT *>(to + Sh::dt) + at(0));
            }
        }
        if constexpr (!VEC && sizeof(DT) == 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i) reinterpret_cast<DT *>(to + Sh::dt)[at(i)] = wd[i];
        }
        if constexpr (!VEC && slow) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                reinterpret_cast<TT *>(to + Sh::x)[at(i)] = wx[i];
                if (READ && zp) reinterpret_cast<TT *>(to + Sh::z)[at(i)] = wz[i];
            }
        }
        if constexpr (slow) {
            if (!bc_vec) {
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    if (id + i * kScanHelpers < NB) reinterpret_cast<TT *>(to + Sh::B)[id + i * kScanHelpers] = wbc[i];
            }
        }
    };
    // four values of this thread's
    auto four = [&](const auto *from, float (&v)[4]) {
        using T = std::remove_const_t<std::remove_pointer_t<decltype(from)>>;
        if constexpr (VEC) {
            Pack<T, 4> q;
            q.load(from + at(0));
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = q.get(i);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = to_f32(from[at(i)]);
        }
    };
    auto put4 = [&](float *to, const float (&v)[4]) {
        if constexpr (VEC) {
            *reinterpret_cast<float4 *>(to + at(0)) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) to[at(i)] = v[i];
        }
    };
    float dsum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    // d and d x of raw values; n: the chunk's tokens
    auto steps = [&](float (&d)[4], float (&x)[4], int n) {
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] += bias[i];
        if (p.softplus)
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i] = softplus<TT>(d[i]);
        if (n < N || width < W) {  // nothing there: states stay as they are
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (!mon || mt + (VEC ? 0 : i) >= n) d[i] = x[i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[i] *= d[i];
            if (!READ) dsum[i] += d[i];
        }
    };
    // B and C in float32: this thread's own values again; states past K are 0
    auto states = [&](const unsigned char *from, int half, int n) {
        const TT *const rb = reinterpret_cast<const TT *>(from + Sh::B);
        auto place = [&](int v) { return v < N * KP ? floats(Sh::fB) + half * N * KP + v : floats(Sh::fC) + half * N * KP + v - N * KP; };
        if (bc_vec) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = 4 * (id + i * kScanHelpers);
                if (v < NB) {
                    Pack<TT, 4> q;
                    q.load(rb + v);
                    const bool some = v % (N * KP) / KP < n;
                    *reinterpret_cast<float4 *>(place(v)) = some ? make_float4(q.get(0), q.get(1), q.get(2), q.get(3)) : make_float4(0, 0, 0, 0);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                const int v = id + i * kScanHelpers, w = v % (N * KP);
                if (v < NB) *place(v) = w / KP < n && w % KP < K ? to_f32(rb[v]) : 0.0f;
            }
        }
    };
    // Turn k finishes chunk k - 1, makes chunk k + 1 ready and asks for chunk k + Dist, which takes the
    // place of chunk k - 2 in the ring: a barrier lies between a place's last use and its next.
    constexpr int Dist = R - 2;
    for (int k = 0; k < Dist; ++k) {
        fetch(k * Sh::stage);
        land(k * Sh::stage);
    }
    cp_async_wait<Dist - 1>();
    {
        float d[4], x[4];
        four(reinterpret_cast<const DT *>(shared + Sh::dt), d);
        four(reinterpret_cast<const TT *>(shared + Sh::x), x);
        steps(d, x, u.len);
        put4(floats(Sh::fd), d);
        put4(floats(Sh::fx), x);
        states(shared, 0, u.len);
    }
    __syncthreads();
    int free_at = (R - 2) * Sh::stage, done_at = (R - 1) * Sh::stage, next_at = Sh::stage;  // chunks k - 2, k - 1 and k + 1 in the ring
    TT *out = READ ? op - (long long)N * p.o_ts : nullptr;
    const long long dout = N * p.o_ts;
    auto ask = [&]() {  // fetch() where the chunk is whole and all values are vectors
        unsigned char *const to = shared + free_at;
        cp_async<4 * (int)sizeof(DT)>(reinterpret_cast<DT *>(to + Sh::dt) + at(0), fd_at);
        cp_async<4 * (int)sizeof(TT)>(reinterpret_cast<TT *>(to + Sh::x) + at(0), fx_at);
        if (READ && zp) cp_async<4 * (int)sizeof(TT)>(reinterpret_cast<TT *>(to + Sh::z) + at(0), fz_at);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = 4 * (id + i * kScanHelpers);
            if (v < NB) {
                cp_async<4 * (int)sizeof(TT)>(reinterpret_cast<TT *>(to + Sh::B) + v, fb_at[i]);
                fb_at[i] += N * (v < N * KP ? p.B_ts : p.C_ts);
            }
        }
        cp_async_commit();
        fx_at += dx;
        fz_at += dz;
        fd_at += dd;
        ahead += N;
    };
    // WHOLE: all three chunks are whole and all values vectors, so that nothing has to be asked
    auto turn = [&](auto whole, int k) {
        constexpr bool WHOLE = decltype(whole)::value;
        if constexpr (WHOLE) ask();
        else fetch(free_at);
        cp_async_wait<Dist - 1>();
        const int half = (k + 1) & 1, left = u.len - k * N;  // both neighbours' half of the buffers in pairs
        [[maybe_unused]] float rx[4], rz[4], y[4];
        [[maybe_unused]] const unsigned char *const done = shared + done_at;
        float d[4], x[4];
        const unsigned char *const next = shared + next_at;
        four(reinterpret_cast<const DT *>(next + Sh::dt), d);
        four(reinterpret_cast<const TT *>(next + Sh::x), x);
        if constexpr (READ) {
            four(reinterpret_cast<const TT *>(done + Sh::x), rx);
            if (zp) four(reinterpret_cast<const TT *>(done + Sh::z), rz);
            const float *const fy = floats(Sh::fy) + half * NW * N * W;
            // a warp's sum, or two warps' where a warp has one group
            constexpr int Q = KT == 2 || (KT == 4 && sizeof(TT) == 2) ? 2 : 1;
#pragma unroll
            for (int w = 0; w < NW; w += Q) {
                float a[4], q[4];
                four(fy + w * N * W, a);
                if constexpr (Q == 2) four(fy + (w + 1) * N * W, q);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if constexpr (Q == 2) a[i] += q[i];
                    y[i] = w ? y[i] + a[i] : a[i];
                }
            }
        }
        steps(d, x, WHOLE ? N : left - N);
        put4(floats(Sh::fd) + half * N * W, d);
        put4(floats(Sh::fx) + half * N * W, x);
        if constexpr (WHOLE) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = 4 * (id + i * kScanHelpers);
                if (v < NB) {
                    Pack<TT, 4> q;
                    q.load(reinterpret_cast<const TT *>(next + Sh::B) + v);
                    *reinterpret_cast<float4 *>(floats(v < N * KP ? Sh::fB : Sh::fC - 4 * N * KP) + half * N * KP + v) =
                        make_float4(q.get(0), q.get(1), q.get(2), q.get(3));
                }
            }
        } else {
            states(next, half, left - N);
        }
        if constexpr (READ) {
            Pack<TT, 4> o;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                y[i] = fmaf(D[i], rx[i], y[i]);
                if (zp) y[i] *= silu(rz[i]);
                o.set(i, y[i]);
            }
            if constexpr (WHOLE) {
                o.store(out);
            } else {
                const int n = mon && k > 0 ? left + N - mt : 0;
                if constexpr (VEC) {
                    if (n > 0) o.store(out);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (i < n) out[i * p.o_ts] = o.u.e[i];
                }
            }
            out += dout;
        }
        if constexpr (!WHOLE) land(free_at);
        free_at = done_at;
        done_at = done_at == (R - 1) * Sh::stage ? 0 : done_at + Sh::stage;
        next_at = next_at == (R - 1) * Sh::stage ? 0 : next_at + Sh::stage;
        __syncthreads();
    };
    // Chunks k - 1 ... k + Dist are whole for 1 <= k <= last.  One step size a head takes the other turns (8 ragged rows
    // x 4096 channels 397 us; with whole turns for it too 385, and 383 instead of 381 for step sizes a channel).
    const int last = VEC && bc_vec && p.dt_es && width == W ? u.len / N - 1 - Dist : 0;
    turn(std::false_type{}, 0);
    int k = 1;
    if constexpr (VEC) {
        for (; k <= last; ++k) turn(std::true_type{}, k);
    }
    for (; k <= chunks; ++k) turn(std::false_type{}, k);
    if (first) {
        // each channel's step sizes, over the threads that have its tokens
        float *const part = floats(0);
        cp_async_wait<0>();
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (VEC) part[at(i)] = dsum[i];
        if (!VEC) part[mt / 4 * W + mc] = dsum[0] + dsum[1] + dsum[2] + dsum[3];
        asm volatile("bar.sync 1, %0;" ::"n"(kScanHelpers) : "memory");
        if (id < width) {
            float s = 0.0f;
            for (int t = 0; t < (VEC ? N : N / 4); ++t) s += part[t * W + id];
            int j;
            const int h = head(id, j);
            p.ws[scan_pieces(p.T, p.seg, p.batch) * p.nv * p.K * p.V + (u.piece * p.nv + h) * (long long)p.V + j] = s;
        }
    }
}

template <typename TT, typename DT, int KT, int NW, bool VEC, bool READ, bool EXACT>
cudaError_t scan_launch(const ScanParams &p, long long rows, int parts, int pass, cudaStream_t s) {
    using Sh = ScanShared<TT, DT, KT, NW>;
    static_assert(Sh::bytes <= 227 << 10, "a block's shared memory");
    constexpr auto kernel = k_scan<TT, DT, KT, NW, VEC, READ, EXACT>;
    static LaunchCache cache;
    LaunchInfo info;
    const cudaError_t e = launch_info(cache, &info, [](LaunchInfo &) {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Sh::bytes);
    });
    if (e != cudaSuccess) return e;
    const long long tiles = ((long long)p.r * p.V + Sh::W - 1) / Sh::W, blocks = rows * p.nk * tiles * parts;
    if (blocks >= 1ll << 31) return cudaErrorInvalidConfiguration;
    kernel<<<(unsigned)blocks, 32 * NW + kScanHelpers, Sh::bytes, s>>>(p, (int)tiles, pass);
    return cudaGetLastError();
}

template <typename TT, typename DT, int KT, int NW, bool VEC, bool EXACT> cudaError_t scan_go(const ScanParams &p, cudaStream_t s) {
    const long long rows = p.seg ? scan_pieces(p.T, p.seg, p.batch) : p.batch;
    cudaError_t e = cudaSuccess;
    if (p.seg && EXACT) {
        // eight states a block, two a warp, whatever K
        if constexpr (EXACT) e = scan_launch<TT, DT, 2, 4, VEC, false, true>(p, p.batch, (p.K + 7) / 8, kOrdered, s);
        if (e != cudaSuccess) return e;
    } else if (p.seg) {
        if constexpr (!EXACT) e = scan_launch<TT, DT, KT, NW, VEC, false, false>(p, rows, 1, kOwn, s);
        if (e != cudaSuccess || (e = launch_scan_join(p, s)) != cudaSuccess) return e;
    }
    return p.out ? scan_launch<TT, DT, KT, NW, VEC, true, EXACT>(p, rows, 1, kMain, s)
                 : scan_launch<TT, DT, KT, NW, VEC, false, EXACT>(p, rows, 1, kMain, s);
}

// States a warp and warps, by K.
template <typename TT, typename DT, bool VEC, bool EXACT> cudaError_t scan_states(const ScanParams &p, cudaStream_t s) {
    if (p.K <= 8) return scan_go<TT, DT, 2, 4, VEC, EXACT>(p, s);
    if (p.K <= 16) return scan_go<TT, DT, 4, 4, VEC, EXACT>(p, s);
    if (p.K <= 32) {
        // Eight warps of four states take half the steps for a token, four of eight read shared memory less often.
        // Measured with 32 states, us: 8 ragged rows x 4096 channels bfloat16 606 / 567, float32 1193 / 1327; 45 blocks
        // of 5 rows of up to 301 tokens, float32 51 / 77.
        const long long tiles = ((long long)p.r * p.V + kScanTile - 1) / kScanTile;
        if (sizeof(TT) == 4 || (long long)p.batch * p.nk * tiles <= 152) return scan_go<TT, DT, 4, 8, VEC, EXACT>(p, s);
        if constexpr (sizeof(TT) == 2) return scan_go<TT, DT, 8, 4, VEC, EXACT>(p, s);
    }
    if (p.K <= 64) return scan_go<TT, DT, 8, 8, VEC, EXACT>(p, s);
    return scan_go<TT, DT, 16, 8, VEC, EXACT>(p, s);
}
template <typename TT, typename DT, bool EXACT = false> cudaError_t scan_vec(const ScanParams &p, bool vec, cudaStream_t s) {
    return vec ? scan_states<TT, DT, true, EXACT>(p, s) : scan_states<TT, DT, false, EXACT>(p, s);
}

}  // namespace gdr
