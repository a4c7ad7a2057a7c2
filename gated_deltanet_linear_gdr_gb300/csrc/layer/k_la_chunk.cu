// Decayed linear attention, chunked form on the tensor cores (bfloat16 tokens).
//
// A row is taken 64 tokens at a time.  With S0 the state before a chunk of n
// tokens, i and j counted inside it:
//
//     P^T[j, i]  = k_j . q_i                                   (K Q^T)
//     P~^T[j, i] = scale lambda^(i-j) P^T[j, i] for j <= i, else 0   -> bfloat16
//     O^T[:, i]  = scale lambda^(i+1) (S0^T q_i)  +  V^T P~^T[:, i]
//     S^T        = lambda^n S0^T + V^T K~,  K~[j] = lambda^(n-1-j) k_j
//
// Everything is kept transposed (value index = tensor memory lane), so that
// the state, which a warp's lanes hold in float32 registers, goes back into
// tensor memory as the A operand of S0^T Q^T, and V^T serves two products.
// Rounding to bfloat16: P~ once (as the output is).  The state operand is split
// into two bfloat16 parts and K~ into two (bfloat16 pool) or three (float32
// pool), which keeps 16 and 24 bits: the state itself never loses any.
//
// One CTA per SM walks (row segment, value head, 128-column tile) units, with
// a warp role for each step: TMA loads three chunks ahead, one thread issues
// the matrix products, 4 warps make K~, 8 warps keep S, 4 warps make P~ and
// write the output.  Roles hand over through mbarriers, so the products of a
// chunk run under the elementwise work of its neighbours.
//
// Bound: a chunk of one head with K = V = 128 moves 64 KiB (1.47 us of an SM's
// share of HBM) and holds the tensor cores for about 1400 (bfloat16 pool) to
// 1660 cycles.
#include "tc.cuh"

#include "layer_internal.h"

namespace gdr {
namespace {

using namespace tc;

constexpr int kC = 64;        // tokens a chunk
constexpr int kStages = 3;
constexpr int kSub = kC * 128;        // bytes of a 64-token x 64-channel operand block
constexpr int kTile = 2 * kSub;       // bytes of a 64-token x 128-channel operand
constexpr int kStage = 3 * kTile;     // Q | K | V
constexpr int kMaxRows = 128;         // rows whose order and segments are worked out in shared memory

constexpr int kWarpsS = 8, kWarpsP = 4, kWarpsK = 4;
constexpr int kWarpMma = kWarpsS + kWarpsP + kWarpsK, kWarpTma = kWarpMma + 1;
constexpr int kThreads = 32 * (kWarpTma + 1);

// tensor memory columns
constexpr uint32_t kColP = 0, kColO1 = 128, kColO2 = 192, kColDS = 256, kColHi = 384, kColLo = 448;

enum Bar {
    kFull = 0, kEmpty = kFull + kStages, kPFull = kEmpty + kStages, kPFree = kPFull + 2, kPtFull = kPFree + 2,
    kSFull, kSFree, kDsFull, kDsFree, kKtFull, kOFull, kOFree, kDrain, kBars
};

struct Smem {
    unsigned char stage[kStages][kStage];
    unsigned char kt[3][kTile];   // K~, its bfloat16 parts
    unsigned char pt[kSub];       // P~^T
    unsigned char ost[kWarpsP][kC * 64];  // output on its way out, [token][32 columns] a warp
    float factor[kWarpsP][2][kC];         // scale lambda^(i+1), by unit parity
    uint64_t bar[kBars];
    int order[kMaxRows], first[kMaxRows + 1];
    uint32_t tmem;
    int gave_up;
};
static_assert(sizeof(Smem) + 1024 <= 232448, "shared memory");

struct ChunkParams {
    LaParams p;
    int seg;    // tokens a segment (a multiple of kC), or 0: rows are whole
    int parts;  // bfloat16 parts of K~
    float *ws;  // start states of the segments [segment, nv, K, V] (seg != 0)
};

// A unit of work, the same for every role: one segment of a row, one head, one column tile.
struct Unit {
    int h, tile, b, slot;
    int t0, len;  // tokens of the segment; len 0: nothing to compute
    int chunks;
    int x;        // segment number
    bool first, last;          // of its row
    int skip_t0, skip_len;     // a skipped row's tokens, whose output is zero
    float lg2;                 // log2 lambda
};

__device__ __forceinline__ float power(float lg2, int n) { return n == 0 ? 1.0f : exp2f(lg2 * (float)n); }

// Walks this CTA's units: positions blockIdx.x, then back and forth, so that
// units sorted by length are dealt evenly.
template <bool STATES> struct Walk {
    const ChunkParams &c;
    const Smem &sm;
    int i = 0;
    __device__ Walk(const ChunkParams &c_, const Smem &sm_) : c(c_), sm(sm_) {}

    __device__ bool next(Unit &u, bool report) {
        const LaParams &p = c.p;
        const unsigned per = (unsigned)(p.nv * p.tiles), G = gridDim.x;
        const long long pos = (long long)i * G + ((i & 1) ? G - 1 - blockIdx.x : blockIdx.x);
        ++i;
        const long long xx = pos / per;
        const int ht = (int)(pos - xx * per);
        u.h = ht / p.tiles;
        u.tile = ht - u.h * p.tiles;
        u.x = (int)xx;
        int seg_i = 0;
        if (p.batch <= kMaxRows) {
            int r = u.x;
            if (c.seg) {
                if (u.x >= sm.first[p.batch]) return false;
                r = 0;
                while (sm.first[r + 1] <= u.x) ++r;
                seg_i = u.x - sm.first[r];
            } else if (u.x >= p.batch) {
                return false;
            }
            u.b = sm.order[r];
        } else {
            if (xx >= p.batch) return false;
            u.b = u.x;
        }
        u.len = u.chunks = u.skip_len = 0;
        u.first = u.last = true;
        const int r0 = p.offsets[u.b], r1 = p.offsets[u.b + 1];
        u.slot = p.slot_idx[u.b];
        const float d = p.decay[(long long)u.h * p.decay_s];
        const bool leader = report && u.h == 0 && u.tile == 0 && seg_i == 0;
        if (r0 < 0 || r1 < r0 || r1 > p.T) {
            if (leader) flag(p.status, GDR_STATUS_BAD_OFFSETS);
            return true;
        }
        const bool too_long = p.max_len > 0 && r1 - r0 > p.max_len;
        const bool decay_ok = p.decay_is_log ? d <= 0.0f : (d >= 0.0f && d <= 1.0f);
        if (r1 > r0 && (u.slot < 0 || u.slot >= p.max_slots || !decay_ok || too_long)) {
            if (too_long) {
                if (leader) flag(p.status, GDR_STATUS_ROW_TOO_LONG);
            } else if (u.slot < -1 || u.slot >= p.max_slots) {
                if (leader) flag(p.status, GDR_STATUS_BAD_SLOT);
            } else if (u.slot >= 0 && report) {
                flag(p.status, GDR_STATUS_BAD_DECAY);
            }
            if (seg_i == 0) {
                u.skip_t0 = r0;
                u.skip_len = r1 - r0;
            }
            return true;
        }
        u.lg2 = p.decay_is_log ? d * 1.44269504088896340736f : log2f(d);
        u.t0 = r0;
        u.len = r1 - r0;
        if (c.seg) {
            const int at = seg_i * c.seg;
            u.first = seg_i == 0;
            u.last = u.len - at <= c.seg;
            u.t0 += at;
            u.len = u.last ? u.len - at : c.seg;
            if (STATES && u.last) u.len = 0;
        }
        u.chunks = (u.len + kC - 1) / kC;
        return true;
    }
};

// Rows by descending length, and the number of each one's first segment.
__device__ __forceinline__ void plan_rows(const ChunkParams &c, Smem &sm) {
    const int B = c.p.batch;
    if (B > kMaxRows) return;
    for (int b = threadIdx.x; b < B; b += kThreads) {
        const int t0 = c.p.offsets[b], t1 = c.p.offsets[b + 1];
        sm.first[b] = t0 < 0 || t1 < t0 || t1 > c.p.T ? 0 : t1 - t0;
    }
    __syncthreads();
    if (threadIdx.x < B) {
        const int b = threadIdx.x, len = sm.first[b];
        int rank = 0;
        for (int o = 0; o < B; ++o) rank += sm.first[o] > len || (sm.first[o] == len && o < b);
        sm.order[rank] = b;
    }
    __syncthreads();
    if (c.seg && threadIdx.x < 32) {  // batch <= 32: one lane a row
        const int lane = threadIdx.x;
        const int n = lane < B ? max(1, (sm.first[sm.order[lane]] + c.seg - 1) / c.seg) : 0;
        int end = n;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int o = __shfl_up_sync(kFull, end, m);
            if (lane >= m) end += o;
        }
        __syncwarp();
        if (lane < B) sm.first[lane + 1] = end;
        if (lane == 0) sm.first[0] = 0;
    }
    __syncthreads();
}

// ---- the roles ----------------------------------------------------------------

struct Ctx {
    const ChunkParams &c;
    Smem &sm;
    uint32_t base;  // shared address of sm
    uint32_t bars;
    uint32_t tmem;
    __device__ uint32_t bar(int i) const { return bars + 8u * (uint32_t)i; }
    __device__ bool wait(int i, uint32_t parity) const { return mbar_wait(bar(i), parity & 1u, &sm.gave_up); }
    __device__ uint32_t stage(unsigned g) const { return base + (uint32_t)(g % kStages) * kStage; }
    // one arrival for the warp, once every lane has got here
    __device__ void arrive(int i) const {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(bar(i));
    }
};

template <bool STATES>
__device__ void role_tma(const Ctx &x, const CUtensorMap *mq, const CUtensorMap *mk, const CUtensorMap *mv) {
    const LaParams &p = x.c.p;
    const int nk = p.K > 64 ? 2 : 1;
    Walk<STATES> walk(x.c, x.sm);
    Unit u;
    unsigned g = 0;
    bool good = true;
    while (good && walk.next(u, false)) {
        const int hk = u.h / p.r, v0 = u.tile * 128, nv = p.V - v0 > 64 ? 2 : 1;
        const uint32_t bytes = (uint32_t)((STATES ? 1 : 2) * nk + nv) * kSub;
        for (int j = 0; j < u.chunks; ++j, ++g) {
            const int s = g % kStages;
            if (g >= kStages && !(good = x.wait(kEmpty + s, g / kStages - 1))) break;
            const uint32_t dst = x.stage(g), full = x.bar(kFull + s);
            mbar_expect(full, bytes);
            const int t = u.t0 + j * kC;
            for (int i = 0; i < nk; ++i) tma_load3(dst + kTile + i * kSub, mk, i * 64, hk, t, full);
            for (int i = 0; i < nv; ++i) tma_load3(dst + 2 * kTile + i * kSub, mv, v0 + i * 64, u.h, t, full);
            if (!STATES)
                for (int i = 0; i < nk; ++i) tma_load3(dst + i * kSub, mq, i * 64, hk, t, full);
        }
    }
    // no copy is in flight when the CTA ends
    for (unsigned o = g > kStages ? g - kStages : 0; o < g; ++o) {
        volatile int never = 0;
        mbar_wait(x.bar(kFull + o % kStages), (o / kStages) & 1u, &never);
    }
}

template <bool STATES> __device__ void role_mma(const Ctx &x) {
    const LaParams &p = x.c.p;
    const int ksteps = p.K / 16;
    const uint32_t id_p = idesc_bf16(64, kC, false, false);    // P^T = K Q^T
    const uint32_t id_o1 = idesc_bf16(128, kC, false, false);  // S0^T Q^T
    const uint32_t id_o2 = idesc_bf16(128, kC, true, true);    // V^T P~^T
    const uint32_t id_s = idesc_bf16(128, p.K, true, true);    // V^T K~
    const uint32_t pt = x.base + offsetof(Smem, pt), kt = x.base + offsetof(Smem, kt);
    auto scores = [&](unsigned g) {
        if (!x.wait(kFull + g % kStages, g / kStages)) return false;
        if (g >= 2 && !x.wait(kPFree + (g & 1), (g >> 1) - 1)) return false;
        fence_after();
        const uint32_t q = x.stage(g), k = q + kTile, d = x.tmem + kColP + (g & 1) * kC;
        for (int i = 0; i < ksteps; ++i) {
            const uint32_t at = (uint32_t)(i >> 2) * kSub + (uint32_t)(i & 3) * 32;
            mma_ss(d, desc128(k + at, 16, 1024), desc128(q + at, 16, 1024), id_p, i > 0);
        }
        mma_commit(x.bar(kPFull + (g & 1)));
        return true;
    };
    Walk<STATES> walk(x.c, x.sm);
    Unit u;
    unsigned g = 0;
    int left = 0;  // chunks of the current unit that are still to do
    bool more = true;
    auto next_unit = [&]() {  // moves on to a unit with chunks
        while (left == 0 && (more = walk.next(u, false))) left = u.chunks;
        return left > 0;
    };
    bool good = next_unit() && (STATES || scores(0));
    while (good) {
        const uint32_t q = x.stage(g), v = q + 2 * kTile;
        // V^T K~ over all parts of K~
        good = x.wait(kKtFull, g) && (g == 0 || x.wait(kDsFree, g - 1));
        if (!good) break;
        fence_after();
        for (int part = 0; part < x.c.parts; ++part)
            for (int i = 0; i < kC / 16; ++i)
                mma_ss(x.tmem + kColDS, desc128(v + i * 2048, kSub, 1024), desc128(kt + part * kTile + i * 2048, kSub, 1024),
                       id_s, part + i > 0);
        mma_commit(x.bar(kDsFull));
        if (STATES) {
            mma_commit(x.bar(kEmpty + g % kStages));
        } else {
            // S0^T Q^T, both parts of the state
            good = x.wait(kSFull, g) && (g == 0 || x.wait(kOFree, g - 1));
            if (!good) break;
            fence_after();
            for (int half = 0; half < 2; ++half)
                for (int i = 0; i < ksteps; ++i) {
                    const uint32_t at = (uint32_t)(i >> 2) * kSub + (uint32_t)(i & 3) * 32;
                    mma_ts(x.tmem + kColO1, x.tmem + (half ? kColLo : kColHi) + i * 8, desc128(q + at, 16, 1024), id_o1,
                           half + i > 0);
                }
            mma_commit(x.bar(kSFree));
            if (!(good = x.wait(kPtFull, g))) break;
            fence_after();
            for (int i = 0; i < kC / 16; ++i)
                mma_ss(x.tmem + kColO2, desc128(v + i * 2048, kSub, 1024), desc128(pt + i * 2048, kSub, 1024), id_o2, i > 0);
            mma_commit(x.bar(kOFull));
            mma_commit(x.bar(kEmpty + g % kStages));
        }
        ++g;
        --left;
        if (!next_unit()) break;
        if (!STATES) good = scores(g);
    }
    // no matrix instruction is in flight when tensor memory is freed
    mma_commit(x.bar(kDrain));
    volatile int never = 0;
    mbar_wait(x.bar(kDrain), 0, &never);
}

// K~[j] = lambda^(n-1-j) k_j in bfloat16 parts, at the places K has in its
// swizzled block: a thread has 16-byte vectors of 4 tokens.  In a row's last
// chunk the tokens past its end, which belong to somebody else, become zero,
// in V as well: a product of zero and infinity would not.
template <bool STATES> __device__ void role_keys(const Ctx &x, int tid) {
    const LaParams &p = x.c.p;
    const int nk = p.K > 64 ? 2 : 1;
    Walk<STATES> walk(x.c, x.sm);
    Unit u;
    unsigned g = 0;
    while (walk.next(u, false)) {
        float w[4];
        const int nv = p.V - u.tile * 128 > 64 ? 2 : 1;
        for (int j = 0; j < u.chunks; ++j, ++g) {
            const int n = min(kC, u.len - j * kC);
            if (j == 0 || n < kC) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int back = n - 1 - (i * 16 + tid / 8);
                    w[i] = back < 0 ? 0.0f : power(u.lg2, back);
                }
            }
            if (!x.wait(kFull + g % kStages, g / kStages)) return;
            if (g > 0 && !x.wait(kDsFull, g - 1)) return;  // the products that read the last K~ are done
            unsigned char *stage = x.sm.stage[g % kStages];
            for (int sub = 0; sub < nk; ++sub) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int at = sub * kSub + (i * 128 + tid) * 16;
                    const uint4 raw = *reinterpret_cast<const uint4 *>(stage + kTile + at);
                    const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
                    const bool keep = i * 16 + tid / 8 < n;
                    uint32_t o[3][4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float a = keep ? __uint_as_float(in[e] << 16) * w[i] : 0.0f;
                        float b = keep ? __uint_as_float(in[e] & 0xffff0000u) * w[i] : 0.0f;
                        o[0][e] = pack_bf16(a, b);
                        a -= __uint_as_float(o[0][e] << 16);
                        b -= __uint_as_float(o[0][e] & 0xffff0000u);
                        o[1][e] = pack_bf16(a, b);
                        if (x.c.parts == 3) {
                            a -= __uint_as_float(o[1][e] << 16);
                            b -= __uint_as_float(o[1][e] & 0xffff0000u);
                            o[2][e] = pack_bf16(a, b);
                        }
                    }
#pragma unroll
                    for (int part = 0; part < 3; ++part)
                        if (part < x.c.parts)
                            *reinterpret_cast<uint4 *>(x.sm.kt[part] + at) =
                                make_uint4(o[part][0], o[part][1], o[part][2], o[part][3]);
                }
            }
            if (n < kC) {
                for (int i = n * 8 + tid; i < kC * 8; i += 32 * kWarpsK)
                    for (int sub = 0; sub < nv; ++sub)
                        *reinterpret_cast<uint4 *>(stage + 2 * kTile + sub * kSub + i * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_async_smem();
            x.arrive(kKtFull);
        }
    }
}

// The state: lane = value index, 64 of its key indices in a thread's
// registers (warps 0-3: 0..63, warps 4-7: 64..127).
template <typename ST, bool STATES> __device__ void role_state(const Ctx &x, int warp, int lane) {
    const LaParams &p = x.c.p;
    const int quad = warp & 3, half = warp >> 2, v = quad * 32 + lane;
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    const bool mine = half * 64 < p.K;
    Walk<STATES> walk(x.c, x.sm);
    Unit u;
    unsigned g = 0;
    float s[64];
    while (walk.next(u, false)) {
        if (u.chunks == 0) continue;
        const bool on = mine && u.tile * 128 + v < p.V;
        const int k0 = half * 64, kn = min(64, p.K - k0);
        ST *pool = static_cast<ST *>(p.state) + (long long)u.slot * p.st_slot + (long long)u.h * p.st_head + u.tile * 128 + v;
        float *ws = x.c.ws + ((long long)u.x * p.nv + u.h) * p.K * p.V + u.tile * 128 + v;
        if (STATES) {
#pragma unroll
            for (int i = 0; i < 64; ++i) s[i] = 0.0f;
        } else if (x.c.seg) {
#pragma unroll
            for (int i = 0; i < 64; ++i) s[i] = on && i < kn ? ws[(long long)(k0 + i) * p.V] : 0.0f;
        } else {
#pragma unroll
            for (int i = 0; i < 64; ++i) s[i] = on && i < kn ? to_f32(pool[(long long)(k0 + i) * p.st_k]) : 0.0f;
        }
        const float lam_c = power(u.lg2, kC);
        for (int j = 0; j < u.chunks; ++j, ++g) {
            const int n = min(kC, u.len - j * kC);
            if (!STATES) {
                // the start state as matrix operand: s = hi + lo to 16 bits
                if (g > 0 && !x.wait(kSFree, g - 1)) return;
                if (mine) {
                    fence_after();
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        uint32_t hi[16], lo[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float a = s[32 * i + 2 * e], b = s[32 * i + 2 * e + 1];
                            hi[e] = pack_bf16(a, b);
                            lo[e] = pack_bf16(a - __uint_as_float(hi[e] << 16), b - __uint_as_float(hi[e] & 0xffff0000u));
                        }
                        tmem_st16(x.tmem + lanes + kColHi + half * 32 + i * 16, hi);
                        tmem_st16(x.tmem + lanes + kColLo + half * 32 + i * 16, lo);
                    }
                    wait_st();
                    fence_before();
                }
                x.arrive(kSFull);
            }
            const float lam_n = n == kC ? lam_c : power(u.lg2, n);
            if (!x.wait(kDsFull, g)) return;
            if (mine) {
                fence_after();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    uint32_t d[16];
                    tmem_ld16(x.tmem + lanes + kColDS + half * 64 + i * 16, d);
                    wait_ld();
#pragma unroll
                    for (int e = 0; e < 16; ++e) s[16 * i + e] = fmaf(lam_n, s[16 * i + e], __uint_as_float(d[e]));
                }
                fence_before();
            }
            x.arrive(kDsFree);
        }
        if (STATES) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
                if (on && i < kn) ws[(long long)(k0 + i) * p.V] = s[i];
        } else if (u.last) {
#pragma unroll
            for (int i = 0; i < 64; ++i)
                if (on && i < kn) pool[(long long)(k0 + i) * p.st_k] = from_f32<ST>(s[i]);
        }
    }
}

// P~ and the output.  A warp has 16 keys of P^T and 32 columns of O^T.
__device__ void role_out(const Ctx &x, int warp, int lane) {
    const LaParams &p = x.c.p;
    uint16_t *const out = static_cast<uint16_t *>(p.out);
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    const int row0 = warp * 16 + lane / 4;  // this thread's keys: row0 and row0 + 8
    const uint32_t pt = x.base + offsetof(Smem, pt);
    unsigned char *const ost = x.sm.ost[warp];
    // stmatrix: lane l names row l % 8 of matrix l / 8: keys +0, +8, +0, +8 of column blocks n, n, n + 1, n + 1
    const int srow = warp * 16 + (lane & 7) + ((lane >> 3) & 1) * 8, sblk = lane >> 4;
    Walk<false> walk(x.c, x.sm);
    Unit u;
    unsigned g = 0;
    int parity = 0;
    uint16_t *prev = nullptr;  // where the chunk before this one goes, its tokens and its factors
    int prev_n = 0, prev_w = 0;
    const float *prev_f = nullptr;
    // O^T of chunk g - 1 -> staging; tensor memory is free again when every lane has read
    auto collect = [&]() {
        if (!x.wait(kOFull, g - 1)) return false;
        fence_after();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t a[16], b[16];
            tmem_ld16(x.tmem + lanes + kColO1 + i * 16, a);
            tmem_ld16(x.tmem + lanes + kColO2 + i * 16, b);
            wait_ld();
            if (i == 3) {
                fence_before();
                x.arrive(kOFree);
            }
#pragma unroll
            for (int e = 0; e < 16; e += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(prev_f + i * 16 + e);
                const float o0 = fmaf(f.x, __uint_as_float(a[e]), __uint_as_float(b[e]));
                const float o1 = fmaf(f.y, __uint_as_float(a[e + 1]), __uint_as_float(b[e + 1]));
                const float o2 = fmaf(f.z, __uint_as_float(a[e + 2]), __uint_as_float(b[e + 2]));
                const float o3 = fmaf(f.w, __uint_as_float(a[e + 3]), __uint_as_float(b[e + 3]));
                const uint32_t lo = pack_bf16(o0, o1), hi = pack_bf16(o2, o3);
                uint16_t *to = reinterpret_cast<uint16_t *>(ost) + (i * 16 + e) * 32 + lane;
                to[0] = (uint16_t)lo;
                to[32] = (uint16_t)(lo >> 16);
                to[64] = (uint16_t)hi;
                to[96] = (uint16_t)(hi >> 16);
            }
        }
        return true;
    };
    auto write = [&]() {
        __syncwarp();
        const int c0 = (lane & 3) * 8;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const int t = r * 8 + lane / 4;
            if (t < prev_n && c0 < prev_w)
                *reinterpret_cast<uint4 *>(prev + (long long)t * p.o_ts + c0) =
                    *reinterpret_cast<const uint4 *>(ost + t * 64 + c0 * 2);
        }
        __syncwarp();
    };
    while (walk.next(u, warp == 0 && lane == 0)) {
        const int col = u.tile * 128 + warp * 32;
        if (u.skip_len) {
            const int w = min(32, p.V - col);
            if (lane < w)
                for (int t = 0; t < u.skip_len; ++t)
                    out[(long long)(u.skip_t0 + t) * p.o_ts + (long long)u.h * p.o_hs + col + lane] = 0;
        }
        if (u.chunks == 0) continue;
        parity ^= 1;
        float *factor = x.sm.factor[warp][parity];
        factor[lane] = p.scale * power(u.lg2, lane + 1);
        factor[lane + 32] = p.scale * power(u.lg2, lane + 33);
        float w[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            const int gap = 8 * (i >> 2) + 2 * (lane & 3) + (i & 1) - (row0 + ((i >> 1) & 1) * 8);
            w[i] = gap < 0 ? 0.0f : p.scale * power(u.lg2, gap);
        }
        __syncwarp();
        for (int j = 0; j < u.chunks; ++j, ++g) {
            const int n = min(kC, u.len - j * kC);
            if (g > 0 && !collect()) return;
            if (!x.wait(kPFull + (g & 1), g >> 1)) return;
            fence_after();
            uint32_t r[32];
            tmem_ld_16x64(x.tmem + lanes + kColP + (g & 1) * kC, r);
            wait_ld();
            fence_before();
            x.arrive(kPFree + (g & 1));
            // masked places are chosen, not multiplied: whatever they hold stays out
            const bool on0 = row0 < n, on1 = row0 + 8 < n;
            uint32_t h[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const bool on = (i & 1) ? on1 : on0;
                const float a = on && w[2 * i] != 0.0f ? __uint_as_float(r[2 * i]) * w[2 * i] : 0.0f;
                const float b = on && w[2 * i + 1] != 0.0f ? __uint_as_float(r[2 * i + 1]) * w[2 * i + 1] : 0.0f;
                h[i] = pack_bf16(a, b);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                stmatrix4(pt + srow * 128 + (((2 * i + sblk) ^ (srow & 7)) << 4), h[4 * i], h[4 * i + 1], h[4 * i + 2],
                          h[4 * i + 3]);
            fence_async_smem();
            x.arrive(kPtFull);
            if (g > 0) write();
            prev = out + (long long)(u.t0 + j * kC) * p.o_ts + (long long)u.h * p.o_hs + col;
            prev_n = n;
            prev_w = p.V - col;
            prev_f = factor;
        }
    }
    if (g > 0 && collect()) write();
}

template <typename ST, bool STATES>
__global__ void __launch_bounds__(kThreads, 1)
    k_la_chunk(const __grid_constant__ ChunkParams c, const __grid_constant__ CUtensorMap mq,
               const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw), pad = (1024u - (raw & 1023u)) & 1023u;
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw + pad);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = raw + pad, bars = base + (uint32_t)offsetof(Smem, bar);
    if (threadIdx.x == 0) {
        sm.gave_up = 0;
        for (int i = 0; i < kBars; ++i) {
            const bool by_p = i == kPFree || i == kPFree + 1 || i == kPtFull || i == kOFree;
            const bool by_s = i == kSFull || i == kDsFree;
            mbar_init(bars + 8 * i, by_p ? kWarpsP : by_s ? kWarpsS : i == kKtFull ? kWarpsK : 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
    }
    if (warp == kWarpMma) tmem_alloc(base + (uint32_t)offsetof(Smem, tmem), 512);
    if (warp == kWarpTma && lane == 0) {
        tma_prefetch_map(&mk);
        tma_prefetch_map(&mv);
        if (!STATES) tma_prefetch_map(&mq);
    }
    plan_rows(c, sm);
    fence_before();
    __syncthreads();
    fence_after();
    const Ctx x{c, sm, base, bars, sm.tmem};
    if (warp < kWarpsS) {
        role_state<ST, STATES>(x, warp, lane);
    } else if (warp < kWarpsS + kWarpsP) {
        if (!STATES) role_out(x, warp - kWarpsS, lane);
    } else if (warp < kWarpMma) {
        role_keys<STATES>(x, (int)threadIdx.x - 32 * (kWarpsS + kWarpsP));
    } else if (warp == kWarpMma) {
        if (lane == 0) role_mma<STATES>(x);
    } else {
        if (lane == 0) role_tma<STATES>(x, &mq, &mk, &mv);
    }
    __syncwarp();
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == kWarpMma) tmem_free(sm.tmem, 512);
    if (threadIdx.x == 0 && sm.gave_up) flag(c.p.status, GDR_STATUS_TIMEOUT);
}

// Start states of a split row's segments, in place over the segments' own
// contributions: S_0 = pool, S_(s+1) = lambda^seg S_s + D_s.
template <typename ST> __global__ void __launch_bounds__(256) k_la_join(const __grid_constant__ ChunkParams c) {
    const LaParams &p = c.p;
    const int h = blockIdx.y, r = blockIdx.z;  // r: rank of the row
    __shared__ int s_len[32];
    const int B = p.batch;
    if (threadIdx.x < 32) {
        int len = -1;
        if ((int)threadIdx.x < B) {
            const int t0 = p.offsets[threadIdx.x], t1 = p.offsets[threadIdx.x + 1];
            len = t0 < 0 || t1 < t0 || t1 > p.T ? 0 : t1 - t0;
        }
        s_len[threadIdx.x] = len;
    }
    __syncthreads();
    // the row of this rank, and the segments of the rows before it
    int b = 0, before = 0;
    for (int o = 0; o < B; ++o) {
        int rank = 0;
        for (int q = 0; q < B; ++q) rank += s_len[q] > s_len[o] || (s_len[q] == s_len[o] && q < o);
        if (rank == r) b = o;
        if (rank < r) before += max(1, (s_len[o] + c.seg - 1) / c.seg);
    }
    const int n = (s_len[b] + c.seg - 1) / c.seg, slot = p.slot_idx[b];
    const float d = p.decay[(long long)h * p.decay_s];
    const bool decay_ok = p.decay_is_log ? d <= 0.0f : (d >= 0.0f && d <= 1.0f);
    if (n == 0 || slot < 0 || slot >= p.max_slots || !decay_ok || (p.max_len > 0 && s_len[b] > p.max_len)) return;
    const float lam = power(p.decay_is_log ? d * 1.44269504088896340736f : log2f(d), c.seg);
    const int i = (blockIdx.x * 256 + threadIdx.x) * 4;  // V is a multiple of 16: four columns of one row
    if (i >= p.K * p.V) return;
    const int k = i / p.V, v = i - k * p.V;
    const ST *pool = static_cast<const ST *>(p.state) + (long long)slot * p.st_slot + (long long)h * p.st_head +
                     (long long)k * p.st_k + v;
    float4 s = make_float4(to_f32(pool[0]), to_f32(pool[1]), to_f32(pool[2]), to_f32(pool[3]));
    const long long step = (long long)p.nv * p.K * p.V;
    float *ws = c.ws + (long long)before * step + (long long)h * p.K * p.V + i;
    for (int j = 0; j < n; ++j, ws += step) {
        const float4 own = j + 1 < n ? *reinterpret_cast<const float4 *>(ws) : make_float4(0, 0, 0, 0);
        *reinterpret_cast<float4 *>(ws) = s;
        s.x = fmaf(lam, s.x, own.x);
        s.y = fmaf(lam, s.y, own.y);
        s.z = fmaf(lam, s.z, own.z);
        s.w = fmaf(lam, s.w, own.w);
    }
}

// ---- host -----------------------------------------------------------------------

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
    static const EncodeFn fn = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult st{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &st) != cudaSuccess ||
            st != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            f = nullptr;
        }
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

// [T, heads, dim] bfloat16 in boxes of 64 tokens x 64 channels of one head; what lies outside reads as zero.
bool encode(EncodeFn fn, CUtensorMap *map, const void *base, int dim, int heads, long long T, long long hs, long long ts) {
    if (heads == 1) hs = (dim + 7) / 8 * 8;  // not used: any valid stride
    if (T == 1) ts = (dim + 7) / 8 * 8;
    if (hs <= 0 || ts <= 0) return false;
    const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)T};
    const cuuint64_t strides[2] = {(cuuint64_t)hs * 2, (cuuint64_t)ts * 2};
    const cuuint32_t box[3] = {64, 1, (cuuint32_t)kC}, one[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, one,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename ST> cudaError_t go(ChunkParams c, const CUtensorMap *m, cudaStream_t s) {
    static LaunchCache cache;
    LaunchInfo li;
    constexpr int smem = (int)sizeof(Smem) + 1024;
    cudaError_t e = launch_info(cache, &li, [](LaunchInfo &) {
        cudaError_t r = cudaFuncSetAttribute(k_la_chunk<ST, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (r == cudaSuccess)
            r = cudaFuncSetAttribute(k_la_chunk<ST, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        return r;
    });
    if (e != cudaSuccess) return e;
    const LaParams &p = c.p;
    const long long per = (long long)p.nv * p.tiles;
    const long long rows = c.seg ? p.batch + p.T / c.seg : p.batch;
    const unsigned grid = (unsigned)(rows * per < li.sms ? rows * per : li.sms);
    if (c.seg) {
        k_la_chunk<ST, true><<<grid, kThreads, smem, s>>>(c, m[0], m[1], m[2]);
        const dim3 jg((unsigned)((p.K * p.V + 1023) / 1024), (unsigned)p.nv, (unsigned)p.batch);
        k_la_join<ST><<<jg, 256, 0, s>>>(c);
    }
    k_la_chunk<ST, false><<<grid, kThreads, smem, s>>>(c, m[0], m[1], m[2]);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_la_chunk(const LaParams &p, bool state_bf16, int seg, void *ws, cudaStream_t s, bool *used) {
    *used = false;
    const EncodeFn fn = encode_fn();
    CUtensorMap m[3];
    if (!fn || !encode(fn, &m[0], p.q, p.K, p.nk, p.T, p.q_hs, p.q_ts) ||
        !encode(fn, &m[1], p.k, p.K, p.nk, p.T, p.k_hs, p.k_ts) || !encode(fn, &m[2], p.v, p.V, p.nv, p.T, p.v_hs, p.v_ts))
        return cudaSuccess;
    *used = true;
    ChunkParams c{p, seg, state_bf16 ? 2 : 3, static_cast<float *>(ws)};
    return state_bf16 ? go<uint16_t>(c, m, s) : go<float>(c, m, s);
}

}  // namespace gdr
