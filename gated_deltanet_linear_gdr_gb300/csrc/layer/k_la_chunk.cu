// Decayed linear attention, chunked form on the tensor cores (bfloat16 tokens).
//
// A row is taken 64 tokens at a time.  With S0 the state before a chunk of n
// tokens, i and j counted inside it:
//
//     P^T[j, i]  = k_j . q_i                                   (K Q^T)
//     P~^T[j, i] = scale lambda^(i-j) P^T[j, i] for j <= i, else 0
//     O^T[:, i]  = scale lambda^(i+1) (S0^T q_i)  +  V^T P~^T[:, i]
//     S^T        = lambda^n S0^T + V^T K~,  K~[j] = lambda^(n-1-j) k_j
//
// Everything is kept transposed (value index = tensor memory lane), so that
// the state, which a warp's lanes hold in float32 registers, goes back into
// tensor memory as the A operand of S0^T Q^T, and V^T serves two products.
// Operands made here go in as bfloat16 parts, each the rounding of what the ones
// before leave: P~ and the state as operand of the readout in two (16 bits), K~
// in two (bfloat16 pool) or three (float32 pool).  So results are rounded once,
// whatever cancels in their sums.  (One part for P~ and the state, 8 bits, made
// outputs off by 2.1e-3 of their norm for 1.7e-3, and by all of it where the
// history cancels; it was 4 to 13% faster with 128 key channels.)
//
// One CTA per SM walks (row segment, value head, 128-column tile) units, with
// a warp role for each step: 8 warps keep S, 4 make K~, 4 make P~, 4 write the
// output, one each issues K Q^T, the state's product and the output's two, and
// one loads three chunks ahead by TMA.  Roles hand over through mbarriers, so
// the products of a chunk run under the elementwise work of its neighbours.
// (One issuing warp for all products of a chunk was the slowest of the roles.)
//
// Bound: what an SM has beside its share of HBM.  A chunk of one head with K = V =
// 128 moves 64 KiB, 1.47 us of that share; with every SM at work it takes 1.95.
// The six roles' code does not fit the nearest instruction cache (17% of stalls),
// and their loads and stores take 43% of shared memory's cycles beside the 45% in
// which the tensor cores read it; the role that makes K~ waits for both most.
// 4 rows of 4096 tokens x 38 heads, a unit an SM, take 126 us with a bfloat16 pool
// (76% of the measured copy rate) and 132 with a float32 pool; heads of 64 x 64 79
// us (60%).  A row alone on its SM takes 1.5 us a chunk (64 x 64: 1.1).  A unit costs
// 5 us to begin and end, of which its state's exchange takes 1.5: rows of one chunk
// are the costly ones.
#include "tc.cuh"

#include "layer_internal.h"

namespace gdr {
namespace {

using namespace tc;

// Key channels are padded to KP = 64 or 128: TMA reads zeros past K, and zeros
// add nothing to any of the products.
constexpr int kC = 64;        // tokens a chunk
constexpr int kSub = kC * 128;        // bytes of a 64-token x 64-channel operand block
constexpr int kTile = 2 * kSub;       // bytes of a 64-token x 128-channel operand
// The chunks on their way in, K | V | Q, or K | V where only states are computed,
// and after them K~ but for its first part, which takes K's place, of two
// chunks: with two parts it fills half of its room, and a state on its way has
// the rest.  Half as many key channels leave room for more chunks, without which
// loads, not roles, set the pace (4 rows of 4096 tokens x 38 heads of 64 x 64: 85
// us with three, 76 with five, both with one part of the readout's operands).
template <int KP, bool STATES> struct Ring {
    static constexpr int KB = KP / 64 * kSub;  // K's bytes, or Q's
    static constexpr int V = KB, Q = KB + kTile, BYTES = STATES ? KB + kTile : 2 * KB + kTile;
    static constexpr int N = KP == 64 ? (STATES ? 6 : 5) : (STATES ? 4 : 3);
    static constexpr int KT = KP == 64 ? 10 * kTile : 9 * kTile;  // of both kinds
    static constexpr int STATE = KT + 2 * KB;
    static constexpr int OST = 12 * kTile;  // with 64 key channels, where output is turned
    static_assert(N * BYTES <= KT && KT + 4 * KB <= (KP == 64 ? OST : 13 * kTile) && STATE + KP * 256 <= (KP == 64 ? OST : 13 * kTile), "ring");
};
constexpr int kMaxStages = 6;
constexpr int kMaxRows = 64, kMaxHeads = 64;  // rows and heads whose facts are kept in shared memory
constexpr int kPlanned = 16;                  // rows whose units are dealt by load

// Warps by role, in warpgroups of 4.  The issuers and the loader come first:
// between ready warps the scheduler prefers the older.
constexpr int kWarpsS = 8, kWarpsO = 4, kWarpsP = 4, kWarpsK = 4;
constexpr int kWarpMma = 0, kWarpS = 4, kWarpO = kWarpS + kWarpsS, kWarpP = kWarpO + kWarpsO, kWarpK = kWarpP + kWarpsP;
constexpr int kThreads = 32 * (kWarpK + kWarpsK);
// Registers a thread: 768 threads are launched with 80, and the roles share them out anew.
constexpr int kRegsS = 112, kRegsO = 96, kRegsP = 80, kRegsK = 48, kRegsRest = 32;
static_assert(2 * kRegsS + kRegsO + kRegsP + kRegsK + kRegsRest == 6 * 80, "shares");

// Without output to make, the warps of P~ and O make K~ too.
template <bool STATES> constexpr int kTeams = STATES ? 3 : 1;

// Tensor memory columns: P^T, S0^T Q^T, V^T P~^T, V^T K~, the start state's two
// parts.  All 512 are in use: with 64 key channels P^T and the start state have
// two places, for one chunk and the next, with 128 only one.
template <int KP> struct Cols {
    static constexpr bool TWO = KP == 64;
    static constexpr uint32_t P = 0, O1 = TWO ? 128 : 64, O2 = O1 + 128, DS = O2 + 64, S = 384, PART = KP / 2;
    static constexpr uint32_t next(uint32_t odd) { return TWO ? odd * 64 : 0; }  // of P^T or the start state
    static_assert(DS + KP <= S && S + (TWO ? 2 : 1) * 2 * PART <= 512, "tensor memory");
};

enum Bar {
    kLoaded = 0, kStageFree = kLoaded + kMaxStages, kPFull = kStageFree + kMaxStages, kPFree = kPFull + 2,
    kPtFull = kPFree + 2, kSFull, kDsFull = kSFull + 2, kDsFree = kDsFull + 2, kKtFull, kOFull = kKtFull + 2,
    kOFree = kOFull + 2, kO1Full, kStateIn = kO1Full + 2, kStateTurn, kDrain, kBars
};

struct Smem {
    unsigned char ring[13 * kTile];       // Ring
    unsigned char pt[kSub];               // P~^T, its first part
    union {
        unsigned char pt_rest[kSub];      // and its second
        int load[kThreads / 4];           // before any: what each CTA has to do so far, in chunks (plan_rows)
    };
    uint64_t bar[kBars];
    int row_t0[kMaxRows], row_len[kMaxRows], row_slot[kMaxRows];  // by rank: the longest row first; len -1: bad offsets
    int first[kMaxRows + 1];                                      // a ranked row's first segment
    float lg2[kMaxHeads];                                         // log2 lambda, NaN where the decay is bad
    int rank[kPlanned];                                           // of this CTA, for each planned row
    int planned;
    uint32_t tmem;
    int gave_up, state_loads, next_len;
    float next_lg2;
};
static_assert(sizeof(Smem) + 1024 <= 232448 && offsetof(Smem, ring) == 0, "shared memory");
// Ordinary accesses are ordered before a TMA copy into the same bytes by a proxy
// fence only; nothing but barriers lies between the deal and the first copies,
// so it keeps to bytes that no copy writes.
static_assert(offsetof(Smem, load) >= sizeof(Smem::ring), "the deal's memory is not TMA's");

struct ChunkParams {
    LaParams p;
    int seg;    // tokens a segment (a multiple of kC), or 0: rows are whole
    float *ws;  // start states of the segments [segment, nv, K, V] (seg != 0)
    FastDiv per, tiles;  // units a segment (nv * tiles), column tiles
};

// A unit of work, the same for every role: one segment of a row, one head, one column tile.
struct Unit {
    int h, tile, slot;
    int t0, len;  // tokens of the segment; len 0: nothing to compute
    int chunks;
    int x;        // segment number
    bool last;                 // of its row
    int skip_t0, skip_len;     // a skipped row's tokens, whose output is zero
    float lg2;                 // log2 lambda
};

__device__ __forceinline__ float power(float lg2, int n) { return n == 0 ? 1.0f : exp2f(lg2 * (float)n); }
// The same to 2^-22, 0 below float32's normal range: for weights that end in bfloat16.
__device__ __forceinline__ float power_fast(float lg2, int n) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(lg2 * (float)n));
    return n == 0 ? 1.0f : y;
}

// A row's length, or -1 where its offsets are not sound.
__device__ __forceinline__ int sound_len(const LaParams &p, int t0, int t1) {
    return t0 < 0 || t1 < t0 || t1 > p.T ? -1 : t1 - t0;
}
// Cut rows, one a lane of a warp: -1 too for a row that begins before an earlier
// one's end.  Rows that lie apart have at most T / seg + batch segments, which
// is what the workspace holds.
__device__ __forceinline__ int apart(int t0, int len) {
    int end = max(len < 0 ? 0 : t0 + len, 0);
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, end, m);
        if ((int)(threadIdx.x & 31) >= m) end = max(end, o);
    }
    const int before = __shfl_up_sync(0xffffffffu, end, 1);
    return (threadIdx.x & 31) && t0 < before ? -1 : len;
}
// log2 of a head's decay; NaN for one outside [0, 1].
__device__ __forceinline__ float log2_lambda(const LaParams &p, int h) {
    const float d = p.decay[(long long)h * p.decay_s];
    const bool ok = p.decay_is_log ? d <= 0.0f : (d >= 0.0f && d <= 1.0f);
    return !ok ? __int_as_float(0x7fffffff) : p.decay_is_log ? d * 1.44269504088896340736f : log2f(d);
}

// Walks this CTA's units.  Few rows: row by row, the longest first, each row's
// units to the CTAs with the least to do so far (plan_rows).  Otherwise
// positions blockIdx.x, then back and forth, so that units sorted by length are
// dealt evenly.
template <bool STATES> struct Walk {
    const ChunkParams &c;
    const Smem &sm;
    int i = 0, row = 0;
    __device__ Walk(const ChunkParams &c_, const Smem &sm_) : c(c_), sm(sm_) {}

    // The next unit; every lane has the same, and the compiler is told so.
    __device__ __forceinline__ bool next(Unit &u, bool report) {
        const bool more = find(u, report);
        u.h = (int)uniform(u.h);
        u.tile = (int)uniform(u.tile);
        u.t0 = (int)uniform(u.t0);
        u.len = (int)uniform(u.len);
        u.chunks = (int)uniform(u.chunks);
        u.x = (int)uniform(u.x);
        u.slot = (int)uniform(u.slot);
        return uniform(more) != 0;
    }
    __device__ bool find(Unit &u, bool report) {
        const LaParams &p = c.p;
        u.t0 = u.x = u.h = u.tile = u.len = u.chunks = u.skip_len = u.slot = 0;
        const unsigned G = gridDim.x;
        unsigned ht;
        if (sm.planned) {
            for (;; ++row, i = 0) {
                if (row >= p.batch) return false;
                ht = (unsigned)sm.rank[row] + (unsigned)i * G;
                if (ht < c.per.d) break;
            }
            ++i;
            u.x = row;
        } else {
            const unsigned pos = (unsigned)i * G + ((i & 1) ? G - 1 - blockIdx.x : blockIdx.x);
            ++i;
            u.x = (int)c.per.div(pos);  // positions are below 2^31 and a walk ends at the first one past the units
            ht = pos - (unsigned)u.x * c.per.d;
        }
        u.h = (int)c.tiles.div(ht);
        u.tile = (int)(ht - (unsigned)u.h * c.tiles.d);
        int seg_i = 0, r0, len;
        if (p.batch <= kMaxRows) {
            int r = u.x;
            if (c.seg) {
                if (u.x >= sm.first[p.batch]) return false;
                r = 0;
                while (sm.first[r + 1] <= u.x) ++r;
                seg_i = u.x - sm.first[r];
            } else if (r >= p.batch) {
                return false;
            }
            r0 = sm.row_t0[r];
            len = sm.row_len[r];
            u.slot = sm.row_slot[r];
        } else {
            if (u.x >= p.batch) return false;
            r0 = p.offsets[u.x];
            len = sound_len(p, r0, p.offsets[u.x + 1]);
            u.slot = p.slot_idx[u.x];
        }
        u.lg2 = u.h < kMaxHeads ? sm.lg2[u.h] : log2_lambda(p, u.h);
        u.last = true;
        const bool leader = report && u.h == 0 && u.tile == 0 && seg_i == 0;
        if (len < 0) {
            if (leader) flag(p.status, GDR_STATUS_BAD_OFFSETS);
            return true;
        }
        const bool too_long = p.max_len > 0 && len > p.max_len, bad_decay = isnan(u.lg2);
        if (len > 0 && (u.slot < 0 || u.slot >= p.max_slots || bad_decay || too_long)) {
            if (too_long) {
                if (leader) flag(p.status, GDR_STATUS_ROW_TOO_LONG);
            } else if (u.slot < -1 || u.slot >= p.max_slots) {
                if (leader) flag(p.status, GDR_STATUS_BAD_SLOT);
            } else if (u.slot >= 0 && report) {
                flag(p.status, GDR_STATUS_BAD_DECAY);
            }
            if (seg_i == 0) {
                u.skip_t0 = r0;
                u.skip_len = len;
            }
            return true;
        }
        u.t0 = r0;
        u.len = len;
        if (c.seg) {
            const int at = seg_i * c.seg;
            u.last = u.len - at <= c.seg;
            u.t0 += at;
            u.len = u.last ? u.len - at : c.seg;
            if (STATES && u.last) u.len = 0;
        }
        u.chunks = pieces(u.len, kC);
        return true;
    }
};

// Facts of the rows, by descending length, and of the heads; the number of each row's first segment.
__device__ __forceinline__ void plan_rows(const ChunkParams &c, Smem &sm) {
    const LaParams &p = c.p;
    const int B = p.batch, tid = threadIdx.x;
    if (tid >= 128 && tid < 128 + min(p.nv, kMaxHeads)) sm.lg2[tid - 128] = log2_lambda(p, tid - 128);
    int len = -1, t0 = 0, slot = -1;
    if (B <= kMaxRows && tid < B) {
        t0 = p.offsets[tid];
        len = sound_len(p, t0, p.offsets[tid + 1]);
        slot = p.slot_idx[tid];
    }
    if (c.seg && tid < 32) len = apart(t0, len);  // batch <= 32
    if (B <= kMaxRows && tid < B) sm.first[tid] = len;
    __syncthreads();
    int rank = 0;
    if (B <= kMaxRows && tid < B) {
        for (int o = 0; o < B; ++o) rank += sm.first[o] > len || (sm.first[o] == len && o < tid);
        sm.row_t0[rank] = t0;
        sm.row_len[rank] = len;
        sm.row_slot[rank] = slot;
    }
    __syncthreads();
    // few rows, one of them long: every CTA works out the same deal.  (Back and
    // forth alone, 8 rows of 512 to 4096 tokens x 32 heads lasted 80 chunks
    // where 66 are possible.)
    const int G = (int)gridDim.x;
    const bool planned = !c.seg && B <= kPlanned && (unsigned)B * c.per.d > gridDim.x && 4 * G <= kThreads && sm.row_len[0] >= 8 * kC;
    if (tid == 0) sm.planned = planned;
    if (planned) {
        int *const load = sm.load;
        const int cta = tid >> 2, part = tid & 3;  // four threads compare for a CTA
        for (int o = tid; o < G; o += kThreads) load[o] = 0;
        __syncthreads();
        for (int r = 0; r < B; ++r) {
            int n = 0;
            if (cta < G) {
                const int mine = load[cta];
                for (int o = part; o < G; o += 4) n += load[o] < mine || (load[o] == mine && o < cta);
            }
            n += __shfl_xor_sync(0xffffffffu, n, 1);
            n += __shfl_xor_sync(0xffffffffu, n, 2);
            __syncthreads();
            if (cta < G && part == 0) {
                const int heads = (int)c.per.d, units = n < heads ? (heads - n - 1) / G + 1 : 0;
                load[cta] += units * (pieces(sm.row_len[r], kC) + 2);  // two chunks' time to begin and end one
                if (cta == (int)blockIdx.x) sm.rank[r] = n;
            }
            __syncthreads();
        }
    }
    if (c.seg && tid < 32) {  // one lane a row
        int end = tid < B ? max(1, pieces(sm.row_len[tid], c.seg)) : 0;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, end, m);
            if (tid >= m) end += o;
        }
        if (tid < B) sm.first[tid + 1] = end;
        if (tid == 0) sm.first[0] = 0;
    }
    __syncthreads();
}

// ---- the roles ----------------------------------------------------------------

// A phase's parity is never ambiguous: a barrier completes its phase for chunk
// g + 1 (of a pair of barriers: g + 2) only after every waiter has passed the
// one for chunk g, since each waiter's own work for g is among what that takes.
struct Ctx {
    const ChunkParams &c;
    Smem &sm;
    uint32_t base;  // shared address of sm
    uint32_t bars;
    uint32_t tmem;
    __device__ uint32_t bar(int i) const { return bars + 8u * (uint32_t)i; }
    // The answer is the warp's, so that loops that end by it keep the warp together.
    __device__ bool wait(int i, uint32_t parity) const {
        return __all_sync(0xffffffffu, mbar_wait(bar(i), parity & 1u, &sm.gave_up));
    }
    // one arrival for the warp, once every lane has got here
    __device__ void arrive(int i) const {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(bar(i));
    }
};

// Chunks in order, into the stages.
template <int KP, bool ST2, bool STATES> struct Loader {  // ST2: a bfloat16 pool
    const Ctx &x;
    const CUtensorMap *mq, *mk, *mv;
    Walk<STATES> walk;
    Unit u;
    int j;
    unsigned g = 0;
    bool more = true;
    __device__ Loader(const Ctx &x_, const CUtensorMap *q, const CUtensorMap *k, const CUtensorMap *v)
        : x(x_), mq(q), mk(k), mv(v), walk(x_.c, x_.sm), j(0) {
        u.chunks = 0;
    }

    // Asks L2 for the unit's start state, which its warps will want in up to
    // three chunks' time: 4 lanes a key index, 128 bytes of it each.
    __device__ void fetch_state() {
        const LaParams &p = x.c.p;
        const int lane = threadIdx.x & 31, es = x.c.seg || !ST2 ? 4 : 2, bytes = min(128, p.V - u.tile * 128) * es;
        const char *from;
        long long step;
        if (x.c.seg) {
            from = reinterpret_cast<const char *>(x.c.ws + ((long long)u.x * p.nv + u.h) * p.K * p.V + u.tile * 128);
            step = (long long)p.V * 4;
        } else {
            from = static_cast<const char *>(p.state) + ((long long)u.slot * p.st_slot + (long long)u.h * p.st_head + u.tile * 128) * es;
            step = p.st_k * es;
        }
        const int at = (lane & 3) * 128;
        if (at < bytes)
            for (int k = lane >> 2; k < p.K; k += 8)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(from + (long long)k * step + at));
    }

    // Loads the next chunk, if there is one, once its stage is free; false where a wait gave up.
    __device__ bool step() {
        while (more && j >= u.chunks) {
            more = walk.next(u, false);
            j = 0;
            if (!STATES && more && u.chunks > 0) fetch_state();
        }
        if (!more) return true;
        using R = Ring<KP, STATES>;
        const int s = g % R::N;
        if (g >= R::N && !x.wait(kStageFree + s, g / R::N - 1)) return false;
        if (elect_one()) {
            const LaParams &p = x.c.p;
            constexpr int nk = KP / 64;
            const int v0 = u.tile * 128, nv = p.V - v0 > 64 ? 2 : 1, hk = u.h / p.r, t = u.t0 + j * kC;
            const uint32_t dst = x.base + s * R::BYTES, full = x.bar(kLoaded + s);
            mbar_expect(full, (uint32_t)((STATES ? 1 : 2) * nk + nv) * kSub);
#pragma unroll
            for (int i = 0; i < nk; ++i) {
                tma_load3(dst + i * kSub, mk, i * 64, hk, t, full);
                if (!STATES) tma_load3(dst + R::Q + i * kSub, mq, i * 64, hk, t, full);
            }
            for (int i = 0; i < nv; ++i) tma_load3(dst + R::V + i * kSub, mv, v0 + i * 64, u.h, t, full);
        }
        __syncwarp();
        ++g;
        ++j;
        return true;
    }
    // No copy is in flight when the CTA ends.
    __device__ void drain() {
        volatile int never = 0;
        constexpr unsigned N = Ring<KP, STATES>::N;
        for (unsigned o = g > N ? g - N : 0; o < g; ++o) mbar_wait(x.bar(kLoaded + o % N), (o / N) & 1u, &never);
    }
};

// The issuing warps.  How many chunks this CTA has:
template <bool STATES> __device__ __forceinline__ unsigned count_chunks(const Ctx &x) {
    Walk<STATES> walk(x.c, x.sm);
    Unit u;
    unsigned total = 0;
    while (walk.next(u, false)) total += (unsigned)u.chunks;
    return total;
}
// No product is under way when tensor memory is freed.
__device__ __forceinline__ void drain_mma(const Ctx &x) {
    __syncwarp();
    mma_commit(elect_one(), x.bar(kDrain));
    volatile int never = 0;
    mbar_wait(x.bar(kDrain), 0, &never);
}

// P^T = K Q^T
template <int KP> __device__ void role_mma_scores(const Ctx &x) {
    using R = Ring<KP, false>;
    const uint32_t id = idesc_bf16(64, kC, false, false);
    const uint64_t d_km = desc128(x.base, 16, 1024);  // stage 0, K-major
    const unsigned total = count_chunks<false>(x);
    for (unsigned g = 0; g < total; ++g) {
        // the place has been read, and the product before last, whose barrier this one's is, seen by both its waiters
        constexpr unsigned ago = Cols<KP>::TWO ? 2 : 1;
        if (g >= ago && !x.wait(kPFree + ((g - ago) & 1), (g - ago) >> 1)) break;
        if (g > 1 && !x.wait(kKtFull + (g & 1), (g >> 1) - 1)) break;
        if (!x.wait(kLoaded + g % R::N, g / R::N)) break;
        fence_after();
        const uint32_t me = elect_one(), st = uniform(g % R::N), odd = uniform(g & 1);
        const uint64_t k = d_km + (st * R::BYTES >> 4), q = k + (R::Q >> 4);
        mma_ss_k<KP / 16>(me, x.tmem + Cols<KP>::P + Cols<KP>::next(odd), k, q, id, kSub);
        mma_commit(me, x.bar(kPFull) + 8 * odd);
    }
    drain_mma(x);
}

// V^T K~.  For a segment's own state (STATES) the weights count to the segment's
// end and all of its chunks add up in tensor memory; else each chunk's is read.
template <int KP, int PARTS, bool STATES> __device__ void role_mma_state(const Ctx &x) {
    using R = Ring<KP, STATES>;
    const uint32_t id = idesc_bf16(128, KP, true, true);
    const uint64_t d_mn = desc128(x.base, kSub, 1024);  // stage 0, MN-major
    const uint64_t d_kt = desc128(x.base + R::KT, kSub, 1024);
    Walk<STATES> walk(x.c, x.sm);
    Unit u;
    unsigned g = 0, reads = 0;
    while (walk.next(u, false)) {
        for (int j = 0; j < u.chunks; ++j, ++g) {
            const bool fresh = !STATES || j == 0;
            if (!x.wait(kLoaded + g % R::N, g / R::N) || !x.wait(kKtFull + (g & 1), g >> 1)) return;
            if (fresh) {
                if (reads > 0 && !x.wait(kDsFree, reads - 1)) return;
                ++reads;
            }
            fence_after();
            const uint32_t me = elect_one(), st = uniform(g % R::N), odd = uniform(g & 1);
            const uint64_t k = d_mn + (st * R::BYTES >> 4), v = k + (R::V >> 4), kt = d_kt + (odd * (PARTS - 1) * R::KB >> 4);
            const uint32_t ds = x.tmem + Cols<KP>::DS;
            if (fresh)
                mma_ss_mn64<false>(me, ds, v, k, id);
            else
                mma_ss_mn64<true>(me, ds, v, k, id);
            mma_ss_mn64<true>(me, ds, v, kt, id);
            if (PARTS == 3) mma_ss_mn64<true>(me, ds, v, kt + (R::KB >> 4), id);
            mma_commit(me, x.bar(kDsFull) + 8 * odd);
            if (STATES && j + 1 == u.chunks) mma_commit(me, x.bar(kOFull));
            mma_commit(me, x.bar(kStageFree) + 8 * st);
        }
    }
}

// S0^T Q^T and V^T P~^T, two parts each.
template <int KP> __device__ void role_mma_out(const Ctx &x) {
    using R = Ring<KP, false>;
    const uint32_t id1 = idesc_bf16(128, kC, false, false), id2 = idesc_bf16(128, kC, true, true);
    const uint64_t d_km = desc128(x.base + R::Q, 16, 1024), d_v = desc128(x.base + R::V, kSub, 1024);
    const uint64_t d_pt = desc128(x.base + (uint32_t)offsetof(Smem, pt), kSub, 1024);
    const uint64_t d_rest = desc128(x.base + (uint32_t)offsetof(Smem, pt_rest), kSub, 1024);
    const unsigned total = count_chunks<false>(x);
    for (unsigned g = 0; g < total; ++g) {
        if (!x.wait(kLoaded + g % R::N, g / R::N) || !x.wait(kSFull + (g & 1), g >> 1)) break;
        fence_after();
        const uint32_t me = elect_one(), st = uniform(g % R::N), odd = uniform(g & 1);
        const uint64_t q = d_km + (st * R::BYTES >> 4), v = d_v + (st * R::BYTES >> 4);
        using C = Cols<KP>;
        const uint32_t o1 = x.tmem + C::O1 + odd * kC;  // read for the chunk before last, as kOFree has said for the last one
        const uint32_t s0 = x.tmem + C::S + C::next(odd);
        mma_ts_k<KP / 16, false>(me, o1, s0, q, id1, kSub);
        mma_ts_k<KP / 16, true>(me, o1, s0 + C::PART, q, id1, kSub);
        mma_commit(me, x.bar(kO1Full) + 8 * odd);
        if (!x.wait(kPtFull, g) || (g > 0 && !x.wait(kOFree, g - 1))) break;
        fence_after();
        mma_ss_mn64<false>(me, x.tmem + C::O2, v, d_pt, id2);
        mma_ss_mn64<true>(me, x.tmem + C::O2, v, d_rest, id2);
        mma_commit(me, x.bar(kOFull) + 8 * odd);
        mma_commit(me, x.bar(kStageFree) + 8 * st);
    }
    drain_mma(x);
}

// In a row's last chunk the tokens past its end belong to somebody else.  They
// are cleared in V, since zero times infinity is not zero, by both roles
// whose products read V, each before its own.
__device__ __forceinline__ void clear_tail(unsigned char *v, int n, int nv, int tid, int threads) {
    for (int i = n * 8 + tid; i < kC * 8; i += threads)
        for (int sub = 0; sub < nv; ++sub) *reinterpret_cast<uint4 *>(v + sub * kSub + i * 16) = make_uint4(0, 0, 0, 0);
}

// K~[j] = w_j k_j, w_j = lambda^(n-1-j), in PARTS bfloat16 parts, at the places K
// has in its swizzled block: a thread has 16-byte vectors of 4 tokens.
// Two parts in bfloat16 arithmetic: with w = a + b (a, b bfloat16, b the rest),
//     hi = rn(k a),  k a - hi exactly (it has 8 bits),  mid = rn(k b + (k a - hi)),
// three instructions a pair, off by 2^-17 of the product.  Three parts in
// float32, each the rounding of what the ones before leave.
// `team` of TEAMS warpgroups takes the 16-token blocks team, team + TEAMS, ..
template <int KP, int PARTS, bool STATES, int TEAMS> __device__ void role_keys(const Ctx &x, int team, int warp, int lane) {
    const LaParams &p = x.c.p;
    const int tid = warp * 32 + lane, row = tid / 8;
    Walk<STATES> walk(x.c, x.sm);
    Unit u;
    unsigned g = 0;
    while (walk.next(u, false)) {
        const int nv = p.V - u.tile * 128 > 64 ? 2 : 1;
        const int last = (3 - team) / TEAMS * TEAMS + team;  // this team's last block
        const float lam_b = power(u.lg2, 16 * TEAMS);
        float w_last = 0.0f;  // weight of this thread's token there
        for (int j = 0; j < u.chunks; ++j, ++g) {
            const int n = min(kC, u.len - j * kC);
            if (STATES || j == 0 || n < kC)
                w_last = power(u.lg2, max((STATES ? u.len - j * kC : n) - 1 - (16 * last + row), 0));
            using R = Ring<KP, STATES>;
            if (!x.wait(kLoaded + g % R::N, g / R::N)) return;
            unsigned char *stage = x.sm.ring + g % R::N * R::BYTES;
            if (__builtin_expect(n < kC, 0)) clear_tail(stage + R::V, n, nv, tid, 32 * kWarpsK);
            if (!STATES && !x.wait(kPFull + (g & 1), g >> 1)) return;           // K Q^T has read K
            if (g > 1 && !x.wait(kDsFull + (g & 1), (g >> 1) - 1)) return;  // and the product before last its K~
            unsigned char *const rest = x.sm.ring + R::KT + (g & 1) * (PARTS - 1) * R::KB;
            // small loops: the roles share the instruction caches
            float w = w_last;
#pragma unroll 1
            for (int i = last; i >= 0; i -= TEAMS) {
                const int back = n - 1 - (i * 16 + row);
                if (n < kC) w = back < 0 ? 0.0f : power(u.lg2, back);
                const __nv_bfloat162 wa = __float2bfloat162_rn(w);
                const __nv_bfloat162 wb = __float2bfloat162_rn(w - __low2float(wa));
#pragma unroll
                for (int sub = 0; sub < KP / 64; ++sub) {
                    const int at = sub * kSub + tid * 16 + i * 2048;
                    uint4 *const here = reinterpret_cast<uint4 *>(stage + at);
                    uint4 raw = *here;
                    if (back < 0) raw = make_uint4(0, 0, 0, 0);
                    const uint32_t in[4] = {raw.x, raw.y, raw.z, raw.w};
                    uint32_t o[3][4];
                    if constexpr (PARTS == 2) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const __nv_bfloat162 k = *reinterpret_cast<const __nv_bfloat162 *>(&in[e]);
                            const __nv_bfloat162 hi = __hmul2_rn(k, wa), mid = __hfma2(k, wb, __hfma2(k, wa, __hneg2(hi)));
                            o[0][e] = *reinterpret_cast<const uint32_t *>(&hi);
                            o[1][e] = *reinterpret_cast<const uint32_t *>(&mid);
                        }
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float2 r = __fmul2_rn(unpack_bf16(in[e]), make_float2(w, w));
                            o[0][e] = pack_bf16(r);
                            r = rest_bf16(r, o[0][e]);
                            o[1][e] = pack_bf16(r);
                            o[2][e] = pack_bf16(rest_bf16(r, o[1][e]));
                        }
                    }
                    *here = make_uint4(o[0][0], o[0][1], o[0][2], o[0][3]);
#pragma unroll
                    for (int part = 1; part < PARTS; ++part)
                        *reinterpret_cast<uint4 *>(rest + (part - 1) * R::KB + at) =
                            make_uint4(o[part][0], o[part][1], o[part][2], o[part][3]);
                }
                w *= lam_b;
            }
            fence_async_smem();
            x.arrive(kKtFull + (g & 1));
        }
    }
}

// The state: lane = value index, half of its key indices in a thread's
// registers (warps 0-3 the first half, warps 4-7 the second).
template <int KP> struct StateRole {
    static constexpr int KEYS = KP / 2, N = KEYS / 2;  // a thread's keys, and pairs of them
    int half, v;
    uint32_t lanes;
    __device__ StateRole(int warp, int lane)
        : half(warp >> 2), v((warp & 3) * 32 + lane), lanes((uint32_t)((warp & 3) * 32) << 16) {}
};

// s = lam s + what V^T K~ has left in tensor memory.
template <int KP>
__device__ __forceinline__ void state_add(const Ctx &x, const StateRole<KP> &r, float2 (&s)[KP / 4], float lam) {
    fence_after();
    const float2 l2 = make_float2(lam, lam);
#pragma unroll
    for (int i = 0; i < r.KEYS / 16; ++i) {
        uint32_t d[16];
        tmem_ld16(x.tmem + r.lanes + Cols<KP>::DS + r.half * r.KEYS + i * 16, d);
        wait_ld();
#pragma unroll
        for (int e = 0; e < 8; ++e)
            s[8 * i + e] = __ffma2_rn(l2, s[8 * i + e], make_float2(__uint_as_float(d[2 * e]), __uint_as_float(d[2 * e + 1])));
    }
    fence_before();
    x.arrive(kDsFree);
}

// A unit's chunks; false where a wait gave up.
template <int KP>
__device__ __forceinline__ bool state_chunks(const Ctx &x, const StateRole<KP> &r, float2 (&s)[KP / 4], unsigned &g, int len,
                                             float lg2) {
    using C = Cols<KP>;
    const float lam_c = power(lg2, kC);
    for (int left = len; left > 0; left -= kC, ++g) {
        // the start state as matrix operand, in two parts, once the product that read its place last is done
        constexpr unsigned ago = C::TWO ? 2 : 1;
        if (g >= ago && !x.wait(kO1Full + ((g - ago) & 1), (g - ago) >> 1)) return false;
        fence_after();
        const uint32_t to = x.tmem + r.lanes + C::S + C::next(g & 1) + r.half * r.N;
#pragma unroll
        for (int i = 0; i < r.N / 8; ++i) {  // in pieces of 8 columns: registers are short
            uint32_t h[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = pack_bf16(s[8 * i + e]);
            tmem_st8(to + i * 8, h);
#pragma unroll
            for (int e = 0; e < 8; ++e) h[e] = pack_bf16(rest_bf16(s[8 * i + e], h[e]));
            tmem_st8(to + C::PART + i * 8, h);
        }
        wait_st();
        fence_before();
        x.arrive(kSFull + (g & 1));
        const float lam_n = left >= kC ? lam_c : power(lg2, left);
        if (!x.wait(kDsFull + (g & 1), g >> 1)) return false;
        state_add<KP>(x, r, s, lam_n);
    }
    return true;
}

// A bfloat16 pool's states come and go through a 32 KiB buffer by TMA: while a
// unit is computed the next one's start state comes in; between units each
// thread takes its elements of that and puts the finished ones in their places,
// and they leave (role_out issues the copies, having time to wait for them, and
// says what the next unit is).  Written from the registers instead, a state's
// 64 stores a thread took 6000 cycles of the 8500 of a unit of one chunk:
// instructions that run once a unit come from far away.
template <int KP> __device__ void role_state_staged(const Ctx &x, int warp, int lane) {
    const StateRole<KP> r(warp, lane);
    const uint32_t buf = x.base + Ring<KP, false>::STATE + (r.half * r.KEYS * 128 + r.v) * 2;  // [KP][128]
    unsigned g = 0;
    float2 s[r.N] = {};
    for (unsigned units = 0;; ++units) {
        if (!x.wait(kStateIn, units)) return;
        const int len = (int)uniform((uint32_t)x.sm.next_len);
        const float lg2 = x.sm.next_lg2;
        // what lies outside the pool's rows and columns came in as zero; the first time nothing finished goes out
#pragma unroll
        for (int i = 0; i < r.N; i += 4) exchange_bf16(buf + 2 * i * 256, s[i], s[i + 1], s[i + 2], s[i + 3]);
        fence_async_smem();
        x.arrive(kStateTurn);
        if (len == 0 || !state_chunks<KP>(x, r, s, g, len, lg2)) return;
    }
}

// Other states: a float32 pool, the segments' start states, and the segments' own (STATES).
template <typename ST, int KP, bool STATES> __device__ void role_state(const Ctx &x, int warp, int lane) {
    const LaParams &p = x.c.p;
    const StateRole<KP> r(warp, lane);
    Walk<STATES> walk(x.c, x.sm);
    Unit u;
    unsigned g = 0;
    float2 s[r.N];
    while (walk.next(u, false)) {
        if (u.chunks == 0) continue;
        const bool on = u.tile * 128 + r.v < p.V;
        const int k0 = r.half * r.KEYS, kn = min(r.KEYS, p.K - k0);
        ST *pool = static_cast<ST *>(p.state) + (long long)u.slot * p.st_slot + (long long)u.h * p.st_head + u.tile * 128 + r.v;
        float *ws = x.c.ws + ((long long)u.x * p.nv + u.h) * p.K * p.V + u.tile * 128 + r.v;
        // in groups of 16 key indices (K is a multiple of 16), each asked for at once
#pragma unroll
        for (int i = 0; i < r.N; ++i) s[i] = make_float2(0.0f, 0.0f);
        if (!STATES && on) {
#pragma unroll
            for (int b = 0; b < r.KEYS / 16; ++b) {
                if (16 * b >= kn) break;
                const float *from;
                long long step;
                if (sizeof(ST) == 2 || x.c.seg) {
                    from = ws + (long long)(k0 + 16 * b) * p.V;
                    step = p.V;
                } else {
                    from = reinterpret_cast<const float *>(pool) + (long long)(k0 + 16 * b) * p.st_k;
                    step = p.st_k;
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) s[8 * b + i] = make_float2(from[2 * i * step], from[(2 * i + 1) * step]);
            }
        }
        if constexpr (STATES) {  // all of the segment's chunks have added up
            if (!x.wait(kOFull, g++)) return;
            state_add<KP>(x, r, s, 0.0f);
        } else {
            if (!state_chunks<KP>(x, r, s, g, u.len, u.lg2)) return;
        }
        if (on && (STATES || u.last)) {
#pragma unroll
            for (int b = 0; b < r.KEYS / 16; ++b) {
                if (16 * b >= kn) break;
                if (STATES) {
                    float *to = ws + (long long)(k0 + 16 * b) * p.V;
#pragma unroll
                    for (int i = 0; i < 16; ++i) to[i * p.V] = (i & 1) ? s[8 * b + i / 2].y : s[8 * b + i / 2].x;
                } else {
                    ST *to = pool + (long long)(k0 + 16 * b) * p.st_k;
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        to[i * p.st_k] = from_f32<ST>((i & 1) ? s[8 * b + i / 2].y : s[8 * b + i / 2].x);
                }
            }
        }
    }
}

// P~: a warp has 16 keys of P^T.  Its blocks of 8 queries are wholly masked
// before its own 16, mixed there, and wholly kept after.
template <int KP> __device__ void role_scores(const Ctx &x, int warp, int lane) {
    using R = Ring<KP, false>;
    const LaParams &p = x.c.p;
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    const int row0 = warp * 16 + lane / 4;  // this thread's keys: row0 and row0 + 8
    const uint32_t pt = x.base + (uint32_t)offsetof(Smem, pt);
    // stmatrix: lane l names row l % 8 of matrix l / 8: keys +0, +8, +0, +8 of query blocks n, n, n + 1, n + 1
    const int srow = warp * 16 + (lane & 7) + ((lane >> 3) & 1) * 8, sblk = lane >> 4;
    Walk<false> walk(x.c, x.sm);
    Unit u;
    unsigned g = 0;
    while (walk.next(u, false)) {
        if (u.chunks == 0) continue;
        float2 w[9];  // of block b and key row0 + 8 i: w[b + 1 - i]
#pragma unroll
        for (int i = 0; i < 9; ++i) {
            const int gap = 8 * (i - 1) + 2 * (lane & 3) - row0;
            w[i].x = gap < 0 ? 0.0f : p.scale * power_fast(u.lg2, gap);
            w[i].y = gap < -1 ? 0.0f : p.scale * power_fast(u.lg2, gap + 1);
        }
        for (int j = 0; j < u.chunks; ++j, ++g) {
            const int n = min(kC, u.len - j * kC);
            if (!x.wait(kPFull + (g & 1), g >> 1)) return;
            fence_after();
            uint32_t r[32];
            tmem_ld_16x64(x.tmem + lanes + Cols<KP>::P + Cols<KP>::next(g & 1), r);
            wait_ld();
            fence_before();
            x.arrive(kPFree + (g & 1));
            uint32_t h[16], rest[16];
#pragma unroll
            for (int b = 0; b < 8; ++b) {
                if (b < 2 * warp) {
                    h[2 * b] = h[2 * b + 1] = rest[2 * b] = rest[2 * b + 1] = 0;
                    continue;
                }
                float2 e[2];
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    e[i] = __fmul2_rn(make_float2(__uint_as_float(r[4 * b + 2 * i]), __uint_as_float(r[4 * b + 2 * i + 1])),
                                      w[b + 1 - i]);
                if (b < 2 * warp + 2) {  // chosen, not multiplied: whatever a masked place holds stays out
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int gap = 8 * b + 2 * (lane & 3) - (row0 + i * 8);
                        if (gap < 0) e[i].x = 0.0f;
                        if (gap < -1) e[i].y = 0.0f;
                    }
                }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    h[2 * b + i] = pack_bf16(e[i]);
                    rest[2 * b + i] = pack_bf16(rest_bf16(e[i], h[2 * b + i]));
                }
            }
            if (__builtin_expect(n < kC, 0)) {
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    if (row0 >= n) h[2 * b] = rest[2 * b] = 0;
                    if (row0 + 8 >= n) h[2 * b + 1] = rest[2 * b + 1] = 0;
                }
                clear_tail(x.sm.ring + g % R::N * R::BYTES + R::V, n, p.V - u.tile * 128 > 64 ? 2 : 1, warp * 32 + lane,
                           32 * kWarpsP);
            }
            auto put = [&](uint32_t to, const uint32_t (&w)[16]) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    stmatrix4(to + srow * 128 + (((2 * i + sblk) ^ (srow & 7)) << 4), w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
            };
            if (g > 0 && !x.wait(kOFull + ((g - 1) & 1), (g - 1) >> 1)) return;  // the product that read the last P~ is done
            put(pt, h);
            put(x.base + (uint32_t)offsetof(Smem, pt_rest), rest);
            fence_async_smem();
            x.arrive(kPtFull);
        }
    }
}

// The copies of a bfloat16 pool's states, in and out of their one buffer.
template <int KP> struct StateCopies {
    const Ctx &x;
    const CUtensorMap *map;
    Walk<false> ahead;
    int now[3], next[3];  // tile, head, slot: of the unit being computed, and of the one whose start state is on its way
    unsigned units = 0;
    __device__ StateCopies(const Ctx &x_, const CUtensorMap *m) : x(x_), map(m), ahead(x_.c, x_.sm) {}
    __device__ uint32_t buf() const { return x.base + Ring<KP, false>::STATE; }

    // Announces the next unit, and that there is none by a length of 0.
    __device__ void load() {
        Unit u;
        bool more;
        while ((more = ahead.next(u, false)) && u.chunks == 0) {
        }
        next[0] = u.tile;
        next[1] = u.h;
        next[2] = u.slot;
        if ((threadIdx.x & 31) == 0) {
            ++x.sm.state_loads;
            x.sm.next_len = more ? u.len : 0;
            x.sm.next_lg2 = u.lg2;
            if (more) {
                mbar_expect(x.bar(kStateIn), KP * 256);
                tma_load4(buf(), map, u.tile * 128, 0, u.h, u.slot, x.bar(kStateIn));
            } else {
                mbar_arrive(x.bar(kStateIn));
            }
        }
        __syncwarp();
    }
    // Once every thread has taken its part of the buffer and put the finished
    // state's there, that leaves; false where a wait gave up.
    __device__ bool store() {
        if (!x.wait(kStateTurn, units)) return false;
        if (units > 0 && (threadIdx.x & 31) == 0) tma_store4(map, now[0] * 128, 0, now[1], now[2], buf());
        __syncwarp();
        ++units;
        return true;
    }
    __device__ bool turn() {
        if (!store()) return false;
        for (int i = 0; i < 3; ++i) now[i] = next[i];
        if ((threadIdx.x & 31) == 0) tma_stores_read();
        __syncwarp();
        load();
        return true;
    }
};

// The output: a warp has 32 columns of O^T, which it turns into rows of 64 bytes
// a token.  With 64 key channels it does so through shared memory; with 128 there is
// no room left beside P~'s second part, and 8x8 blocks are turned in registers,
// which takes 400 cycles more.
template <int KP> __device__ void role_out(const Ctx &x, int warp, int lane, StateCopies<KP> *states) {
    const LaParams &p = x.c.p;
    uint16_t *const out = static_cast<uint16_t *>(p.out);
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    constexpr bool kStaged = KP == 64;
    unsigned char *const ost = x.sm.ring + Ring<KP, false>::OST + warp * (32 * 64);  // 32 tokens x 32 columns
    const uint32_t ost_a = x.base + Ring<KP, false>::OST + warp * (32 * 64);
    // staging: 16-byte block c of token t lies at block c ^ (t / 2 % 4) of its 64 bytes
    const int st_tok = (lane >> 4) * 8 + (lane & 7), st_blk = (lane >> 3) & 1;
    Walk<false> walk(x.c, x.sm);
    Unit u;
    unsigned g = 0;
    if (states) states->load();
    while (walk.next(u, warp == 0 && lane == 0)) {
        const int col = u.tile * 128 + warp * 32;
        if (col + (lane & 3) * 8 < p.V)
            for (unsigned t = lane / 4; t < (unsigned)u.skip_len; t += 8)
                *reinterpret_cast<uint4 *>(out + ((long long)u.skip_t0 + t) * p.o_ts + (long long)u.h * p.o_hs + col +
                                           (lane & 3) * 8) = make_uint4(0, 0, 0, 0);
        if (u.chunks == 0) continue;
        if (states && !states->turn()) return;
        float2 f0[4];  // of the first 32 tokens; the others' are lambda^32 of theirs
#pragma unroll
        for (int b = 0; b < 4; ++b) {
            const int i = 8 * b + 2 * (lane & 3);
            f0[b] = make_float2(p.scale * power_fast(u.lg2, i + 1), p.scale * power_fast(u.lg2, i + 2));
        }
        const float lam32 = power_fast(u.lg2, 32);
        const bool on = col + (lane & 3) * 8 < p.V;
        const bool on2[2] = {col < p.V, col + 16 < p.V};  // V is a multiple of 16
        uint16_t *to = out + (long long)(u.t0 + lane / 4) * p.o_ts + (long long)u.h * p.o_hs + col +
                       (kStaged ? (lane & 3) * 8 : (lane & 1) * 8 + (lane & 2) * 2);
        for (int j = 0; j < u.chunks; ++j, ++g) {
            const int n = min(kC, u.len - j * kC);
            if (!x.wait(kOFull + (g & 1), g >> 1)) return;
            fence_after();
            // 32 tokens, packed; the first 32 leave the warp's registers before the others are read
            uint32_t h[16];
            auto collect = [&](int ch) {
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {  // 16 of the columns
                    uint32_t a[16], b[16];
                    tmem_ld_16x32(x.tmem + lanes + ((uint32_t)(hh * 16) << 16) + Cols<KP>::O1 + (g & 1) * kC + ch * 32, a);
                    tmem_ld_16x32(x.tmem + lanes + ((uint32_t)(hh * 16) << 16) + Cols<KP>::O2 + ch * 32, b);
                    wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        h[hh * 8 + i] =
                            pack_bf16(__ffma2_rn(ch ? __fmul2_rn(f0[i / 2], make_float2(lam32, lam32)) : f0[i / 2],
                                                 make_float2(__uint_as_float(a[2 * i]), __uint_as_float(a[2 * i + 1])),
                                                 make_float2(__uint_as_float(b[2 * i]), __uint_as_float(b[2 * i + 1]))));
                }
            };
            auto stage = [&]() {
                __syncwarp();
#pragma unroll
                for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const int t = i * 16 + st_tok;
                        const uint32_t *w = h + hh * 8 + i * 4;
                        stmatrix4_t(ost_a + t * 64 + (((hh * 2 + st_blk) ^ ((t >> 1) & 3)) << 4), w[0], w[1], w[2], w[3]);
                    }
                __syncwarp();
            };
            auto write = [&](int ch) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int t = r * 8 + lane / 4;
                    uint16_t *const here = to + (long long)(ch * 32 + r * 8) * p.o_ts;
                    if constexpr (kStaged) {
                        if (on && ch * 32 + t < n)
                            *reinterpret_cast<uint4 *>(here) =
                                *reinterpret_cast<const uint4 *>(ost + t * 64 + (((lane & 3) ^ ((t >> 1) & 3)) << 4));
                    } else {
#pragma unroll
                        for (int hh = 0; hh < 2; ++hh) {  // 16 columns: words 0, 1 or 2, 3 of one of their two blocks
                            uint32_t w0 = turn8x8(h[hh * 8 + r * 2]), w1 = turn8x8(h[hh * 8 + r * 2 + 1]);
                            const uint32_t got = __shfl_xor_sync(0xffffffffu, lane & 1 ? w0 : w1, 1);
                            (lane & 1 ? w0 : w1) = got;
                            if (on2[hh] && ch * 32 + t < n) *reinterpret_cast<uint2 *>(here + hh * 16) = make_uint2(w0, w1);
                        }
                    }
                }
            };
            collect(0);
            if constexpr (kStaged) stage(); else write(0);
            collect(1);
            fence_before();
            x.arrive(kOFree);
            if constexpr (kStaged) {
                write(0);
                stage();
            }
            write(1);
            to += (long long)kC * p.o_ts;
        }
    }
    if (states) states->store();
}

// STAGED: a bfloat16 pool's states by TMA; compiled apart from the other form of
// the state's role, beside which neither has the registers it needs (4 rows of
// 4096 tokens x 38 heads, bfloat16 pool: 136 us together).
template <typename ST, int KP, bool STATES, bool STAGED>
__global__ void __launch_bounds__(kThreads, 1)
    k_la_chunk(const __grid_constant__ ChunkParams c, const __grid_constant__ CUtensorMap mq,
               const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
               const __grid_constant__ CUtensorMap ms) {
    constexpr int PARTS = sizeof(ST) == 2 ? 2 : 3;  // bfloat16 parts of K~
    extern __shared__ unsigned char smem_raw[];
    const uint32_t raw = smem_addr(smem_raw), pad = (1024u - (raw & 1023u)) & 1023u;
    Smem &sm = *reinterpret_cast<Smem *>(smem_raw + pad);
    const int warp = (int)uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
    const uint32_t base = raw + pad, bars = base + (uint32_t)offsetof(Smem, bar);
    if (threadIdx.x == 0) {
        sm.gave_up = sm.state_loads = 0;
        for (int i = 0; i < kBars; ++i) {
            int n = 1;
            if (i >= kStageFree && i < kStageFree + kMaxStages) n = STATES ? 1 : 2;  // the products that read a stage last
            if (i == kPFree || i == kPFree + 1 || i == kPtFull) n = kWarpsP;
            if (i == kDrain) n = STATES ? 1 : 3;
            if (i == kSFull || i == kSFull + 1 || i == kDsFree || i == kStateTurn) n = kWarpsS;
            if (i == kKtFull || i == kKtFull + 1) n = kWarpsK * kTeams<STATES>;
            if (i == kOFree) n = kWarpsO;
            mbar_init(bars + 8 * i, n);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async_smem();
    }
    if (warp == kWarpMma) tmem_alloc(base + (uint32_t)offsetof(Smem, tmem), 512);
    if (warp == kWarpMma + 3 && lane == 0) {
        tma_prefetch_map(&mk);
        tma_prefetch_map(&mv);
        if (!STATES) tma_prefetch_map(&mq);
    }
    plan_rows(c, sm);
    fence_before();
    __syncthreads();
    fence_after();
    const Ctx x{c, sm, base, bars, uniform(sm.tmem)};
    if (warp < kWarpS) {
        regs_down<kRegsRest>();
        if (warp == kWarpMma) {
            role_mma_state<KP, PARTS, STATES>(x);
            drain_mma(x);
        } else if (warp == kWarpMma + 1) {
            if (!STATES) role_mma_out<KP>(x);
        } else if (warp == kWarpMma + 2) {
            if (!STATES) role_mma_scores<KP>(x);
        } else {
            Loader<KP, sizeof(ST) == 2, STATES> load(x, &mq, &mk, &mv);
            while (load.more && load.step()) {
            }
            load.drain();
        }
    } else if (warp < kWarpO) {
        regs_up<kRegsS>();
        if constexpr (STAGED)
            role_state_staged<KP>(x, warp - kWarpS, lane);
        else
            role_state<ST, KP, STATES>(x, warp - kWarpS, lane);
    } else if (warp < kWarpP) {
        if (kRegsO > 80) regs_up<kRegsO>();
        if constexpr (!STATES) {
            StateCopies<KP> states(x, &ms);
            const bool mine = STAGED && warp == kWarpO;
            role_out<KP>(x, warp - kWarpO, lane, mine ? &states : nullptr);
            if (mine && lane == 0 && sm.state_loads) {  // no state's copy is in flight when the CTA ends
                volatile int never = 0;
                mbar_wait(x.bar(kStateIn), (uint32_t)(sm.state_loads - 1) & 1u, &never);
                tma_stores_done();
            }
        } else {
            role_keys<KP, PARTS, STATES, kTeams<STATES>>(x, 2, warp - kWarpO, lane);
        }
    } else if (warp < kWarpK) {
        if (kRegsP > 80) regs_up<kRegsP>();
        if constexpr (STATES)
            role_keys<KP, PARTS, STATES, kTeams<STATES>>(x, 1, warp - kWarpP, lane);
        else
            role_scores<KP>(x, warp - kWarpP, lane);
    } else {
        regs_down<kRegsK>();
        role_keys<KP, PARTS, STATES, kTeams<STATES>>(x, 0, warp - kWarpK, lane);
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
        int t0 = 0, len = -1;
        if ((int)threadIdx.x < B) {
            t0 = p.offsets[threadIdx.x];
            len = sound_len(p, t0, p.offsets[threadIdx.x + 1]);
        }
        s_len[threadIdx.x] = apart(t0, len);
    }
    __syncthreads();
    // the row of this rank, and the segments of the rows before it
    int b = 0, before = 0;
    for (int o = 0; o < B; ++o) {
        int rank = 0;
        for (int q = 0; q < B; ++q) rank += s_len[q] > s_len[o] || (s_len[q] == s_len[o] && q < o);
        if (rank == r) b = o;
        if (rank < r) before += max(1, pieces(s_len[o], c.seg));
    }
    const int n = pieces(s_len[b], c.seg), slot = p.slot_idx[b];
    const float lg2 = log2_lambda(p, h);
    if (n <= 0 || slot < 0 || slot >= p.max_slots || isnan(lg2) || (p.max_len > 0 && s_len[b] > p.max_len)) return;
    const float lam = power(lg2, c.seg);
    const int i = (blockIdx.x * 256 + threadIdx.x) * 4;  // V is a multiple of 16: four columns of one row
    if (i >= p.K * p.V) return;
    const int k = i / p.V, v = i - k * p.V;
    const ST *pool = static_cast<const ST *>(p.state) + (long long)slot * p.st_slot + (long long)h * p.st_head +
                     (long long)k * p.st_k + v;
    float4 s = make_float4(to_f32(pool[0]), to_f32(pool[1]), to_f32(pool[2]), to_f32(pool[3]));
    const long long step = (long long)p.nv * p.K * p.V;
    float *ws = c.ws + (long long)before * step + (long long)h * p.K * p.V + i;
    // eight segments' loads at a time: one after the other they took 33 us for 14 segments
    for (int j0 = 0; j0 < n; j0 += 8, ws += 8 * step) {
        float4 own[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            own[j] = j0 + j + 1 < n ? *reinterpret_cast<const float4 *>(ws + j * step) : make_float4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (j0 + j >= n) break;
            *reinterpret_cast<float4 *>(ws + j * step) = s;
            s.x = fmaf(lam, s.x, own[j].x);
            s.y = fmaf(lam, s.y, own[j].y);
            s.z = fmaf(lam, s.z, own[j].z);
            s.w = fmaf(lam, s.w, own[j].w);
        }
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

// A bfloat16 pool [slots, nv, K, V] in boxes of one head's 128 columns.
bool encode_pool(EncodeFn fn, CUtensorMap *map, const LaParams &p) {
    const cuuint64_t dims[4] = {(cuuint64_t)p.V, (cuuint64_t)p.K, (cuuint64_t)p.nv, (cuuint64_t)p.max_slots};
    const cuuint64_t strides[3] = {(cuuint64_t)p.st_k * 2, (cuuint64_t)p.st_head * 2, (cuuint64_t)p.st_slot * 2};
    const cuuint32_t box[4] = {128, p.K > 64 ? 128u : 64u, 1, 1}, one[4] = {1, 1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, p.state, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename ST, int KP> cudaError_t go(ChunkParams c, const CUtensorMap *m, cudaStream_t s) {
    static LaunchCache cache;
    LaunchInfo li;
    constexpr int smem = (int)sizeof(Smem) + 1024;
    constexpr bool kStages = sizeof(ST) == 2;
    cudaError_t e = launch_info(cache, &li, [](LaunchInfo &) {
        cudaError_t r = cudaSuccess;
        for (const void *f : {(const void *)k_la_chunk<ST, KP, false, false>, (const void *)k_la_chunk<ST, KP, true, false>,
                              (const void *)k_la_chunk<ST, KP, false, kStages>})
            if (r == cudaSuccess) r = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        return r;
    });
    if (e != cudaSuccess) return e;
    const LaParams &p = c.p;
    const long long per = (long long)p.nv * p.tiles;
    const long long rows = c.seg ? p.batch + p.T / c.seg : p.batch;
    const unsigned grid = (unsigned)(rows * per < li.sms ? rows * per : li.sms);
    if (c.seg) {
        k_la_chunk<ST, KP, true, false><<<grid, kThreads, smem, s>>>(c, m[0], m[1], m[2], m[3]);
        const dim3 jg((unsigned)((p.K * p.V + 1023) / 1024), (unsigned)p.nv, (unsigned)p.batch);
        k_la_join<ST><<<jg, 256, 0, s>>>(c);
        k_la_chunk<ST, KP, false, false><<<grid, kThreads, smem, s>>>(c, m[0], m[1], m[2], m[3]);
    } else {
        k_la_chunk<ST, KP, false, kStages><<<grid, kThreads, smem, s>>>(c, m[0], m[1], m[2], m[3]);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_la_chunk(const LaParams &p, bool state_bf16, int seg, void *ws, cudaStream_t s, bool *used) {
    *used = false;
    const EncodeFn fn = encode_fn();
    CUtensorMap m[4] = {};
    if (!fn || !encode(fn, &m[0], p.q, p.K, p.nk, p.T, p.q_hs, p.q_ts) ||
        !encode(fn, &m[1], p.k, p.K, p.nk, p.T, p.k_hs, p.k_ts) || !encode(fn, &m[2], p.v, p.V, p.nv, p.T, p.v_hs, p.v_ts))
        return cudaSuccess;
    if (state_bf16 && !seg && !encode_pool(fn, &m[3], p)) return cudaSuccess;
    *used = true;
    const ChunkParams c{p, seg, static_cast<float *>(ws), FastDiv((unsigned)(p.nv * p.tiles)),
                        FastDiv((unsigned)p.tiles)};
    if (p.K > 64) return state_bf16 ? go<uint16_t, 128>(c, m, s) : go<float, 128>(c, m, s);
    return state_bf16 ? go<uint16_t, 64>(c, m, s) : go<float, 64>(c, m, s);
}

}  // namespace gdr
