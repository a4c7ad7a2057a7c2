// Verification of drafted tokens: how many drafts of a row the target lets through,
// and the token drawn behind them.
//
// A row needs a handful of single probabilities and then one whole row of the
// target's (and of the drafter's, where a draft was refused): a sum, and the place
// where the running sum passes its share.  The sum is HBM bound, or bound by its
// chain of dependent steps where rows are few.  A row is a cluster of blocks, as
// many as it takes to fill the GPU; every warp sums one stretch of the vocabulary,
// the blocks exchange their sums through distributed shared memory, and the block
// whose stretch has the place reads that stretch (out of L2) once more, all of its
// threads side by side.
//
// The token has to be the one that exact arithmetic finds: with a vocabulary of
// 1e5 a float32 sum would miss it in a few draws of a hundred.  Differences are
// kept as (difference, its rounding error) and sums as (sum, error) of float32 pairs by
// two-sum (Knuth, The Art of Computer Programming 2, 4.2.2), good to 46 bits and
// more; the FP64 pipes (2 operations a cycle and multiprocessor) would take 2.5 times as long as
// the memory.  What is left of a stretch's sums is added up in double.
#include <cooperative_groups.h>

#include "../gdr_device.cuh"
#include "layer_internal.h"

namespace gdr {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 16, kThreads = 32 * kWarps;

// Probabilities count from 0 up; negative, infinite and NaN ones do not.
__device__ __forceinline__ float clean(float p) { return p > 0.0f && p < __int_as_float(0x7f800000) ? p : 0.0f; }

// A sum of float32 values and what its roundings lost.
struct Sum {
    float s = 0.0f, c = 0.0f;
    __device__ __forceinline__ void add(float w, float low) {
        const float t = __fadd_rn(s, w), b = __fsub_rn(t, s);
        const float e = __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(w, b));
        c = __fadd_rn(c, __fadd_rn(e, low));
        s = t;
    }
};

enum Weight { kTarget, kDifference };  // p (0 at a refused token that was not drawn); max(p - q, 0)

// One token's weight as (value, rounding error).
template <Weight M> __device__ __forceinline__ void add_weight(Sum &a, float p, float q) {
    p = clean(p);
    if constexpr (M == kDifference) {
        q = clean(q);
        const float w = __fsub_rn(p, q), b = __fsub_rn(w, p);
        const float e = __fsub_rn(__fsub_rn(p, __fsub_rn(w, b)), __fadd_rn(q, b));
        const bool some = w > 0.0f;
        a.add(some ? w : 0.0f, some ? e : 0.0f);
    } else {
        a.add(p, 0.0f);
    }
}

template <Weight M> __device__ __forceinline__ double exact_weight(float p, float q) {
    p = clean(p);
    if constexpr (M == kDifference) {
        q = clean(q);
        return p > q ? (double)p - (double)q : 0.0;
    } else {
        return (double)p;
    }
}

// C neighbouring probabilities from i on; those outside [0, end) count as 0.
template <typename PT, int C> __device__ __forceinline__ void take(const PT *row, int i, int end, bool vec, float (&v)[C]) {
    if (vec && i >= 0 && i + C <= end) {
        Pack<PT, C> w;
        w.load(row + i);
#pragma unroll
        for (int j = 0; j < C; ++j) v[j] = w.get(j);
    } else {
#pragma unroll
        for (int j = 0; j < C; ++j) v[j] = i + j >= 0 && i + j < end ? to_f32(row[i + j]) : 0.0f;
    }
}

// What a row's draw goes by: weights of tokens [0, vocab), read in vectors from an index at or
// before 0 that is aligned in memory.
template <typename PT> struct Weights {
    static constexpr int C = 16 / (int)sizeof(PT);
    const PT *p, *q;
    Weight mode;
    int no, vocab;
    bool vec;
    // C neighbouring weights as (value, rounding error)
    __device__ __forceinline__ void load(int i, int end, float (&pv)[C], float (&qv)[C]) const {
        take<PT, C>(p, i, end, vec, pv);
        if (mode == kDifference) take<PT, C>(q, i, end, vec, qv);
    }
    __device__ __forceinline__ void add(Sum &a, int i, const float (&pv)[C], const float (&qv)[C]) const {
        if (mode == kDifference) {
#pragma unroll
            for (int j = 0; j < C; ++j) add_weight<kDifference>(a, pv[j], qv[j]);
        } else {
#pragma unroll
            for (int j = 0; j < C; ++j) add_weight<kTarget>(a, i + j == no ? 0.0f : pv[j], 0.0f);
        }
    }
    __device__ __forceinline__ double exact(int i, float pv, float qv) const {
        if (mode == kDifference) return exact_weight<kDifference>(pv, qv);
        return i == no ? 0.0 : exact_weight<kTarget>(pv, 0.0f);
    }
};

// The sum of a warp's stretch [i0, i1), in every lane.
template <typename PT> __device__ __forceinline__ double stretch(const Weights<PT> &w, int i0, int i1, int lane) {
    constexpr int C = Weights<PT>::C, U = 2;
    Sum a;
    for (int i = i0 + lane * C; i < i1; i += 32 * C * U) {
        float pv[U][C], qv[U][C];
#pragma unroll
        for (int k = 0; k < U; ++k) w.load(i + k * 32 * C, i1, pv[k], qv[k]);
#pragma unroll
        for (int k = 0; k < U; ++k) w.add(a, i + k * 32 * C, pv[k], qv[k]);
    }
#pragma unroll
    for (int m = 16; m; m >>= 1) {
        const float s = __shfl_xor_sync(kFull, a.s, m), c = __shfl_xor_sync(kFull, a.c, m);
        a.add(s, c);
    }
    return (double)a.s + (double)a.c;
}

template <typename PT> __global__ void __launch_bounds__(kThreads, 2) k_accept(const __grid_constant__ AcceptParams p) {
    __shared__ double sums[kWarps];  // of this block's stretches, then of a stretch's parts
    __shared__ double block_sum;
    __shared__ int first_refused, first_none, found, last;
    cg::cluster_group cluster = cg::this_cluster();
    const int blocks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int b = (int)(blockIdx.x / (unsigned)blocks), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const long long lo = p.offsets[b], hi = p.offsets[b + 1];
    const bool inside = lo >= 0 && hi >= lo && hi <= p.T, fits = inside && hi - lo <= p.width;
    if (rank == 0 && tid == 0 && !fits) flag(p.status, inside ? GDR_STATUS_ROW_TOO_LONG : GDR_STATUS_BAD_OFFSETS);
    int *const out = p.out + (long long)b * p.o_ts;
    if (!fits || hi == lo) {  // the same in every block of the cluster
        if (rank == 0) {
            for (int i = tid; i < p.width; i += kThreads) out[i] = -1;
            if (tid == 0) p.counts[b] = 0;
        }
        return;
    }
    // which drafts pass
    const int drafts = (int)(hi - lo) - 1;
    const float v = p.row_u[b];
    if (tid == 0) {
        first_refused = first_none = drafts;
        found = 0x7fffffff;
        last = -1;
    }
    __syncthreads();
    const PT *const target = static_cast<const PT *>(p.target), *const draft = static_cast<const PT *>(p.draft);
    for (int i = tid; i < drafts; i += kThreads) {
        const long long t = lo + i;
        const int d = p.tokens[t + 1];
        const float u = p.u[t];
        if (d < 0 || d >= p.vocab) {
            atomicMin(&first_none, i);
            continue;
        }
        const float pd = clean(to_f32(target[t * p.t_ts + d])), qd = draft ? clean(to_f32(draft[t * p.d_ts + d])) : 1.0f;
        if (!((double)u * (double)qd < (double)pd)) atomicMin(&first_refused, i);
    }
    __syncthreads();
    const int accepted = min(first_refused, first_none);
    const bool refused = first_refused < first_none;
    const long long t = lo + accepted;
    Weights<PT> w;
    constexpr int C = Weights<PT>::C;
    w.p = target + t * p.t_ts;
    w.q = draft ? draft + t * p.d_ts : w.p;
    w.mode = !refused ? kTarget : draft ? kDifference : kTarget;
    w.no = refused && !draft ? p.tokens[t + 1] : -1;
    w.vocab = p.vocab;
    const int off_p = (int)(reinterpret_cast<uintptr_t>(w.p) % 16), off_q = (int)(reinterpret_cast<uintptr_t>(w.q) % 16);
    w.vec = w.mode == kTarget || off_p == off_q;
    const int start = -(off_p / (int)sizeof(PT));  // aligned, at most C - 1 before the first token

    // the sums: a stretch of whole vectors a warp
    const int each = ((p.vocab - start - 1) / (blocks * kWarps) + C) / C * C;
    const long long from = (long long)(rank * kWarps + warp) * each + start;
    const int i0 = (int)(from < p.vocab ? from : p.vocab), i1 = p.vocab - i0 < each ? p.vocab : i0 + each;
    double total = 0.0, before = 0.0, share = 0.0;
    int owner = -1;
    for (int pass = 0; pass < 2; ++pass) {
        const double s = stretch(w, i0, i1, lane);
        if (lane == 0) sums[warp] = s;
        __syncthreads();
        if (warp == 0) {
            double all = lane < kWarps ? sums[lane] : 0.0;
#pragma unroll
            for (int m = kWarps / 2; m; m >>= 1) all += __shfl_xor_sync(kFull, all, m);
            if (lane == 0) block_sum = all;
        }
        cluster.sync();
        // every warp adds up the blocks' sums alike: lane r has block r's
        const double mine = lane < blocks ? *cluster.map_shared_rank(&block_sum, lane) : 0.0;
        double upto = mine;
#pragma unroll
        for (int m = 1; m < 8; m <<= 1) {
            const double o = __shfl_up_sync(kFull, upto, m);
            if (lane >= m) upto += o;
        }
        total = __shfl_sync(kFull, upto, 7);
        if (total > 0.0) {
            // the block whose part passes the share; the last one with a weight where none does
            share = v > 0.0f ? (double)v * total : 0.0;
            const unsigned some = __ballot_sync(kFull, mine > 0.0), past = __ballot_sync(kFull, mine > 0.0 && upto > share);
            owner = past ? __ffs(past) - 1 : 31 - __clz(some);
            before = __shfl_sync(kFull, upto - mine, owner);
        }
        if (total > 0.0 || (w.mode == kTarget && w.no < 0)) break;
        w.mode = kTarget;  // nothing left over of the target: drawn from the target itself
        w.no = -1;
        w.vec = true;
        cluster.sync();  // before the sums are written again
    }
    if (owner == rank) {
        // the stretch, the same way
        const double mine = lane < kWarps ? sums[lane] : 0.0;
        double upto = mine;
#pragma unroll
        for (int m = 1; m < kWarps; m <<= 1) {
            const double o = __shfl_up_sync(kFull, upto, m);
            if (lane >= m) upto += o;
        }
        const unsigned some = __ballot_sync(kFull, mine > 0.0), past = __ballot_sync(kFull, mine > 0.0 && before + upto > share);
        const int which = past ? __ffs(past) - 1 : 31 - __clz(some);
        double base = before + __shfl_sync(kFull, upto - mine, which);
        const long long s0 = (long long)(rank * kWarps + which) * each + start;
        const int end = (int)(s0 + each < p.vocab ? s0 + each : p.vocab);
        // and its least token at which the running sum passes, by all threads
        for (int i = (int)s0; i < end; i += C * kThreads) {
            const int at = i + tid * C;
            float pv[C], qv[C];
            double own = 0.0;
#pragma unroll
            for (int j = 0; j < C; ++j) pv[j] = qv[j] = 0.0f;
            if (at < end) w.load(at, end, pv, qv);
#pragma unroll
            for (int j = 0; j < C; ++j) own += w.exact(at + j, pv[j], qv[j]);
            double sum = own;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const double o = __shfl_up_sync(kFull, sum, m);
                if (lane >= m) sum += o;
            }
            __syncthreads();  // sums is read no more
            if (lane == 31) sums[warp] = sum;
            __syncthreads();
            double ahead = lane < warp ? sums[lane] : 0.0, all = lane < kWarps ? sums[lane] : 0.0;
#pragma unroll
            for (int m = kWarps / 2; m; m >>= 1) {
                ahead += __shfl_xor_sync(kFull, ahead, m);
                all += __shfl_xor_sync(kFull, all, m);
            }
            double run = base + ahead + (sum - own);
            int here = -1, positive = -1;
#pragma unroll
            for (int j = 0; j < C; ++j) {
                const double x = w.exact(at + j, pv[j], qv[j]);
                run += x;
                if (x > 0.0) {
                    positive = at + j;
                    if (here < 0 && run > share) here = at + j;
                }
            }
            if (here >= 0) atomicMin(&found, here);
            if (positive >= 0) atomicMax(&last, positive);
            __syncthreads();
            if (found != 0x7fffffff) break;
            base += all;
        }
        if (tid == 0) out[accepted] = found != 0x7fffffff ? found : last;
    }
    if (rank == 0) {
        for (int i = tid; i < p.width; i += kThreads)
            if (i != accepted) out[i] = i < accepted ? p.tokens[lo + 1 + i] : -1;
        if (tid == 0) {
            p.counts[b] = accepted + 1;
            if (owner < 0) {
                out[accepted] = -1;
                flag(p.status, GDR_STATUS_NO_MASS);
            }
        }
    }
    if (blocks > 1) cluster.sync();  // a block's shared memory stays while others read it
}

template <typename PT> cudaError_t go(const AcceptParams &p, cudaStream_t s) {
    // blocks a row: as many as run at once (two a multiprocessor), up to the largest portable cluster
    int blocks = 1;
    while (blocks < 8 && (long long)p.batch * blocks * 2 <= 2 * 152) blocks *= 2;
    if ((long long)p.batch * blocks >= 1ll << 31) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t c{};
    c.gridDim = dim3((unsigned)p.batch * (unsigned)blocks);
    c.blockDim = dim3(kThreads);
    c.stream = s;
    cudaLaunchAttribute a[1];
    a[0].id = cudaLaunchAttributeClusterDimension;
    a[0].val.clusterDim.x = (unsigned)blocks;
    a[0].val.clusterDim.y = a[0].val.clusterDim.z = 1;
    c.attrs = a;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, k_accept<PT>, p);
}

}  // namespace

cudaError_t launch_accept(const AcceptParams &p, bool bf16, cudaStream_t s) {
    return bf16 ? go<uint16_t>(p, s) : go<float>(p, s);
}

}  // namespace gdr
