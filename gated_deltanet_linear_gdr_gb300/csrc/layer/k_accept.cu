// Verification of drafted tokens: how many drafts of a row the target lets through,
// and the token drawn behind them.
//
// A row needs a handful of single probabilities and then one whole row of the
// target's (and of the drafter's, where a draft was refused), twice: a sum, and
// the place where the running sum passes its share.  The first reading is HBM
// bound, the second finds its values in L2 and looks at one warp's part only.  A
// row is a cluster of blocks, as many as it takes to fill the GPU with few rows;
// every warp sums one stretch of the vocabulary, the blocks exchange their sums
// through distributed shared memory, and the warp whose stretch has the place walks
// through it.
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

enum Weight { kTarget, kDifference, kWithout };  // p; max(p - q, 0); p but 0 at the refused token

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

// C neighbouring probabilities from i on; those at `end` and behind it count as 0.
template <typename PT, int C> __device__ __forceinline__ void take(const PT *row, int i, int end, bool vec, float (&v)[C]) {
    if (vec && i + C <= end) {
        Pack<PT, C> w;
        w.load(row + i);
#pragma unroll
        for (int j = 0; j < C; ++j) v[j] = w.get(j);
    } else {
#pragma unroll
        for (int j = 0; j < C; ++j) v[j] = i + j < end ? to_f32(row[i + j]) : 0.0f;
    }
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
    for (int m = 16; m; m >>= 1) v += __shfl_xor_sync(kFull, v, m);
    return v;
}

// The sum of a warp's stretch [i0, i1).
template <typename PT, Weight M>
__device__ __forceinline__ double stretch(const PT *p, const PT *q, int no, int i0, int i1, bool vec, int lane) {
    constexpr int C = 16 / (int)sizeof(PT), U = 4;
    Sum a;
    for (int i = i0 + lane * C; i < i1; i += 32 * C * U) {
        float pv[U][C], qv[U][C];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            take<PT, C>(p, i + k * 32 * C, i1, vec, pv[k]);
            if (M == kDifference) take<PT, C>(q, i + k * 32 * C, i1, vec, qv[k]);
        }
#pragma unroll
        for (int k = 0; k < U; ++k)
#pragma unroll
            for (int j = 0; j < C; ++j) {
                if (M == kWithout && i + k * 32 * C + j == no) pv[k][j] = 0.0f;
                add_weight<M>(a, pv[k][j], M == kDifference ? qv[k][j] : 0.0f);
            }
    }
    return warp_sum((double)a.s + (double)a.c);
}

// The least token of a stretch where base and the running sum pass `share`; its last one with a weight where none does.
template <typename PT, Weight M>
__device__ __forceinline__ int find(const PT *p, const PT *q, int no, int i0, int i1, bool vec, int lane, double base, double share) {
    constexpr int C = 16 / (int)sizeof(PT);
    int last = -1;
    for (int at = i0; at < i1; at += 32 * C) {
        const int i = at + lane * C;
        float pv[C], qv[C];
        take<PT, C>(p, i, i1, vec, pv);
        if (M == kDifference) take<PT, C>(q, i, i1, vec, qv);
        double w[C], own = 0.0;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            if (M == kWithout && i + j == no) pv[j] = 0.0f;
            w[j] = exact_weight<M>(pv[j], M == kDifference ? qv[j] : 0.0f);
            own += w[j];
        }
        double upto = own;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const double o = __shfl_up_sync(kFull, upto, m);
            if (lane >= m) upto += o;
        }
        double run = base + (upto - own);
        int here = -1;
#pragma unroll
        for (int j = 0; j < C; ++j) {
            run += w[j];
            if (here < 0 && w[j] > 0.0 && run > share) here = i + j;
        }
        const unsigned found = __ballot_sync(kFull, here >= 0);
        if (found) return __shfl_sync(kFull, here, __ffs(found) - 1);
        int mine = -1;
#pragma unroll
        for (int j = 0; j < C; ++j)
            if (w[j] > 0.0) mine = i + j;
        const int most = __reduce_max_sync(kFull, mine);
        last = most > last ? most : last;
        base += __shfl_sync(kFull, upto, 31);
    }
    return last;
}

template <typename PT> __global__ void __launch_bounds__(kThreads) k_accept(const __grid_constant__ AcceptParams p) {
    __shared__ double sums[kWarps];  // of this block's stretches
    __shared__ double block_sum;
    __shared__ int first_refused, first_none;
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
    if (tid == 0) first_refused = first_none = drafts;
    __syncthreads();
    const PT *const target = static_cast<const PT *>(p.target), *const draft = static_cast<const PT *>(p.draft);
    for (int i = tid; i < drafts; i += kThreads) {
        const long long t = lo + i;
        const int d = p.tokens[t + 1];
        if (d < 0 || d >= p.vocab) {
            atomicMin(&first_none, i);
            continue;
        }
        const float pd = clean(to_f32(target[t * p.t_ts + d])), qd = draft ? clean(to_f32(draft[t * p.d_ts + d])) : 1.0f;
        if (!((double)p.u[t] * (double)qd < (double)pd)) atomicMin(&first_refused, i);
    }
    __syncthreads();
    const int accepted = min(first_refused, first_none);
    const bool refused = first_refused < first_none;
    const long long t = lo + accepted;
    const int no = refused ? p.tokens[t + 1] : -1;
    const PT *const tp = target + t * p.t_ts, *const dp = draft ? draft + t * p.d_ts : nullptr;
    Weight mode = !refused ? kTarget : draft ? kDifference : kWithout;

    // the sums: stretches of whole vectors
    const int each = ((p.vocab - 1) / (blocks * kWarps) + 8) / 8 * 8;
    const long long from = (long long)(rank * kWarps + warp) * each;
    const int i0 = (int)(from < p.vocab ? from : p.vocab), i1 = p.vocab - i0 < each ? p.vocab : i0 + each;
    const bool vec = p.vec != 0;
    double total = 0.0, before = 0.0;
    int owner = -1;
    const float v = p.row_u[b];
    double share = 0.0;
    for (int pass = 0; pass < 2; ++pass) {
        const double s = mode == kTarget       ? stretch<PT, kTarget>(tp, dp, no, i0, i1, vec, lane)
                         : mode == kDifference ? stretch<PT, kDifference>(tp, dp, no, i0, i1, vec, lane)
                                               : stretch<PT, kWithout>(tp, dp, no, i0, i1, vec, lane);
        if (lane == 0) sums[warp] = s;
        __syncthreads();
        if (tid == 0) {
            double all = 0.0;
            for (int w = 0; w < kWarps; ++w) all += sums[w];
            block_sum = all;
        }
        cluster.sync();
        total = 0.0;
        for (int r = 0; r < blocks; ++r) total += *cluster.map_shared_rank(&block_sum, r);
        if (total > 0.0 || mode == kTarget) break;
        mode = kTarget;  // nothing left over of the target: drawn from the target itself
        cluster.sync();  // before the sums are written again
    }
    if (total > 0.0) {
        // the block, and then the warp, whose stretch passes the share; the last one with a weight where none does
        share = v > 0.0f ? (double)v * total : 0.0;
        double run = 0.0;
        bool passed = false;
        for (int r = 0; r < blocks && !passed; ++r) {
            const double s = *cluster.map_shared_rank(&block_sum, r);
            if (!(s > 0.0)) continue;
            owner = r;
            before = run;
            run += s;
            passed = run > share;
        }
    }
    if (owner == rank) {
        int mine = -1;
        double run = before, base = 0.0;
        bool passed = false;
        for (int w = 0; w < kWarps && !passed; ++w) {
            if (!(sums[w] > 0.0)) continue;
            mine = w;
            base = run;
            run += sums[w];
            passed = run > share;
        }
        if (mine == warp) {
            const int x = mode == kTarget       ? find<PT, kTarget>(tp, dp, no, i0, i1, vec, lane, base, share)
                          : mode == kDifference ? find<PT, kDifference>(tp, dp, no, i0, i1, vec, lane, base, share)
                                                : find<PT, kWithout>(tp, dp, no, i0, i1, vec, lane, base, share);
            if (lane == 0) out[accepted] = x;
        }
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
    cluster.sync();  // a block's shared memory stays while others read it
}

template <typename PT> cudaError_t go(const AcceptParams &p, cudaStream_t s) {
    // blocks a row: enough to fill the GPU twice over, up to the largest portable cluster
    int blocks = 1;
    while (blocks < 8 && (long long)p.batch * blocks < 2 * 152) blocks *= 2;
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
