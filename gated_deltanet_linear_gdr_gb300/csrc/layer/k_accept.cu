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
// two-sum (Knuth, The Art of Computer Programming 2, 4.2.2): 14 additions a token, which
// the FP32 pipes do while memory delivers it; the FP64 pipes (2 operations a cycle and
// multiprocessor) would take several times as long.  The error is itself a sum that is
// rounded: after n additions it has lost n^2/2 2^-48 of the sum at worst.  So a lane
// begins a new pair every 64 tokens: good to 2^-36 at worst, to 2^-45 by chance, however
// many tokens there are.  Beside that only single warps, at the joints, work in double.
//
// Measured, float32 probabilities: 256 rows of 5 to 8 tokens against 32000 tokens 24 us (9.3 at the copy rate), one
// row against 131072 15 us, of which the host takes 11.
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
    // p - q where that is positive, as (difference, its rounding error)
    __device__ __forceinline__ void add_difference(float p, float q) {
        const float w = __fsub_rn(p, q), b = __fsub_rn(w, p);
        const float e = __fsub_rn(__fsub_rn(p, __fsub_rn(w, b)), __fadd_rn(q, b));
        const bool some = w > 0.0f;
        add(some ? w : 0.0f, some ? e : 0.0f);
    }
    __device__ __forceinline__ Sum over_warp() const {
        Sum a = *this;
#pragma unroll
        for (int m = 16; m; m >>= 1) {
            const float os = __shfl_xor_sync(kFull, a.s, m), oc = __shfl_xor_sync(kFull, a.c, m);
            a.add(os, oc);
        }
        return a;
    }
    __device__ __forceinline__ double value() const { return (double)s + (double)c; }
};

// A lane's sum over any number of tokens: pairs of kFold of them at most, added up as normalised pairs (each of which
// adds 3 2^-48 at most: Joldes, Muller and Popescu 2017, tight and rigorous error bounds for basic building blocks of
// double-word arithmetic), kFold of those at most in double.
constexpr int kFold = 64;
struct LongSum {
    Sum part, mid;
    double all = 0.0;
    int folds = 0;
    __device__ __forceinline__ void fold() {
        const float h = __fadd_rn(part.s, part.c), l = __fsub_rn(part.c, __fsub_rn(h, part.s));
        const float t = __fadd_rn(mid.s, h), b = __fsub_rn(t, mid.s);
        const float e = __fadd_rn(__fsub_rn(mid.s, __fsub_rn(t, b)), __fsub_rn(h, b));
        const float w = __fadd_rn(e, __fadd_rn(mid.c, l));
        mid.s = __fadd_rn(t, w);
        mid.c = __fsub_rn(w, __fsub_rn(mid.s, t));
        part = Sum();
        if (++folds % kFold == 0) {
            all += mid.value();
            mid = Sum();
        }
    }
    __device__ __forceinline__ Sum pair() {
        if (folds == 0) return part;
        fold();
        if (folds <= kFold) return mid;
        all += mid.value();
        mid.s = (float)all;
        mid.c = (float)(all - (double)mid.s);
        return mid;
    }
};

// What a row's draw goes by: the weights of tokens [0, vocab).
template <typename PT> struct Weights {
    static constexpr int C = 16 / (int)sizeof(PT);  // tokens of a vector
    const PT *p, *q;
    bool difference;  // max(p - q, 0); else p
    int no;           // a token whose weight is 0, or -1
    int start;        // the first vector's place, where p is aligned: at or up to C - 1 before token 0
    bool vec;         // q is aligned where p is

    __device__ __forceinline__ double exact(int i) const {
        const float pi = clean(to_f32(p[i]));
        if (!difference) return i == no ? 0.0 : (double)pi;
        const float qi = clean(to_f32(q[i]));
        return pi > qi ? (double)pi - (double)qi : 0.0;
    }
    __device__ __forceinline__ void one(Sum &a, int i) const {
        const float pi = clean(to_f32(p[i]));
        if (difference) a.add_difference(pi, clean(to_f32(q[i])));
        else a.add(i == no ? 0.0f : pi, 0.0f);
    }
    // The sum of a lane's part of [i0, i1), C tokens or one at a time.
    __device__ __forceinline__ Sum slow(int i0, int i1, int lane) const {
        LongSum a;
        int n = 0;
        for (int i = i0 + lane; i < i1; i += 32) {
            if (i >= 0) one(a.part, i);
            if (++n % kFold == 0) a.fold();
        }
        return a.pair();
    }
    // The same by vectors.  Values that do not count leave a NaN in `odd`: then the sum is not to be used.
    template <bool DIFF> __device__ __forceinline__ Sum fast(int i0, int i1, int lane, float &odd) const {
        constexpr int U = 2;
        LongSum sum;
        Sum &a = sum.part;
        int n = 0;
        // whole vectors lie in [a0, a1); before them there are tokens only at the row's beginning, behind them only at its end
        const int a0 = i0 < 0 ? i0 + C : i0, a1 = i1 - (i1 - start) % C;
        if (i0 < 0 && lane < a0 && lane < i1) one(a, lane);
        if (a1 >= a0 && lane < i1 - a1) one(a, a1 + lane);
        for (int i = a0 + lane * C; i < a1; i += 32 * C * U) {
            Pack<PT, C> pv[U], qv[U];
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int at = i + k * 32 * C;
                if (at < a1) {
                    pv[k].load(p + at);
                    if (DIFF) qv[k].load(q + at);
                }
            }
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int at = i + k * 32 * C, gone = DIFF ? -1 : no - at;
                if (at >= a1) break;
#pragma unroll
                for (int j = 0; j < C; ++j) {
                    float x = pv[k].get(j);
                    odd = fmaf(x, 0.0f, odd);
                    x = fmaxf(x, 0.0f);
                    if constexpr (DIFF) {
                        const float y = qv[k].get(j);
                        odd = fmaf(y, 0.0f, odd);
                        a.add_difference(x, fmaxf(y, 0.0f));
                    } else {
                        a.add(j == gone ? 0.0f : x, 0.0f);
                    }
                }
            }
            if (++n % (kFold / (C * U)) == 0) sum.fold();
        }
        return sum.pair();
    }
    // The sum of a warp's stretch [i0, i1), in every lane.
    __device__ __forceinline__ Sum stretch(int i0, int i1, int lane) const {
        Sum a;
        float odd = 0.0f;
        if (vec && i0 < i1) a = difference ? fast<true>(i0, i1, lane, odd) : fast<false>(i0, i1, lane, odd);
        if (!vec || __any_sync(kFull, odd != 0.0f)) a = slow(i0, i1, lane);
        return a.over_warp();
    }
};

// Of up to 32 parts, part `lane`'s weight `mine`: the one at which `before` and the running sum pass `share`,
// the last one with a weight where none does, -1 where there is no weight; `base`: the sum ahead of it, which is at
// most the share, although the running sums' roundings may put it above; `passed`: whether one does.
__device__ __forceinline__ int part_of(double mine, double before, double share, int lane, double &base, bool &passed) {
    double upto = mine;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const double o = __shfl_up_sync(kFull, upto, m);
        if (lane >= m) upto += o;
    }
    const unsigned some = __ballot_sync(kFull, mine > 0.0), past = __ballot_sync(kFull, mine > 0.0 && before + upto > share);
    const int which = past ? __ffs(past) - 1 : 31 - __clz(some);
    passed = past != 0;
    base = fmin(before + __shfl_sync(kFull, upto - mine, which < 0 ? 0 : which), share);
    return which;
}

template <typename PT> __global__ void __launch_bounds__(kThreads, 2) k_accept(const __grid_constant__ AcceptParams p) {
    __shared__ Sum sums[kWarps];  // of this block's stretches, then of a stretch's parts
    __shared__ double block_sum, joint_base, joint_share, joint_sum;
    __shared__ int first_refused, first_none, joint_owner, joint_part;
    __shared__ bool joint_passed;
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
    if (tid == 0) first_refused = first_none = drafts;
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
    w.difference = refused && draft;
    w.no = refused && !draft ? p.tokens[t + 1] : -1;
    const int off_p = (int)(reinterpret_cast<uintptr_t>(w.p) % 16), off_q = (int)(reinterpret_cast<uintptr_t>(w.q) % 16);
    w.vec = !w.difference || off_p == off_q;
    w.start = -(off_p / (int)sizeof(PT));

    // the sums: a stretch of whole vectors a warp
    const int each = ((p.vocab - w.start - 1) / (blocks * kWarps) + C) / C * C;
    const long long from = (long long)(rank * kWarps + warp) * each + w.start;
    const int i0 = (int)(from < p.vocab ? from : p.vocab), i1 = p.vocab - i0 < each ? p.vocab : i0 + each;
    for (int pass = 0; pass < 2; ++pass) {
        const Sum s = w.stretch(i0, i1, lane);
        if (lane == 0) sums[warp] = s;
        __syncthreads();
        if (warp == 0) {
            double all = lane < kWarps ? sums[lane].value() : 0.0;
#pragma unroll
            for (int m = kWarps / 2; m; m >>= 1) all += __shfl_xor_sync(kFull, all, m);
            if (lane == 0) block_sum = all;
        }
        if (blocks > 1) cluster.sync();
        if (warp == 0) {
            // lane r has block r's sum: every block finds the same place
            const double mine = blocks == 1 ? (lane == 0 ? block_sum : 0.0) : lane < blocks ? *cluster.map_shared_rank(&block_sum, lane) : 0.0;
            double total = mine, base;
            bool passed;
#pragma unroll
            for (int m = 4; m; m >>= 1) total += __shfl_xor_sync(kFull, total, m);
            total = __shfl_sync(kFull, total, 0);
            const double share = v > 0.0f ? (double)v * total : 0.0;
            const int owner = part_of(mine, 0.0, share, lane, base, passed);
            if (owner == rank) {
                const int part = part_of(lane < kWarps ? sums[lane].value() : 0.0, base, share, lane, base, passed);
                if (lane == 0) joint_part = part;
            }
            if (lane == 0) {
                joint_owner = owner;
                joint_base = base;
                joint_share = share;
            }
        }
        __syncthreads();
        if (joint_owner >= 0 || (!w.difference && w.no < 0)) break;
        w.difference = false;  // nothing left over of the target: drawn from the target itself
        w.no = -1;
        w.vec = true;
        if (blocks > 1) cluster.sync();  // before the sums are written again
    }
    const int owner = joint_owner;
    if (owner == rank) {
        // the stretch again, in parts of a vector a lane: the warp's part, then the lane's, then the token
        const double share = joint_share;
        double base = joint_base;
        const long long s0 = (long long)(rank * kWarps + joint_part) * each + w.start;
        const int end = (int)(s0 + each < p.vocab ? s0 + each : p.vocab);
        for (int i = (int)s0; i < end; i += C * kThreads) {
            const int at = i + tid * C;
            Sum own;
#pragma unroll
            for (int j = 0; j < C; ++j)
                if (at + j >= 0 && at + j < end) w.one(own, at + j);
            const Sum part = own.over_warp();
            __syncthreads();  // sums, and what hangs on it, are read no more
            if (lane == 0) sums[warp] = part;
            __syncthreads();
            if (warp == 0) {
                double next;
                bool passed;
                const double mine = lane < kWarps ? sums[lane].value() : 0.0;
                const int which = part_of(mine, base, share, lane, next, passed);
                double all = mine;
#pragma unroll
                for (int m = 16; m; m >>= 1) all += __shfl_xor_sync(kFull, all, m);
                if (lane == 0) {
                    joint_part = which;
                    joint_base = next;
                    joint_sum = all;
                    joint_passed = passed;
                }
            }
            __syncthreads();
            const int which = joint_part;
            const double ahead = joint_base;
            if (which == warp) {
                double first;
                bool passed;
                const int l = part_of(own.value(), ahead, share, lane, first, passed);
                // the token past the share: the last one with a weight and no more than the share ahead of it, as the
                // lane's first weight has it in any case
                int found = -1;
                if (lane == l) {
#pragma unroll
                    for (int j = 0; j < C; ++j) {
                        const double x = at + j >= 0 && at + j < end ? w.exact(at + j) : 0.0;
                        if (x > 0.0 && !(first > share)) found = at + j;
                        first += x;
                    }
                    out[accepted] = found;
                }
            }
            if (joint_passed) break;
            base = fmin(base + joint_sum, share);  // not passed, but for the roundings of this sum
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
    if (blocks > 1) cluster.sync();  // a block's shared memory stays while others read it
}

template <typename PT> cudaError_t go(const AcceptParams &p, cudaStream_t s) {
    // blocks a row: as many as run at once (two a multiprocessor), up to the largest portable cluster.  Measured, against
    // one block a row: one row of 131072 tokens 15 / 33 us, 33 rows of 50257 15 / 16 (the host's call is 11 of each).
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
