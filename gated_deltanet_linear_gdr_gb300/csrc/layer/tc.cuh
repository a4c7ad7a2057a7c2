// Tensor core (tcgen05), TMA and mbarrier instructions as inline PTX.
//
// Every wait is bounded: after kWaitLimit clock cycles (about a second), or once
// another warp of the CTA has given up, it returns false and the caller leaves
// its loop.
#pragma once

#include <cuda.h>

#include "../gdr_device.cuh"

namespace gdr {
namespace tc {

constexpr unsigned kWaitLimit = 2000000000u;

__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// One attempt; the hardware may suspend the warp for up to about a millisecond.
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(1000000u)
        : "memory");
    return ok != 0;
}
// Waits for the phase of this parity; false if the limit ran out or *gave_up is set.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, volatile int *gave_up) {
    const unsigned start = (unsigned)clock();
    while (!mbar_try(bar, parity)) {
        if (*gave_up) return false;
        if ((unsigned)clock() - start > kWaitLimit) {
            *gave_up = 1;
            return false;
        }
    }
    return true;
}

// Generic-proxy writes to shared memory become visible to TMA and the tensor cores.
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// One box of a 3-dimensional tensor map; x * element size is a multiple of 16 bytes.
__device__ __forceinline__ void tma_load3(uint32_t dst, const CUtensorMap *map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}
// The same in 4 dimensions, and back.  Stores of a thread are waited for by that thread.
__device__ __forceinline__ void tma_load4(uint32_t dst, const CUtensorMap *map, int x, int y, int z, int w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
        ::"r"(dst), "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void tma_store4(const CUtensorMap *map, int x, int y, int z, int w, uint32_t src) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3, %4}], [%5];" ::"l"(map),
                 "r"(x), "r"(y), "r"(z), "r"(w), "r"(src)
                 : "memory");
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
__device__ __forceinline__ void tma_stores_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void tma_stores_done() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
// Takes the eight bfloat16 values at a, a + 256, ... and puts the roundings of
// x there; x becomes what was taken.  One piece, so that each value keeps its
// register and the loads wait once.
__device__ __forceinline__ void exchange_bf16(uint32_t a, float2 &x, float2 &y, float2 &z, float2 &w) {
    asm volatile(
        "{\n\t.reg .b16 p<8>, q<8>, z;\n\t.reg .b32 w;\n\tmov.b16 z, 0;\n\t"
        "ld.shared.b16 p0, [%8+0];\n\t"
        "ld.shared.b16 p1, [%8+256];\n\t"
        "ld.shared.b16 p2, [%8+512];\n\t"
        "ld.shared.b16 p3, [%8+768];\n\t"
        "ld.shared.b16 p4, [%8+1024];\n\t"
        "ld.shared.b16 p5, [%8+1280];\n\t"
        "ld.shared.b16 p6, [%8+1536];\n\t"
        "ld.shared.b16 p7, [%8+1792];\n\t"
        "cvt.rn.bf16x2.f32 w, %1, %0;\n\t"
        "mov.b32 {q0, q1}, w;\n\t"
        "cvt.rn.bf16x2.f32 w, %3, %2;\n\t"
        "mov.b32 {q2, q3}, w;\n\t"
        "cvt.rn.bf16x2.f32 w, %5, %4;\n\t"
        "mov.b32 {q4, q5}, w;\n\t"
        "cvt.rn.bf16x2.f32 w, %7, %6;\n\t"
        "mov.b32 {q6, q7}, w;\n\t"
        "st.shared.b16 [%8+0], q0;\n\t"
        "st.shared.b16 [%8+256], q1;\n\t"
        "st.shared.b16 [%8+512], q2;\n\t"
        "st.shared.b16 [%8+768], q3;\n\t"
        "st.shared.b16 [%8+1024], q4;\n\t"
        "st.shared.b16 [%8+1280], q5;\n\t"
        "st.shared.b16 [%8+1536], q6;\n\t"
        "st.shared.b16 [%8+1792], q7;\n\t"
        "mov.b32 w, {z, p0};\n\t"
        "mov.b32 %0, w;\n\t"
        "mov.b32 w, {z, p1};\n\t"
        "mov.b32 %1, w;\n\t"
        "mov.b32 w, {z, p2};\n\t"
        "mov.b32 %2, w;\n\t"
        "mov.b32 w, {z, p3};\n\t"
        "mov.b32 %3, w;\n\t"
        "mov.b32 w, {z, p4};\n\t"
        "mov.b32 %4, w;\n\t"
        "mov.b32 w, {z, p5};\n\t"
        "mov.b32 %5, w;\n\t"
        "mov.b32 w, {z, p6};\n\t"
        "mov.b32 %6, w;\n\t"
        "mov.b32 w, {z, p7};\n\t"
        "mov.b32 %7, w;\n\t"
        "}"
        : "+f"(x.x), "+f"(x.y), "+f"(y.x), "+f"(y.y), "+f"(z.x), "+f"(z.y), "+f"(w.x), "+f"(w.y)
        : "r"(a)
        : "memory");
}
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap *map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// ---- tensor memory ------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc(uint32_t slot, uint32_t cols) {  // whole warp
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(slot), "r"(cols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {  // whole warp
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 lanes x 16 columns: thread = lane, r[i] = column i.
__device__ __forceinline__ void tmem_ld16(uint32_t a, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(a));
}
// The same back, 8 columns.
__device__ __forceinline__ void tmem_st8(uint32_t a, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(a), "r"(r[0]), "r"(r[1]),
                 "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
// 16 lanes x 64 columns in the layout of an m16n8 accumulator, eight times over:
// r[4n], r[4n+1]: lane t/4, columns 8n + 2(t%4), +1; r[4n+2], r[4n+3]: lane t/4 + 8.
__device__ __forceinline__ void tmem_ld_16x64(uint32_t a, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(a));
}

// The same for 32 columns.
__device__ __forceinline__ void tmem_ld_16x32(uint32_t a, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(a));
}

// True in one lane of a converged warp.
__device__ __forceinline__ uint32_t elect_one() {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(ok));
    return ok;
}

// Moves a warpgroup's registers a thread; every warp of it executes this, and
// the shares of all warpgroups add up to no more than the launch gave out.
template <int N> __device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// The value of lane 0, for all lanes: tells the compiler that a number is the
// same in the whole warp, so that descriptors made from it stay in uniform
// registers (a matrix instruction takes no others).
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// ---- matrix instructions --------------------------------------------------------
// Shared-memory operand of 128-byte rows in 8-row swizzled atoms (1024 bytes,
// 1024-byte aligned).  K-major: sbo = bytes between groups of 8 rows.
// MN-major: rows run along K; sbo = bytes between groups of 8 rows, lbo =
// bytes between blocks of 64 MN elements.
__device__ __forceinline__ uint64_t desc128(uint32_t addr, uint32_t lbo, uint32_t sbo) {
    return (uint64_t)((addr & 0x3ffff) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(sbo >> 4) << 32) |
           (1ull << 46) | (2ull << 61);
}
// bfloat16 operands, float32 accumulator; *_mn: the operand is MN-major.
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, bool a_mn, bool b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
// `me`: elect_one() of a converged warp.  The instruction is predicated, not
// branched around, so that the warp stays converged and the operands, which
// have to lie in uniform registers, are computed there: behind a branch each
// of them is moved over first, which measured 60 to 110 cycles a product of 32.
template <bool ACC> __device__ __forceinline__ void mma_ss(uint32_t me, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc),
        "n"(ACC ? 1 : 0), "r"(me)
        : "memory");
}
template <bool ACC> __device__ __forceinline__ void mma_ts(uint32_t me, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc),
        "n"(ACC ? 1 : 0), "r"(me)
        : "memory");
}
// D = A B over STEPS steps of 16 along K, both operands K-major in blocks of 64
// (`block` bytes apart).  Written out by the compiler: a counted loop costs
// about as much a step as the product itself.
template <int STEPS> __device__ __forceinline__ void mma_ss_k(uint32_t me, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                                             uint32_t block) {
    mma_ss<false>(me, d, a, b, idesc);
#pragma unroll
    for (int i = 1; i < STEPS; ++i) {
        const uint32_t at = ((uint32_t)(i >> 2) * block + (uint32_t)(i & 3) * 32) >> 4;
        mma_ss<true>(me, d, a + at, b + at, idesc);
    }
}
// The same with A in tensor memory, 8 columns a step.
template <int STEPS, bool ACC>
__device__ __forceinline__ void mma_ts_k(uint32_t me, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t block) {
    mma_ts<ACC>(me, d, a, b, idesc);
#pragma unroll
    for (int i = 1; i < STEPS; ++i)
        mma_ts<true>(me, d, a + i * 8, b + (((uint32_t)(i >> 2) * block + (uint32_t)(i & 3) * 32) >> 4), idesc);
}
// D = A B over 64 along K, both operands MN-major (2048 bytes a step of 16).
template <bool ACC> __device__ __forceinline__ void mma_ss_mn64(uint32_t me, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
    mma_ss<ACC>(me, d, a, b, idesc);
#pragma unroll
    for (int i = 1; i < 4; ++i) mma_ss<true>(me, d, a + (i * 2048 >> 4), b + (i * 2048 >> 4), idesc);
}
// The barrier gets one arrival once every matrix instruction this thread has issued is done.
__device__ __forceinline__ void mma_commit(uint32_t me, uint32_t bar) {
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(me)
        : "memory");
}

__device__ __forceinline__ void stmatrix4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
                 "r"(d)
                 : "memory");
}
// An 8x8 matrix of 16-bit values, two neighbours of row lane / 4 in a lane, transposed.
__device__ __forceinline__ uint32_t turn8x8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
// stmatrix4 with each 8x8 matrix transposed.
__device__ __forceinline__ void stmatrix4_t(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b),
                 "r"(c), "r"(d)
                 : "memory");
}
// A pair of bfloat16 in one register, lower half first, and back.
__device__ __forceinline__ float2 unpack_bf16(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack_bf16(float2 x) {
    const __nv_bfloat162 h2 = __floats2bfloat162_rn(x.x, x.y);
    return *reinterpret_cast<const uint32_t *>(&h2);
}
// x - (what its bfloat16 rounding w holds): exact
__device__ __forceinline__ float2 rest_bf16(float2 x, uint32_t w) {
    return __ffma2_rn(unpack_bf16(w), make_float2(-1.0f, -1.0f), x);
}

}  // namespace tc
}  // namespace gdr
