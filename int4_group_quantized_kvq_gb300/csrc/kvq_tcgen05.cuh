// kvq_tcgen05.cuh -- the fifth-generation tensor cores in inline PTX: tensor memory, the MMA of f16
// operands into f32 accumulators, its completion on mbarriers, and the operand layout used here.
//
// Every operand tile in shared memory is a set of chunks of [rows][64 f16] in the 128-byte swizzle: row
// t of a chunk is 128 bytes at 128 t, its 16-byte piece p stored at piece p ^ (t & 7); chunks start on
// 1024-byte boundaries.  Such a tile serves as a K-major operand (rows are M or N, the 64 values run
// along K) and, unchanged, as an MN-major one (rows run along K, the values are M or N).
#pragma once

#include <cstdint>

#include "kvq_device.cuh"

namespace kvq {

// Byte offset of 16-byte piece `piece` (0 .. 7) of row `row` of a chunk.
__device__ __forceinline__ uint32_t swizzled(uint32_t row, uint32_t piece) {
    return row * 128u + ((piece ^ (row & 7u)) << 4);
}

// Shared-memory matrix descriptor, 128-byte swizzle, 1024 bytes from one group of 8 rows to the next.  Its
// low word holds the address (in 16 bytes) and lbo: MN-major, the bytes from one chunk of 64 values to
// the next (K-major: unused).  Steps within a tile add to the low word.
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) {
    return ((addr & 0x3FFFFu) >> 4) | (lbo >> 4) << 16;
}
__device__ __forceinline__ uint64_t smem_desc(uint32_t lo) {
    constexpr uint32_t kHi = (1024u >> 4) | (1u << 14) | (2u << 29);
    return static_cast<uint64_t>(kHi) << 32 | lo;
}
// Instruction descriptor: f16 x f16 -> f32, M x N, MN-major flags of A and B.
constexpr uint32_t mma_idesc(int M, int N, bool a_mn, bool b_mn) {
    return (1u << 4) | (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
           (static_cast<uint32_t>(N / 8) << 17) | (static_cast<uint32_t>(M / 16) << 24);
}

__device__ __forceinline__ void tmem_alloc(uint32_t smem_result, uint32_t columns) {  // one whole warp
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_result), "r"(columns)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t columns) {  // the same warp
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(columns) : "memory");
}

// One thread of a converged warp, known as such to the compiler: operands of the instructions below sit
// in uniform registers, and behind any other condition it builds a loop over the threads for each.
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(one));
    return one != 0;
}

// A value that is the same in the whole warp, made known as such to the compiler (what follows from such
// values alone is computed in uniform registers, where the MMAs take their operands from).
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// D[tmem] (+)= A[smem] B[smem], 16 along K; by one thread.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d), "l"(a),
        "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
}
// The same with A in tensor memory (two f16 of K to a column).
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{ .reg .pred p; setp.ne.u32 p, %4, 0; tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p; }" ::"r"(d), "r"(a),
        "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(accumulate))
        : "memory");
}
// An arrival on `bar` once every MMA this thread has issued is complete.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 32 columns of the warp's 32 lanes, a lane's row in its registers.  The values are there after
// tmem_wait_ld, to which the caller ties their use (tmem_touch).
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
        "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t addr, uint32_t (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(addr)
        : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
        "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr)
        : "memory");
}
// Keeps uses of r behind the tmem_wait_ld before it.
template <int N>
__device__ __forceinline__ void tmem_touch(uint32_t (&r)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// Two fp32 values in a register pair, and arithmetic on both in one instruction (each rounded once).
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void split_pair(uint64_t x, float& a, float& b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x));
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

template <int N>
__device__ __forceinline__ void regs_more() {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_less() {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// A wait of these kernels on an mbarrier, by a whole warp: bounded (by p.wait_ns), and over at once when any
// thread of the CTA has given up (*stop).  A thread that gives up raises the flag and goes on through its loops
// without waiting, so the CTA's barriers stay matched; the issuers of copies and MMAs issue nothing more, and
// wait for what they have issued before the CTA leaves (finish_products; load_pages in chunk_shared.cuh).
constexpr uint32_t kWaitNs = 250000000;
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile("{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
                 : "=r"(done)
                 : "r"(bar), "r"(parity)
                 : "memory");
    return done != 0;
}
template <class P>
__device__ __forceinline__ bool wait_or_stop(uint32_t bar, uint32_t parity, volatile int* stop, const P& p) {
    bool there = mbar_try(bar, parity);
    if (!there) {
        uint64_t t0 = 0;
        for (uint32_t tries = 1; !(there = mbar_try(bar, parity)); ++tries) {
            // (a short wait reads neither: *stop behind the first try took 4% of a call of drafted tokens, every fourth one
            // 1% of a part of a prompt)
            if (tries % 16) continue;
            if (*stop) break;
            const uint64_t t = global_timer_ns();
            if (t0 == 0) t0 = t;
            if (t - t0 > p.wait_ns) {
                *stop = 1;
                raise_flag(p.status, KVQ_FLAG_WAIT_TIMEOUT);
                break;
            }
        }
    }
    return __all_sync(0xffffffffu, there);  // false: given up
}

// The end of a CTA, behind a barrier of all its threads (which all call this).  Once a wait has been given up,
// nobody has waited for the last products: they may still read shared memory, write tensor memory and arrive on
// barriers.  Each warp that issued some waits for all of its own (`bar`: a barrier of its own, of one arrival;
// the elected thread is the same every time), and nobody leaves before.
__device__ __forceinline__ void finish_products(bool issuer, uint32_t bar, volatile int* stop) {
    if (!*stop) return;
    if (issuer) {
        if (elect_one()) mma_commit(bar);
        __syncwarp();
        mbar_wait(bar, 0, kWaitNs);
    }
    __syncthreads();
}

}  // namespace kvq
