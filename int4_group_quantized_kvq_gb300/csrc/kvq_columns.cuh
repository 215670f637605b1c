// kvq_columns.cuh -- softmax over scores that lie transposed in tensor memory (positions along the lanes,
// lines along the columns), by 256 threads: two have a position, half of the lines each.
#pragma once

#include <cstdint>

#include "kvq_device.cuh"
#include "kvq_tcgen05.cuh"

namespace kvq {

__device__ __forceinline__ float warp_max(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}
// Barrier of the softmax warps that tells whether any thread's x holds.
__device__ __forceinline__ bool any_of_softmax(bool x) {
    uint32_t r;
    asm volatile(
        "{ .reg .pred p, q; setp.ne.u32 p, %1, 0; barrier.cta.red.or.pred q, 2, 256, p; selp.u32 %0, 1, 0, q; }"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(x))
        : "memory");
    return r != 0;
}
__device__ __forceinline__ void softmax_barrier() { asm volatile("barrier.cta.sync 1, 256;" ::: "memory"); }

// Sums over the warp's lanes of N values each: halving the values a lane keeps at each exchange, N - 1
// shuffles and a few.  Afterwards v[0] of a lane is the sum of column first_column (N up to 32).
template <int N>
__device__ __forceinline__ void warp_sums(float (&v)[N], int lane) {
    int n = N;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        if (n > 1) {
            n /= 2;
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                if (i >= n) break;
                const float keep = lane & off ? v[i + n] : v[i], send = lane & off ? v[i] : v[i + n];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, send, off);
            }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], off);
        }
    }
}
template <int N>
__device__ __forceinline__ int first_column(int lane) {
    int n = N, c = 0;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        if (n > 1) {
            n /= 2;
            if (lane & off) c += n;
        }
    return c;
}

template <int N>
__device__ __forceinline__ void load_columns(uint32_t addr, uint32_t (&v)[N]) {
    if constexpr (N == 8) tmem_ld8(addr, v);
    if constexpr (N == 16) tmem_ld16(addr, v);
    if constexpr (N == 32) tmem_ld32(addr, v);
    tmem_wait_ld();
    tmem_touch(v);
}

// The dimension at position x (of 8) in the order the unpack leaves.
__device__ __forceinline__ int dim_of(int x) { return (x & ~7) + ((x & 7) >> 1) + 4 * (x & 1); }

}  // namespace kvq
