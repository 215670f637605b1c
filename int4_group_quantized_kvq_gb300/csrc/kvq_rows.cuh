// kvq_rows.cuh -- what the kernels over a ragged batch of rows share: which sequence a row
// belongs to, and the quantization of 8 values a lane holds.
//
// A ragged batch: rows cu_rows[b] .. cu_rows[b + 1] - 1 belong to sequence b, rows from
// cu_rows[B] on to none (a padded batch).
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

#include "kvq_device.cuh"
#include "kvq_quant.cuh"

namespace kvq {

// The sequence of row `row`, by the whole warp: the last b with cu_rows[b] <= row, or -1 for a
// row of no sequence.  Each round narrows the candidates 32-fold (one load and one vote), so a
// batch of up to 1023 sequences takes two dependent loads where a bisection takes ten.
// Offsets that do not ascend give some b in [-1, B).
__device__ __forceinline__ int warp_find_seq(const int32_t* cu_rows, int B, int row, int lane) {
    int lo = 0, n = B + 1;
    while (true) {
        const int step = (n + 31) / 32;
        const int at = lane * step;
        const bool le = at < n && __ldg(cu_rows + lo + at) <= row;
        const int cnt = __popc(__ballot_sync(0xffffffffu, le));
        if (cnt == 0) return -1;  // (only offsets that do not ascend: cu_rows[0] is 0)
        lo += (cnt - 1) * step;
        if (step == 1) break;
        n = min(step, n - (cnt - 1) * step);
    }
    return lo < B ? lo : -1;
}

// fp32(1/7): fp16_rne(a * kSeventh) == fp16_rne(fp32_rn(a / 7)) for every fp16 a >= 0 (see quantize.cu).
constexpr float kSeventh = 0.142857149f;

__device__ __forceinline__ void halves_to_floats(uint4 r, float (&x)[8]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

// The largest magnitude of 8 values, NaN ignored (as fmaxf does).
__device__ __forceinline__ float amax8(const float (&x)[8]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
    return m;
}

// A group's scale from its largest magnitude: fp16_rne(amax / 7), 1 where that is zero.
__device__ __forceinline__ __half scale_of(float amax_seventh) {
    __half s16 = __float2half_rn(amax_seventh);
    if ((__half_as_ushort(s16) & 0x7fffu) == 0) s16 = __ushort_as_half(0x3c00u);
    return s16;
}

// The codes of 8 values as a word of nibbles (code + 8, low nibble first), s the group's scale and
// amax its largest magnitude: the two-step arithmetic of quant_lane16 (quantize.cu), for 8 values.
// With rs = rcp(s) within 2 ulp of 1/s, m = fma(x, rs, 1.5 2^23 + 8) rounds x rs + 8 once, and
// e = x rs - (m - ..) tells how far from a half-integer it is.  Off by less than 2^-19, the quotient
// rounds to the same integer when every |e| <= 1/2 - 2^-16; else (or where a clamp is possible, or
// for NaN and infinities) the quotient itself decides: F16 values take the exact half-integer check,
// values of fp32 the IEEE division.
template <bool F16>
__device__ __forceinline__ uint32_t quant_word8(const float (&x)[8], float s, float amax) {
    float rs;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rs) : "f"(s));
    constexpr float kMagic8 = 12582920.0f;        // 1.5 * 2^23 + 8
    constexpr float kBand = 0.4999847412109375f;  // 1/2 - 2^-16
    uint32_t m[8];
    float emax = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float mi = fmaf(x[i], rs, kMagic8);
        emax = max_abs_nan(emax, fmaf(x[i], rs, kMagic8 - mi));
        m[i] = __float_as_uint(mi);
    }
    // bits 4 .. 21 of m are zero and its low four bits are the nibble: shift-adds pack them
    const uint32_t lo = m[0] + 16u * m[1] + 256u * (m[2] + 16u * m[3]);
    const uint32_t hi = m[4] + 16u * m[5] + 256u * (m[6] + 16u * m[7]);
    uint32_t word = prmt(lo, hi, 0x5410u);
    if (amax * rs > 7.49f || !(emax <= kBand)) {
        if (F16) {
            bool plain = isinf(s);
#pragma unroll
            for (int i = 0; i < 8; ++i) plain |= x[i] != x[i];
            word = quant8(x, s, plain);
        } else {
            word = quant8(x, s, true);
        }
    }
    return word;
}

// Eight codes times their scale, rounded to fp16 (the product is exact in fp32).
__device__ __forceinline__ void codes_to_floats(uint32_t word, float s, float (&v)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = static_cast<float>(static_cast<int>((word >> (4 * k)) & 0xFu) - 8) * s;
}
__device__ __forceinline__ uint4 floats_to_halves(const float (&v)[8]) {
    return make_uint4(pack_h2(v[0], v[1]), pack_h2(v[2], v[3]), pack_h2(v[4], v[5]), pack_h2(v[6], v[7]));
}

// (a, b) turned by (c, n): (a c - b n, b c + a n), every operation rounded once to fp32.
__device__ __forceinline__ void turn(float& a, float& b, float c, float n) {
    const float u = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, n));
    b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, n));
    a = u;
}

}  // namespace kvq
