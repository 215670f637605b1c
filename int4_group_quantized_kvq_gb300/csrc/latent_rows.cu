// latent_rows.cu -- the rows of a latent cache: one latent vector and one rotary key per token,
// shared by all query heads.  The latent part is normalised (RMS norm, optional) and quantized to 4
// bits in groups, the rotary key turned by its position and kept in fp16; the queries' rotary parts
// are turned in the same pass.
#include <cuda_fp16.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "kvq_rows.cuh"

namespace kvq {
namespace {

// A sum held as two floats, hi + lo with |lo| <= half a step of hi (Knuth's two-sum keeps what each
// addition rounds off), so the sum of L squares is off by about 2^-44 of itself.  A code next to a
// half-integer follows the norm's last bit: with an exact sum and a reciprocal root rounded once, the
// stored codes are a function of the row, whatever the order of the additions.
struct TwoFloat {
    float hi, lo;
    __device__ __forceinline__ void add(float x) {
        const float s = __fadd_rn(hi, x);
        const float t = __fsub_rn(s, hi);
        lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, t)), __fsub_rn(x, t)));
        hi = s;
    }
    __device__ __forceinline__ void renormalise() {
        const float s = __fadd_rn(hi, lo);
        lo = __fsub_rn(lo, __fsub_rn(s, hi));
        hi = s;
    }
};

// 1 / sqrt(m.hi + m.lo), rounded once (nearly always: one Newton step on the approximate root, its
// residual 1 - m r^2 formed with fmas, leaves an error of about 2^-42 before the last rounding).
__device__ __forceinline__ float rsqrt_two(const TwoFloat& m) {
    const float r = rsqrtf(m.hi);
    const float p = __fmul_rn(r, r);
    const float pl = fmaf(r, r, -p);
    float t = fmaf(-m.hi, p, 1.f);
    t = fmaf(-m.hi, pl, t);
    t = fmaf(-m.lo, p, t);
    return fmaf(0.5f * r, t, r);
}

// A warp takes a row: its latent values, L / 32 to a lane, are read once, summed, normalised, quantized and
// stored, its rotary key and the row's query heads turned in between; with few rows the heads are shared
// out over further warps.  A stream of bytes: 18 000 rows of L = 512 with 32 heads, 178 MB, take 43 us
// (4.1 TB/s) at 40% of the issue slots; what is missing is the chain of lookups and of the sum over the row
// ahead of its stores.  Rows in runs, their lookups side by side in the lanes of a warp, took 73 us instead
// of 54 for the whole case.
template <int L, bool INTER>
__global__ void __launch_bounds__(256, 3) latent_append_kernel(LatentAppendArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");  // (and no early start of the next kernel: q_out may be its q)
    constexpr int E = L / 32;  // latent values per lane
    constexpr int R = 64;      // rotary part
    const int lane = threadIdx.x & 31;
    const int qheads = a.q_pe != nullptr ? a.H : 0;
    // with one slice a warp does the whole row; with more, slice 0 the row's cache entry and the others
    // its query heads
    const int per = a.slices == 1 ? qheads : (qheads + a.slices - 2) / (a.slices - 1);
    const long long tasks = static_cast<long long>(a.rows) * a.slices;
    const long long warps = static_cast<long long>(gridDim.x) * (blockDim.x / 32);
    for (long long task = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) / 32; task < tasks;
         task += warps) {
        const int row = static_cast<int>(task / a.slices);
        const int slice = static_cast<int>(task - static_cast<long long>(row) * a.slices);
        const bool entry = slice == 0;
        const int h0 = a.slices == 1 ? 0 : max(0, slice - 1) * per;
        const int h1 = a.slices == 1 ? qheads : entry ? 0 : min(qheads, h0 + per);
        uint4 raw[E / 8];
        const __half* src = a.x + row * a.x_stride;
        if (entry) {  // (before the lookups: rows behind the last sequence are read too, and dropped)
#pragma unroll
            for (int i = 0; i < E / 8; ++i) raw[i] = __ldcs(reinterpret_cast<const uint4*>(src + lane * E) + i);
        }
        const int b = warp_find_seq(a.cu_rows, a.B, row, lane);
        if (b < 0) continue;
        const long long pos = static_cast<long long>(__ldg(a.start_pos + b)) + (row - __ldg(a.cu_rows + b));
        // the angles of the lane's pairs 4 (lane % 8) .. + 3: eight lanes turn a head
        const int p0 = 4 * (lane & 7);
        const long long tp = a.positions != nullptr ? __ldg(a.positions + row) : pos;
        if (tp < 0 || tp >= a.table_len) {
            if (lane == 0) raise_flag(a.status, KVQ_FLAG_BAD_POSITION);
            continue;
        }
        const float4 c4 = __ldg(reinterpret_cast<const float4*>(a.table + tp * R + p0));
        const float4 n4 = __ldg(reinterpret_cast<const float4*>(a.table + tp * R + R / 2 + p0));
        const float c[4] = {c4.x, c4.y, c4.z, c4.w}, n[4] = {n4.x, n4.y, n4.z, n4.w};
        auto turn_head = [&](const __half* in, __half* out) {
            float u[4], w[4];
            if (INTER) {
                uint4 r = *reinterpret_cast<const uint4*>(in + 2 * p0);
                float x[8];
                halves_to_floats(r, x);
#pragma unroll
                for (int i = 0; i < 4; ++i) turn(x[2 * i], x[2 * i + 1], c[i], n[i]);
                *reinterpret_cast<uint4*>(out + 2 * p0) = floats_to_halves(x);
            } else {
                const uint2 ra = *reinterpret_cast<const uint2*>(in + p0);
                const uint2 rb = *reinterpret_cast<const uint2*>(in + R / 2 + p0);
                const float2 a0 = __half22float2(*reinterpret_cast<const __half2*>(&ra.x));
                const float2 a1 = __half22float2(*reinterpret_cast<const __half2*>(&ra.y));
                const float2 b0 = __half22float2(*reinterpret_cast<const __half2*>(&rb.x));
                const float2 b1 = __half22float2(*reinterpret_cast<const __half2*>(&rb.y));
                u[0] = a0.x, u[1] = a0.y, u[2] = a1.x, u[3] = a1.y;
                w[0] = b0.x, w[1] = b0.y, w[2] = b1.x, w[3] = b1.y;
#pragma unroll
                for (int i = 0; i < 4; ++i) turn(u[i], w[i], c[i], n[i]);
                *reinterpret_cast<uint2*>(out + p0) = make_uint2(pack_h2(u[0], u[1]), pack_h2(u[2], u[3]));
                *reinterpret_cast<uint2*>(out + R / 2 + p0) = make_uint2(pack_h2(w[0], w[1]), pack_h2(w[2], w[3]));
            }
        };
#pragma unroll 2
        for (int h = h0 + lane / 8; h < h1; h += 4)
            turn_head(a.q_pe + row * a.q_pe_stride + static_cast<long long>(h) * R,
                      a.q_out + (static_cast<long long>(row) * a.H + h) * (L + R) + L);
        if (!entry) continue;
        const long long pidx = pos >> a.lg_p;
        if (pos < 0 || pidx >= a.max_blocks) {
            if (lane == 0) raise_flag(a.status, KVQ_FLAG_BAD_POSITION);
            continue;
        }
        const int page = __ldg(a.block_table + static_cast<long long>(b) * a.max_blocks + pidx);
        if (page < 0 || page >= a.num_pages) {
            if (lane == 0) raise_flag(a.status, KVQ_FLAG_BAD_PAGE);
            continue;
        }
        const int slot = static_cast<int>(pos & ((1 << a.lg_p) - 1));
        uint8_t* blk = a.pool + static_cast<long long>(page) * a.lay.bytes;
        if (lane < 8)
            turn_head(src + L, reinterpret_cast<__half*>(blk + a.lay.rope) + static_cast<long long>(slot) * R);
        float x[E];
#pragma unroll
        for (int i = 0; i < E / 8; ++i) halves_to_floats(raw[i], *reinterpret_cast<float(*)[8]>(&x[8 * i]));
        if (a.gain != nullptr) {
            TwoFloat s{0.f, 0.f};
#pragma unroll
            for (int i = 0; i < E; ++i) s.add(__fmul_rn(x[i], x[i]));  // (a product of two fp16 values is exact)
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) {
                const float oh = __shfl_xor_sync(0xffffffffu, s.hi, off);
                const float ol = __shfl_xor_sync(0xffffffffu, s.lo, off);
                // two-sum of the lanes' hi parts: the larger first in both lanes, so both get the same
                const float big = fmaxf(s.hi, oh), small = fminf(s.hi, oh);
                const float lo = __fadd_rn(s.lo, ol);
                s.hi = big;
                s.lo = lo;
                s.add(small);
            }
            s.renormalise();
            s.hi *= 1.f / L;  // (a power of two)
            s.lo *= 1.f / L;
            s.add(a.eps);
            s.renormalise();
            const float r = rsqrt_two(s);
            const float4* g = reinterpret_cast<const float4*>(a.gain + lane * E);
#pragma unroll
            for (int i = 0; i < E / 4; ++i) {
                const float4 w = __ldg(g + i);
                x[4 * i] = __fmul_rn(__fmul_rn(x[4 * i], r), w.x);
                x[4 * i + 1] = __fmul_rn(__fmul_rn(x[4 * i + 1], r), w.y);
                x[4 * i + 2] = __fmul_rn(__fmul_rn(x[4 * i + 2], r), w.z);
                x[4 * i + 3] = __fmul_rn(__fmul_rn(x[4 * i + 3], r), w.w);
            }
        }
        float amax = 0.f;
#pragma unroll
        for (int i = 0; i < E; ++i) amax = fmaxf(amax, fabsf(x[i]));
#pragma unroll
        for (int off = 1; off < 128 / E; off <<= 1) {
            const float t = __shfl_xor_sync(0xffffffffu, amax, off);
            if (off * E < a.lay.G) amax = fmaxf(amax, t);
        }
        const __half s16 = scale_of(__fdiv_rn(amax, 7.f));
        const float sc = __half2float(s16);
        uint32_t words[E / 8];
#pragma unroll
        for (int i = 0; i < E / 8; ++i)
            words[i] = quant_word8<false>(*reinterpret_cast<const float(*)[8]>(&x[8 * i]), sc, amax);
        uint8_t* codes = blk + slot * (L / 2) + lane * (E / 2);
        if constexpr (E == 16) *reinterpret_cast<uint2*>(codes) = make_uint2(words[0], words[1]);
        else *reinterpret_cast<uint32_t*>(codes) = words[0];
        if (lane * E % a.lay.G == 0)
            reinterpret_cast<__half*>(blk + a.lay.scales)[slot * (L / a.lay.G) + lane * E / a.lay.G] = s16;
    }
}

// The way back, a warp a row: 28 MB in 12 us, of which the launch and one chain of lookups are half.
template <int L>
__global__ void __launch_bounds__(256) latent_dequantize_kernel(LatentDequantArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int E = L / 32, R = 64;
    const int lane = threadIdx.x & 31;
    const int warps = gridDim.x * (blockDim.x / 32);
    for (int row = (blockIdx.x * blockDim.x + threadIdx.x) / 32; row < a.rows; row += warps) {
        const int b = warp_find_seq(a.cu_rows, a.B, row, lane);
        if (b < 0) continue;
        const long long pos = static_cast<long long>(__ldg(a.start_pos + b)) + (row - __ldg(a.cu_rows + b));
        const long long pidx = pos >> a.lg_p;
        __half* out = a.out + static_cast<long long>(row) * (L + R);
        if (pos < 0 || pidx >= a.max_blocks) {  // zero rows, as kvq_dequantize
            if (lane == 0) raise_flag(a.status, KVQ_FLAG_BAD_POSITION);
            for (int i = lane; i < (L + R) / 8; i += 32) reinterpret_cast<uint4*>(out)[i] = make_uint4(0, 0, 0, 0);
            continue;
        }
        int page = __ldg(a.block_table + static_cast<long long>(b) * a.max_blocks + pidx);
        if (page < 0 || page >= a.num_pages) {
            if (lane == 0) raise_flag(a.status, KVQ_FLAG_BAD_PAGE);
            page = 0;
        }
        const int slot = static_cast<int>(pos & ((1 << a.lg_p) - 1));
        const uint8_t* blk = a.pool + static_cast<long long>(page) * a.lay.bytes;
        const float s = __half2float(
            reinterpret_cast<const __half*>(blk + a.lay.scales)[slot * (L / a.lay.G) + lane * E / a.lay.G]);
        const uint32_t* codes = reinterpret_cast<const uint32_t*>(blk + slot * (L / 2) + lane * (E / 2));
        uint32_t w[E / 8];
        if constexpr (E == 16) {
            const uint2 t = __ldg(reinterpret_cast<const uint2*>(codes));
            w[0] = t.x, w[1] = t.y;
        } else {
            w[0] = __ldg(codes);
        }
        uint4 rope = make_uint4(0, 0, 0, 0);
        if (lane < R / 8)
            rope = __ldg(reinterpret_cast<const uint4*>(blk + a.lay.rope + slot * (2 * R)) + lane);
#pragma unroll
        for (int i = 0; i < E / 8; ++i) {
            float v[8];
            codes_to_floats(w[i], s, v);
            reinterpret_cast<uint4*>(out + lane * E)[i] = floats_to_halves(v);
        }
        if (lane < R / 8) reinterpret_cast<uint4*>(out + L)[lane] = rope;
    }
}

}  // namespace

cudaError_t launch_latent_append(LatentAppendArgs a, cudaStream_t stream) {
    const int parts = a.q_pe != nullptr ? 1 + (a.H + 3) / 4 : 1;
    const int blocks = rows_grid(a.rows, parts, 24, &a.slices);
    const void* k = a.lay.L == 512 ? (a.inter ? (const void*)latent_append_kernel<512, true>
                                              : (const void*)latent_append_kernel<512, false>)
                                   : (a.inter ? (const void*)latent_append_kernel<256, true>
                                              : (const void*)latent_append_kernel<256, false>);
    void* args[] = {&a};
    return launch_rows(k, blocks, 256, args, stream);
}

cudaError_t launch_latent_dequantize(LatentDequantArgs a, cudaStream_t stream) {
    int slices = 1;
    const int blocks = rows_grid(a.rows, 1, 32, &slices);
    void* args[] = {&a};
    return launch_rows(a.lay.L == 512 ? (const void*)latent_dequantize_kernel<512> : (const void*)latent_dequantize_kernel<256>,
                       blocks, 256, args, stream);
}

}  // namespace kvq
