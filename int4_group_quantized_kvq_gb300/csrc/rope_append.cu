// rope_append.cu -- rotary positions and quantize-on-append in one pass over the rows of a
// projection, and the way back: a ragged batch of cached rows, dequantized.
//
// A rotary pair (a, b) of a head turns by the angle of the row's position: (a c - b n, b c + a n)
// with c, n read from a table of cosines and sines, in fp32, then rounded to fp16.  q rows go to
// q_out; k rows, turned and rounded, and v rows, as they are, to their pages as kvq_quantize_append
// stores them, bit for bit.
#include <cuda_fp16.h>

#include <algorithm>

#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "kvq_rows.cuh"

namespace kvq {
namespace {

// A warp takes a row (or one of `slices` parts of its heads, when there are few rows): one lookup of
// the sequence, the page and the angles serves all of them, and a lane keeps the angles of its 8
// rotary pairs in registers.  LPR = D / 16 lanes hold a head, two pieces of 8 values each; a lane of
// the rotary part of a head split in halves holds both halves of its pairs (so no value moves
// between lanes), any other lane 16 values in a row.
//
// A stream of bytes: 668 MB take 147 us (4.5 TB/s, two thirds of the copy rate) for 32768 rows of 32 + 8 + 8
// heads of 128, at 56% of the issue slots.  What is missing is the chain of lookups ahead of a row's loads
// and the scattered stores of the codes (4 bytes a lane).  Three CTAs an SM (80 registers, of which 52 to 60 bytes
// spill): with four, or 16 warps, more spills or fewer loads are in flight (232 us).  Runs of rows a warp, their
// lookups side by side in its lanes, took 211 to 302 us for both kernels of the case instead of 200.
template <int D, bool INTER>
__global__ void __launch_bounds__(256, 3) rope_append_kernel(RopeAppendArgs a) {
    // Starts while the kernel ahead drains, and touches nothing before that one has finished.  It does
    // not let the next kernel start early: a decode grid may read its q before its own wait, and
    // q_out may be that q.
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int LPR = D / 16;
    constexpr int TEAMS = 32 / LPR;
    const int lane = threadIdx.x & 31;
    const int team = lane / LPR;
    const int tl = lane % LPR;
    const bool turned = tl < a.rot / 16;
    const bool split = turned && !INTER;
    const int half = a.rot / 2;
    const int o0 = split ? 8 * tl : 16 * tl;
    const int o1 = split ? half + 8 * tl : 16 * tl + 8;
    const int heads = a.Hq + 2 * a.Hkv;
    const int per = (heads + a.slices - 1) / a.slices;
    const long long tasks = static_cast<long long>(a.rows) * a.slices;
    const long long warps = static_cast<long long>(gridDim.x) * (blockDim.x / 32);
    for (long long task = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) / 32; task < tasks;
         task += warps) {
        const int row = static_cast<int>(task / a.slices);
        const int h0 = static_cast<int>(task - static_cast<long long>(row) * a.slices) * per;
        const int h1 = min(heads, h0 + per);
        const __half* qr = a.q + row * a.q_stride;
        const __half* kr = a.k + row * a.k_stride;
        const __half* vr = a.v + row * a.v_stride;
        auto load = [&](int h, uint4 (&r)[2]) {
            r[0] = r[1] = make_uint4(0, 0, 0, 0);
            if (h >= h1) return;
            const __half* src = h < a.Hq ? qr + h * D : h < a.Hq + a.Hkv ? kr + (h - a.Hq) * D : vr + (h - a.Hq - a.Hkv) * D;
            r[0] = __ldcs(reinterpret_cast<const uint4*>(src + o0));
            r[1] = __ldcs(reinterpret_cast<const uint4*>(src + o1));
        };
        // the first values are on their way while the row's place is looked up (a chain of dependent loads)
        uint4 raw[2], nxt[2];
        load(h0 + team, raw);
        const int b = warp_find_seq(a.cu_rows, a.B, row, lane);
        if (b < 0) continue;  // behind the last sequence
        const long long pos = static_cast<long long>(__ldg(a.start_pos + b)) + (row - __ldg(a.cu_rows + b));
        // the angles of the lane's pairs 8 tl .. 8 tl + 7
        float c[8], n[8];
        bool bad = false;
        if (a.axes == 1) {
            const long long p = a.positions != nullptr ? __ldg(a.positions + row) : pos;
            bad = p < 0 || p >= a.table_len;
            if (turned && !bad) {
                const float* t = a.table + p * a.rot + 8 * tl;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    reinterpret_cast<float4*>(c)[i] = __ldg(reinterpret_cast<const float4*>(t) + i);
                    reinterpret_cast<float4*>(n)[i] = __ldg(reinterpret_cast<const float4*>(t + half) + i);
                }
            }
        } else {
            int p[3] = {0, 0, 0};
#pragma unroll
            for (int x = 0; x < 3; ++x) {
                if (x < a.axes) p[x] = __ldg(a.positions + static_cast<long long>(x) * a.rows + row);
                bad |= p[x] < 0 || p[x] >= a.table_len;
            }
            auto axis_of = [&](int pair) { return pair < a.bound0 ? p[0] : pair < a.bound1 ? p[1] : p[2]; };
            const int at0 = axis_of(8 * tl);
            if (turned && !bad) {
                const float* t = a.table + static_cast<long long>(at0) * a.rot + 8 * tl;
                const bool one = (8 * tl < a.bound0) == (8 * tl + 7 < a.bound0) && (8 * tl < a.bound1) == (8 * tl + 7 < a.bound1);
                if (one) {  // the lane's pairs turn with one axis
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        reinterpret_cast<float4*>(c)[i] = __ldg(reinterpret_cast<const float4*>(t) + i);
                        reinterpret_cast<float4*>(n)[i] = __ldg(reinterpret_cast<const float4*>(t + half) + i);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float* ti = a.table + static_cast<long long>(axis_of(8 * tl + i)) * a.rot + 8 * tl + i;
                        c[i] = __ldg(ti);
                        n[i] = __ldg(ti + half);
                    }
                }
            }
        }
        if (bad) {  // no angle: nothing of the row is written
            if (lane == 0) raise_flag(a.status, KVQ_FLAG_BAD_POSITION);
            continue;
        }
        uint8_t* blk = nullptr;  // the row's page, its first kv head's block
        int slot = 0;
        if (h1 > a.Hq) {
            const long long pidx = pos >> a.lg_p;
            if (pos < 0 || pidx >= a.max_blocks) {
                if (lane == 0) raise_flag(a.status, KVQ_FLAG_BAD_POSITION);
            } else {
                const int page = __ldg(a.block_table + static_cast<long long>(b) * a.max_blocks + pidx);
                if (page < 0 || page >= a.num_pages) {
                    if (lane == 0) raise_flag(a.status, KVQ_FLAG_BAD_PAGE);
                } else {
                    blk = a.pool + static_cast<long long>(page) * a.Hkv * a.L.bytes;
                    slot = static_cast<int>(pos & ((1 << a.lg_p) - 1));
                }
            }
        }
#pragma unroll 1
        for (int hb = h0; hb < h1; hb += TEAMS) {  // (the warp's teams take heads hb .. hb + TEAMS - 1)
            const int h = hb + team;
            load(h + TEAMS, nxt);
            float x0[8], x1[8];
            halves_to_floats(raw[0], x0);
            halves_to_floats(raw[1], x1);
            if (turned && h < a.Hq + a.Hkv) {
                if (INTER) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        turn(x0[2 * i], x0[2 * i + 1], c[i], n[i]);
                        turn(x1[2 * i], x1[2 * i + 1], c[4 + i], n[4 + i]);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) turn(x0[i], x1[i], c[i], n[i]);
                }
                raw[0] = floats_to_halves(x0);
                raw[1] = floats_to_halves(x1);
            }
            if (h < min(a.Hq, h1)) {
                __half* dst = a.q_out + row * a.q_out_stride + h * D;
                *reinterpret_cast<uint4*>(dst + o0) = raw[0];
                *reinterpret_cast<uint4*>(dst + o1) = raw[1];
            }
            if (hb + TEAMS > a.Hq) {  // (the whole warp) some team holds a kv row
                halves_to_floats(raw[0], x0);
                halves_to_floats(raw[1], x1);
                const bool is_v = h >= a.Hq + a.Hkv;
                const int G = is_v ? a.L.Gv : a.L.Gk;
                // the group maxima of both pieces.  Where a group lies within one half of the rotary part its
                // pieces are one of each of G / 8 lanes; elsewhere both pieces of G / 16 lanes
                float m0 = amax8(x0), m1 = amax8(x1);
                const bool apart = split && G <= half;
                if (!apart) m0 = m1 = fmaxf(m0, m1);
                const int width = apart ? G / 8 : G / 16;
#pragma unroll
                for (int off = 1; off < LPR; off <<= 1) {
                    const float t0 = __shfl_xor_sync(0xffffffffu, m0, off);
                    const float t1 = __shfl_xor_sync(0xffffffffu, m1, off);
                    if (off < width) {
                        m0 = fmaxf(m0, t0);
                        m1 = fmaxf(m1, t1);
                    }
                }
                if (h >= a.Hq && h < h1 && blk != nullptr) {
                    const __half s0 = scale_of(m0 * kSeventh), s1 = scale_of(m1 * kSeventh);
                    uint8_t* dst = blk + static_cast<long long>(h - a.Hq - (is_v ? a.Hkv : 0)) * a.L.bytes;
                    uint8_t* codes = dst + (is_v ? a.L.v_codes : 0) + slot * (D / 2);
                    __half* scales = reinterpret_cast<__half*>(dst + (is_v ? a.L.v_scales : a.L.k_scales)) + slot * (D / G);
                    *reinterpret_cast<uint32_t*>(codes + o0 / 2) = quant_word8<true>(x0, __half2float(s0), m0);
                    *reinterpret_cast<uint32_t*>(codes + o1 / 2) = quant_word8<true>(x1, __half2float(s1), m1);
                    if ((o0 & (G - 1)) == 0) scales[o0 / G] = s0;
                    if ((o1 & (G - 1)) == 0) scales[o1 / G] = s1;
                }
                __syncwarp();
            }
            raw[0] = nxt[0];
            raw[1] = nxt[1];
        }
    }
}

// The way back: a warp takes a row (or a part of its heads), a lane 16 values of a head's K or V row
// at a time.  The same 32768 rows of 8 heads take 46 us: 35 MB read and 134 MB written (of which L2 keeps a
// part), at 61% of the issue slots.
template <bool F32>
__global__ void __launch_bounds__(256) dequantize_rows_kernel(DequantRowsArgs a) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int d = a.L.d, lpr = d / 16;
    const int jobs = 2 * a.Hkv * lpr;  // (kv head, K or V, piece)
    const int per = (jobs + a.slices - 1) / a.slices;
    const long long tasks = static_cast<long long>(a.rows) * a.slices;
    const long long warps = static_cast<long long>(gridDim.x) * (blockDim.x / 32);
    for (long long task = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) / 32; task < tasks;
         task += warps) {
        const int row = static_cast<int>(task / a.slices);
        const int j0 = static_cast<int>(task - static_cast<long long>(row) * a.slices) * per;
        const int b = warp_find_seq(a.cu_rows, a.B, row, lane);
        if (b < 0) continue;
        const long long pos = static_cast<long long>(__ldg(a.start_pos + b)) + (row - __ldg(a.cu_rows + b));
        const long long pidx = pos >> a.lg_p;
        const bool inside = pos >= 0 && pidx < a.max_blocks;  // else zero rows
        int page = 0;
        if (!inside) {
            if (lane == 0) raise_flag(a.status, KVQ_FLAG_BAD_POSITION);
        } else {
            page = __ldg(a.block_table + static_cast<long long>(b) * a.max_blocks + pidx);
            if (page < 0 || page >= a.num_pages) {
                if (lane == 0) raise_flag(a.status, KVQ_FLAG_BAD_PAGE);
                page = 0;
            }
        }
        const int slot = static_cast<int>(pos & ((1 << a.lg_p) - 1));
        const uint8_t* blk = a.pool + static_cast<long long>(page) * a.Hkv * a.L.bytes;
#pragma unroll 2
        for (int j = j0 + lane; j < min(jobs, j0 + per); j += 32) {
            const int piece = j % lpr;
            const int hv = j / lpr;  // K of every head, then V
            const bool is_v = hv >= a.Hkv;
            const int h = is_v ? hv - a.Hkv : hv;
            const int G = is_v ? a.L.Gv : a.L.Gk;
            uint2 w = make_uint2(0x88888888u, 0x88888888u);
            float s = 0.f;
            if (inside) {
                const uint8_t* src = blk + static_cast<long long>(h) * a.L.bytes;
                w = __ldg(reinterpret_cast<const uint2*>(src + (is_v ? a.L.v_codes : 0) + slot * (d / 2)) + piece);
                s = __half2float(reinterpret_cast<const __half*>(src + (is_v ? a.L.v_scales : a.L.k_scales))[slot * (d / G) +
                                                                                                     16 * piece / G]);
            }
            float v0[8], v1[8];
            codes_to_floats(w.x, s, v0);
            codes_to_floats(w.y, s, v1);
            const long long o = (static_cast<long long>(row) * a.Hkv + h) * d + 16 * piece;
            void* out = is_v ? a.out_v : a.out_k;
            if (F32) {
                float4* p = reinterpret_cast<float4*>(static_cast<float*>(out) + o);
                p[0] = make_float4(v0[0], v0[1], v0[2], v0[3]);
                p[1] = make_float4(v0[4], v0[5], v0[6], v0[7]);
                p[2] = make_float4(v1[0], v1[1], v1[2], v1[3]);
                p[3] = make_float4(v1[4], v1[5], v1[6], v1[7]);
            } else {
                uint4* p = reinterpret_cast<uint4*>(static_cast<__half*>(out) + o);
                p[0] = floats_to_halves(v0);
                p[1] = floats_to_halves(v1);
            }
        }
    }
}

}  // namespace

int rows_grid(long long tasks_per_slice, int most_slices, int warps_per_sm, int* slices) {
    int dev = 0, sms = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (sms < 1) sms = 1;
    const long long room = static_cast<long long>(sms) * warps_per_sm;
    *slices = static_cast<int>(std::max(1ll, std::min<long long>(most_slices, room / std::max(1ll, tasks_per_slice))));
    const long long warps = std::min(tasks_per_slice * *slices, room);
    return static_cast<int>((warps + 7) / 8);
}

cudaError_t launch_rows(const void* kernel, int blocks, int threads, void** args, cudaStream_t stream) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(blocks));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelExC(&cfg, kernel, args);
}

cudaError_t launch_rope_append(RopeAppendArgs a, cudaStream_t stream) {
    const int teams = 32 / (a.L.d / 16);
    const int blocks = rows_grid(a.rows, (a.Hq + 2 * a.Hkv + teams - 1) / teams, 24, &a.slices);
    const void* k = nullptr;
    switch (a.L.d) {
        case 64: k = a.inter ? (const void*)rope_append_kernel<64, true> : (const void*)rope_append_kernel<64, false>; break;
        case 128: k = a.inter ? (const void*)rope_append_kernel<128, true> : (const void*)rope_append_kernel<128, false>; break;
        case 256: k = a.inter ? (const void*)rope_append_kernel<256, true> : (const void*)rope_append_kernel<256, false>; break;
        default: return cudaErrorInvalidValue;
    }
    void* args[] = {&a};
    return launch_rows(k, blocks, 256, args, stream);
}

cudaError_t launch_dequantize_rows(DequantRowsArgs a, cudaStream_t stream) {
    const int jobs = 2 * a.Hkv * (a.L.d / 16);
    const int blocks = rows_grid(a.rows, (jobs + 31) / 32, 32, &a.slices);
    void* args[] = {&a};
    return launch_rows(a.out_fp32 ? (const void*)dequantize_rows_kernel<true> : (const void*)dequantize_rows_kernel<false>,
                       blocks, 256, args, stream);
}

}  // namespace kvq
