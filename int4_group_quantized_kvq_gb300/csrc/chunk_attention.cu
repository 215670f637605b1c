// chunk_attention.cu -- causal attention of a ragged batch of query rows (prompts, parts of prompts,
// a few drafted tokens) over the packed INT4 cache.
#include <cuda_fp16.h>

#include <cmath>

#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "kvq_rows.cuh"

namespace kvq {
namespace {

// One warp per (row, query head): a lane holds D / 32 dimensions, a position's score is a shuffle
// reduction, the softmax runs online.
template <int D>
__global__ void __launch_bounds__(256) chunk_kernel(ChunkArgs a) {
    constexpr int E = D / 32;
    uint32_t* status = reinterpret_cast<uint32_t*>(a.workspace);
    const int lane = threadIdx.x & 31;
    const long long tasks = static_cast<long long>(a.rows) * a.Hq;
    const long long warps = static_cast<long long>(gridDim.x) * 8;
    for (long long task = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) / 32; task < tasks; task += warps) {
        const int row = static_cast<int>(task / a.Hq), hq = static_cast<int>(task % a.Hq), h = hq / (a.Hq / a.Hkv);
        const int b = warp_find_seq(a.cu_rows, a.B, row, lane);
        if (b < 0) continue;
        const int most = static_cast<int>(min(static_cast<long long>(a.max_len), static_cast<long long>(a.max_blocks) << a.lg_p));
        int len = a.seq_lens[b];
        if (len > most) {
            if (lane == 0) raise_flag(status, KVQ_FLAG_BAD_POSITION);
            len = most;
        }
        // (offsets that do not ascend must not lead behind the sequence)
        const int pos = min(max(len, 0) - 1, max(len, 0) - (a.cu_rows[b + 1] - a.cu_rows[b]) + (row - a.cu_rows[b]));
        float q[E], o[E];
        for (int i = 0; i < E; ++i) {
            q[i] = __half2float(a.q[task * D + lane * E + i]) * a.softmax_scale;
            o[i] = 0.f;
        }
        float m = -INFINITY, l = 0.f;
        for (int t = 0; t <= pos; ++t) {
            int page = a.block_table[static_cast<long long>(b) * a.max_blocks + (t >> a.lg_p)];
            if (page < 0 || page >= a.num_pages) {
                if (lane == 0) raise_flag(status, KVQ_FLAG_BAD_PAGE);
                page = 0;
            }
            const int slot = t & ((1 << a.lg_p) - 1);
            const uint8_t* blk = a.pool + (static_cast<long long>(page) * a.Hkv + h) * a.L.bytes;
            const float sk = __half2float(reinterpret_cast<const __half*>(blk + a.L.k_scales)[slot * (D / a.L.Gk) + lane * E / a.L.Gk]);
            const float sv = __half2float(reinterpret_cast<const __half*>(blk + a.L.v_scales)[slot * (D / a.L.Gv) + lane * E / a.L.Gv]);
            float z = 0.f, v[E];
            for (int i = 0; i < E; ++i) {
                const int at = lane * E + i, sh = 4 * (at & 1);
                z += q[i] * static_cast<float>(((blk[slot * (D / 2) + at / 2] >> sh) & 15) - 8) * sk;
                v[i] = static_cast<float>(((blk[a.L.v_codes + slot * (D / 2) + at / 2] >> sh) & 15) - 8) * sv;
            }
            for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
            const float mn = fmaxf(m, z), al = expf(m - mn), p = expf(z - mn);
            l = l * al + p;
            for (int i = 0; i < E; ++i) o[i] = o[i] * al + p * v[i];
            m = mn;
        }
        for (int i = 0; i < E; ++i)
            a.out[task * D + lane * E + i] = __float2half_rn(pos < 0 ? 0.f : o[i] / l);
    }
}

}  // namespace

size_t chunk_workspace_bytes(const ChunkArgs&) { return 256; }

cudaError_t launch_chunk_attention(const ChunkArgs& a, cudaStream_t stream) {
    int slices;
    const int blocks = rows_grid(static_cast<long long>(a.rows) * a.Hq, 1, 32, &slices);
    if (a.L.d == 64) chunk_kernel<64><<<blocks, 256, 0, stream>>>(a);
    else chunk_kernel<128><<<blocks, 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace kvq
