// latent_attention.cu -- attention whose keys and values are one shared latent vector per token
// (absorbed form), over the packed latent cache.
#include <cuda_fp16.h>

#include <cmath>

#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "kvq_rows.cuh"

namespace kvq {
namespace {

// One warp per (row, query head): a lane holds L / 32 latent values and two of the rotary part.
template <int L>
__global__ void __launch_bounds__(256) latent_kernel(LatentAttnArgs a) {
    constexpr int E = L / 32, R = 64;
    uint32_t* status = reinterpret_cast<uint32_t*>(a.workspace);
    const int lane = threadIdx.x & 31;
    const long long tasks = static_cast<long long>(a.rows) * a.H;
    const long long warps = static_cast<long long>(gridDim.x) * 8;
    for (long long task = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) / 32; task < tasks; task += warps) {
        const int row = static_cast<int>(task / a.H);
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
        const __half* qr = a.q + task * (L + R);
        float q[E], o[E], qp[2];
        for (int i = 0; i < E; ++i) {
            q[i] = __half2float(qr[lane * E + i]) * a.softmax_scale;
            o[i] = 0.f;
        }
        for (int i = 0; i < 2; ++i) qp[i] = __half2float(qr[L + 2 * lane + i]) * a.softmax_scale;
        float m = -INFINITY, l = 0.f;
        for (int t = 0; t <= pos; ++t) {
            int page = a.block_table[static_cast<long long>(b) * a.max_blocks + (t >> a.lg_p)];
            if (page < 0 || page >= a.num_pages) {
                if (lane == 0) raise_flag(status, KVQ_FLAG_BAD_PAGE);
                page = 0;
            }
            const int slot = t & ((1 << a.lg_p) - 1);
            const uint8_t* blk = a.pool + static_cast<long long>(page) * a.lay.bytes;
            const float s = __half2float(reinterpret_cast<const __half*>(blk + a.lay.scales)[slot * (L / a.lay.G) + lane * E / a.lay.G]);
            const __half* rope = reinterpret_cast<const __half*>(blk + a.lay.rope) + slot * R;
            float z = qp[0] * __half2float(rope[2 * lane]) + qp[1] * __half2float(rope[2 * lane + 1]), v[E];
            for (int i = 0; i < E; ++i) {
                const int at = lane * E + i;
                v[i] = static_cast<float>(((blk[slot * (L / 2) + at / 2] >> (4 * (at & 1))) & 15) - 8) * s;
                z += q[i] * v[i];
            }
            for (int off = 16; off > 0; off >>= 1) z += __shfl_xor_sync(0xffffffffu, z, off);
            const float mn = fmaxf(m, z), al = expf(m - mn), p = expf(z - mn);
            l = l * al + p;
            for (int i = 0; i < E; ++i) o[i] = o[i] * al + p * v[i];
            m = mn;
        }
        for (int i = 0; i < E; ++i)
            a.out[task * L + lane * E + i] = __float2half_rn(pos < 0 ? 0.f : o[i] / l);
    }
}

}  // namespace

size_t latent_workspace_bytes(const LatentAttnArgs&) { return 256; }

cudaError_t launch_latent_attention(const LatentAttnArgs& a, cudaStream_t stream) {
    int slices;
    const int blocks = rows_grid(static_cast<long long>(a.rows) * a.H, 1, 32, &slices);
    if (a.lay.L == 256) latent_kernel<256><<<blocks, 256, 0, stream>>>(a);
    else latent_kernel<512><<<blocks, 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace kvq
