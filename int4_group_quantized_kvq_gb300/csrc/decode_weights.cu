// decode_weights.cu -- accumulation of the attention weight each cached position received.
//
// With z the score of a position in log2 units, M and 1/L the row's maximum and reciprocal
// sum from the combine, the position's softmax weight for a query head is 2^(z - M) / L, and
//     weights[b][h][t] = decay * weights[b][h][t] + sum over the r query heads of kv head h.
// The scores lie as [b][h][t][query head], so a position's r scores are adjacent and a warp
// reads whole lines.  The sum runs over the query heads in order: results do not depend on
// timing.  Bound by latency and by the L2: the scores were written by the decode grid just
// ahead and are mostly still in the L2 cache.
#include <algorithm>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

struct WeightsParams {
    const float* scores;
    const float2* stat;
    const int32_t* seq_lens;
    float* weights;
    int32_t score_ld, weights_ld, max_pos, Hkv, r;  // max_pos: positions of the block table
    float decay;
};

constexpr int kThreads = 256;
constexpr int kPerThread = 4;  // positions per thread, kThreads apart

__global__ void __launch_bounds__(kThreads) accumulate_weights_kernel(WeightsParams p) {
    asm volatile("griddepcontrol.launch_dependents;");
    const int h = blockIdx.y, b = blockIdx.z;
    int L = p.seq_lens[b];
    L = min(min(L, p.score_ld), p.max_pos);
    const long long head = static_cast<long long>(b) * p.Hkv + h;
    const int t0 = blockIdx.x * (kThreads * kPerThread) + threadIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    float sum[kPerThread];
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) sum[k] = 0.f;
    const float* z = p.scores + (head * p.score_ld + t0) * p.r;
    for (int g = 0; g < p.r; ++g) {
        const float2 st = __ldcg(p.stat + head * p.r + g);
#pragma unroll
        for (int k = 0; k < kPerThread; ++k)
            if (t0 + k * kThreads < L)
                sum[k] = fmaf(fast_exp2(__ldcg(z + static_cast<long long>(k) * kThreads * p.r + g) - st.x), st.y, sum[k]);
    }
    float* w = p.weights + head * p.weights_ld + t0;
#pragma unroll
    for (int k = 0; k < kPerThread; ++k)
        if (t0 + k * kThreads < L) w[k * kThreads] = p.decay == 0.f ? sum[k] : fmaf(p.decay, w[k * kThreads], sum[k]);
}

}  // namespace

cudaError_t launch_accumulate_weights(const DecodeArgs& a, const DecodePlan& plan, cudaStream_t stream) {
    if (a.max_len <= 0) return cudaSuccess;
    WeightsParams p;
    p.scores = reinterpret_cast<const float*>(a.workspace + plan.ws_score_offset);
    p.stat = reinterpret_cast<const float2*>(a.workspace + plan.ws_stat_offset);
    p.seq_lens = a.seq_lens;
    p.weights = a.weights;
    p.score_ld = a.max_len;
    p.weights_ld = a.weights_ld;
    p.max_pos = static_cast<int32_t>(std::min<long long>(static_cast<long long>(a.max_blocks) * a.L.P, 0x7fffffff));
    p.Hkv = a.Hkv;
    p.r = a.Hq / a.Hkv;
    p.decay = a.decay;
    // launched while the combine runs; the kernel waits for it before it reads anything the
    // decode kernels write
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    const int per = kThreads * kPerThread;
    cfg.gridDim = dim3(static_cast<unsigned>((a.max_len + per - 1) / per), static_cast<unsigned>(a.Hkv),
                       static_cast<unsigned>(a.B));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t err = cudaLaunchKernelEx(&cfg, accumulate_weights_kernel, p);
    return err != cudaSuccess ? err : cudaGetLastError();
}

}  // namespace kvq
