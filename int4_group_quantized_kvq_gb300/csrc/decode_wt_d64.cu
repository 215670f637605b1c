// decode_wt_d64.cu -- attention-with-weights kernel instances for head_dim 64 (INT4) and for the
// INT8 per-row cache (head_dim 128).
#include "decode_impl.cuh"

#define KVQ_WT_D64_CASES(CALL)                 \
    KVQ_WEIGHTS_CASES(64, 32, 32, false, CALL)  \
    KVQ_WEIGHTS_CASES(64, 32, 64, false, CALL)  \
    KVQ_WEIGHTS_CASES(64, 64, 32, false, CALL)  \
    KVQ_WEIGHTS_CASES(64, 64, 64, false, CALL)
KVQ_DECODE_TU_OF(KVQ_WT_D64_CASES, KVQ_WEIGHTS_RUN, KVQ_WEIGHTS_OCC, decode_run_wt_d64, decode_occupancy_wt_d64)

namespace kvq {

cudaError_t decode_run_wt_int8(const DecodeArgs& a, const DecodePlan& plan, cudaStream_t s) {
    if (plan.hk != 1 || a.L.d != 128 || a.window > 0) return cudaErrorInvalidValue;
    const bool p16 = a.L.P == 16;
    if (plan.hs == 1)
        return p16 ? decode::run<128, 128, 128, 1, 1, false, true, 1, 1>(a, plan, s)
                   : decode::run<128, 128, 128, 1, 1, false, false, 1, 1>(a, plan, s);
    return p16 ? decode::run<128, 128, 128, 1, 2, false, true, 1, 1>(a, plan, s)
               : decode::run<128, 128, 128, 1, 2, false, false, 1, 1>(a, plan, s);
}

int decode_occupancy_wt_int8(const DecodeArgs& a, const DecodePlan& plan, size_t smem) {
    if (plan.hk != 1 || a.L.d != 128 || a.window > 0) return 0;
    const bool p16 = a.L.P == 16;
    if (plan.hs == 1)
        return p16 ? decode::occupancy<128, 128, 128, 1, 1, false, true, 1, 1>(smem)
                   : decode::occupancy<128, 128, 128, 1, 1, false, false, 1, 1>(smem);
    return p16 ? decode::occupancy<128, 128, 128, 1, 2, false, true, 1, 1>(smem)
               : decode::occupancy<128, 128, 128, 1, 2, false, false, 1, 1>(smem);
}

}  // namespace kvq
