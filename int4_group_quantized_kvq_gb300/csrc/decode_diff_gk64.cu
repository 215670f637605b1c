// decode_diff_gk64.cu -- differential-attention kernel instances for head_dim 128, K groups of 64.
#include "decode_impl.cuh"

#define KVQ_DIFF_GK64_CASES(CALL)               \
    KVQ_DIFF_CASES(128, 64, 32, false, CALL)    \
    KVQ_DIFF_CASES(128, 64, 64, false, CALL)    \
    KVQ_DIFF_CASES(128, 64, 128, false, CALL)
KVQ_DECODE_TU_OF(KVQ_DIFF_GK64_CASES, KVQ_DIFF_RUN, KVQ_DIFF_OCC, decode_run_diff_gk64, decode_occupancy_diff_gk64)
