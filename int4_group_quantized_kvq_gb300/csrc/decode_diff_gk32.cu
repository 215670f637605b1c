// decode_diff_gk32.cu -- differential-attention kernel instances for K groups of 32: head_dim 128 and 64.
#include "decode_impl.cuh"

#define KVQ_DIFF_GK32_CASES(CALL)               \
    KVQ_DIFF_CASES(128, 32, 32, false, CALL)    \
    KVQ_DIFF_CASES(128, 32, 64, false, CALL)    \
    KVQ_DIFF_CASES(128, 32, 128, false, CALL)
KVQ_DECODE_TU_OF(KVQ_DIFF_GK32_CASES, KVQ_DIFF_RUN, KVQ_DIFF_OCC, decode_run_diff_gk32, decode_occupancy_diff_gk32)

#define KVQ_DIFF_D64_CASES(CALL)                \
    KVQ_DIFF_CASES(64, 32, 32, false, CALL)     \
    KVQ_DIFF_CASES(64, 32, 64, false, CALL)
KVQ_DECODE_TU_OF(KVQ_DIFF_D64_CASES, KVQ_DIFF_RUN, KVQ_DIFF_OCC, decode_run_diff_d64, decode_occupancy_diff_d64)
