// decode_diff_d256.cu -- differential-attention kernel instances for head_dim 256 (up to 2 query
// heads per kv head: four virtual ones).
#include "decode_impl.cuh"

#define KVQ_DIFF_D256_CASES(CALL)                  \
    KVQ_DIFF_CASES_4(256, 64, 32, false, CALL)  \
    KVQ_DIFF_CASES_4(256, 64, 64, false, CALL)  \
    KVQ_DIFF_CASES_4(256, 64, 128, false, CALL) \
    KVQ_DIFF_CASES_4(256, 128, 32, false, CALL) \
    KVQ_DIFF_CASES_4(256, 128, 64, false, CALL) \
    KVQ_DIFF_CASES_4(256, 128, 128, false, CALL)
KVQ_DECODE_TU_OF(KVQ_DIFF_D256_CASES, KVQ_DIFF_RUN, KVQ_DIFF_OCC, decode_run_diff_d256, decode_occupancy_diff_d256)
