// decode_wt_d256.cu -- attention-with-weights kernel instances for head_dim 256.
#include "decode_impl.cuh"

#define KVQ_WT_D256_CASES(CALL)                    \
    KVQ_DECODE_CASES_1H(256, 64, 32, false, CALL)  \
    KVQ_DECODE_CASES_1H(256, 64, 64, false, CALL)  \
    KVQ_DECODE_CASES_1H(256, 64, 128, false, CALL) \
    KVQ_DECODE_CASES_1H(256, 128, 32, false, CALL) \
    KVQ_DECODE_CASES_1H(256, 128, 64, false, CALL) \
    KVQ_DECODE_CASES_1H(256, 128, 128, false, CALL)
KVQ_DECODE_TU_OF(KVQ_WT_D256_CASES, KVQ_WEIGHTS_RUN, KVQ_WEIGHTS_OCC, decode_run_wt_d256, decode_occupancy_wt_d256)
