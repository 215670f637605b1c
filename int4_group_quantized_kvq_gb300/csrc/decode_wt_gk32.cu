// decode_wt_gk32.cu -- attention-with-weights kernel instances for head_dim 128, K groups of 32.
#include "decode_impl.cuh"

#define KVQ_WT_GK32_CASES(CALL)                 \
    KVQ_WEIGHTS_CASES(128, 32, 32, false, CALL)  \
    KVQ_WEIGHTS_CASES(128, 32, 64, false, CALL)  \
    KVQ_WEIGHTS_CASES(128, 32, 128, false, CALL)
KVQ_DECODE_TU_OF(KVQ_WT_GK32_CASES, KVQ_WEIGHTS_RUN, KVQ_WEIGHTS_OCC, decode_run_wt_gk32, decode_occupancy_wt_gk32)
