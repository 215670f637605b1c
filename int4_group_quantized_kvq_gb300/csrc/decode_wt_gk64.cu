// decode_wt_gk64.cu -- attention-with-weights kernel instances for head_dim 128, K groups of 64.
#include "decode_impl.cuh"

#define KVQ_WT_GK64_CASES(CALL)                 \
    KVQ_WEIGHTS_CASES(128, 64, 32, false, CALL)  \
    KVQ_WEIGHTS_CASES(128, 64, 64, false, CALL)  \
    KVQ_WEIGHTS_CASES(128, 64, 128, false, CALL)
KVQ_DECODE_TU_OF(KVQ_WT_GK64_CASES, KVQ_WEIGHTS_RUN, KVQ_WEIGHTS_OCC, decode_run_wt_gk64, decode_occupancy_wt_gk64)
