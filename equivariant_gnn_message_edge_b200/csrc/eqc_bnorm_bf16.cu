#define EQC_BN_TYPE __nv_bfloat16
#define EQC_BN_NAME run_bf16
#define EQC_BN_STAGED staged_bf16
#include "eqc_bnorm_inst.cuh"
