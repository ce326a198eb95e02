#define EQC_BN_TYPE __half
#define EQC_BN_NAME run_f16
#define EQC_BN_STAGED staged_f16
#include "eqc_bnorm_inst.cuh"
