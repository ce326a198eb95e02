#define EQC_BN_TYPE float
#define EQC_BN_NAME run_f32
#define EQC_BN_STAGED staged_f32
#include "eqc_bnorm_inst.cuh"
