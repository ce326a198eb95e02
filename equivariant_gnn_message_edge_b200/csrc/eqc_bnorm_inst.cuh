// Instances of the block norm for one element type: EQC_BN_TYPE, EQC_BN_NAME.
// p.first receives the CTAs of each degree.
#include "eqc_bnorm_staged.cuh"

namespace eqc {
namespace bn {

cudaError_t EQC_BN_NAME(BnParams& p, const Shape& s, bool bwd, cudaStream_t st) {
    using T = EQC_BN_TYPE;
    if (s.V) return bwd ? launch_for<T, true>(p, s, st) : launch_for<T, false>(p, s, st);
    const float rows[4] = {1.f, 3.f, 5.f, 7.f};
    split_ctas(p, kStreamCtas, rows);
    if (bwd) {
        // the kernel's limit is set once and for every C: threads that call at once must not lower each other's
        static bool done[64] = {};
        const cudaError_t e = allow_smem(bn_bwd_stream<T>, done);
        if (e != cudaSuccess) return e;
        const int smem = 2 * p.C * (int)sizeof(float);
        bn_bwd_stream<T><<<p.first[p.L + 1], 256, smem, st>>>(p);
    } else {
        bn_fwd_stream<T><<<p.first[p.L + 1], 256, 0, st>>>(p);
    }
    count_launch();
    return cudaGetLastError();
}

cudaError_t EQC_BN_STAGED(const StagedParams& s, const Staged& h, int grid, bool bwd, cudaStream_t st) {
    using T = EQC_BN_TYPE;
    if (h.apart) return bwd ? staged_for<T, true, true>(s, h, grid, st) : staged_for<T, false, true>(s, h, grid, st);
    return bwd ? staged_for<T, true, false>(s, h, grid, st) : staged_for<T, false, false>(s, h, grid, st);
}

}  // namespace bn
}  // namespace eqc
