// Test-only build of the block norm (bf16) whose waits for bulk copies cannot
// complete (not part of libeqconv; tests/test_gpu_layers_wait.py loads it).
//
// Every phase here expects 16 bytes more than its copies carry, so none ever
// completes, and the wait limit is cut to 2 ms.  The kernels must give up on
// their first wait, set status bit 4, wait (bounded) for the copies on their
// way and return: the same code as the library's, with only these two
// constants changed.
#define EQC_BULK_WAIT_LIMIT_NS 2000000ull
#define EQC_TEST_BULK_DEFICIT 16

#include "../eqc_bnorm.cu"
#include "../eqc_bnorm_bf16.cu"

namespace eqc {
void count_launch() {}
namespace bn {
cudaError_t run_f32(BnParams&, const Shape&, bool, cudaStream_t) { return cudaErrorNotSupported; }
cudaError_t run_f16(BnParams&, const Shape&, bool, cudaStream_t) { return cudaErrorNotSupported; }
cudaError_t staged_f32(const StagedParams&, const Staged&, int, bool, cudaStream_t) { return cudaErrorNotSupported; }
cudaError_t staged_f16(const StagedParams&, const Staged&, int, bool, cudaStream_t) { return cudaErrorNotSupported; }
}  // namespace bn
}  // namespace eqc

// p: x, b, gate, w_post, w_pre, x_out, h, stats, g_x, g_h, dx, db, dgate, dw_post, dw_pre, workspace, status
extern "C" __attribute__((visibility("default"))) int eqc_probe_block_norm(int N, int L, int C, int backward,
                                                                           void* const* p, void* stream) {
    eqc::BlockNormArgs a{};
    a.N = N;
    a.L = L;
    a.C = C;
    a.type = EQCONV_BF16;
    a.gate_kind = EQCONV_GATE_SIGMOID;
    a.eps = 1e-6f;
    a.scale = 1.f;
    a.x = p[0];
    a.b = p[1];
    a.gate = p[2];
    a.w_post = static_cast<const float*>(p[3]);
    a.w_pre = static_cast<const float*>(p[4]);
    a.x_out = p[5];
    a.h = p[6];
    a.stats = static_cast<float*>(p[7]);
    a.status = static_cast<unsigned*>(p[16]);
    if (!backward) return (int)eqc::block_norm_forward(a, static_cast<cudaStream_t>(stream));
    a.x_out = a.h = nullptr;
    a.g_x = p[8];
    a.g_h = p[9];
    a.dx = p[10];
    a.db = p[11];
    a.dgate = p[12];
    a.dw_post = static_cast<float*>(p[13]);
    a.dw_pre = static_cast<float*>(p[14]);
    a.part = static_cast<float*>(p[15]);
    return (int)eqc::block_norm_backward(a, static_cast<cudaStream_t>(stream));
}

// Whether the staged kernels take the case: `tensors` as large as x, of elements of `bytes`.
extern "C" __attribute__((visibility("default"))) int eqc_probe_block_norm_staged(int N, int L, int C, int bytes,
                                                                                  int tensors, int gated, int backward,
                                                                                  int aligned) {
    return eqc::bn::staged_shape(N, L, C, bytes, tensors, gated != 0, backward != 0, aligned != 0).slots;
}
