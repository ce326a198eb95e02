// Host entry points of the node-level operators (contracts in include/eqconv.h).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "eqconv.h"

namespace eqc {

struct EmbedArgs {
    int64_t V, padding;
    int C, in_type, out_type, id_bits;
    int64_t N;
    const void* ids;
    float scale;
    unsigned* status;
};
cudaError_t embed_forward(const EmbedArgs& a, const void* table, int64_t table_stride, void* y, int64_t y_stride,
                          cudaStream_t st);
size_t embed_workspace(int64_t V, int C, int64_t N);
cudaError_t embed_backward(const EmbedArgs& a, const void* gy, int64_t gy_stride, void* dtable, void* ws,
                           cudaStream_t st);

struct BlockNormArgs {
    int N, L, C, type, gate_kind;
    float eps, scale;
    const void *x, *b, *gate;
    const float *w_post, *w_pre;
    void *x_out, *h;
    float* stats;
    // backward only
    const void *g_x, *g_h;
    void *dx, *db, *dgate;
    float *dw_post, *dw_pre;
    float* part;
    unsigned* status;
};
cudaError_t block_norm_forward(const BlockNormArgs& a, cudaStream_t st);
size_t block_norm_workspace(int L, int C, int N);
cudaError_t block_norm_backward(const BlockNormArgs& a, cudaStream_t st);

size_t clip_workspace(int n, const eqconv_tensor_t* t);
// scale false: the norm alone
cudaError_t clip_gradients(int n, const eqconv_tensor_t* t, bool scale, float max_norm, float eps, float* norm,
                           void* ws, cudaStream_t st);

}  // namespace eqc
