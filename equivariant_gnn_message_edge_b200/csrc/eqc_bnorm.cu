// Host side of the block norm: the shape of a launch, and the weight gradients'
// last sum (kernels in eqc_bnorm.cuh, instances in eqc_bnorm_<type>.cu).
#include "eqc_bnorm.cuh"

namespace eqc {
namespace bn {

cudaError_t run_f32(BnParams& p, const Shape& s, bool bwd, cudaStream_t st);
cudaError_t run_bf16(BnParams& p, const Shape& s, bool bwd, cudaStream_t st);
cudaError_t run_f16(BnParams& p, const Shape& s, bool bwd, cudaStream_t st);

namespace {

// dw[l, c]: the CTAs' partial rows in CTA order, 8 equal runs of them by the
// block's 8 warps and the warps' sums in order.
__global__ void __launch_bounds__(256) bn_dw_reduce(const BnParams p, float* dw_post, float* dw_pre) {
    __shared__ float s[8][32];
    const int x = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + x, l = blockIdx.y;
    float* dw = blockIdx.z ? dw_pre : dw_post;
    if (!dw) return;
    const int share = (p.first[l + 1] - p.first[l] + 7) / 8;
    const int t0 = p.first[l] + w * share, t1 = t0 + share < p.first[l + 1] ? t0 + share : p.first[l + 1];
    float v = 0.f;
    if (c < p.C)
#pragma unroll 8
        for (int t = t0; t < t1; ++t) v += p.part[((int64_t)t * 2 + blockIdx.z) * p.C + c];
    s[w][x] = v;
    __syncthreads();
    if (w != 0 || c >= p.C) return;
    for (int i = 1; i < 8; ++i) v += s[i][x];
    dw[l * p.C + c] = v;
}

BnParams params_of(const BlockNormArgs& a) {
    BnParams p{};
    p.N = a.N;
    p.C = a.C;
    p.L = a.L;
    p.gate_kind = a.gate_kind;
    p.eps = a.eps;
    p.scale = a.scale;
    p.x = a.x;
    p.b = a.b;
    p.gate = a.gate;
    p.w_post = a.w_post;
    p.w_pre = a.w_pre;
    p.x_out = a.x_out;
    p.h = a.h;
    p.stats = a.stats;
    p.g_x = a.g_x;
    p.g_h = a.g_h;
    p.dx = a.dx;
    p.db = a.db;
    p.dgate = a.dgate;
    p.part = a.part;
    return p;
}

// Channels a thread may move at once: 16 bytes, else 2, else 1, by C and the
// tensors' starts.
Shape shape_for(const BlockNormArgs& a) {
    const int es = type_bytes(a.type);
    uintptr_t all = 0;
    for (const void* q : {a.x, a.b, a.gate, (const void*)a.x_out, (const void*)a.h, a.g_x, a.g_h,
                          (const void*)a.dx, (const void*)a.db, (const void*)a.dgate})
        all |= reinterpret_cast<uintptr_t>(q);
    for (const int V : {16 / es, 2, 1})
        if (a.C % V == 0 && all % (V * es) == 0) return shape_of(a.L, a.C, V);
    return Shape{0, 0, 0, 0};
}

cudaError_t run(BnParams& p, const BlockNormArgs& a, bool bwd, cudaStream_t st) {
    const Shape s = shape_for(a);
    switch (a.type) {
        case EQCONV_F32: return run_f32(p, s, bwd, st);
        case EQCONV_BF16: return run_bf16(p, s, bwd, st);
        default: return run_f16(p, s, bwd, st);
    }
}

}  // namespace
}  // namespace bn

cudaError_t block_norm_forward(const BlockNormArgs& a, cudaStream_t st) {
    if (a.N == 0) return cudaSuccess;
    bn::BnParams p = bn::params_of(a);
    return bn::run(p, a, false, st);
}

size_t block_norm_workspace(int L, int C, int N) {
    // the most CTAs of any shape that C allows
    int most = bn::cta_cap(bn::Shape{0, 0, 0, 0});
    for (const int V : {8, 4, 2, 1}) {
        if (C % V) continue;
        const int k = bn::cta_cap(bn::shape_of(L, C, V));
        if (k > most) most = k;
    }
    int64_t ctas = (int64_t)bn::kSMs * most;
    if (ctas > (int64_t)N * (L + 1)) ctas = (int64_t)N * (L + 1);
    return (size_t)(ctas + L + 1) * 2 * C * sizeof(float);
}

cudaError_t block_norm_backward(const BlockNormArgs& a, cudaStream_t st) {
    cudaError_t err;
    const size_t wbytes = (size_t)(a.L + 1) * a.C * sizeof(float);
    if (a.N == 0) {
        if (a.dw_post && (err = cudaMemsetAsync(a.dw_post, 0, wbytes, st)) != cudaSuccess) return err;
        if (a.dw_pre && (err = cudaMemsetAsync(a.dw_pre, 0, wbytes, st)) != cudaSuccess) return err;
        return cudaSuccess;
    }
    bn::BnParams p = bn::params_of(a);
    if ((err = bn::run(p, a, true, st)) != cudaSuccess || (!a.dw_post && !a.dw_pre)) return err;
    bn::bn_dw_reduce<<<dim3((a.C + 31) / 32, a.L + 1, 2), 256, 0, st>>>(p, a.dw_post, a.dw_pre);
    count_launch();
    return cudaGetLastError();
}

}  // namespace eqc
