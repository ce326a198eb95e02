// Block norm: the root-mean-square norms before and after a layer, fused with
// the layer's gate, its residual scale and the residual sum.
//
// A node's rows of one degree l (2l + 1 rows of C channels, contiguous) are
// normalised on their own, so the work splits into groups (node, l) that share
// nothing but the weights w[l, :].  With M = (2l + 1) C, mean over the group:
//   s_b = rsqrt(mean b^2 + eps)            u = b s_b w_post
//   y   = x + scale a(gate) u  (= x_out)   s_y = rsqrt(mean y^2 + eps)   h = y s_y w_pre
// and backward, from g_x and g_h (gradients of x_out and h):
//   p = g_h w_pre     t = g_x + s_y (p - y s_y^2 mean(p y))      dx = t
//   q = scale a(gate) t w_post     db = s_b (q - b s_b^2 mean(q b))
//   dgate[c] = scale a'(gate) sum_m t u
//   dw_post[l, c] = sum over nodes, m of scale a(gate) t b s_b
//   dw_pre[l, c]  = sum over nodes, m of g_h y s_y
// y is made again from x, b and gate, so the backward reads no saved tensor
// but the two statistics of each group.
#include <cuda_runtime.h>

#include <cstdint>

#include "eqc_elem.cuh"
#include "eqc_layers.h"

namespace eqc {

void count_launch();

namespace {

constexpr int kSMs = 148;
constexpr int kMaxCtas = 4 * kSMs;   // persistent CTAs of one launch

struct BnParams {
    int N, C, L;
    int first[5];        // CTAs of degree l: [first[l], first[l + 1])
    int gate_kind;
    float eps, scale;
    const void *x, *b, *gate;
    const float *w_post, *w_pre;
    void *x_out, *h;
    float* stats;        // [2][N][L + 1]: s_b, then s_y
    const void *g_x, *g_h;
    void *dx, *db, *dgate;
    float* part;         // [CTAs][2][C]: dw_post, dw_pre
    bool want_post, want_pre;
};

// a(g) and a'(g) of the gate kinds (EQCONV_GATE_*).
__device__ __forceinline__ void gate_value(int kind, float g, float& a, float& da) {
    if (kind == 3) {
        a = tanhf(g);
        da = 1.f - a * a;
    } else {
        const float s = 1.f / (1.f + expf(-g));
        a = kind == 1 ? s : g * s;
        da = kind == 1 ? s * (1.f - s) : s * (1.f + g * (1.f - s));
    }
}

__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
    for (int w = 0; w < (int)blockDim.x / 32; ++w) v += red[w];
    return v;
}

// The degree and the first group of this CTA.
__device__ __forceinline__ int degree_of(const BnParams& p, int cta) {
    int l = 0;
    while (l < p.L && cta >= p.first[l + 1]) ++l;
    return l;
}

// Streaming forward: one CTA walks nodes of one degree, three passes over a
// group's channels (the later ones hit L1 or L2).
template <class T>
__global__ void __launch_bounds__(256) bn_fwd_stream(const BnParams p) {
    __shared__ float red[8];
    const int l = degree_of(p, blockIdx.x), K = 2 * l + 1, D = (p.L + 1) * (p.L + 1);
    const int step = p.first[l + 1] - p.first[l];
    const T* x_ = static_cast<const T*>(p.x);
    const T* b_ = static_cast<const T*>(p.b);
    const T* g_ = static_cast<const T*>(p.gate);
    const float inv_m = 1.f / ((float)K * (float)p.C);
    for (int n = blockIdx.x - p.first[l]; n < p.N; n += step) {
        const int64_t at = ((int64_t)n * D + l * l) * p.C, ga = ((int64_t)n * (p.L + 1) + l) * p.C;
        float sb = 0.f;
        if (b_) {
            float s = 0.f;
            for (int c = threadIdx.x; c < p.C; c += 256)
                for (int m = 0; m < K; ++m) {
                    const float v = to_float(b_[at + (int64_t)m * p.C + c]);
                    s += v * v;
                }
            sb = rsqrtf(block_sum(s, red) * inv_m + p.eps);
        }
        float s = 0.f;
        for (int pass = 0; pass < 2; ++pass) {
            if (pass == 1 && !p.w_pre) break;
            float sy = 0.f;
            if (pass == 1) sy = rsqrtf(block_sum(s, red) * inv_m + p.eps);
            for (int c = threadIdx.x; c < p.C; c += 256) {
                float a = 1.f, da;
                if (g_) gate_value(p.gate_kind, to_float(g_[ga + c]), a, da);
                const float k = b_ ? p.scale * a * sb * p.w_post[l * p.C + c] : 0.f;
                for (int m = 0; m < K; ++m) {
                    const int64_t i = at + (int64_t)m * p.C + c;
                    float y = to_float(x_[i]);
                    if (b_) y += k * to_float(b_[i]);
                    if (pass == 0) {
                        s += y * y;
                        if (p.x_out) static_cast<T*>(p.x_out)[i] = from_float<T>(y);
                    } else {
                        static_cast<T*>(p.h)[i] = from_float<T>(y * sy * p.w_pre[l * p.C + c]);
                    }
                }
            }
            if (pass == 1 && p.stats && threadIdx.x == 0)
                p.stats[((int64_t)p.N + n) * (p.L + 1) + l] = sy;
        }
        if (p.stats && b_ && threadIdx.x == 0) p.stats[(int64_t)n * (p.L + 1) + l] = sb;
    }
}

// Streaming backward: the weight gradients of the CTA's nodes are summed in
// shared memory, each channel by the thread that owns it.
template <class T>
__global__ void __launch_bounds__(256) bn_bwd_stream(const BnParams p) {
    extern __shared__ float acc[];   // [2][C]
    __shared__ float red[8];
    const int l = degree_of(p, blockIdx.x), K = 2 * l + 1, D = (p.L + 1) * (p.L + 1);
    const int step = p.first[l + 1] - p.first[l];
    const T* x_ = static_cast<const T*>(p.x);
    const T* b_ = static_cast<const T*>(p.b);
    const T* g_ = static_cast<const T*>(p.gate);
    const T* gx_ = static_cast<const T*>(p.g_x);
    const T* gh_ = static_cast<const T*>(p.g_h);
    const float inv_m = 1.f / ((float)K * (float)p.C);
    for (int c = threadIdx.x; c < 2 * p.C; c += 256) acc[c] = 0.f;
    __syncthreads();
    for (int n = blockIdx.x - p.first[l]; n < p.N; n += step) {
        const int64_t at = ((int64_t)n * D + l * l) * p.C, ga = ((int64_t)n * (p.L + 1) + l) * p.C;
        const float sb = b_ ? p.stats[(int64_t)n * (p.L + 1) + l] : 0.f;
        const float sy = gh_ ? p.stats[((int64_t)p.N + n) * (p.L + 1) + l] : 0.f;
        float mean_py = 0.f, mean_qb = 0.f;
        for (int pass = gh_ ? 0 : 1; pass < 3; ++pass) {
            if (pass == 2 && !b_) break;
            float s = 0.f;
            for (int c = threadIdx.x; c < p.C; c += 256) {
                float a = 1.f, da = 0.f;
                if (g_) gate_value(p.gate_kind, to_float(g_[ga + c]), a, da);
                const float wo = b_ ? p.w_post[l * p.C + c] : 0.f;
                const float wi = gh_ ? p.w_pre[l * p.C + c] : 0.f;
                const float k = p.scale * a * sb * wo;
                float tb = 0.f, gy = 0.f;
                for (int m = 0; m < K; ++m) {
                    const int64_t i = at + (int64_t)m * p.C + c;
                    const float b = b_ ? to_float(b_[i]) : 0.f;
                    float t = gx_ ? to_float(gx_[i]) : 0.f;
                    if (gh_) {
                        float y = to_float(x_[i]);
                        if (b_) y += k * b;
                        const float gh = to_float(gh_[i]), pp = gh * wi;
                        if (pass == 0) s += pp * y;
                        gy += gh * y;
                        t += sy * (pp - y * (sy * sy) * mean_py);
                    }
                    if (pass == 1) {
                        static_cast<T*>(p.dx)[i] = from_float<T>(t);
                        tb += t * b;
                        s += p.scale * a * t * wo * b;
                    } else if (pass == 2) {
                        const float q = p.scale * a * t * wo;
                        static_cast<T*>(p.db)[i] = from_float<T>(sb * (q - b * (sb * sb) * mean_qb));
                    }
                }
                if (pass == 1) {
                    if (g_) static_cast<T*>(p.dgate)[ga + c] = from_float<T>(p.scale * da * tb * sb * wo);
                    acc[c] += p.scale * a * tb * sb;
                    acc[p.C + c] += gy * sy;
                }
            }
            if (pass == 0) mean_py = block_sum(s, red) * inv_m;
            if (pass == 1 && b_) mean_qb = block_sum(s, red) * inv_m;
        }
    }
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * p.C; c += 256) p.part[(int64_t)blockIdx.x * 2 * p.C + c] = acc[c];
}

// dw[l, c]: the CTAs' partial sums added in CTA order.
__global__ void bn_dw_reduce(const BnParams p, float* dw_post, float* dw_pre) {
    const int c = blockIdx.x * blockDim.x + threadIdx.x, l = blockIdx.y;
    if (c >= p.C) return;
    for (int which = 0; which < 2; ++which) {
        float* dw = which ? dw_pre : dw_post;
        if (!dw) continue;
        float s = 0.f;
        for (int t = p.first[l]; t < p.first[l + 1]; ++t) s += p.part[((int64_t)t * 2 + which) * p.C + c];
        dw[l * p.C + c] = s;
    }
}

// CTAs in proportion to the degrees' rows, at least one each.
void split_ctas(BnParams& p, int64_t most) {
    const int D = (p.L + 1) * (p.L + 1);
    p.first[0] = 0;
    for (int l = 0; l <= p.L; ++l) {
        int64_t k = most * (2 * l + 1) / D;
        if (k > p.N) k = p.N;
        if (k < 1) k = 1;
        p.first[l + 1] = p.first[l] + (int)k;
    }
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
    split_ctas(p, kMaxCtas);
    return p;
}

}  // namespace

cudaError_t block_norm_forward(const BlockNormArgs& a, cudaStream_t st) {
    if (a.N == 0) return cudaSuccess;
    const BnParams p = params_of(a);
    return with_type(a.type, [&](auto tv) {
        using T = decltype(tv);
        bn_fwd_stream<T><<<p.first[p.L + 1], 256, 0, st>>>(p);
        count_launch();
        return cudaGetLastError();
    });
}

size_t block_norm_workspace(int L, int C, int N) {
    BnParams p{};
    p.N = N;
    p.C = C;
    p.L = L;
    split_ctas(p, kMaxCtas);
    return (size_t)p.first[L + 1] * 2 * C * sizeof(float);
}

cudaError_t block_norm_backward(const BlockNormArgs& a, cudaStream_t st) {
    cudaError_t err;
    const size_t wbytes = (size_t)(a.L + 1) * a.C * sizeof(float);
    if (a.N == 0) {
        if (a.dw_post && (err = cudaMemsetAsync(a.dw_post, 0, wbytes, st)) != cudaSuccess) return err;
        if (a.dw_pre && (err = cudaMemsetAsync(a.dw_pre, 0, wbytes, st)) != cudaSuccess) return err;
        return cudaSuccess;
    }
    const BnParams p = params_of(a);
    const int smem = 2 * a.C * (int)sizeof(float);
    err = with_type(a.type, [&](auto tv) {
        using T = decltype(tv);
        if (smem > 48 * 1024) {
            const cudaError_t e =
                cudaFuncSetAttribute(bn_bwd_stream<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
        }
        bn_bwd_stream<T><<<p.first[p.L + 1], 256, smem, st>>>(p);
        count_launch();
        return cudaGetLastError();
    });
    if (err != cudaSuccess || (!a.dw_post && !a.dw_pre)) return err;
    bn_dw_reduce<<<dim3((a.C + 127) / 128, a.L + 1), 128, 0, st>>>(p, a.dw_post, a.dw_pre);
    count_launch();
    return cudaGetLastError();
}

}  // namespace eqc
