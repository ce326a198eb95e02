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
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "eqc_elem.cuh"
#include "eqc_layers.h"

namespace eqc {

void count_launch();

namespace bn {

constexpr int kSMs = 148;
constexpr int kStreamCtas = 4 * kSMs;

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
    int width;           // staged kernels: threads across the channels of a node (a power of two up to 32, or whole warps)
};

// 2^x and 1/x by the hardware's approximations (2 and 1 units in the last
// place of fp32); results below the normal range become 0.
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// a(g) and a'(g) of V gates (pairs), of one kind (EQCONV_GATE_*).  The error is
// a few units in the last place of fp32, and |g| more of them through the
// rounded argument of the power, in a' too: where a is close to 1, 1 - a is
// taken from the power and not from a.  For the sigmoid s = 1 / (1 + e) with
// e = exp(-g), 1 - s = e s (1 where s is 0 and e infinite: min(NaN, 1)).  tanh is
// (1 - q) / (1 + q) of q = exp(-2 |g|), 1 - tanh^2 is 4 q / (1 + q)^2, and near
// 0, where the first cancels, tanh is its Taylor series: for |g| < 0.25 up to a
// term below 2^-28 of the value.  16-bit gates take g itself below 2^-8, which
// leaves 2^-17 of the value there and above: 2^-6 of their own type's rounding
// or less, for a third fewer instructions in rows that these bound.
template <int V, bool SHORT = false>
__device__ __forceinline__ void gate_values(int kind, const F2 (&g)[V / 2], F2 (&a)[V / 2], F2 (&da)[V / 2]) {
    constexpr float kLog2e = 1.4426950408889634f;
    const F2 one(1.f), minus(-1.f);
    if (kind == 3) {
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            float x, y;
            g[i].split(x, y);
            const float qx = exp2_fast(-2.f * kLog2e * fabsf(x)), qy = exp2_fast(-2.f * kLog2e * fabsf(y));
            const F2 q(qx, qy);
            float nx, ny, dx, dy, sx, sy, fx, fy;
            fma2(q, minus, one).split(nx, ny);
            add2(q, one).split(dx, dy);
            dx = rcp_fast(dx);
            dy = rcp_fast(dy);
            fx = copysignf(nx * dx, x);
            fy = copysignf(ny * dy, y);
            if constexpr (SHORT) {
                a[i] = F2(fabsf(x) < 0x1p-8f ? x : fx, fabsf(y) < 0x1p-8f ? y : fy);
            } else {
                const F2 g2 = mul2(g[i], g[i]);
                F2 c = fma2(g2, F2(-1382.f / 155925.f), F2(62.f / 2835.f));
                c = fma2(g2, c, F2(-17.f / 315.f));
                c = fma2(g2, c, F2(2.f / 15.f));
                c = fma2(g2, c, F2(-1.f / 3.f));
                fma2(mul2(g[i], g2), c, g[i]).split(sx, sy);
                a[i] = F2(fabsf(x) < 0.25f ? sx : fx, fabsf(y) < 0.25f ? sy : fy);
            }
            const F2 d2(2.f * dx, 2.f * dy);
            da[i] = mul2(mul2(q, d2), d2);
        }
    } else {
        F2 s[V / 2], r[V / 2];      // the sigmoid, and 1 minus it
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            float x, y;
            g[i].split(x, y);
            const float ex = exp2_fast(-kLog2e * x), ey = exp2_fast(-kLog2e * y);
            const float sx = rcp_fast(1.f + ex), sy = rcp_fast(1.f + ey);
            s[i] = F2(sx, sy);
            r[i] = F2(fminf(ex * sx, 1.f), fminf(ey * sy, 1.f));
        }
        if (kind == 1) {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                a[i] = s[i];
                da[i] = mul2(s[i], r[i]);
            }
        } else {
            // s (1 + g (1 - s)): the error of 1 - s counts |g| times beside 1
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                a[i] = mul2(g[i], s[i]);
                da[i] = mul2(s[i], fma2(g[i], fma2(s[i], minus, one), one));
            }
        }
    }
}

template <int V>
__device__ __forceinline__ void gate_values(int kind, const float (&g)[V], float (&a)[V], float (&da)[V]) {
    constexpr int W = (V + 1) / 2 * 2;
    F2 gv[W / 2], av[W / 2], dv[W / 2];
#pragma unroll
    for (int i = 0; i < W / 2; ++i) gv[i] = F2(g[2 * i], 2 * i + 1 < V ? g[2 * i + 1] : 0.f);
    gate_values<W>(kind, gv, av, dv);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        float x, y;
        av[e / 2].split(x, y);
        a[e] = e & 1 ? y : x;
        dv[e / 2].split(x, y);
        da[e] = e & 1 ? y : x;
    }
}

__device__ __forceinline__ void gate_value(int kind, float g, float& a, float& da) {
    float gv[1] = {g}, av[1], dv[1];
    gate_values(kind, gv, av, dv);
    a = av[0];
    da = dv[0];
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

// Streaming, for groups that fit neither shared memory nor registers: one CTA
// walks nodes of one degree, three passes over a group's channels (the later
// ones hit L1 or L2), and is bound by their latency (3000 fp32 rows of 6001:
// forward 350 us, backward 525 us; 3000 lmax3 nodes of 509: backward 486 us).
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
    let_next_start();
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


// ---------------------------------------------------------------------------
// Resident kernels, for groups too large to be staged: a group's elements stay
// in registers between the sums.  A CTA owns a group of one degree; a thread
// owns V neighbouring channels, J times a CTA's width apart, in all K = 2l + 1
// rows, of NB nodes at a time.  Bound by memory: every tensor is moved once,
// all loads of a batch are in flight together.  The weights and the sums of
// their gradients stay in the thread that owns the channel for the whole
// persistent loop over nodes.  3000 lmax3 nodes of 512 fp32 channels: backward
// 198 us (3.2 TB/s), since loads, sums and stores of a group follow one another.

// Sums of NB values over the worker's threads; every thread gets them.
template <int NB>
struct WorkerSum {
    float* red;          // [2][NB][16], only for workers of several warps
    int width, flip;
    __device__ __forceinline__ void operator()(float (&v)[NB]) {
#pragma unroll
        for (int o = 16; o; o >>= 1)
            if (o < width)
#pragma unroll
                for (int i = 0; i < NB; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        if (width <= 32) return;
        float* r = red + flip * NB * 16;
        flip ^= 1;       // the next sum's buffer: one barrier a sum is enough
        if ((threadIdx.x & 31) == 0)
#pragma unroll
            for (int i = 0; i < NB; ++i) r[i * 16 + (threadIdx.x >> 5)] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int warps = width >> 5;
            float s = 0.f;
            for (int w = 0; w < warps; ++w) s += r[i * 16 + w];
            v[i] = s;
        }
    }
};

// Nodes at a time: more where a group is small, within the registers.
template <int V, int K, int J, bool BWD>
constexpr int batch_of() {
    return BWD ? (K * J == 1 && V < 8 ? 2 : 1) : K * J >= 4 ? 1 : (K * J >= 2 || V == 8) ? 2 : 4;
}

template <class T, int V, int K, int J>
__device__ __forceinline__ void fwd_groups(const BnParams& p, int l, float* red) {
    constexpr int NB = batch_of<V, K, J, false>();
    const int D = (p.L + 1) * (p.L + 1);
    const int x0 = threadIdx.x, width = blockDim.x;
    const bool post = p.b != nullptr, pre = p.w_pre != nullptr, gated = p.gate != nullptr;
    const float inv_m = 1.f / ((float)K * (float)p.C);
    const int64_t step = (int64_t)(p.first[l + 1] - p.first[l]) * NB;
    WorkerSum<NB> sum{red, width, 0};
    Pack<float, V> wo[J], wi[J];
    bool own[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int c = (x0 + j * width) * V;
        own[j] = c < p.C;
        if (own[j] && post)
#pragma unroll
            for (int e = 0; e < V; ++e) wo[j].e[e] = __ldg(p.w_post + l * p.C + c + e);
        if (own[j] && pre)
#pragma unroll
            for (int e = 0; e < V; ++e) wi[j].e[e] = __ldg(p.w_pre + l * p.C + c + e);
    }
    for (int64_t nw = (int64_t)(blockIdx.x - p.first[l]) * NB; nw < p.N; nw += step) {
        Pack<T, V> x[NB][K][J], b[NB][K][J], g[NB][J];
        const auto at = [&](int i, int m, int j) {
            return ((nw + i) * D + l * l + m) * p.C + (x0 + j * width) * V;
        };
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (!own[j] || nw + i >= p.N) continue;
#pragma unroll
                for (int m = 0; m < K; ++m) {
                    x[i][m][j].load(static_cast<const T*>(p.x) + at(i, m, j));
                    if (post) b[i][m][j].load(static_cast<const T*>(p.b) + at(i, m, j));
                }
                if (gated)
                    g[i][j].load(static_cast<const T*>(p.gate) + ((nw + i) * (p.L + 1) + l) * p.C + (x0 + j * width) * V);
            }
        float sb[NB], sy[NB];
#pragma unroll
        for (int i = 0; i < NB; ++i) sb[i] = sy[i] = 0.f;
        if (post) {
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int j = 0; j < J; ++j)
                    if (own[j] && nw + i < p.N)
#pragma unroll
                        for (int m = 0; m < K; ++m)
#pragma unroll
                            for (int e = 0; e < V; ++e) sb[i] += b[i][m][j].get(e) * b[i][m][j].get(e);
            sum(sb);
#pragma unroll
            for (int i = 0; i < NB; ++i) sb[i] = rsqrtf(sb[i] * inv_m + p.eps);
        }
        float k[NB][J][V];        // y = x + k b
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (!own[j] || nw + i >= p.N) continue;
                float a[V], da[V];
                if (gated) {
                    float gv[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) gv[e] = g[i][j].get(e);
                    gate_values(p.gate_kind, gv, a, da);
                }
#pragma unroll
                for (int e = 0; e < V; ++e)
                    k[i][j][e] = post ? p.scale * (gated ? a[e] : 1.f) * sb[i] * wo[j].e[e] : 0.f;
#pragma unroll
                for (int m = 0; m < K; ++m) {
                    Pack<T, V> o;
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        float y = x[i][m][j].get(e);
                        if (post) y += k[i][j][e] * b[i][m][j].get(e);
                        sy[i] += y * y;
                        o.set(e, y);
                    }
                    if (post) o.store(static_cast<T*>(p.x_out) + at(i, m, j));
                }
            }
        if (pre) {
            sum(sy);
#pragma unroll
            for (int i = 0; i < NB; ++i) {
                sy[i] = rsqrtf(sy[i] * inv_m + p.eps);
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    if (!own[j] || nw + i >= p.N) continue;
#pragma unroll
                    for (int m = 0; m < K; ++m) {
                        Pack<T, V> o;
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            float y = x[i][m][j].get(e);
                            if (post) y += k[i][j][e] * b[i][m][j].get(e);
                            o.set(e, y * sy[i] * wi[j].e[e]);
                        }
                        o.store(static_cast<T*>(p.h) + at(i, m, j));
                    }
                }
            }
        }
        if (p.stats && x0 == 0)
#pragma unroll
            for (int i = 0; i < NB; ++i)
                if (nw + i < p.N) {
                    if (post) p.stats[(nw + i) * (p.L + 1) + l] = sb[i];
                    if (pre) p.stats[((int64_t)p.N + nw + i) * (p.L + 1) + l] = sy[i];
                }
    }
}

template <class T, int V, int K, int J>
__device__ __forceinline__ void bwd_groups(const BnParams& p, int l, float* red) {
    constexpr int NB = batch_of<V, K, J, true>();
    const int D = (p.L + 1) * (p.L + 1);
    const int x0 = threadIdx.x, width = blockDim.x;
    const bool post = p.b != nullptr, pre = p.g_h != nullptr, gated = p.gate != nullptr, more = p.g_x != nullptr;
    const float inv_m = 1.f / ((float)K * (float)p.C);
    const int64_t step = (int64_t)(p.first[l + 1] - p.first[l]) * NB;
    WorkerSum<NB> sum{red, width, 0};
    Pack<float, V> wo[J], wi[J];
    float dwo[J][V], dwi[J][V];
    bool own[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int c = (x0 + j * width) * V;
        own[j] = c < p.C;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            dwo[j][e] = dwi[j][e] = 0.f;
            wo[j].e[e] = own[j] && post ? __ldg(p.w_post + l * p.C + c + e) : 0.f;
            wi[j].e[e] = own[j] && pre ? __ldg(p.w_pre + l * p.C + c + e) : 0.f;
        }
    }
    for (int64_t nw = (int64_t)(blockIdx.x - p.first[l]) * NB; nw < p.N; nw += step) {
        Pack<T, V> x[NB][K][J], b[NB][K][J], gx[NB][K][J], gh[NB][K][J], g[NB][J];
        float sb[NB], sy[NB];
        const auto at = [&](int i, int m, int j) {
            return ((nw + i) * D + l * l + m) * p.C + (x0 + j * width) * V;
        };
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            sb[i] = post && nw + i < p.N ? __ldg(p.stats + (nw + i) * (p.L + 1) + l) : 0.f;
            sy[i] = pre && nw + i < p.N ? __ldg(p.stats + ((int64_t)p.N + nw + i) * (p.L + 1) + l) : 0.f;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (!own[j] || nw + i >= p.N) continue;
#pragma unroll
                for (int m = 0; m < K; ++m) {
                    if (pre) x[i][m][j].load(static_cast<const T*>(p.x) + at(i, m, j));
                    if (post) b[i][m][j].load(static_cast<const T*>(p.b) + at(i, m, j));
                    if (more) gx[i][m][j].load(static_cast<const T*>(p.g_x) + at(i, m, j));
                    if (pre) gh[i][m][j].load(static_cast<const T*>(p.g_h) + at(i, m, j));
                }
                if (gated)
                    g[i][j].load(static_cast<const T*>(p.gate) + ((nw + i) * (p.L + 1) + l) * p.C + (x0 + j * width) * V);
            }
        }
        float sa[NB][J][V], da[NB][J][V];      // scale a(gate), scale a'(gate)
        float mpy[NB], mqb[NB];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            mpy[i] = mqb[i] = 0.f;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (!own[j] || nw + i >= p.N) continue;
                if (gated) {
                    float gv[V];
#pragma unroll
                    for (int e = 0; e < V; ++e) gv[e] = g[i][j].get(e);
                    gate_values(p.gate_kind, gv, sa[i][j], da[i][j]);
                }
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    sa[i][j][e] = gated ? p.scale * sa[i][j][e] : p.scale;
                    da[i][j][e] = gated ? p.scale * da[i][j][e] : 0.f;
                }
                if (pre)
#pragma unroll
                    for (int m = 0; m < K; ++m)
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            float y = x[i][m][j].get(e);
                            if (post) y += sa[i][j][e] * sb[i] * wo[j].e[e] * b[i][m][j].get(e);
                            mpy[i] += gh[i][m][j].get(e) * wi[j].e[e] * y;
                        }
            }
        }
        if (pre) {
            sum(mpy);
#pragma unroll
            for (int i = 0; i < NB; ++i) mpy[i] *= inv_m * sy[i] * sy[i];
        }
        // t, the gradient of x_out in all
        const auto grad = [&](int i, int m, int j, int e) {
            float t = more ? gx[i][m][j].get(e) : 0.f;
            if (pre) {
                float y = x[i][m][j].get(e);
                if (post) y += sa[i][j][e] * sb[i] * wo[j].e[e] * b[i][m][j].get(e);
                t += sy[i] * (gh[i][m][j].get(e) * wi[j].e[e] - y * mpy[i]);
            }
            return t;
        };
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (!own[j] || nw + i >= p.N) continue;
                float tb[V], gy[V];
#pragma unroll
                for (int e = 0; e < V; ++e) tb[e] = gy[e] = 0.f;
#pragma unroll
                for (int m = 0; m < K; ++m) {
                    Pack<T, V> o;
#pragma unroll
                    for (int e = 0; e < V; ++e) {
                        const float t = grad(i, m, j, e);
                        o.set(e, t);
                        if (post) tb[e] += t * b[i][m][j].get(e);
                        if (pre) {
                            float y = x[i][m][j].get(e);
                            if (post) y += sa[i][j][e] * sb[i] * wo[j].e[e] * b[i][m][j].get(e);
                            gy[e] += gh[i][m][j].get(e) * y;
                        }
                    }
                    o.store(static_cast<T*>(p.dx) + at(i, m, j));
                }
                Pack<T, V> o;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    mqb[i] += sa[i][j][e] * wo[j].e[e] * tb[e];
                    dwo[j][e] += sa[i][j][e] * sb[i] * tb[e];
                    dwi[j][e] += sy[i] * gy[e];
                    o.set(e, da[i][j][e] * sb[i] * wo[j].e[e] * tb[e]);
                }
                if (gated)
                    o.store(static_cast<T*>(p.dgate) + ((nw + i) * (p.L + 1) + l) * p.C + (x0 + j * width) * V);
            }
        if (!post) continue;
        sum(mqb);
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            mqb[i] *= inv_m * sb[i] * sb[i];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (!own[j] || nw + i >= p.N) continue;
#pragma unroll
                for (int m = 0; m < K; ++m) {
                    Pack<T, V> o;
#pragma unroll
                    for (int e = 0; e < V; ++e)
                        o.set(e, sb[i] * (sa[i][j][e] * wo[j].e[e] * grad(i, m, j, e) - b[i][m][j].get(e) * mqb[i]));
                    o.store(static_cast<T*>(p.db) + at(i, m, j));
                }
            }
        }
    }
    float* part = p.part + (int64_t)blockIdx.x * 2 * p.C;
#pragma unroll
    for (int j = 0; j < J; ++j)
        if (own[j])
#pragma unroll
            for (int e = 0; e < V; ++e) {
                part[(x0 + j * width) * V + e] = dwo[j][e];
                part[p.C + (x0 + j * width) * V + e] = dwi[j][e];
            }
}

// LMAX: the plan's L; J > 1 only for L = 0.  One CTA works on one degree.
template <class T, int V, int LMAX, int J>
__global__ void __launch_bounds__(LMAX == 0 ? 512 : 256) bn_fwd_kernel(const BnParams p) {
    __shared__ float red[2 * 4 * 16];
    const int l = degree_of(p, blockIdx.x);
    if (l == 0) return fwd_groups<T, V, 1, J>(p, 0, red);
    if constexpr (LMAX >= 1)
        if (l == 1) return fwd_groups<T, V, 3, 1>(p, 1, red);
    if constexpr (LMAX >= 2)
        if (l == 2) return fwd_groups<T, V, 5, 1>(p, 2, red);
    if constexpr (LMAX >= 3) return fwd_groups<T, V, 7, 1>(p, 3, red);
}

template <class T, int V, int LMAX, int J>
__global__ void __launch_bounds__(LMAX == 0 ? 512 : 256) bn_bwd_kernel(const BnParams p) {
    let_next_start();
    __shared__ float red[2 * 4 * 16];
    const int l = degree_of(p, blockIdx.x);
    if (l == 0) return bwd_groups<T, V, 1, J>(p, 0, red);
    if constexpr (LMAX >= 1)
        if (l == 1) return bwd_groups<T, V, 3, 1>(p, 1, red);
    if constexpr (LMAX >= 2)
        if (l == 2) return bwd_groups<T, V, 5, 1>(p, 2, red);
    if constexpr (LMAX >= 3) return bwd_groups<T, V, 7, 1>(p, 3, red);
}

// How a launch is cut: V channels a thread (0: the streaming kernels), J
// times, `threads` a CTA.
struct Shape {
    int V, J, threads;
};

// Groups that fit a CTA's registers: 16 bytes a thread and row in one piece,
// four for L = 0 (rows wider than the staged kernels take: up to 512 threads),
// and for the backward at L = 3 also 8 bytes (rows of no whole 16 bytes of which
// two nodes do not fit shared memory: 3000 nodes of 1020 bf16 channels 338 us,
// streaming 861 us).  pieces: bytes all rows start on.
inline Shape shape_of(int L, int C, int es, bool bwd, int pieces) {
    Shape s{16 / es, L == 0 ? 4 : 1, 0};
    if (pieces % 16 != 0 || C * es % 16 != 0) {
        if (!(L == 3 && bwd && pieces % 8 == 0 && C * es % 8 == 0)) return Shape{0, 0, 0};
        s.V = 8 / es;
    }
    const int across = (C / s.V + s.J - 1) / s.J;
    if (across > (L == 0 ? 512 : 256) || (L == 1 && es == 4)) return Shape{0, 0, 0};
    s.threads = (across + 31) / 32 * 32;
    return s;
}

// CTAs in proportion to the degrees' shares of the time, at least one each and
// no more than there are nodes.
inline void split_ctas(BnParams& p, int most, const float (&share)[4]) {
    float all = 0.f;
    for (int l = 0; l <= p.L; ++l) all += share[l];
    p.first[0] = 0;
    for (int l = 0; l <= p.L; ++l) {
        int64_t k = (int64_t)(most * share[l] / all);
        if (k > p.N) k = p.N;
        if (k < 1) k = 1;
        p.first[l + 1] = p.first[l] + (int)k;
    }
}

// Most CTAs an SM runs of a launch; partial sums are sized by it.
inline int cta_cap(const Shape& s) {
    if (!s.V) return kStreamCtas / kSMs;
    const int k = 1024 / s.threads;
    return k < 1 ? 1 : k > 8 ? 8 : k;
}

template <class T, int V, int LMAX, int J, bool BWD>
cudaError_t launch(BnParams& p, const Shape& s, cudaStream_t st) {
    void (*kernel)(BnParams) = nullptr;
    if constexpr (BWD) kernel = bn_bwd_kernel<T, V, LMAX, J>;
    else kernel = bn_fwd_kernel<T, V, LMAX, J>;
    static int regs = 0;                     // of this kernel, asked for once
    if (!regs) {
        cudaFuncAttributes a;
        const cudaError_t e = cudaFuncGetAttributes(&a, kernel);
        if (e != cudaSuccess) return e;
        regs = a.numRegs;
    }
    int resident = 65536 / (((regs + 7) / 8 * 8) * s.threads);
    resident = resident < 1 ? 1 : resident;
    const int cap = cta_cap(s);
    // a batch of nodes takes its rows' time and about that of six rows more, waiting for its loads and sums
    constexpr int n0 = batch_of<V, 1, J, BWD>(), n1 = batch_of<V, 3, 1, BWD>(), n2 = batch_of<V, 5, 1, BWD>();
    const float share[4] = {1.f + 6.f / n0, 3.f + 6.f / n1, 5.f + 6.f / n2, 7.f + 6.f};
    split_ctas(p, kSMs * (resident < cap ? resident : cap), share);
    kernel<<<p.first[p.L + 1], s.threads, 0, st>>>(p);
    count_launch();
    return cudaGetLastError();
}

template <class T, bool BWD>
cudaError_t launch_for(BnParams& p, const Shape& s, cudaStream_t st) {
    constexpr int W = 16 / sizeof(T);
    if (p.L == 0) return launch<T, W, 0, 4, BWD>(p, s, st);
    if constexpr (W == 8)
        if (p.L == 1) return launch<T, W, 1, 1, BWD>(p, s, st);
    if (p.L == 2) return launch<T, W, 2, 1, BWD>(p, s, st);
    if constexpr (BWD)
        if (s.V < W) return launch<T, W / 2, 3, 1, BWD>(p, s, st);
    return launch<T, W, 3, 1, BWD>(p, s, st);
}

}  // namespace bn
}  // namespace eqc
