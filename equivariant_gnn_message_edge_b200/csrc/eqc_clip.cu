// The norm of many tensors together, and their scaling to a bound:
//   n = sqrt(sum over all tensors and elements of g^2)
//   k = min(1, max_norm / (n + eps))       g <- k g
// Bound by memory: every element read once for the norm, and read and written
// once for the scaling.  Squares are summed in fp64 (at the memory's rate an SM
// has some 6 fp32 elements a clock to add, a tenth of what its fp64 units do),
// so no gradient is so large or so small that its square leaves the range, and
// the order of the sums is fixed.  564 MB of bf16 with some fp32: norm 100 us
// (5.6 TB/s), norm and scaling 287 us (5.9 TB/s, a part of the reads from L2).
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "eqc_elem.cuh"
#include "eqc_layers.h"

namespace eqc {

void count_launch();

namespace {

constexpr int kThreads = 256;
constexpr int kChunkBytes = 32768;        // of a tensor, from 16-byte boundary to boundary
// CTAs an SM holds of each kernel at once: the chunks are dealt out to as many, in one wave.
constexpr int kNormPerSm = 6, kScalePerSm = 5;
constexpr int kMaxBlocks = 148 * kNormPerSm;

// The tensors of one launch, by value in the kernel's parameters.
template <int MAXT>
struct Table {
    const void* in[MAXT];
    void* out[MAXT];
    int64_t n[MAXT];
    int chunk0[MAXT + 1];     // first chunk of each tensor
    uint8_t type[MAXT];
    int count;
};

// The tensor of a chunk.
template <int MAXT>
__device__ __forceinline__ int tensor_of(const Table<MAXT>& t, int chunk) {
    int lo = 0, hi = t.count;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (t.chunk0[mid] <= chunk) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ double block_sum(double v, double* red) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) v += red[w];
    return v;
}

// Calls f(pack, first element, elements valid from, to) for this thread's
// 16-byte vectors of the chunk.  A chunk inside the tensor has all its loads in
// flight together; in one at an end, vectors that reach over it are filled
// element by element (zeros outside).
template <class T, class F>
__device__ __forceinline__ void over_chunk(const void* base, int64_t n, int chunk, F&& f) {
    constexpr int VE = 16 / sizeof(T);
    constexpr int kVecs = kChunkBytes / 16;
    const T* p = static_cast<const T*>(base);
    const int off = (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
    const T* origin = p - off;                 // 16-byte boundary at or before p
    const int64_t v0 = (int64_t)chunk * kVecs;
    if (v0 * VE >= off && (v0 + kVecs) * VE <= n + off) {
        Pack<T, VE> k[kVecs / kThreads];
#pragma unroll
        for (int j = 0; j < kVecs / kThreads; ++j) k[j].load_rw(origin + (v0 + threadIdx.x + j * kThreads) * VE);
#pragma unroll
        for (int j = 0; j < kVecs / kThreads; ++j) f(k[j], (v0 + threadIdx.x + j * kThreads) * VE - off, 0, VE);
        return;
    }
    const int64_t vecs = (n + off + VE - 1) / VE;
    for (int j = threadIdx.x; j < kVecs; j += kThreads) {
        const int64_t v = v0 + j;
        if (v >= vecs) break;
        const int64_t e0 = v * VE - off;       // first element of the vector
        Pack<T, VE> k;
        const int from = e0 < 0 ? (int)-e0 : 0, to = n - e0 < VE ? (int)(n - e0) : VE;
#pragma unroll
        for (int e = 0; e < VE; ++e) k.set(e, e >= from && e < to ? to_float(p[e0 + e]) : 0.f);
        f(k, e0, from, to);
    }
}

// The sum of squares of this thread's elements of a chunk.  fp32 elements go
// to fp64 one by one.  Of 16-bit ones, two squares are added in fp32 first (the
// squares have 22 bits at most, so that x^2 + y^2 is rounded once), which halves
// the conversions to fp64; where such sums may have left the range of fp32,
// above 2^100 or below 2^-80, the thread adds its elements again in fp64.
template <class T>
__device__ __forceinline__ double chunk_squares(const void* base, int64_t n, int chunk) {
    constexpr int VE = 16 / sizeof(T);
    const auto wide = [&] {
        double s[4] = {};        // four sums: an addition in fp64 waits for the last of its own only
        over_chunk<T>(base, n, chunk, [&](const Pack<T, VE>& k, int64_t, int, int) {
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const double v = (double)k.get(e);
                s[e & 3] += v * v;
            }
        });
        return (s[0] + s[1]) + (s[2] + s[3]);
    };
    if constexpr (sizeof(T) == 4) {
        return wide();
    } else {
        double s[4] = {};
        over_chunk<T>(base, n, chunk, [&](const Pack<T, VE>& k, int64_t, int, int) {
#pragma unroll
            for (int e = 0; e < VE / 2; ++e) {
                const float x = k.get(2 * e), y = k.get(2 * e + 1);
                s[e & 3] += (double)fmaf(x, x, y * y);
            }
        });
        const double v = (s[0] + s[1]) + (s[2] + s[3]);
        return v >= 0x1p-80 && v <= 0x1p100 ? v : wide();
    }
}

template <class T>
__device__ __forceinline__ void scale_chunk(const void* base, void* out_, int64_t n, int chunk, float k) {
    constexpr int VE = 16 / sizeof(T);
    T* out = static_cast<T*>(out_);
    const bool same = ((reinterpret_cast<uintptr_t>(base) ^ reinterpret_cast<uintptr_t>(out_)) & 15) == 0;
    over_chunk<T>(base, n, chunk, [&](const Pack<T, VE>& in, int64_t e0, int from, int to) {
        Pack<T, VE> o;
#pragma unroll
        for (int e = 0; e < VE; ++e) o.set(e, in.get(e) * k);
        if (same && from == 0 && to == VE) {
            o.store(out + e0);
        } else {
#pragma unroll
            for (int e = 0; e < VE; ++e)
                if (e >= from && e < to) out[e0 + e] = o.e[e];
        }
    });
}

// part[first + block] = sum of squares of the block's chunks.
template <int MAXT>
__global__ void __launch_bounds__(kThreads, kNormPerSm) clip_norm_kernel(const __grid_constant__ Table<MAXT> t, double* part) {
    let_next_start();
    __shared__ double red[kThreads / 32];
    double s = 0.0;
    for (int chunk = blockIdx.x; chunk < t.chunk0[t.count]; chunk += gridDim.x) {
        const int i = tensor_of(t, chunk), j = chunk - t.chunk0[i];
        s += t.type[i] == 0 ? chunk_squares<float>(t.in[i], t.n[i], j)
                            : (t.type[i] == 1 ? chunk_squares<__nv_bfloat16>(t.in[i], t.n[i], j)
                                              : chunk_squares<__half>(t.in[i], t.n[i], j));
    }
    s = block_sum(s, red);
    if (threadIdx.x == 0) part[blockIdx.x] = s;
}

__device__ __forceinline__ double total_norm(const double* part, int parts, double* red) {
    double s = 0.0;
    for (int i = threadIdx.x; i < parts; i += kThreads) s += part[i];
    return sqrt(block_sum(s, red));
}

__global__ void __launch_bounds__(kThreads) clip_total_kernel(const double* part, int parts, float* norm) {
    wait_for_last();
    __shared__ double red[kThreads / 32];
    const double n = total_norm(part, parts, red);
    if (threadIdx.x == 0) *norm = (float)n;
}

template <int MAXT>
__global__ void __launch_bounds__(kThreads, kScalePerSm) clip_scale_kernel(const __grid_constant__ Table<MAXT> t,
                                                              const double* part, int parts, float max_norm,
                                                              float eps, float* norm) {
    wait_for_last();
    let_next_start();
    __shared__ double red[kThreads / 32];
    const double n = total_norm(part, parts, red);
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = (float)n;
    const double ratio = (double)max_norm / (n + (double)eps);
    const float k = ratio < 1.0 ? (float)ratio : (ratio == ratio ? 1.f : (float)ratio);   // NaN stays NaN
    const int chunks = t.chunk0[t.count];
    // from the back: the chunks read last for the norm are still in L2
    for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
        const int chunk = chunks - 1 - c;
        const int i = tensor_of(t, chunk), j = chunk - t.chunk0[i];
        if (k == 1.f && t.in[i] == t.out[i]) continue;   // nothing to change in place
        if (t.type[i] == 0) scale_chunk<float>(t.in[i], t.out[i], t.n[i], j, k);
        else if (t.type[i] == 1) scale_chunk<__nv_bfloat16>(t.in[i], t.out[i], t.n[i], j, k);
        else scale_chunk<__half>(t.in[i], t.out[i], t.n[i], j, k);
    }
}

int64_t chunks_of(const eqconv_tensor_t& t) {
    const int64_t es = type_bytes(t.type);
    const int64_t bytes = t.n * es + (int64_t)(reinterpret_cast<uintptr_t>(t.in) & 15);
    return t.n > 0 ? (bytes + kChunkBytes - 1) / kChunkBytes : 0;
}

inline int blocks_for(int64_t chunks, int per_sm) { return (int)(chunks < 148 * per_sm ? chunks : 148 * per_sm); }

// Tensors [from, to) of one launch: at most MAXT that have elements, and 2^30
// chunks.  Empty tensors behind the last one belong to the same launch, so that
// every table but an empty list's has a tensor.
template <int MAXT>
int fill(Table<MAXT>& t, int n, const eqconv_tensor_t* ts, int from) {
    int64_t chunks = 0;
    int i = from;
    t.count = 0;
    t.chunk0[0] = 0;
    for (; i < n && t.count < MAXT; ++i) {
        const int64_t k = chunks_of(ts[i]);
        if (k == 0) continue;
        if (chunks + k > (int64_t(1) << 30)) break;
        chunks += k;
        t.in[t.count] = ts[i].in;
        t.out[t.count] = ts[i].out;
        t.n[t.count] = ts[i].n;
        t.type[t.count] = (uint8_t)ts[i].type;
        t.chunk0[++t.count] = (int)chunks;
    }
    while (i < n && chunks_of(ts[i]) == 0) ++i;
    return i;
}

// Lists of up to 96 tensors (the 2.8 KB of a few layers' gradients) launch with
// small parameters, longer ones with 30 KB, which take the host 5 us more a
// call.  Time of a call's two launches on the host, by list and limit:
//                    18 tensors   41 to 96     97 to 128
//   limit 40            5.1 us       9.9 us       9.8 us
//   limit 96            4.8 us       4.6 us       9.5 us
//   limit 128           5.7 us       5.4 us       5.5 us
constexpr int kFew = 96, kMany = 1024;

template <int MAXT>
cudaError_t run(int n, const eqconv_tensor_t* ts, bool scale, float max_norm, float eps, float* norm, double* part,
                cudaStream_t st) {
    Table<MAXT> t;
    int parts = 0, tables = 0;
    for (int from = 0; from < n;) {
        from = fill(t, n, ts, from);
        if (t.count == 0) continue;
        const int blocks = blocks_for(t.chunk0[t.count], kNormPerSm);
        clip_norm_kernel<MAXT><<<blocks, kThreads, 0, st>>>(t, part + parts);
        count_launch();
        parts += blocks;
        ++tables;
    }
    if (!scale || tables == 0) {
        const cudaError_t err = launch_after(clip_total_kernel, 1, kThreads, st, part, parts, norm);
        count_launch();
        return err == cudaSuccess ? cudaGetLastError() : err;
    }
    bool first = true;
    for (int from = 0; from < n;) {
        if (tables > 1) from = fill(t, n, ts, from);
        else from = n;
        if (t.count == 0) continue;
        const cudaError_t err = launch_after(clip_scale_kernel<MAXT>, blocks_for(t.chunk0[t.count], kScalePerSm), kThreads,
                                             st, t, part, parts, max_norm, eps, first ? norm : nullptr);
        count_launch();
        if (err != cudaSuccess) return err;
        first = false;
    }
    return cudaGetLastError();
}

}  // namespace

size_t clip_workspace(int n, const eqconv_tensor_t* ts) {
    // an upper bound for any split into launches
    size_t parts = 1;
    int64_t chunks = 0;
    for (int i = 0; i < n; ++i) chunks += chunks_of(ts[i]);
    const int64_t launches = n / kMany + 1 + (chunks >> 29);
    const int64_t most = launches * kMaxBlocks;
    parts += (size_t)(chunks < most ? chunks : most);
    return parts * sizeof(double);
}

cudaError_t clip_gradients(int n, const eqconv_tensor_t* ts, bool scale, float max_norm, float eps, float* norm,
                           void* ws, cudaStream_t st) {
    double* part = static_cast<double*>(ws);
    if (n <= kFew) return run<kFew>(n, ts, scale, max_norm, eps, norm, part, st);
    return run<kMany>(n, ts, scale, max_norm, eps, norm, part, st);
}

}  // namespace eqc
