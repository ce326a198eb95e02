// Type embedding: rows of a table gathered and scaled, and the gradient of the
// table summed over the nodes of each type in node order.
#include <cuda_runtime.h>

#include <cstdint>

#include "eqc_elem.cuh"
#include "eqc_graph.h"
#include "eqc_layers.h"

namespace eqc {

void count_launch();

namespace {

inline int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

template <class ID>
__device__ __forceinline__ int64_t id_at(const void* ids, int64_t i) {
    return (int64_t)__ldg(reinterpret_cast<const ID*>(ids) + i);
}

// y[i, :] = scale * T[id_i, :].  Bound by memory: N C elements written and the
// rows read once (repeats of a row hit L2).  A block is LX lanes across the
// channels x 256 / LX rows; every thread keeps kRows rows in flight.
constexpr int kRows = 4;

template <class T, class O, int VE, class ID>
__global__ void __launch_bounds__(256) embed_fwd_kernel(const void* ids, int64_t N, int64_t V, int C, const T* table,
                                                        int64_t ldt, float scale, O* y, int64_t ldy, int lx_log2,
                                                        unsigned* status) {
    const int lx = 1 << lx_log2, x = threadIdx.x & (lx - 1), r = threadIdx.x >> lx_log2, ly = 256 >> lx_log2;
    const int64_t row0 = (int64_t)blockIdx.x * ly * kRows + r;
    int64_t id[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        const int64_t i = row0 + (int64_t)k * ly;
        id[k] = i < N ? id_at<ID>(ids, i) : -1;
        if (i < N && (uint64_t)id[k] >= (uint64_t)V) {
            id[k] = -1;
            if (x == 0) atomicOr(status, 1u);
        }
    }
    for (int c = (blockIdx.y * lx + x) * VE; c < C; c += gridDim.y * lx * VE) {
        Pack<T, VE> in[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k)
            if (id[k] >= 0) in[k].load(table + id[k] * ldt + c);
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const int64_t i = row0 + (int64_t)k * ly;
            if (i >= N) continue;
            Pack<O, VE> out;
#pragma unroll
            for (int e = 0; e < VE; ++e) out.set(e, id[k] >= 0 ? in[k].get(e) * scale : 0.f);
            out.store(y + i * ldy + c);
        }
    }
}

// int32 sort keys: the id, or V for ids that give no gradient.
template <class ID>
__global__ void embed_keys_kernel(const void* ids, int64_t N, int64_t V, int64_t padding, int* keys,
                                  unsigned* status) {
    const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= N) return;
    const int64_t id = id_at<ID>(ids, i);
    const bool ok = (uint64_t)id < (uint64_t)V;
    if (!ok) atomicOr(status, 1u);
    keys[i] = ok && id != padding ? (int)id : (int)V;
}

// dT[v, :] = scale * sum over the type's nodes, in node order.
template <class T, class O, int VE>
__global__ void embed_bwd_kernel(const int* ptr, const int* perm, int64_t V, int C, const O* gy, int64_t ldg,
                                 float scale, T* dtable) {
    const int c = (blockIdx.y * 32 + threadIdx.x) * VE;
    const int64_t v = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
    if (v >= V || c >= C) return;
    float acc[VE];
#pragma unroll
    for (int e = 0; e < VE; ++e) acc[e] = 0.f;
    for (int p = ptr[v]; p < ptr[v + 1]; ++p) {
        Pack<O, VE> in;
        in.load(gy + (int64_t)perm[p] * ldg + c);
#pragma unroll
        for (int e = 0; e < VE; ++e) acc[e] += in.get(e);
    }
    Pack<T, VE> out;
#pragma unroll
    for (int e = 0; e < VE; ++e) out.set(e, acc[e] * scale);
    out.store(dtable + v * C + c);
}

// Calls f with the largest of 8 (16-bit outputs), 4, 2 and 1 elements a vector
// such that every row of both tensors starts on the vector's boundary (16
// bytes at most) and C is whole vectors.
template <class T, class O, class F>
cudaError_t with_width(int C, const void* a, int64_t lda, const void* b, int64_t ldb, F&& f) {
    const auto ok = [&](int ve) {
        const auto fits = [&](const void* p, int64_t ld, size_t es) {
            const size_t piece = ve * es < 16 ? ve * es : 16;
            return reinterpret_cast<uintptr_t>(p) % piece == 0 && (size_t)ld * es % piece == 0;
        };
        return C % ve == 0 && fits(a, lda, sizeof(T)) && fits(b, ldb, sizeof(O));
    };
    constexpr int kWide = sizeof(O) == 2 ? 8 : 4;
    if (ok(kWide)) return f(std::integral_constant<int, kWide>{});
    if (ok(2)) return f(std::integral_constant<int, 2>{});
    return f(std::integral_constant<int, 1>{});
}

}  // namespace

cudaError_t embed_forward(const EmbedArgs& a, const void* table, int64_t table_stride, void* y, int64_t y_stride,
                          cudaStream_t st) {
    if (a.N == 0) return cudaSuccess;
    return with_type(a.in_type, [&](auto tv) {
        using T = decltype(tv);
        return with_type(a.out_type, [&](auto ov) {
            using O = decltype(ov);
            return with_width<T, O>(a.C, table, table_stride, y, y_stride, [&](auto wv) {
                constexpr int VE = decltype(wv)::value;
                const int vecs = a.C / VE;
                int lg = 0;
                while (lg < 8 && (1 << lg) < vecs) ++lg;
                const int ly = 256 >> lg;
                const dim3 grid(cdiv(a.N, (int64_t)ly * kRows), 1);
                if (a.id_bits == 32)
                    embed_fwd_kernel<T, O, VE, int32_t><<<grid, 256, 0, st>>>(
                        a.ids, a.N, a.V, a.C, static_cast<const T*>(table), table_stride, a.scale, static_cast<O*>(y),
                        y_stride, lg, a.status);
                else
                    embed_fwd_kernel<T, O, VE, int64_t><<<grid, 256, 0, st>>>(
                        a.ids, a.N, a.V, a.C, static_cast<const T*>(table), table_stride, a.scale, static_cast<O*>(y),
                        y_stride, lg, a.status);
                count_launch();
                return cudaGetLastError();
            });
        });
    });
}

namespace {
struct EmbedWs {
    size_t keys, ptr, perm, sort, total;
};
EmbedWs embed_layout(int64_t V, int64_t N) {
    const auto up = [](size_t b) { return (b + 255) & ~(size_t)255; };
    EmbedWs w{};
    size_t o = 0;
    w.keys = o; o += up(4 * (size_t)N);
    w.ptr = o;  o += up(4 * (size_t)(V + 2));
    w.perm = o; o += up(4 * (size_t)N);
    w.sort = o; o += csr_workspace_bytes((int)(V + 1), (int)N);
    w.total = o;
    return w;
}
}  // namespace

size_t embed_workspace(int64_t V, int, int64_t N) { return embed_layout(V, N).total; }

cudaError_t embed_backward(const EmbedArgs& a, const void* gy, int64_t gy_stride, void* dtable, void* ws,
                           cudaStream_t st) {
    const EmbedWs w = embed_layout(a.V, a.N);
    char* base = static_cast<char*>(ws);
    int* keys = reinterpret_cast<int*>(base + w.keys);
    int* ptr = reinterpret_cast<int*>(base + w.ptr);
    int* perm = reinterpret_cast<int*>(base + w.perm);
    if (a.N > 0) {
        if (a.id_bits == 32)
            embed_keys_kernel<int32_t><<<cdiv(a.N, 256), 256, 0, st>>>(a.ids, a.N, a.V, a.padding, keys, a.status);
        else
            embed_keys_kernel<int64_t><<<cdiv(a.N, 256), 256, 0, st>>>(a.ids, a.N, a.V, a.padding, keys, a.status);
        count_launch();
    }
    cudaError_t err = cudaGetLastError();
    if (err != cudaSuccess) return err;
    err = csr_build(keys, (int)(a.V + 1), (int)a.N, ptr, perm, base + w.sort, a.status, st);
    if (err != cudaSuccess) return err;
    return with_type(a.in_type, [&](auto tv) {
        using T = decltype(tv);
        return with_type(a.out_type, [&](auto ov) {
            using O = decltype(ov);
            return with_width<T, O>(a.C, dtable, a.C, gy, gy_stride, [&](auto wv) {
                constexpr int VE = decltype(wv)::value;
                const dim3 grid(cdiv(a.V, 8), cdiv(a.C, 32 * VE));
                embed_bwd_kernel<T, O, VE><<<grid, dim3(32, 8), 0, st>>>(ptr, perm, a.V, a.C,
                                                                        static_cast<const O*>(gy), gy_stride, a.scale,
                                                                        static_cast<T*>(dtable));
                count_launch();
                return cudaGetLastError();
            });
        });
    });
}

}  // namespace eqc
