// Element types of the node-level operators (embedding, block norm, gradient
// clipping): fp32, bf16 and fp16 tensors read and written as vectors of VE
// elements; all arithmetic is fp32 or wider, with one rounding at the store.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstring>
#include <type_traits>

namespace eqc {

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }

template <class T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ float from_float<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float<__half>(float v) { return __float2half_rn(v); }

// The bits of VE elements, moved in pieces of at most 16 bytes.
template <class T, int VE>
struct Pack {
    static constexpr int kBytes = VE * (int)sizeof(T);
    static constexpr int kPiece = kBytes < 16 ? kBytes : 16;
    static_assert(kBytes % kPiece == 0, "whole pieces");
    union {
        T e[VE];
        uint4 q[(kBytes + 15) / 16];
        uint2 d;
        uint32_t w;
        uint16_t s;
    };
    __device__ __forceinline__ Pack() {}
    // p is aligned to kPiece bytes
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (kPiece == 16) {
#pragma unroll
            for (int i = 0; i < kBytes / 16; ++i) q[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
        } else if constexpr (kPiece == 8) {
            d = __ldg(reinterpret_cast<const uint2*>(p));
        } else if constexpr (kPiece == 4) {
            w = __ldg(reinterpret_cast<const uint32_t*>(p));
        } else {
            s = __ldg(reinterpret_cast<const uint16_t*>(p));
        }
    }
    // as load, for memory that the same kernel also writes, or that the kernel
    // before it writes while this one already waits (launch_after)
    __device__ __forceinline__ void load_rw(const T* p) {
        if constexpr (kPiece == 16) {
#pragma unroll
            for (int i = 0; i < kBytes / 16; ++i) q[i] = reinterpret_cast<const uint4*>(p)[i];
        } else if constexpr (kPiece == 8) {
            d = *reinterpret_cast<const uint2*>(p);
        } else if constexpr (kPiece == 4) {
            w = *reinterpret_cast<const uint32_t*>(p);
        } else {
            s = *reinterpret_cast<const uint16_t*>(p);
        }
    }
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (kPiece == 16) {
#pragma unroll
            for (int i = 0; i < kBytes / 16; ++i) reinterpret_cast<uint4*>(p)[i] = q[i];
        } else if constexpr (kPiece == 8) {
            *reinterpret_cast<uint2*>(p) = d;
        } else if constexpr (kPiece == 4) {
            *reinterpret_cast<uint32_t*>(p) = w;
        } else {
            *reinterpret_cast<uint16_t*>(p) = s;
        }
    }
    __device__ __forceinline__ float get(int i) const { return to_float(e[i]); }
    __device__ __forceinline__ void set(int i, float v) { e[i] = from_float<T>(v); }
};

// Two fp32 values in a 64-bit register pair: one instruction per pair for
// products and sums, each half rounded as fp32.
struct F2 {
    unsigned long long v;
    __device__ __forceinline__ F2() {}
    __device__ __forceinline__ F2(float x, float y) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y)); }
    __device__ __forceinline__ explicit F2(float x) : F2(x, x) {}
    __device__ __forceinline__ void split(float& x, float& y) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
    __device__ __forceinline__ float sum() const {
        float x, y;
        split(x, y);
        return x + y;
    }
};
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return d;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}

// V elements of shared memory as pairs (p on the vector's boundary, 16 bytes at most), and pairs to memory.
template <class T, int V>
__device__ __forceinline__ void load2(F2 (&v)[V / 2], const T* p) {
    constexpr int kWords = V * (int)sizeof(T) / 4;
    uint32_t w[kWords];
    if constexpr (kWords % 4 == 0) {
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
            const uint4 q = reinterpret_cast<const uint4*>(p)[i];
            w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
        }
    } else {
        static_assert(kWords == 2, "8 bytes");
        const uint2 q = *reinterpret_cast<const uint2*>(p);
        w[0] = q.x, w[1] = q.y;
    }
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        if constexpr (sizeof(T) == 4) {
            v[i] = F2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
        } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
            v[i] = F2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
        } else {
            __half2 h;
            memcpy(&h, &w[i], 4);
            const float2 f = __half22float2(h);
            v[i] = F2(f.x, f.y);
        }
    }
}
template <class T, int V>
__device__ __forceinline__ void store2(T* p, const F2 (&v)[V / 2]) {
    constexpr int kWords = V * (int)sizeof(T) / 4;
    uint32_t w[kWords];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        float x, y;
        v[i].split(x, y);
        if constexpr (sizeof(T) == 4) {
            w[2 * i] = __float_as_uint(x), w[2 * i + 1] = __float_as_uint(y);
        } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(x, y);
            memcpy(&w[i], &b, 4);
        } else {
            const __half2 h = __floats2half2_rn(x, y);
            memcpy(&w[i], &h, 4);
        }
    }
    if constexpr (kWords % 4 == 0) {
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i)
            reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else {
        *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    }
}

// Kernels of one call that follow one another: the next one's CTAs may take
// their places on the SMs while the last CTAs of this one still run
// (let_next_start), and wait there until it has ended and its writes are seen
// (wait_for_last, before anything else).  launch_after starts such a next one.
// What the kernel before it wrote is read by plain loads: a read-only load
// (__ldg) asks for memory that nobody writes as long as its kernel lives.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;"); }
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <class... P, class... A>
inline cudaError_t launch_after(void (*kernel)(P...), dim3 grid, int threads, cudaStream_t st, A&&... args) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.stream = st;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// Bytes of one element of a type code (0: unknown code).
inline int type_bytes(int code) { return code == 0 ? 4 : (code == 1 || code == 2) ? 2 : 0; }

// Calls f with a value of the element type of the code (EQCONV_F32, _BF16, _F16).
template <class F>
inline cudaError_t with_type(int code, F&& f) {
    switch (code) {
        case 0: return f(float{});
        case 1: return f(__nv_bfloat16{});
        case 2: return f(__half{});
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace eqc
