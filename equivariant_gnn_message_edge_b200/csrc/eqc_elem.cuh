// Element types of the node-level operators (embedding, block norm, gradient
// clipping): fp32, bf16 and fp16 tensors read and written as vectors of VE
// elements; all arithmetic is fp32 or wider, with one rounding at the store.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

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
    // as load, for memory that the same kernel also writes
    __device__ __forceinline__ void load_rw(const T* p) {
        static_assert(kPiece == 16, "whole 16-byte pieces");
#pragma unroll
        for (int i = 0; i < kBytes / 16; ++i) q[i] = reinterpret_cast<const uint4*>(p)[i];
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
