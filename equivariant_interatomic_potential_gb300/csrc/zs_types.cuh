// Element types of the training operators: 16-byte pieces of fp32, bf16 or
// fp16 read into and written from fp32 registers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "zs_common.cuh"

namespace zs {

inline bool known_dtype(int32_t d) { return d == ZS_F32 || d == ZS_BF16 || d == ZS_F16; }
inline int dtype_bytes(int32_t d) { return d == ZS_F32 ? 4 : 2; }

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);   // elements of a 16-byte piece

// A 16-byte piece as it travels, and its elements in fp32.
template <typename T>
union Piece {
    uint4 raw;
    T e[kVec<T>];
};

__device__ __forceinline__ uint4 ld_piece(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}
__device__ __forceinline__ void st_piece(void* p, uint4 v) {
    asm volatile("st.global.v4.u32 [%0], {%1,%2,%3,%4};" :: "l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

template <typename T>
__device__ __forceinline__ void unpack(uint4 raw, float (&f)[kVec<T>]) {
    Piece<T> p;
    p.raw = raw;
#pragma unroll
    for (int i = 0; i < kVec<T>; ++i) f[i] = to_f32(p.e[i]);
}
template <typename T>
__device__ __forceinline__ uint4 pack(const float (&f)[kVec<T>]) {
    Piece<T> p;
#pragma unroll
    for (int i = 0; i < kVec<T>; ++i) p.e[i] = from_f32<T>(f[i]);
    return p.raw;
}

}  // namespace zs
