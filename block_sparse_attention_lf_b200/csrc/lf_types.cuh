// lf_types.cuh -- loads and stores of 16-bit and 32-bit floating types, 8 elements
// (or one 16-byte vector) at a time, with fp32 arithmetic between them.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace lf {

// dtype codes of the C ABI (lf_dtype)
enum : int { DT_F32 = 0, DT_BF16 = 1, DT_F16 = 2 };

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }

// round to nearest even, once, at the store
template <typename T> __device__ __forceinline__ T from_f32(float x);
template <> __device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <> __device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }

// Elements of a 16-byte vector of T, unpacked to fp32 and packed back.
template <typename T> constexpr int VEC_ELEMS = 16 / static_cast<int>(sizeof(T));

__device__ __forceinline__ void unpack2(uint32_t u, float& a, float& b, __nv_bfloat16)
{
    a = __uint_as_float(u << 16);
    b = __uint_as_float(u & 0xFFFF0000u);
}
__device__ __forceinline__ void unpack2(uint32_t u, float& a, float& b, __half)
{
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&u));
    a = f.x;
    b = f.y;
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename T>
__device__ __forceinline__ void unpack(const uint4& u, float (&v)[VEC_ELEMS<T>])
{
    if constexpr (sizeof(T) == 4) {
        v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y);
        v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
    } else {
        unpack2(u.x, v[0], v[1], T()); unpack2(u.y, v[2], v[3], T());
        unpack2(u.z, v[4], v[5], T()); unpack2(u.w, v[6], v[7], T());
    }
}

template <typename T>
__device__ __forceinline__ uint4 pack(const float (&v)[VEC_ELEMS<T>])
{
    if constexpr (sizeof(T) == 4)
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    else
        return make_uint4(pack2(v[0], v[1], T()), pack2(v[2], v[3], T()), pack2(v[4], v[5], T()), pack2(v[6], v[7], T()));
}

}  // namespace lf
