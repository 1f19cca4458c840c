// dtype.cuh -- 16-byte vectors of the decoder-side element types, held as fp32 in registers.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace vitk {

__device__ __forceinline__ void unpack2(uint32_t u, float &a, float &b, __nv_bfloat16) {
    a = __uint_as_float(u << 16);
    b = __uint_as_float(u & 0xFFFF0000u);
}
__device__ __forceinline__ void unpack2(uint32_t u, float &a, float &b, __half) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u));
    a = f.x;
    b = f.y;
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __nv_bfloat16) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint32_t pack2(float a, float b, __half) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// kVec elements of T per 16-byte vector; values are rounded once, to nearest even, when packed
template <typename T>
struct Vec {
    static constexpr int kVec = 8;
    __device__ static __forceinline__ void unpack(const uint4 &v, float *f) {
        unpack2(v.x, f[0], f[1], T());
        unpack2(v.y, f[2], f[3], T());
        unpack2(v.z, f[4], f[5], T());
        unpack2(v.w, f[6], f[7], T());
    }
    __device__ static __forceinline__ uint4 pack(const float *f) {
        return make_uint4(pack2(f[0], f[1], T()), pack2(f[2], f[3], T()), pack2(f[4], f[5], T()),
                          pack2(f[6], f[7], T()));
    }
};
template <>
struct Vec<float> {
    static constexpr int kVec = 4;
    __device__ static __forceinline__ void unpack(const uint4 &v, float *f) {
        f[0] = __uint_as_float(v.x);
        f[1] = __uint_as_float(v.y);
        f[2] = __uint_as_float(v.z);
        f[3] = __uint_as_float(v.w);
    }
    __device__ static __forceinline__ uint4 pack(const float *f) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};

__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_float(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_float(float x) { return x; }

}  // namespace vitk
