// Loads and stores of fp32, bf16 and fp16 tensors as fp32 values.  A store rounds once,
// to nearest even.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

namespace sk {

__device__ __forceinline__ float2 unpack2(unsigned w, const __nv_bfloat16 *)
{
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

__device__ __forceinline__ float2 unpack2(unsigned w, const __half *)
{
    return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

__device__ __forceinline__ unsigned pack2(float a, float b, const __nv_bfloat16 *)
{
    const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const unsigned *>(&r);
}

__device__ __forceinline__ unsigned pack2(float a, float b, const __half *)
{
    const __half2 r = __floats2half2_rn(a, b);
    return *reinterpret_cast<const unsigned *>(&r);
}

// 4 values as they lie in memory (read-only path; 16- or 8-byte aligned), and as fp32
template <class T>
struct Raw4 {
    typedef uint2 type;
};
template <>
struct Raw4<float> {
    typedef float4 type;
};

__device__ __forceinline__ float4 load4_raw(const float *p) { return __ldg(reinterpret_cast<const float4 *>(p)); }

template <class T>
__device__ __forceinline__ uint2 load4_raw(const T *p)
{
    return __ldg(reinterpret_cast<const uint2 *>(p));
}

__device__ __forceinline__ float4 values(float4 w, const float *) { return w; }

template <class T>
__device__ __forceinline__ float4 values(uint2 w, const T *p)
{
    const float2 a = unpack2(w.x, p), b = unpack2(w.y, p);
    return make_float4(a.x, a.y, b.x, b.y);
}

__device__ __forceinline__ void store1(float *p, float x) { *p = x; }
__device__ __forceinline__ void store1(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void store1(__half *p, float x) { *p = __float2half_rn(x); }

__device__ __forceinline__ void store4(float *p, float4 x) { *reinterpret_cast<float4 *>(p) = x; }
template <class T>
__device__ __forceinline__ void store4(T *p, float4 x)
{
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack2(x.x, x.y, p), pack2(x.z, x.w, p));
}

// 8 values as they lie in memory (16-byte aligned; plain loads, so that an output may be its own
// input), and as fp32
template <class T>
struct Raw8 {
    uint4 w[sizeof(T) / 2];
};

template <class T>
__device__ __forceinline__ void load8_raw(const T *p, Raw8<T> &x)
{
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) x.w[i] = reinterpret_cast<const uint4 *>(p)[i];
}

__device__ __forceinline__ void values8(const Raw8<float> &r, float2 (&x)[4], const float *)
{
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        x[2 * i] = make_float2(__uint_as_float(r.w[i].x), __uint_as_float(r.w[i].y));
        x[2 * i + 1] = make_float2(__uint_as_float(r.w[i].z), __uint_as_float(r.w[i].w));
    }
}

template <class T>
__device__ __forceinline__ void values8(const Raw8<T> &r, float2 (&x)[4], const T *p)
{
    x[0] = unpack2(r.w[0].x, p);
    x[1] = unpack2(r.w[0].y, p);
    x[2] = unpack2(r.w[0].z, p);
    x[3] = unpack2(r.w[0].w, p);
}

__device__ __forceinline__ void store8(float *p, const float2 (&x)[4])
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0].x, x[0].y, x[1].x, x[1].y);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[2].x, x[2].y, x[3].x, x[3].y);
}

template <class T>
__device__ __forceinline__ void store8(T *p, const float2 (&x)[4])
{
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack2(x[0].x, x[0].y, p), pack2(x[1].x, x[1].y, p), pack2(x[2].x, x[2].y, p),
                                               pack2(x[3].x, x[3].y, p));
}

}  // namespace sk
