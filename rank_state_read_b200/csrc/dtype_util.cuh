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

// 4 values (read-only path; 16- or 8-byte aligned)
__device__ __forceinline__ float4 load4(const float *p) { return __ldg(reinterpret_cast<const float4 *>(p)); }

template <class T>
__device__ __forceinline__ float4 load4(const T *p)
{
    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(p));
    const float2 a = unpack2(w.x, p), b = unpack2(w.y, p);
    return make_float4(a.x, a.y, b.x, b.y);
}

__device__ __forceinline__ void store1(float *p, float x) { *p = x; }
__device__ __forceinline__ void store1(__nv_bfloat16 *p, float x) { *p = __float2bfloat16_rn(x); }
__device__ __forceinline__ void store1(__half *p, float x) { *p = __float2half_rn(x); }

// 8 values (16-byte aligned; plain loads, so that an output may be its own input)
__device__ __forceinline__ void load8(const float *p, float (&x)[8])
{
    const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}

template <class T>
__device__ __forceinline__ void load8(const T *p, float (&x)[8])
{
    const uint4 w = *reinterpret_cast<const uint4 *>(p);
    const unsigned v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = unpack2(v[i], p);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

__device__ __forceinline__ void store8(float *p, const float (&x)[8])
{
    reinterpret_cast<float4 *>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4 *>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}

template <class T>
__device__ __forceinline__ void store8(T *p, const float (&x)[8])
{
    *reinterpret_cast<uint4 *>(p) =
        make_uint4(pack2(x[0], x[1], p), pack2(x[2], x[3], p), pack2(x[4], x[5], p), pack2(x[6], x[7], p));
}

}  // namespace sk
