// The gated norm behind a layer's read: RMS over groups of `width` values, a weight, and
// a gate that multiplies after the norm (Gated DeltaNet) or before it (Mamba-2).
//
//     norm first:  out = x r w act(z),          r = 1 / sqrt(mean x^2 + eps)
//     gate first:  u = x act(z),  out = u r w,  r = 1 / sqrt(mean u^2 + eps)
//
// One pass: a group's values stay in registers between the sum of squares and the store,
// so the kernel moves x, z and out once and is bound by HBM.  A group belongs to LANES
// lanes (8 to 32, the width / 8 vectors of 8 values dealt out round robin), so that short
// groups share a warp; groups of more than 512 values belong to a CTA.  Above 8192 values a thread has 64
// of them, which spill in part.  Of the measured copy rate: 32768 x 32 x 128 bf16 0.88, 16384 x 32 x 128
// fp32 0.96, 8192 groups of 16384 bf16 0.68, fp32 0.39.  Sums and products are fp32; the only rounding to
// fewer bits is that of the stored value.
#include <atomic>

#include "device_util.cuh"
#include "dtype_util.cuh"
#include "internal.cuh"

namespace sk {
namespace {

constexpr int GN_THREADS = 256;

// -inf becomes the lowest finite value, NaN stays
__device__ __forceinline__ float gn_finite(float z)
{
    float r;
    asm("max.NaN.f32 %0, %1, 0fFF7FFFFF;" : "=f"(r) : "f"(z));
    return r;
}

// Gate of one value, by expf and a division: exp(-|z|) stays in fp32's range, as exp(-z) does not below
// -88.7, and leaves its normal numbers where the result does.
__device__ __forceinline__ float gn_gate(float z, bool sigmoid)
{
    const float t = expf(-fabsf(z)), s = (z < 0.f ? t : 1.f) / (1.f + t);
    return sigmoid ? s : gn_finite(z) * s;  // silu(-inf) = 0, not -inf * 0
}

// Gates of two values.  Where the result is rounded to 16 bits, by the hardware's exponential and
// reciprocal (a few 2^-22), in pairs, since at 128 columns of bf16 the instructions bound the kernel next
// to HBM (162 us for 32768 x 32 x 128 element by element).  The value and the exponential are scaled by
// 2^-8 there (140 instead of 138 us): the reciprocal then stays a normal number down to z = -92.9, and
// SiLU is one down to -91.9.
template <bool FAST>
__device__ __forceinline__ float2 gn_gates(float2 z, bool sigmoid)
{
    if (!FAST) return make_float2(gn_gate(z.x, sigmoid), gn_gate(z.y, sigmoid));
    const float2 scale = make_float2(0x1p-8f, 0x1p-8f);
    const float2 e = __ffma2_rn(z, make_float2(-1.44269504f, -1.44269504f), make_float2(-8.f, -8.f));
    float2 x, s;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(x.x) : "f"(e.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(x.y) : "f"(e.y));
    x = __fadd2_rn(x, scale);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(x.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(x.y));
    return __fmul2_rn(sigmoid ? scale : __fmul2_rn(make_float2(gn_finite(z.x), gn_finite(z.y)), scale), s);
}

// VECS vectors of 8 values a lane; LANES lanes (a power of two up to 32) or, with
// LANES = 0, all of a CTA of as many warps as it takes hold one group.  The CTAs stay and go through the groups, the
// next one's values on their way (as they are in memory) while one is worked on.
template <class TX, class T, int VECS, int LANES>
__global__ void __launch_bounds__(GN_THREADS) gated_norm_kernel(const NormArgs A)
{
    constexpr bool WHOLE = LANES == 0;
    const int lanes = WHOLE ? blockDim.x : LANES, PER = WHOLE ? 1 : GN_THREADS / (WHOLE ? 1 : LANES);
    const int lane = WHOLE ? threadIdx.x : threadIdx.x % (WHOLE ? 1 : LANES);
    const int nvec = A.width / 8;
    const unsigned items = (unsigned)A.items, step = gridDim.x * PER;
    Raw8<TX> xr[VECS];
    Raw8<T> zr[VECS];
    unsigned row = 0, group = 0;  // of the values in xr, zr
    auto load = [&](unsigned item) {
        if (item < items) {
            row = item / (unsigned)A.groups;
            group = item - row * (unsigned)A.groups;
            const TX *x = static_cast<const TX *>(A.x) + row * A.x_stride + (long long)group * A.width;
            const T *z = static_cast<const T *>(A.z) + row * A.z_stride + (long long)group * A.width;
#pragma unroll
            for (int i = 0; i < VECS; ++i) {
                const int v = lane + i * lanes;
                if (v < nvec) {
                    load8_raw(x + 8 * v, xr[i]);
                    if (A.z) load8_raw(z + 8 * v, zr[i]);
                }
            }
        }
    };
    unsigned item = blockIdx.x * PER + (WHOLE ? 0 : threadIdx.x / (WHOLE ? 1 : LANES));
    load(item);
    // (a CTA's threads leave the loop together: its first thread has its smallest item)
    for (unsigned base = blockIdx.x * PER; base < items; base += step, item += step) {
        const bool there = item < items;
        float2 u[VECS][4], g[VECS][4];
        T *out = static_cast<T *>(A.out) + row * A.out_stride + (long long)group * A.width;
        const float *w = A.weight + (A.weight_groups > 1 ? (long long)group * A.width : 0);
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            values8(xr[i], u[i], (const TX *)nullptr);
            values8(zr[i], g[i], (const T *)nullptr);
        }
        load(item + step);
        float2 sum2 = make_float2(0.f, 0.f);
        auto gates = [&](bool sigmoid) {
#pragma unroll
            for (int i = 0; i < VECS; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) g[i][e] = gn_gates<sizeof(T) == 2>(g[i][e], sigmoid);
        };
        if (!A.z) {
#pragma unroll
            for (int i = 0; i < VECS; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) g[i][e] = make_float2(1.f, 1.f);
        } else if (A.sigmoid) {
            gates(true);
        } else {
            gates(false);
        }
        if (A.gate_first) {
#pragma unroll
            for (int i = 0; i < VECS; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    u[i][e] = __fmul2_rn(u[i][e], g[i][e]);
                    g[i][e] = make_float2(1.f, 1.f);
                }
        }
#pragma unroll
        for (int i = 0; i < VECS; ++i)
            if (there && lane + i * lanes < nvec) {
#pragma unroll
                for (int e = 0; e < 4; ++e) sum2 = __ffma2_rn(u[i][e], u[i][e], sum2);
            }
        float sum = sum2.x + sum2.y;
        if (!WHOLE) {
#pragma unroll
            for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        } else {
            __shared__ float part[2][GN_THREADS / 32];
            float *p = part[(base - blockIdx.x * PER) / step & 1];
            sum = warp_sum(sum);
            if ((threadIdx.x & 31) == 0) p[threadIdx.x >> 5] = sum;
            __syncthreads();
            sum = 0.f;
#pragma unroll
            for (int i = 0; i < GN_THREADS / 32; ++i)
                if (32 * i < lanes) sum += p[i];
        }
        const float r = rsqrtf(sum / (float)A.width + A.eps);
#pragma unroll
        for (int i = 0; i < VECS; ++i) {
            const int v = lane + i * lanes;
            if (there && v < nvec) {
                const float4 w0 = ldg4(w + 8 * v), w1 = ldg4(w + 8 * v + 4);
                const float2 ww[4] = {make_float2(w0.x, w0.y), make_float2(w0.z, w0.w), make_float2(w1.x, w1.y),
                                      make_float2(w1.z, w1.w)};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    u[i][e] = __fmul2_rn(__fmul2_rn(u[i][e], __fmul2_rn(ww[e], make_float2(r, r))), g[i][e]);
                store8(out + 8 * v, u[i]);
            }
        }
    }
}

template <class TX, class T, int VECS, int LANES>
cudaError_t launch_shape(const NormArgs &a, cudaStream_t stream)
{
    const int warps = LANES ? GN_THREADS / 32 : (a.width / 8 + 32 * VECS - 1) / (32 * VECS);
    const int per = LANES ? GN_THREADS / (LANES ? LANES : 1) : 1;
    const long long blocks = (a.items + per - 1) / per;
    // CTAs of each size that one SM holds, asked for once
    static std::atomic<int> resident[GN_THREADS / 32 + 1];
    int n = resident[warps].load(std::memory_order_relaxed);
    if (n == 0) {
        cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, gated_norm_kernel<TX, T, VECS, LANES>, 32 * warps, 0);
        if (e != cudaSuccess) return e;
        if (n < 1) n = 1;
        resident[warps].store(n, std::memory_order_relaxed);
    }
    const long long most = (long long)n * a.sms;
    gated_norm_kernel<TX, T, VECS, LANES><<<(unsigned)(blocks < most ? blocks : most), 32 * warps, 0, stream>>>(a);
    return cudaGetLastError();
}

template <class TX, class T>
cudaError_t launch_types(const NormArgs &a, cudaStream_t stream)
{
    const int nvec = a.width / 8;
    if (nvec <= 8) return launch_shape<TX, T, 1, 8>(a, stream);
    if (nvec <= 16) return launch_shape<TX, T, 1, 16>(a, stream);
    if (nvec <= 32) return launch_shape<TX, T, 1, 32>(a, stream);
    if (nvec <= 64) return launch_shape<TX, T, 2, 32>(a, stream);
    if (nvec <= GN_THREADS) return launch_shape<TX, T, 1, 0>(a, stream);
    if (nvec <= 2 * GN_THREADS) return launch_shape<TX, T, 2, 0>(a, stream);
    if (nvec <= 4 * GN_THREADS) return launch_shape<TX, T, 4, 0>(a, stream);
    return launch_shape<TX, T, 8, 0>(a, stream);
}

template <class TX>
cudaError_t launch_x(const NormArgs &a, cudaStream_t stream)
{
    switch (a.dtype) {
    case SKETCHSSM_BF16: return launch_types<TX, __nv_bfloat16>(a, stream);
    case SKETCHSSM_F16: return launch_types<TX, __half>(a, stream);
    default: return launch_types<TX, float>(a, stream);
    }
}

}  // namespace

cudaError_t launch_gated_norm(const NormArgs &a, cudaStream_t stream)
{
    if (a.items == 0) return cudaSuccess;
    switch (a.x_dtype) {
    case SKETCHSSM_BF16: return launch_x<__nv_bfloat16>(a, stream);
    case SKETCHSSM_F16: return launch_x<__half>(a, stream);
    default: return launch_x<float>(a, stream);
    }
}

}  // namespace sk
