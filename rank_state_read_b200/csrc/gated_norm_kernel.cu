// The gated norm behind a layer's read: RMS over groups of `width` values, a weight, and
// a gate that multiplies after the norm (Gated DeltaNet) or before it (Mamba-2).
//
//     norm first:  out = x r w act(z),          r = 1 / sqrt(mean x^2 + eps)
//     gate first:  u = x act(z),  out = u r w,  r = 1 / sqrt(mean u^2 + eps)
//
// One pass: a group's values stay in registers between the sum of squares and the store,
// so the kernel moves x, z and out once and is bound by HBM.  A group belongs to LANES
// lanes (8 to 32, the width / 8 vectors of 8 values dealt out round robin), so that short
// groups share a warp; groups of more than 2048 values belong to a CTA.  Sums and
// products are fp32; the only rounding to fewer bits is that of the stored value.
#include "device_util.cuh"
#include "dtype_util.cuh"
#include "internal.cuh"

namespace sk {
namespace {

constexpr int GN_THREADS = 256;
constexpr int GN_WARP_MAX = 2048;  // widest group of one warp: 8 vectors a lane

__device__ __forceinline__ float gn_act(float z, int sigmoid)
{
    const float s = 1.f / (1.f + expf(-z));
    // silu(-inf) = 0, not -inf * 0
    return sigmoid ? s : (s == 0.f ? 0.f : z * s);
}

// VECS vectors of 8 values a lane; LANES lanes (a power of two up to 32) or, with
// LANES = GN_THREADS, the whole CTA hold one group.
template <class TX, class T, int VECS, int LANES>
__global__ void __launch_bounds__(GN_THREADS) gated_norm_kernel(const NormArgs A)
{
    const long long item = ((long long)blockIdx.x * GN_THREADS + threadIdx.x) / LANES;
    const int lane = threadIdx.x % LANES;
    const bool there = item < A.items;
    const long long row = there ? item / A.groups : 0;
    const int group = there ? (int)(item - row * A.groups) : 0;
    const int nvec = A.width / 8;
    const TX *x = static_cast<const TX *>(A.x) + row * A.x_stride + (long long)group * A.width;
    const T *z = A.z ? static_cast<const T *>(A.z) + row * A.z_stride + (long long)group * A.width : nullptr;
    const float *w = A.weight + (A.weight_groups > 1 ? (long long)group * A.width : 0);
    T *out = static_cast<T *>(A.out) + row * A.out_stride + (long long)group * A.width;

    float u[VECS][8], g[VECS][8];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        const int v = lane + i * LANES;
        if (there && v < nvec) {
            load8(x + 8 * v, u[i]);
            if (z) load8(z + 8 * v, g[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        const int v = lane + i * LANES;
        if (there && v < nvec) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                g[i][e] = z ? gn_act(g[i][e], A.sigmoid) : 1.f;
                if (A.gate_first) u[i][e] *= g[i][e];
                sum = fmaf(u[i][e], u[i][e], sum);
            }
        }
    }
    if (LANES <= 32) {
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    } else {
        __shared__ float part[GN_THREADS / 32];
        sum = warp_sum(sum);
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = sum;
        __syncthreads();
        sum = 0.f;
#pragma unroll
        for (int i = 0; i < GN_THREADS / 32; ++i) sum += part[i];
    }
    const float r = rsqrtf(sum / (float)A.width + A.eps);
#pragma unroll
    for (int i = 0; i < VECS; ++i) {
        const int v = lane + i * LANES;
        if (there && v < nvec) {
            const float4 w0 = ldg4(w + 8 * v), w1 = ldg4(w + 8 * v + 4);
            const float ww[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                u[i][e] *= r * ww[e];
                if (!A.gate_first) u[i][e] *= g[i][e];
            }
            store8(out + 8 * v, u[i]);
        }
    }
}

template <class TX, class T, int VECS, int LANES>
cudaError_t launch_shape(const NormArgs &a, cudaStream_t stream)
{
    constexpr int PER = GN_THREADS / LANES;
    gated_norm_kernel<TX, T, VECS, LANES><<<(unsigned)((a.items + PER - 1) / PER), GN_THREADS, 0, stream>>>(a);
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
    if (nvec <= 128) return launch_shape<TX, T, 4, 32>(a, stream);
    if (a.width <= GN_WARP_MAX) return launch_shape<TX, T, 8, 32>(a, stream);
    if (nvec <= 4 * GN_THREADS) return launch_shape<TX, T, 4, GN_THREADS>(a, stream);
    return launch_shape<TX, T, 8, GN_THREADS>(a, stream);
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
