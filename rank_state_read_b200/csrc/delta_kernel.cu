// The gated delta rule token by token: single tokens of a decode batch, and packed
// prompts of the types and lengths that the chunked kernel does not take.
//
//     u_t = beta_t (v_t - a_t S_{t-1}^T k_t),   S_t = a_t S_{t-1} + k_t u_t^T,
//     y_t = S_t^T q_t = a_t S_{t-1}^T q_t + (q_t . k_t) u_t
//
// Both reductions over the key dimension read the same S_{t-1}, so a token costs one
// pass over the state in registers.  Unit-length q and k come out of the same pass: the
// raw rows enter the products and the factors 1 / |q|, 1 / |k| are applied to the sums.
//
// One CTA of 2 VS threads per (row, head, slab of VS state columns); thread (ks, c4)
// holds the float4 column chunk c4 of the 16 state rows 4 ks + 32 q + e in registers from
// the first token to the last.  The sums over the 8 row slices of a column chunk are a
// reduce-scatter over lane bits 0..2: 8 values (4 columns of k^T S and of q^T S) leave
// one each in 8 lanes with 7 shuffles.  The next token's rows are loaded before this
// token's products.  States are fp32 and every sum is taken in fp32.
//
// A row whose slot or bounds are bad, or whose slot an earlier row names too, is left
// alone and reported through the plan's status word; a negative slot is padding.
#include "device_util.cuh"
#include "dtype_util.cuh"
#include "internal.cuh"

namespace sk {
namespace {

constexpr int DELTA_MAXT = 160;  // slabs of at most 80 columns

// Where a row's tokens lie and which state it has; false: nothing to do.  Every thread
// of the CTA calls it.
__device__ __forceinline__ bool delta_row(const DeltaArgs &A, int row, long long &first, int &len, long long &slot)
{
    first = row;
    len = 1;
    slot = A.slot ? __ldg(A.slot + row) : row;
    bool bad = false;
    if (A.cu) {
        const int c0 = __ldg(A.cu + row), c1 = __ldg(A.cu + row + 1);
        first = c0;
        len = c1 - c0;
        bad = c0 < 0 || c1 < c0 || c1 > A.tokens;
        if (!bad && len == 0) return false;
    }
    if (slot < 0) return false;
    bad = bad || slot >= A.slots;
    if (A.slot)
        for (int i = threadIdx.x; i < row; i += blockDim.x) bad = bad || __ldg(A.slot + i) == slot;
    if (__syncthreads_or(bad)) {
        if (threadIdx.x == 0) atomicOr(A.status, SK_STATUS_BAD_ROW);
        return false;
    }
    return true;
}

// A token's rows as this thread needs them: 16 values of k and q, 4 of v, a, beta.
struct DeltaToken {
    float4 k[4], q[4], v;
    float a, beta;
};

template <class T>
__device__ __forceinline__ void delta_load(const DeltaArgs &A, long long t, int h, int hq, int ks, int col, DeltaToken &x)
{
    const T *k = static_cast<const T *>(A.k) + t * A.k_stride + hq * KDIM + 4 * ks;
    const T *q = static_cast<const T *>(A.q) + t * A.q_stride + hq * KDIM + 4 * ks;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x.k[i] = load4(k + 32 * i);
        x.q[i] = load4(q + 32 * i);
    }
    x.v = load4(static_cast<const T *>(A.v) + t * A.v_stride + (long long)h * A.V + col);
    x.a = __ldg(A.a + t * A.H + h);
    x.beta = __ldg(A.beta + t * A.H + h);
}

template <class T>
__global__ void __launch_bounds__(DELTA_MAXT, 2) delta_kernel(const DeltaArgs A)
{
    const int nslab = A.V / A.VS;
    const long long item = blockIdx.x;
    const int slab = (int)(item % nslab);
    const int h = (int)(item / nslab % A.H), row = (int)(item / nslab / A.H);
    const int hq = h / A.hpq;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int ks = lane & 7, col = slab * A.VS + (warp * 4 + (lane >> 3)) * 4;
    constexpr unsigned FULL = 0xffffffffu;

    long long first, slot;
    int len;
    if (!delta_row(A, row, first, len, slot)) return;

    float *Sg = A.S + ((slot * A.H + h) * KDIM + 4 * ks) * A.V + col;
    float4 s[16];
#pragma unroll
    for (int i = 0; i < 16; ++i)
        s[i] = *reinterpret_cast<const float4 *>(Sg + (long long)(32 * (i >> 2) + (i & 3)) * A.V);
    DeltaToken x;
    delta_load<T>(A, first, h, hq, ks, col, x);

    for (int t = 0; t < len; ++t) {
        const DeltaToken c = x;
        if (t + 1 < len) delta_load<T>(A, first + t + 1, h, hq, ks, col, x);

        float kk = 0.f, qq = 0.f, qk = 0.f;
        float4 d = zero4(), p = zero4();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            kk += dot4(c.k[i], c.k[i]);
            qq += dot4(c.q[i], c.q[i]);
            qk += dot4(c.q[i], c.k[i]);
            fma4(d, c.k[i].x, s[4 * i + 0]);
            fma4(d, c.k[i].y, s[4 * i + 1]);
            fma4(d, c.k[i].z, s[4 * i + 2]);
            fma4(d, c.k[i].w, s[4 * i + 3]);
            fma4(p, c.q[i].x, s[4 * i + 0]);
            fma4(p, c.q[i].y, s[4 * i + 1]);
            fma4(p, c.q[i].z, s[4 * i + 2]);
            fma4(p, c.q[i].w, s[4 * i + 3]);
        }
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
            kk += __shfl_xor_sync(FULL, kk, o);
            qq += __shfl_xor_sync(FULL, qq, o);
            qk += __shfl_xor_sync(FULL, qk, o);
        }
        const float rk = A.normalize ? rsqrtf(kk + DELTA_QK_EPS) : 1.f;
        const float rq = A.scale * (A.normalize ? rsqrtf(qq + DELTA_QK_EPS) : 1.f);
        // lanes with bit 0 clear take k^T S, the others q^T S; then bits 1 and 2 pick the
        // column: lane bits (b2 b1) end with column 2 b1 + b2 of the chunk
        const bool b0 = ks & 1, b1 = ks & 2, b2 = ks & 4;
        float4 m, o4;
        m.x = b0 ? p.x : d.x;
        m.y = b0 ? p.y : d.y;
        m.z = b0 ? p.z : d.z;
        m.w = b0 ? p.w : d.w;
        o4.x = b0 ? d.x : p.x;
        o4.y = b0 ? d.y : p.y;
        o4.z = b0 ? d.z : p.z;
        o4.w = b0 ? d.w : p.w;
        m.x += __shfl_xor_sync(FULL, o4.x, 1);
        m.y += __shfl_xor_sync(FULL, o4.y, 1);
        m.z += __shfl_xor_sync(FULL, o4.z, 1);
        m.w += __shfl_xor_sync(FULL, o4.w, 1);
        float m0 = b1 ? m.z : m.x, m1 = b1 ? m.w : m.y;
        m0 += __shfl_xor_sync(FULL, b1 ? m.x : m.z, 2);
        m1 += __shfl_xor_sync(FULL, b1 ? m.y : m.w, 2);
        float sum = b2 ? m1 : m0;
        sum += __shfl_xor_sync(FULL, b2 ? m0 : m1, 4);
        // u of the lane's column (lanes with bit 0 set compute it of garbage and take it
        // from their neighbour)
        const float vc = b1 ? (b2 ? c.v.w : c.v.z) : (b2 ? c.v.y : c.v.x);
        float u = c.beta * (vc - c.a * rk * sum);
        u = __shfl_sync(FULL, u, lane & ~1);
        if (b0) {
            const float y = rq * fmaf(c.a, sum, rk * qk * u);
            store1(static_cast<T *>(A.y) + (first + t) * A.y_stride + (long long)h * A.V + col + (b1 ? 2 : 0) + (b2 ? 1 : 0), y);
        }
        const int base = lane & ~7;
        float4 u4;
        u4.x = rk * __shfl_sync(FULL, u, base);
        u4.y = rk * __shfl_sync(FULL, u, base + 4);
        u4.z = rk * __shfl_sync(FULL, u, base + 2);
        u4.w = rk * __shfl_sync(FULL, u, base + 6);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float4 k4 = c.k[i >> 2];
            const float kv = (i & 3) == 0 ? k4.x : (i & 3) == 1 ? k4.y : (i & 3) == 2 ? k4.z : k4.w;
            s[i].x = fmaf(kv, u4.x, c.a * s[i].x);
            s[i].y = fmaf(kv, u4.y, c.a * s[i].y);
            s[i].z = fmaf(kv, u4.z, c.a * s[i].z);
            s[i].w = fmaf(kv, u4.w, c.a * s[i].w);
        }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) st4(Sg + (long long)(32 * (i >> 2) + (i & 3)) * A.V, s[i]);
}

}  // namespace

cudaError_t launch_delta(const DeltaArgs &a, cudaStream_t stream)
{
    if (a.rows == 0) return cudaSuccess;
    const unsigned items = (unsigned)((long long)a.rows * a.H * (a.V / a.VS));
    switch (a.dtype) {
    case SKETCHSSM_BF16: delta_kernel<__nv_bfloat16><<<items, 2 * a.VS, 0, stream>>>(a); break;
    case SKETCHSSM_F16: delta_kernel<__half><<<items, 2 * a.VS, 0, stream>>>(a); break;
    default: delta_kernel<float><<<items, 2 * a.VS, 0, stream>>>(a); break;
    }
    return cudaGetLastError();
}

}  // namespace sk
