// The gated delta rule on packed prompts of 16-bit tokens, 64 tokens at a time on the
// 5th-generation tensor cores (tcgen05).
//
// With G_i the sum of log a over the chunk's tokens up to i and S the state before it, the
// recurrence S_i = a_i (I - beta_i k_i k_i^T) S_{i-1} + beta_i k_i v_i^T unrolls to
//
//     u_i = beta_i (v_i - exp(G_i) S^T k_i - sum_{j<i} exp(G_i - G_j) (k_i . k_j) u_j)
//     =>  U = T R,   T = (I + A)^-1,  A_ij = beta_i exp(G_i - G_j) k_i . k_j  (j < i),
//         R = diag(beta) (V - diag(exp G) K S)
//     Y = diag(exp G) Q S + P U,     P_ij = exp(G_i - G_j) q_i . k_j  (j <= i)
//     S <- exp(G_C) S + sum_j exp(G_C - G_j) k_j u_j^T
//
// so that the chain from chunk to chunk is three matrix products.  All exponents are
// differences with j <= i, never positive; a decay of 0 counts as 2^-150.
//
// One CTA per (sequence, head, slice of 128 value columns), persistent.  Everything on the
// chain is taken transposed: tensor-memory lane = value column.  A column's state (fp32)
// lives in the registers of two threads, its 64 token values pass through them, and the
// left operands S^T, R^T, U^T are written straight into tensor memory, with no shared
// memory, no transposition and no sum across threads.
//   warps 0-7   the chain: warps w and w + 4 share 32 lanes (columns), each half the tokens
//               (or key rows);
//   warps 8-11  one chunk ahead: bring q, k, v in, and form A, P and T;
//   warp 12     issues the chain's MMAs (its warp group gives its registers to the others).
//
// Precision.  The state is held, and its errors count, in fp32.  An operand x of the state's
// path is split into two fp16 parts, x = 2^-e (hi + lo) (1 + 2^-22), e from the largest value
// of its row, and products are taken hi hi + hi lo + lo hi in fp32; q and k, 8 or 11 bits
// wide, are exact in fp16 after a row's power of two.  (fp16 pairs hold 22 bits where bf16
// pairs hold 16 and bf16 triples 24 for half as many products again.)  y goes back to 16
// bits: bf16 outputs take hi alone (2^-12), fp16 outputs the pair.
#include <cstddef>

#include "device_util.cuh"
#include "dtype_util.cuh"
#include "internal.cuh"
#include "ptx_util.cuh"

namespace sk {
namespace {

constexpr int DC_C = 64;        // tokens of a chunk
constexpr int DC_VW = 128;      // value columns of a slice
constexpr int DC_CHAIN = 256, DC_PREP = 128;
constexpr int DC_THREADS = DC_CHAIN + DC_PREP + 128;
// registers a thread after the split: 2 x 128 x 160 + 128 x 152 + 128 x 40 = 512 x 128
constexpr int DC_REG_CHAIN = 160, DC_REG_PREP = 152, DC_REG_ISSUE = 40;
constexpr int DC_KV = 3, DC_TP = 2;  // stages of q, k, v and of T, P

// tensor memory columns
constexpr uint32_t TM_A = 0;     // K S^T, then U^T (64); with the next 64: the state's increment
constexpr uint32_t TM_Q = 128;   // Q S^T (64)
constexpr uint32_t TM_PU = 192;  // P U (64)
constexpr uint32_t TM_S = 256;   // S hi, lo (64 each); then U~ hi, lo, U hi, lo (32 each)
constexpr uint32_t TM_R = 384;   // R hi, lo (32 each)
constexpr uint32_t TM_KK = 448;  // [K; Q] K^T (64)

struct DcSmem {
    // 1024-byte aligned operand tiles, rows of 128 bytes, 128-byte swizzle
    uint8_t kq[DC_KV][2][128 * 128];  // k dims 0-63 | 64-127; rows 0-63 k, 64-127 q
    uint8_t tp[DC_TP][4][64 * 128];   // T hi, T lo (before that A and T in fp32), P hi, P lo
    uint16_t v[DC_KV][DC_C][DC_VW];
    float ab[DC_KV][128];             // beta, a of the chunk's tokens
    // per token, by T / P stage: factors of v and K S in R; of U; of U for the state; of Q S; of P U
    float fv[DC_TP][DC_C], fks[DC_TP][DC_C], fu[DC_TP][DC_C], fw[DC_TP][DC_C], fqs[DC_TP][DC_C], fp[DC_TP][DC_C];
    alignas(16) float fac[128];       // value of a unit of each k and q row
    alignas(16) float Gh[DC_C], Gl[DC_C];  // G in base 2, high and low parts
    float gC[DC_TP];                  // the whole chunk's decay
    float x[32][36];                  // products on the way to T
    float mx[2][2][2][DC_VW];         // column maxima of the two chain halves
    uint64_t b_kq[DC_KV], b_free[DC_KV], b_tp[DC_TP], b_out[DC_TP];
    uint64_t b_S, b_KS, b_QS, b_R, b_U, b_W, b_D, b_PU, b_KK, b_end;
    uint32_t taddr;
    int stop;
    uint32_t dup[DC_MAX_SEQS / 32];
    uint16_t order[DC_MAX_SEQS];      // sequences, longest first
};

// ---- tcgen05 forms of this kernel ----

// instruction descriptor: fp16 x fp16 -> fp32, A K-major, B K-major or (mn) N-major
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, bool mn)
{
    return (1u << 4) | (mn ? 1u << 16 : 0u) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// shared-memory descriptor, 128-byte swizzle: `lbo`: between blocks of 64 along N (N-major
// only), `sbo`: between groups of 8 rows
__device__ __forceinline__ uint64_t sdesc_sw128(uint32_t addr, uint32_t lbo, uint32_t sbo)
{
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) |
           ((uint64_t)((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// 32 columns of the warp's 32 lanes; tmem_ld_wait before the values are used
__device__ __forceinline__ void tmem_ld32(uint32_t addr, float *x)
{
    uint32_t *r = reinterpret_cast<uint32_t *>(x);
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,"
        "%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr)
        : "memory");
}

__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void named_sync(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// ---- splitting ----

// The power of two that brings the largest magnitude `m` into [2^14, 2^15), and its inverse.
// Magnitudes below 2^-112 stay below (their products do not count in fp32); infinities and
// NaN pass on.
__device__ __forceinline__ void pow2_scale(float m, float &mul, float &inv)
{
    int e = (int)(__float_as_uint(m) >> 23);
    e = e < 15 ? 15 : e;
    mul = __uint_as_float((uint32_t)(268 - e) << 23);
    inv = __uint_as_float((uint32_t)(e - 14) << 23);
}

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *reinterpret_cast<uint32_t *>(&h); }

// hi and lo fp16 parts of two scaled values
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo)
{
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    hi = h2_bits(h);
    lo = h2_bits(__floats2half2_rn(a - f.x, b - f.y));
}

// ---- which chunk comes next ----

static_assert(sizeof(DcSmem) <= 232448, "shared memory of one CTA");
static_assert(offsetof(DcSmem, kq) % 1024 == 0 && offsetof(DcSmem, tp) % 1024 == 0, "swizzled tiles");
static_assert(offsetof(DcSmem, v) % 16 == 0 && offsetof(DcSmem, fac) % 16 == 0 && offsetof(DcSmem, Gh) % 16 == 0 &&
                  offsetof(DcSmem, Gl) % 16 == 0 && offsetof(DcSmem, b_kq) % 8 == 0,
              "vector accesses");

struct DcWalk {
    int round, chunk;   // of this CTA's items; chunk of the item
    int h, slice, len;
    long long first, slot;
    bool there;
};

__device__ __forceinline__ void dc_fetch(const DeltaArgs &A, const DcSmem &sm, DcWalk &w)
{
    const int nslice = (A.V + DC_VW - 1) / DC_VW, per = A.H * nslice;
    const int items = A.rows * per, G = gridDim.x;
    w.chunk = 0;
    for (;; ++w.round) {
        // items go round back and forth, so that a CTA that gets a longer one gets a shorter
        // one next
        const long long k = (long long)w.round * G + ((w.round & 1) ? G - 1 - (int)blockIdx.x : (int)blockIdx.x);
        if ((long long)w.round * G >= items) {
            w.there = false;
            return;
        }
        if (k >= items) continue;
        const int row = sm.order[k / per], rest = (int)(k % per);
        const int c0 = __ldg(A.cu + row), c1 = __ldg(A.cu + row + 1), slot = A.slot ? __ldg(A.slot + row) : row;
        if (c0 < 0 || c1 <= c0 || c1 > A.tokens || slot < 0 || slot >= A.slots || (sm.dup[row >> 5] >> (row & 31) & 1))
            continue;
        w.there = true;
        w.first = c0;
        w.len = c1 - c0;
        w.slot = slot;
        w.h = rest / nslice;
        w.slice = rest % nslice;
        return;
    }
}

__device__ __forceinline__ void dc_next(const DeltaArgs &A, const DcSmem &sm, DcWalk &w)
{
    if (!w.there) return;
    if (++w.chunk * DC_C < w.len) return;
    ++w.round;
    dc_fetch(A, sm, w);
}

// ---- waits: bounded; past the plan's limit recorded, past the default limit given up, after
// which nothing waits any more and the kernel runs out ----
__device__ __forceinline__ void dc_wait_long(const DeltaArgs &A, DcSmem &sm, uint64_t *bar, uint32_t parity)
{
    if (*(volatile int *)&sm.stop) return;
    atomicOr(A.status, SK_STATUS_DELTA_TIMEOUT);
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity))
        if (clock64() - t0 > DEFAULT_WAIT_CYCLES || *(volatile int *)&sm.stop) {
            *(volatile int *)&sm.stop = 1;
            return;
        }
}

__device__ __forceinline__ void dc_wait(const DeltaArgs &A, DcSmem &sm, uint64_t *bar, uint32_t parity)
{
    if (mbar_test_wait(bar, parity)) return;
    if (!mbar_wait_bounded(bar, parity, A.wait_limit)) dc_wait_long(A, sm, bar, parity);
}

// one arrival for a warp whose lanes have all done their part
__device__ __forceinline__ void warp_arrive(uint64_t *bar)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// ---- warps 8-11 ----

// cp.async of 16 bytes, or 16 zero bytes
__device__ __forceinline__ void cp_async16_zfill(void *dst, const void *src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(there ? 16 : 0)
                 : "memory");
}

// k, q, v, beta and a of the walk's chunk into stage `st`; rows past the sequence's end are zeros
template <class T>
__device__ __forceinline__ void dc_load(const DeltaArgs &A, DcSmem &sm, const DcWalk &w, int st, int r)
{
    const long long t0 = w.first + (long long)w.chunk * DC_C;
    const int left = w.len - w.chunk * DC_C;
    const int hq = w.h / A.hpq;
    const int vw = min(DC_VW, A.V - w.slice * DC_VW);
    // 16 threads a row of k or q, 8 rows a pass
    const int c = r & 15, r0 = r >> 4;
    const T *kp = static_cast<const T *>(A.k) + hq * KDIM + c * 8, *qp = static_cast<const T *>(A.q) + hq * KDIM + c * 8;
    uint8_t *dst = sm.kq[st][c >> 3];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int t = i * 8 + r0;  // t & 7 == r0
        const bool there = t < left;
        const long long tok = t0 + (there ? t : 0);
        const int off = t * 128 + (((c & 7) ^ r0) << 4);
        cp_async16_zfill(dst + off, kp + tok * A.k_stride, there);
        cp_async16_zfill(dst + 64 * 128 + off, qp + tok * A.q_stride, there);
    }
    if (c * 8 < vw) {
        const T *vp = static_cast<const T *>(A.v) + (long long)w.h * A.V + w.slice * DC_VW + c * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int t = i * 8 + r0;
            const bool there = t < left;
            cp_async16_zfill(&sm.v[st][t][c * 8], vp + (t0 + (there ? t : 0)) * A.v_stride, there);
        }
    }
    const int t = r & 63;
    if (t < left) cp_async4(&sm.ab[st][r], (r < 64 ? A.beta : A.a) + (t0 + t) * A.H + w.h);
}

// where A and T lie in fp32: rows of 64 floats, 16-byte chunks permuted by the row
__device__ __forceinline__ int tri(int i, int j) { return i * 64 + ((((j >> 2) ^ i) & 15) << 2) + (j & 3); }

__device__ __forceinline__ float tf32_round(float x)
{
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
    return __uint_as_float(r);
}

__device__ __forceinline__ void mma_tf32(float (&d)[4], const float (&a)[4], const float (&b)[2])
{
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(__float_as_uint(a[0])), "r"(__float_as_uint(a[1])), "r"(__float_as_uint(a[2])),
                   "r"(__float_as_uint(a[3])), "r"(__float_as_uint(b[0])), "r"(__float_as_uint(b[1])));
}

// D (MT tiles of 16 rows x 8 columns) += L[16 MT x 8 KT] B[8 KT x 8], three tf32 products each:
// fp32 accuracy.  l(i, k), b(k, n): the operands' elements.
template <int MT, int KT, class FL, class FB>
__device__ __forceinline__ void mul_tri(float (&d)[MT][4], FL l, FB b)
{
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int ks = 0; ks < KT; ++ks) {
        float bh[2], bl[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float x = b(8 * ks + t + 4 * e, g);
            bh[e] = tf32_round(x);
            bl[e] = x - bh[e];
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            float ah[4], al[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = l(16 * m + g + 8 * (e & 1), 8 * ks + t + 4 * (e >> 1));
                ah[e] = tf32_round(x);
                al[e] = x - ah[e];
            }
            mma_tf32(d[m], al, bh);
            mma_tf32(d[m], ah, bl);
            mma_tf32(d[m], ah, bh);
        }
    }
}

// T = (I + A)^-1 in place, A strictly lower triangular (zeros elsewhere), by the four warps of
// the group: the 16 x 16 blocks on the diagonal by substitution (a column a lane), then
// T21 = -T22 A21 T11 for blocks of 16 and of 32.  Substitution in blocks is as stable as
// substitution; the powers of A that a product form needs would not be.
__device__ __forceinline__ void invert(float *M, float (&X)[32][36], int r)
{
    const int wq = r >> 5, lane = r & 31, g = lane >> 2, t = lane & 3;
    {
        const int o = 16 * wq, j = lane & 15;
        float x[16];
        x[0] = j == 0 ? 1.f : 0.f;
#pragma unroll
        for (int i = 1; i < 16; ++i) {
            float s = 0.f;
#pragma unroll
            for (int k4 = 0; k4 < i; k4 += 4) {
                const float4 a = lds4(M + tri(o + i, o + k4));
                s = fmaf(a.x, x[k4], s);
                if (k4 + 1 < i) s = fmaf(a.y, x[k4 + 1], s);
                if (k4 + 2 < i) s = fmaf(a.z, x[k4 + 2], s);
                if (k4 + 3 < i) s = fmaf(a.w, x[k4 + 3], s);
            }
            x[i] = (i == j ? 1.f : 0.f) - s;
        }
        __syncwarp();
        if (lane < 16) {
#pragma unroll
            for (int i = 0; i < 16; ++i) M[tri(o + i, o + j)] = x[i];
        }
    }
    named_sync(5, DC_PREP);
    {
        const int o = 32 * (wq >> 1), n0 = 8 * (wq & 1), xr = 16 * (wq >> 1);
        float d[1][4] = {};
        mul_tri<1, 2>(d, [&](int i, int k) { return M[tri(o + 16 + i, o + k)]; },
                      [&](int k, int n) { return M[tri(o + k, o + n0 + n)]; });
#pragma unroll
        for (int e = 0; e < 4; ++e) X[xr + g + 8 * (e >> 1)][n0 + 2 * t + (e & 1)] = d[0][e];
        __syncwarp();
        float f[1][4] = {};
        mul_tri<1, 2>(f, [&](int i, int k) { return M[tri(o + 16 + i, o + 16 + k)]; },
                      [&](int k, int n) { return X[xr + k][n0 + n]; });
        named_sync(5, DC_PREP);  // A21 has been read
#pragma unroll
        for (int e = 0; e < 4; ++e) M[tri(o + 16 + g + 8 * (e >> 1), o + n0 + 2 * t + (e & 1))] = -f[0][e];
    }
    named_sync(5, DC_PREP);
    {
        const int n0 = 8 * wq;
        float d[2][4] = {};
        mul_tri<2, 4>(d, [&](int i, int k) { return M[tri(32 + i, k)]; }, [&](int k, int n) { return M[tri(k, n0 + n)]; });
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) X[16 * m + g + 8 * (e >> 1)][n0 + 2 * t + (e & 1)] = d[m][e];
        __syncwarp();
        float f[2][4] = {};
        mul_tri<2, 4>(f, [&](int i, int k) { return M[tri(32 + i, 32 + k)]; }, [&](int k, int n) { return X[k][n0 + n]; });
        named_sync(5, DC_PREP);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) M[tri(32 + 16 * m + g + 8 * (e >> 1), n0 + 2 * t + (e & 1))] = -f[m][e];
    }
    named_sync(5, DC_PREP);
}

// 64 scaled values as fp16 hi (and lo) parts into row `t` of a swizzled tile
template <bool LO>
__device__ __forceinline__ void put_row(uint8_t *hi, uint8_t *lo, int t, const float (&x)[64], float mul)
{
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        uint32_t h[4], l[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) split2(x[8 * c + 2 * e] * mul, x[8 * c + 2 * e + 1] * mul, h[e], l[e]);
        const int off = t * 128 + ((c ^ (t & 7)) << 4);
        *reinterpret_cast<uint4 *>(hi + off) = make_uint4(h[0], h[1], h[2], h[3]);
        if (LO) *reinterpret_cast<uint4 *>(lo + off) = make_uint4(l[0], l[1], l[2], l[3]);
    }
}

template <class T, bool LO>
__device__ __forceinline__ void dc_prep(const DeltaArgs &A, DcSmem &sm, uint32_t tmem)
{
    const int r = threadIdx.x - DC_CHAIN, wq = r >> 5, lane = r & 31;
    const int t = r & 63;        // token of this thread's row
    const bool is_q = r >= 64;
    DcWalk w, ahead;
    w.round = 0;
    dc_fetch(A, sm, w);
    ahead = w;
    for (int i = 0; i < 2; ++i) {
        if (ahead.there) dc_load<T>(A, sm, ahead, i, r);
        cp_async_commit();
        dc_next(A, sm, ahead);
    }
    for (int n = 0; w.there; ++n, dc_next(A, sm, w)) {
        const int st = n % DC_KV, tp = n % DC_TP;
        const int left = w.len - w.chunk * DC_C;
        cp_async_wait<1>();
        named_sync(5, DC_PREP);

        // this thread's row of k or q: its norm, and fp16 values at a power of two of their own
        {
            uint4 raw[16];
#pragma unroll
            for (int c = 0; c < 16; ++c)
                raw[c] = *reinterpret_cast<const uint4 *>(&sm.kq[st][c >> 3][r * 128 + (((c & 7) ^ (r & 7)) << 4)]);
            float ss = 0.f, m = 0.f;
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                const uint32_t v[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = unpack2(v[e], (const T *)nullptr);
                    ss = fmaf(f.x, f.x, fmaf(f.y, f.y, ss));
                    m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));
                }
            }
            float mul, inv;
            pow2_scale(m, mul, inv);
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                const uint32_t v[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
                uint32_t o[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 f = unpack2(v[e], (const T *)nullptr);
                    o[e] = h2_bits(__floats2half2_rn(f.x * mul, f.y * mul));
                }
                *reinterpret_cast<uint4 *>(&sm.kq[st][c >> 3][r * 128 + (((c & 7) ^ (r & 7)) << 4)]) =
                    make_uint4(o[0], o[1], o[2], o[3]);
            }
            if (A.normalize) inv *= rsqrtf(ss + DELTA_QK_EPS);
            if (is_q) inv *= A.scale;
            sm.fac[r] = inv;
        }
        if (wq == 0) {
            // G of tokens 2 l and 2 l + 1, base 2, summed in 64 bits
            const float a0 = 2 * lane < left ? sm.ab[st][64 + 2 * lane] : 1.f;
            const float a1 = 2 * lane + 1 < left ? sm.ab[st][65 + 2 * lane] : 1.f;
            const double l0 = (double)fmaxf(log2f(a0), -150.f), l1 = (double)fmaxf(log2f(a1), -150.f);
            double s = l0 + l1;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double up = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += up;
            }
            const double g0 = s - l1;
            sm.Gh[2 * lane] = (float)g0;
            sm.Gl[2 * lane] = (float)(g0 - (double)(float)g0);
            sm.Gh[2 * lane + 1] = (float)s;
            sm.Gl[2 * lane + 1] = (float)(s - (double)(float)s);
        }
        fence_async_smem();
        tc_fence_before();
        named_sync(5, DC_PREP);
        warp_arrive(&sm.b_kq[st]);
        if (r == 0) {
            tc_fence_after();
            const uint32_t idesc = idesc_f16(128, 64, false);
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                const uint64_t d = sdesc_sw128(smem_addr(sm.kq[st][ks >> 2]) + (ks & 3) * 32, 16, 1024);
                mma_ss(tmem + TM_KK, d, d, idesc, ks > 0);
            }
            umma_commit(&sm.b_KK);
        }
        // this stage's T, P and factors are free once the chunk two before has given its outputs
        if (n >= DC_TP) dc_wait(A, sm, &sm.b_out[tp], (n / DC_TP - 1) & 1);
        const float Gh = sm.Gh[t], Gl = sm.Gl[t];
        const float beta = t < left ? sm.ab[st][t] : 0.f, f_own = sm.fac[r];
        const float decay = exp2f(Gh + Gl);
        float *M = reinterpret_cast<float *>(sm.tp[tp][0]);
        dc_wait(A, sm, &sm.b_KK, n & 1);
        tc_fence_after();
        {
            float x[64];
            tmem_ld32(tmem + TM_KK + ((uint32_t)(wq * 32) << 16), x);
            tmem_ld32(tmem + TM_KK + 32 + ((uint32_t)(wq * 32) << 16), x + 32);
            tmem_ld_wait();
            const float f = is_q ? f_own : f_own * beta;
            const int last = is_q ? t : t - 1;
            float m = 0.f;
#pragma unroll
            for (int j4 = 0; j4 < 64; j4 += 4) {
                const float4 gh = lds4(sm.Gh + j4), gl = lds4(sm.Gl + j4), fj = lds4(sm.fac + j4);
                const float h[4] = {gh.x, gh.y, gh.z, gh.w}, l[4] = {gl.x, gl.y, gl.z, gl.w}, fk[4] = {fj.x, fj.y, fj.z, fj.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int j = j4 + e;
                    const float d = exp2f((Gh - h[e]) + (Gl - l[e]));
                    // factor by factor: k and q rows may be large where their product is not
                    x[j] = j <= last ? x[j] * fk[e] * f * d : 0.f;
                    m = fmaxf(m, fabsf(x[j]));
                }
            }
            if (is_q) {
                float mul, inv;
                pow2_scale(m, mul, inv);
                put_row<LO>(sm.tp[tp][2], sm.tp[tp][3], t, x, mul);
                sm.fp[tp][t] = inv;
                sm.fqs[tp][t] = decay * f_own;
            } else {
#pragma unroll
                for (int j4 = 0; j4 < 64; j4 += 4) st4(M + tri(t, j4), make_float4(x[j4], x[j4 + 1], x[j4 + 2], x[j4 + 3]));
                sm.fv[tp][t] = beta;
                sm.fks[tp][t] = beta * decay * f_own;
                sm.fw[tp][t] = exp2f((sm.Gh[63] - Gh) + (sm.Gl[63] - Gl)) * f_own;
                if (t == 63) sm.gC[tp] = decay;
            }
        }
        named_sync(5, DC_PREP);
        invert(M, sm.x, r);
        {
            float x[64];
            float m = 0.f;
            if (!is_q) {
#pragma unroll
                for (int j4 = 0; j4 < 64; j4 += 4) {
                    const float4 v = lds4(M + tri(t, j4));
                    x[j4] = v.x, x[j4 + 1] = v.y, x[j4 + 2] = v.z, x[j4 + 3] = v.w;
                }
#pragma unroll
                for (int j = 0; j < 64; ++j) m = fmaxf(m, fabsf(x[j]));
            }
            named_sync(5, DC_PREP);  // the fp32 form has been read: its place takes the parts
            if (!is_q) {
                float mul, inv;
                pow2_scale(m, mul, inv);
                put_row<true>(sm.tp[tp][0], sm.tp[tp][1], t, x, mul);
                sm.fu[tp][t] = inv;
            }
        }
        fence_async_smem();
        tc_fence_before();
        warp_arrive(&sm.b_tp[tp]);

        // the chunk after the next, once the chain is through with the chunk before this one
        if (ahead.there) {
            if (n >= 1) dc_wait(A, sm, &sm.b_free[(n + 2) % DC_KV], ((n - 1) / DC_KV) & 1);
            dc_load<T>(A, sm, ahead, (n + 2) % DC_KV, r);
        }
        cp_async_commit();
        dc_next(A, sm, ahead);
    }
}

// ---- warp 12 ----

template <bool LO>
__device__ __forceinline__ void dc_issue(const DeltaArgs &A, DcSmem &sm, uint32_t tmem)
{
    DcWalk w;
    w.round = 0;
    dc_fetch(A, sm, w);
    const uint32_t i64 = idesc_f16(128, 64, false), i128 = idesc_f16(128, 128, true);
    for (int n = 0; w.there; ++n, dc_next(A, sm, w)) {
        const int st = n % DC_KV, tp = n % DC_TP;
        const uint32_t kq[2] = {smem_addr(sm.kq[st][0]), smem_addr(sm.kq[st][1])};
        // K S
        dc_wait(A, sm, &sm.b_kq[st], (n / DC_KV) & 1);
        dc_wait(A, sm, &sm.b_S, n & 1);
        tc_fence_after();
#pragma unroll
        for (int p = 1; p >= 0; --p)
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
                mma_ts(tmem + TM_A, tmem + TM_S + 64 * p + 8 * ks, sdesc_sw128(kq[ks >> 2] + (ks & 3) * 32, 16, 1024), i64,
                       p == 0 || ks > 0);
        umma_commit(&sm.b_KS);
        // Q S, once the chunk before has read its own
        if (n >= 1) dc_wait(A, sm, &sm.b_out[(n - 1) % DC_TP], ((n - 1) / DC_TP) & 1);
        tc_fence_after();
#pragma unroll
        for (int p = LO ? 1 : 0; p >= 0; --p)
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
                mma_ts(tmem + TM_Q, tmem + TM_S + 64 * p + 8 * ks,
                       sdesc_sw128(kq[ks >> 2] + 64 * 128 + (ks & 3) * 32, 16, 1024), i64, (LO && p == 0) || ks > 0);
        umma_commit(&sm.b_QS);
        // U = T R
        dc_wait(A, sm, &sm.b_R, n & 1);
        tc_fence_after();
        const uint32_t th = smem_addr(sm.tp[tp][0]), tl = smem_addr(sm.tp[tp][1]);
#pragma unroll
        for (int p = 0; p < 3; ++p)  // lo hi, hi lo, hi hi
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
                mma_ts(tmem + TM_A, tmem + TM_R + (p == 0 ? 32 : 0) + 8 * ks, sdesc_sw128((p == 1 ? tl : th) + ks * 32, 16, 1024),
                       i64, p > 0 || ks > 0);
        umma_commit(&sm.b_U);
        // the state's increment: k as the right operand, tokens along K
        dc_wait(A, sm, &sm.b_W, n & 1);
        tc_fence_after();
#pragma unroll
        for (int p = 1; p >= 0; --p)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
                mma_ts(tmem + TM_A, tmem + TM_S + 32 * p + 8 * ks, sdesc_sw128(kq[0] + ks * 2048, 128 * 128, 1024), i128,
                       p == 0 || ks > 0);
        umma_commit(&sm.b_D);
        umma_commit(&sm.b_free[st]);
        // P U
        const uint32_t ph = smem_addr(sm.tp[tp][2]), pl = smem_addr(sm.tp[tp][3]);
#pragma unroll
        for (int p = LO ? 0 : 2; p < 3; ++p)
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
                mma_ts(tmem + TM_PU, tmem + TM_S + 64 + (p == 0 ? 32 : 0) + 8 * ks,
                       sdesc_sw128((p == 1 ? pl : ph) + ks * 32, 16, 1024), i64, (LO && p > 0) || ks > 0);
        umma_commit(&sm.b_PU);
    }
    if (*(volatile int *)&sm.stop) {  // a wait was given up: let what is in flight end before tensor memory goes
        umma_commit(&sm.b_end);
        mbar_wait_bounded(&sm.b_end, 0, DEFAULT_WAIT_CYCLES);
    }
}

// ---- warps 0-7 ----

template <class T, bool LO>
__device__ __forceinline__ void dc_chain(const DeltaArgs &A, DcSmem &sm, uint32_t tmem)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quad = warp & 3, g = warp >> 2;  // lanes 32 quad .. + 31; tokens 32 g .., key rows 64 g ..
    const int col = quad * 32 + lane;
    const uint32_t tm = tmem + ((uint32_t)(quad * 32) << 16);
    int flip = 0;  // which of the two exchange buffers comes next
    // maxima over both halves of this lane's column
    auto both = [&](float &a, float &b) {
        sm.mx[flip][g][0][col] = a;
        sm.mx[flip][g][1][col] = b;
        named_sync(1 + quad, 64);
        a = fmaxf(a, sm.mx[flip][g ^ 1][0][col]);
        b = fmaxf(b, sm.mx[flip][g ^ 1][1][col]);
        flip ^= 1;
    };
    DcWalk w;
    w.round = 0;
    dc_fetch(A, sm, w);
    float S[64];
    float sS = 0.f;  // value of a unit of S's parts
    for (int n = 0; w.there;) {
        const int vw = min(DC_VW, A.V - w.slice * DC_VW);
        const bool own = col < vw;
        const int vcol = w.slice * DC_VW + col;
        float *Sg = A.S + ((w.slot * A.H + w.h) * KDIM + 64 * g) * A.V + vcol;
        // parts of S to tensor memory, once nothing reads what lay there
        auto put_state = [&](bool busy) {
            float m = 0.f, unused = 0.f, mul;
#pragma unroll
            for (int i = 0; i < 64; ++i) m = fmaxf(m, fabsf(S[i]));
            both(m, unused);
            pow2_scale(m, mul, sS);
            if (busy) dc_wait(A, sm, &sm.b_PU, (n - 1) & 1);
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) split2(S[32 * b + 2 * i] * mul, S[32 * b + 2 * i + 1] * mul, hi[i], lo[i]);
                tmem_st16(tm + TM_S + 32 * g + 16 * b, hi);
                tmem_st16(tm + TM_S + 64 + 32 * g + 16 * b, lo);
            }
            tmem_st_wait();
            tc_fence_before();
            warp_arrive(&sm.b_S);
        };
#pragma unroll
        for (int i = 0; i < 64; ++i) S[i] = own ? Sg[(long long)i * A.V] : 0.f;
        put_state(false);

        const int chunks = (w.len + DC_C - 1) / DC_C;
        for (int c = 0; c < chunks; ++c, ++n) {
            const int st = n % DC_KV, tp = n % DC_TP;
            const int left = w.len - c * DC_C;
            const float s_old = sS;
            float x[32];
            float mr = 0.f, unused = 0.f, mul, sR;
            // R
            dc_wait(A, sm, &sm.b_tp[tp], (n / DC_TP) & 1);
            dc_wait(A, sm, &sm.b_KS, n & 1);
            tc_fence_after();
            tmem_ld32(tm + TM_A + 32 * g, x);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const int t = 32 * g + i;
                const uint16_t raw = own ? sm.v[st][t][col] : (uint16_t)0;
                const float2 v = unpack2(raw, (const T *)nullptr);
                x[i] = fmaf(-sm.fks[tp][t], sS * x[i], sm.fv[tp][t] * v.x);
                mr = fmaxf(mr, fabsf(x[i]));
            }
            both(mr, unused);
            pow2_scale(mr, mul, sR);
            {
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) split2(x[2 * i] * mul, x[2 * i + 1] * mul, hi[i], lo[i]);
                tmem_st16(tm + TM_R + 16 * g, hi);
                tmem_st16(tm + TM_R + 32 + 16 * g, lo);
            }
            tmem_st_wait();
            tc_fence_before();
            warp_arrive(&sm.b_R);
            // U, and U as the state takes it
            dc_wait(A, sm, &sm.b_U, n & 1);
            tc_fence_after();
            tmem_ld32(tm + TM_A + 32 * g, x);
            tmem_ld_wait();
            float mu = 0.f, mw = 0.f, sU, sW, mulw;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const int t = 32 * g + i;
                x[i] *= sR * sm.fu[tp][t];
                mu = fmaxf(mu, fabsf(x[i]));
                mw = fmaxf(mw, fabsf(x[i] * sm.fw[tp][t]));
            }
            both(mu, mw);
            pow2_scale(mu, mul, sU);
            pow2_scale(mw, mulw, sW);
            dc_wait(A, sm, &sm.b_QS, n & 1);  // S's parts have been read
            tc_fence_after();
            {
                uint32_t hi[16], lo[16];
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int t = 32 * g + 2 * i;
                    split2(x[2 * i] * sm.fw[tp][t] * mulw, x[2 * i + 1] * sm.fw[tp][t + 1] * mulw, hi[i], lo[i]);
                }
                tmem_st16(tm + TM_S + 16 * g, hi);
                tmem_st16(tm + TM_S + 32 + 16 * g, lo);
#pragma unroll
                for (int i = 0; i < 16; ++i) split2(x[2 * i] * mul, x[2 * i + 1] * mul, hi[i], lo[i]);
                tmem_st16(tm + TM_S + 64 + 16 * g, hi);
                if (LO) tmem_st16(tm + TM_S + 96 + 16 * g, lo);
            }
            tmem_st_wait();
            tc_fence_before();
            warp_arrive(&sm.b_W);
            // the new state
            const float gC = sm.gC[tp];
            dc_wait(A, sm, &sm.b_D, n & 1);
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                tmem_ld32(tm + TM_A + 64 * g + 32 * b, x);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i) S[32 * b + i] = fmaf(sW, x[i], gC * S[32 * b + i]);
            }
            ++n;
            if (c + 1 < chunks)
                put_state(true);
            else
                dc_wait(A, sm, &sm.b_PU, (n - 1) & 1);
            --n;
            // the outputs, while the next chunk's K S runs
            tc_fence_after();
            float q[32];
            tmem_ld32(tm + TM_Q + 32 * g, q);
            tmem_ld32(tm + TM_PU + 32 * g, x);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const int t = 32 * g + i;
                x[i] = fmaf(s_old * sm.fqs[tp][t], q[i], sU * sm.fp[tp][t] * x[i]);
            }
            tc_fence_before();
            warp_arrive(&sm.b_out[tp]);
            if (own) {
                T *yp = static_cast<T *>(A.y) + (w.first + (long long)c * DC_C + 32 * g) * A.y_stride + (long long)w.h * A.V + vcol;
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    if (32 * g + i < left) store1(yp + i * A.y_stride, x[i]);
            }
        }
        if (own) {
#pragma unroll
            for (int i = 0; i < 64; ++i) Sg[(long long)i * A.V] = S[i];
        }
        ++w.round;
        dc_fetch(A, sm, w);
    }
}

// The order in which sequences are taken (longest first) and those whose slot an earlier one
// names; block 0 reports bad ones.
__device__ __forceinline__ void dc_order(const DeltaArgs &A, DcSmem &sm)
{
    for (int i = threadIdx.x; i < (A.rows + 31) / 32; i += DC_THREADS) sm.dup[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < A.rows; i += DC_THREADS) {
        const int c0 = __ldg(A.cu + i), c1 = __ldg(A.cu + i + 1), slot = A.slot ? __ldg(A.slot + i) : i;
        const int len = c1 - c0;
        int rank = 0;
        bool dup = false;
        int d0 = __ldg(A.cu);
        for (int j = 0; j < A.rows; ++j) {
            const int d1 = __ldg(A.cu + j + 1), other = d1 - d0;
            d0 = d1;
            rank += other > len || (other == len && j < i);
            if (A.slot && j < i) dup = dup || __ldg(A.slot + j) == slot;
        }
        dup = dup && slot >= 0;
        sm.order[rank] = (uint16_t)i;
        if (dup) atomicOr(&sm.dup[i >> 5], 1u << (i & 31));
        const bool bad = c0 < 0 || c1 < c0 || c1 > A.tokens;
        if (blockIdx.x == 0 && (bad || (len > 0 && slot >= 0 && (dup || slot >= A.slots))))
            atomicOr(A.status, SK_STATUS_BAD_ROW);
    }
}

template <class T, bool LO>
__global__ void __launch_bounds__(DC_THREADS, 1) delta_chunk_kernel(const DeltaArgs A)
{
    extern __shared__ __align__(1024) unsigned char raw_smem[];
    DcSmem &sm = *reinterpret_cast<DcSmem *>(raw_smem);
    const int warp = threadIdx.x >> 5;
    if (warp == 0) {
        tmem_alloc(&sm.taddr, 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        sm.stop = 0;
        for (int i = 0; i < DC_KV; ++i) {
            mbar_init(&sm.b_kq[i], DC_PREP / 32);
            mbar_init(&sm.b_free[i], 1);
        }
        for (int i = 0; i < DC_TP; ++i) {
            mbar_init(&sm.b_tp[i], DC_PREP / 32);
            mbar_init(&sm.b_out[i], DC_CHAIN / 32);
        }
        mbar_init(&sm.b_S, DC_CHAIN / 32);
        mbar_init(&sm.b_R, DC_CHAIN / 32);
        mbar_init(&sm.b_W, DC_CHAIN / 32);
        mbar_init(&sm.b_KS, 1);
        mbar_init(&sm.b_QS, 1);
        mbar_init(&sm.b_U, 1);
        mbar_init(&sm.b_D, 1);
        mbar_init(&sm.b_PU, 1);
        mbar_init(&sm.b_KK, 1);
        mbar_init(&sm.b_end, 1);
        mbar_fence_init();
    }
    dc_order(A, sm);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sm.taddr;
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(DC_REG_CHAIN));
        dc_chain<T, LO>(A, sm, tmem);
    } else if (warp < 12) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(DC_REG_PREP));
        dc_prep<T, LO>(A, sm, tmem);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(DC_REG_ISSUE));
        if (threadIdx.x == DC_CHAIN + DC_PREP) dc_issue<LO>(A, sm, tmem);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

template <class T, bool LO>
cudaError_t launch_type(const DeltaArgs &a, int sms, cudaStream_t stream)
{
    const long long items = (long long)a.rows * a.H * ((a.V + DC_VW - 1) / DC_VW);
    cudaError_t e = cudaFuncSetAttribute(delta_chunk_kernel<T, LO>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)sizeof(DcSmem));
    if (e != cudaSuccess) return e;
    delta_chunk_kernel<T, LO><<<(unsigned)(items < sms ? items : sms), DC_THREADS, sizeof(DcSmem), stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

bool delta_chunk_fits(const DeltaArgs &a)
{
    return a.cu && a.dtype != SKETCHSSM_F32 && a.rows <= DC_MAX_SEQS;
}

cudaError_t launch_delta_chunk(const DeltaArgs &a, int sms, cudaStream_t stream)
{
    return a.dtype == SKETCHSSM_BF16 ? launch_type<__nv_bfloat16, true>(a, sms, stream)
                                     : launch_type<__half, true>(a, sms, stream);
}

}  // namespace sk
