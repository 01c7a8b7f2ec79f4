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
// one each in 8 lanes with 7 shuffles.  States are fp32 and every sum is taken in fp32.
//
// A row whose slot or bounds are bad, or whose slot an earlier row names too, is left
// alone and reported through the plan's status word; a negative slot is padding.
#include <climits>

#include "device_util.cuh"
#include "dtype_util.cuh"
#include "internal.cuh"
#include "ptx_util.cuh"
#include "wait_rule.cuh"

namespace sk {
namespace {

constexpr int DELTA_MAXVS = 80;  // columns of a slab at most
constexpr int DELTA_AHEAD = 4;   // tokens between a line's way into L2 and its use
// Most sequences that are taken longest first: each CTA ranks them by itself.  (32 heads of 128,
// in order / longest first: 24 of 1500 tokens 311 / 265 us, 64 of 1280 243 / 235, 64 of 6400
// 982 / 907; 100 of 900 220 / 232.)
constexpr int DELTA_SORT = 64;

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

// The sequence of rank `r` by length, longest first (up to DELTA_SORT of them).
__device__ __forceinline__ int delta_ranked(const DeltaArgs &A, int r)
{
    __shared__ int4 len4[DELTA_SORT / 4];
    __shared__ int found;
    int *len = reinterpret_cast<int *>(len4);
    for (int i = threadIdx.x; i < (A.rows + 3) / 4 * 4; i += blockDim.x)
        len[i] = i < A.rows ? (int)((unsigned)__ldg(A.cu + i + 1) - (unsigned)__ldg(A.cu + i))  // (bad bounds may be any numbers)
                            : INT_MIN;
    __syncthreads();
    for (int i = threadIdx.x; i < A.rows; i += blockDim.x) {
        const int mine = len[i];
        int rank = 0;
        for (int j = 0; j < A.rows; j += 4) {
            const int4 o = len4[j / 4];
            rank += (o.x > mine || (o.x == mine && j < i)) + (o.y > mine || (o.y == mine && j + 1 < i)) +
                    (o.z > mine || (o.z == mine && j + 2 < i)) + (o.w > mine || (o.w == mine && j + 3 < i));
        }
        if (rank == r) found = i;
    }
    __syncthreads();
    return found;
}

// A token's rows as this thread needs them, as they came: 16 values of k and q, 4 of v, a, beta.
template <class T>
struct DeltaToken {
    typename Raw4<T>::type k[4], q[4], v;
    float a, beta;
};

template <class T>
__device__ __forceinline__ void delta_load(const DeltaArgs &A, long long t, int h, int hq, int ks, int col, DeltaToken<T> &x)
{
    const T *k = static_cast<const T *>(A.k) + t * A.k_stride + hq * KDIM + 4 * ks;
    const T *q = static_cast<const T *>(A.q) + t * A.q_stride + hq * KDIM + 4 * ks;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x.k[i] = load4_raw(k + 32 * i);
        x.q[i] = load4_raw(q + 32 * i);
    }
    x.v = load4_raw(static_cast<const T *>(A.v) + t * A.v_stride + (long long)h * A.V + col);
    x.a = __ldg(A.a + t * A.H + h);
    x.beta = __ldg(A.beta + t * A.H + h);
}

// The pair i (rows 2 i, 2 i + 1) of this thread's 16 values of q or k.
template <class T>
__device__ __forceinline__ float2 pair_of(const typename Raw4<T>::type (&x)[4], int i)
{
    const float4 w = values(x[i >> 1], (const T *)nullptr);
    return i & 1 ? make_float2(w.z, w.w) : make_float2(w.x, w.y);
}

// One token: y written (by the lanes with bit 0 of the row slice set), the state s moved on; s[i][c]: the
// rows 2 i, 2 i + 1 of column c, so that packed products take pairs of k and q as they are.  y: this
// thread's 4 columns.
template <class T>
__device__ __forceinline__ void delta_token(const DeltaArgs &A, const DeltaToken<T> &c, float2 (&s)[8][4], T *y)
{
    constexpr unsigned FULL = 0xffffffffu;
    const int lane = threadIdx.x & 31, ks = lane & 7;
    const float4 cv = values(c.v, (const T *)nullptr);
    float2 kk2 = make_float2(0.f, 0.f), qq2 = kk2, qk2 = kk2, d2[4] = {}, p2[4] = {};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float2 k = pair_of<T>(c.k, i), q = pair_of<T>(c.q, i);
        kk2 = __ffma2_rn(k, k, kk2);
        qq2 = __ffma2_rn(q, q, qq2);
        qk2 = __ffma2_rn(q, k, qk2);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            d2[e] = __ffma2_rn(k, s[i][e], d2[e]);
            p2[e] = __ffma2_rn(q, s[i][e], p2[e]);
        }
    }
    float kk = kk2.x + kk2.y, qq = qq2.x + qq2.y, qk = qk2.x + qk2.y;
    const float4 d = make_float4(d2[0].x + d2[0].y, d2[1].x + d2[1].y, d2[2].x + d2[2].y, d2[3].x + d2[3].y);
    const float4 p = make_float4(p2[0].x + p2[0].y, p2[1].x + p2[1].y, p2[2].x + p2[2].y, p2[3].x + p2[3].y);
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
    const float vc = b1 ? (b2 ? cv.w : cv.z) : (b2 ? cv.y : cv.x);
    float u = c.beta * (vc - c.a * rk * sum);
    u = __shfl_sync(FULL, u, lane & ~1);
    if (b0) store1(y + (b1 ? 2 : 0) + (b2 ? 1 : 0), rq * fmaf(c.a, sum, rk * qk * u));
    const int base = lane & ~7;
    const int from[4] = {0, 4, 2, 6};
    const float2 a2 = make_float2(c.a, c.a);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float ue = rk * __shfl_sync(FULL, u, base + from[e]);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            s[i][e] = __ffma2_rn(pair_of<T>(c.k, i), make_float2(ue, ue), __fmul2_rn(a2, s[i][e]));
    }
}

// Sequences, and single tokens of few rows: one CTA of 2 VS threads per (row, head, slab); the next
// token's rows are loaded before this token's products, and the lines of tokens further ahead are
// brought into L2.  32 heads of 128, fp32: one prompt of 500 tokens 214 us, 0.43 us a token, which its
// 370 instructions and their latencies bound; 24 prompts of 1500 tokens in all 265 us.  Without the
// lines brought ahead 282 and 315 us; in the order that the prompts come in 311 for the 24; with a
// column's rows one by one 282 and 334.  Tokens seven ahead in shared memory, two ahead in
// registers, two a turn of the loop, or 8 state rows a thread were slower.
template <class T>
__global__ void __launch_bounds__(DELTA_MAXVS * 2, 2) delta_kernel(const DeltaArgs A)
{
    const int nslab = A.V / A.VS;
    const long long item = blockIdx.x;
    const int slab = (int)(item % nslab);
    const int h = (int)(item / nslab % A.H);
    int row = (int)(item / nslab / A.H);
    if (A.sort) row = delta_ranked(A, row);
    const int hq = h / A.hpq;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int ks = lane & 7, col = slab * A.VS + (warp * 4 + (lane >> 3)) * 4;
    long long first, slot;
    int len;
    if (!delta_row(A, row, first, len, slot)) return;

    float *Sg = A.S + ((slot * A.H + h) * KDIM + 4 * ks) * A.V + col;
    float2 s[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float *r = Sg + (long long)(32 * (i >> 1) + 2 * (i & 1)) * A.V;
        const float4 x = *reinterpret_cast<const float4 *>(r), z = *reinterpret_cast<const float4 *>(r + A.V);
        s[i][0] = make_float2(x.x, z.x);
        s[i][1] = make_float2(x.y, z.y);
        s[i][2] = make_float2(x.z, z.z);
        s[i][3] = make_float2(x.w, z.w);
    }
    DeltaToken<T> x;
    delta_load<T>(A, first, h, hq, ks, col, x);
    T *y = static_cast<T *>(A.y) + first * A.y_stride + (long long)h * A.V + col;
    // lanes 0-11 of the first warp bring the lines of tokens further ahead into L2: 4 pieces of k and of
    // q, 2 of v, a and beta
    const char *ahead = nullptr;
    long long ahead_step = 0;
    if (len > DELTA_AHEAD && warp == 0 && lane < 12) {
        const int part = lane < 8 ? lane >> 2 : lane < 10 ? 2 : lane - 7, piece = lane < 8 ? lane & 3 : lane & 1;
        const long long width = part < 2 ? KDIM / 4 : A.VS / 2;
        ahead_step = (part == 0 ? A.k_stride : part == 1 ? A.q_stride : part == 2 ? A.v_stride : A.H) *
                     (part < 3 ? (long long)sizeof(T) : 4);
        ahead = part < 2 ? (const char *)(part ? A.q : A.k) + (hq * KDIM + piece * width) * sizeof(T)
                : part == 2 ? (const char *)A.v + ((long long)h * A.V + slab * A.VS + piece * width) * sizeof(T)
                            : (const char *)((part == 3 ? A.a : A.beta) + h);
        ahead += (first + DELTA_AHEAD) * ahead_step;
    }
    for (int t = 0; t < len; ++t, y += A.y_stride) {
        const DeltaToken<T> c = x;
        if (t + 1 < len) delta_load<T>(A, first + t + 1, h, hq, ks, col, x);
        if (ahead && t + DELTA_AHEAD < len) asm volatile("prefetch.global.L2 [%0];" ::"l"(ahead));
        ahead += ahead_step;
        delta_token<T>(A, c, s, y);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float *r = Sg + (long long)(32 * (i >> 1) + 2 * (i & 1)) * A.V;
        st4(r, make_float4(s[i][0].x, s[i][1].x, s[i][2].x, s[i][3].x));
        st4(r + A.V, make_float4(s[i][0].y, s[i][1].y, s[i][2].y, s[i][3].y));
    }
}

// Single tokens of many rows: the states are all that counts, so the kernel is a stream of them.
// Persistent CTAs of 8 warps, one per SM, take runs of neighbouring (row, head) items; a state of
// up to 128 columns is one bulk copy, and three of them are on their way or in use, so that some
// 128 KB a CTA are always in flight.  A warp has 16 rows of the state, a lane 4 columns of each:
// every access is a run of whole lines.  512 rows of 32 heads of 128, bf16: 350 us,
// 6.2 TB/s of states and tokens, 0.94 of the measured copy rate.  (The kernel
// above takes 556 us for them, its layout with the next item's state loaded into registers 548 us; an
// item index in 64 bits, whose divisions every thread waits for, cost 45 us.)
constexpr int DS_THREADS = 256, DS_STAGES = 3, DS_VW = 128, DS_LEAST_V = 64;

struct DsSmem {
    float part[2][8][2][DS_VW];  // the warps' shares of k^T S and q^T S
    uint64_t full[DS_STAGES];
    int slot[DS_STAGES], first[DS_STAGES];  // slot -1: a row to leave alone
};

// 16 values of a row that all lanes of a warp want
template <class T>
struct Row16 {
    uint4 w[sizeof(T)];
};
template <class T>
__device__ __forceinline__ void row16_load(const T *p, Row16<T> &x)
{
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) x.w[i] = __ldg(reinterpret_cast<const uint4 *>(p) + i);
}
__device__ __forceinline__ void row16_get(const Row16<float> &x, int i, float (&f)[4])  // values 4 i ..
{
    f[0] = __uint_as_float(x.w[i].x), f[1] = __uint_as_float(x.w[i].y), f[2] = __uint_as_float(x.w[i].z), f[3] = __uint_as_float(x.w[i].w);
}
template <class T>
__device__ __forceinline__ void row16_get(const Row16<T> &x, int i, float (&f)[4])
{
    const uint4 w = x.w[i >> 1];
    const float2 a = unpack2(i & 1 ? w.z : w.x, (const T *)nullptr), b = unpack2(i & 1 ? w.w : w.y, (const T *)nullptr);
    f[0] = a.x, f[1] = a.y, f[2] = b.x, f[3] = b.y;
}

template <class T>
__global__ void __launch_bounds__(DS_THREADS, 1) delta_step_kernel(const DeltaArgs A)
{
    extern __shared__ __align__(128) unsigned char raw[];
    DsSmem &sm = *reinterpret_cast<DsSmem *>(raw);
    float *states = reinterpret_cast<float *>(raw + (sizeof(DsSmem) + 127) / 128 * 128);
    const int V = A.V;
    const int items = A.rows * A.H;  // the host has checked that it fits
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r0 = warp * 16;
    const bool on = 4 * lane < V;
    const int from = (int)((long long)items * blockIdx.x / gridDim.x), to = (int)((long long)items * (blockIdx.x + 1) / gridDim.x);
    if (threadIdx.x == 0) {
        for (int i = 0; i < DS_STAGES; ++i) mbar_init(&sm.full[i], 1);
        mbar_fence_init();
    }
    __syncthreads();

    // item i's state on its way to its stage (all threads: a new row's slot is checked together)
    int row = -1;
    long long first = 0, slot = 0;
    bool good = false;
    RingPhases ring;
    auto bring = [&](int i) {
        const int st = (i - from) % DS_STAGES;
        const int r = i / A.H, h = i - r * A.H;
        if (r != row) {
            int len;
            row = r;
            good = delta_row(A, row, first, len, slot);
        }
        if (good) ring.issued(st);
        if (warp == 0) {
            if (lane == 0) {
                sm.slot[st] = good ? (int)slot : -1;
                sm.first[st] = (int)first;
                if (good) mbar_arrive_expect_tx(&sm.full[st], (uint32_t)(KDIM * V * 4));
            }
            __syncwarp();
            if (good && lane < KDIM / 8)  // 8 rows a copy: 4% faster than one copy
                bulk_copy_g2s(states + (st * KDIM + 8 * lane) * V, A.S + ((slot * A.H + h) * KDIM + 8 * lane) * V,
                              (uint32_t)(8 * V * 4), &sm.full[st]);
        }
    };
    for (int i = from; i < from + DS_STAGES && i < to; ++i) bring(i);
    __syncthreads();

    for (int i = from; i < to; ++i) {
        const int st = (i - from) % DS_STAGES, pb = (i - from) & 1;
        const int h = i % A.H, col = 4 * lane;
        const int sl = sm.slot[st];
        const long long tok = sm.first[st];
        float4 s[16], v = zero4();
        Row16<T> kr, qr;
        float qk = 0.f, kk = 0.f, qq = 0.f, a = 0.f, beta = 0.f;
        bool lost = false;
        if (sl >= 0) {
            const T *k = static_cast<const T *>(A.k) + tok * A.k_stride + h / A.hpq * KDIM;
            const T *q = static_cast<const T *>(A.q) + tok * A.q_stride + h / A.hpq * KDIM;
            row16_load(k + r0, kr);
            row16_load(q + r0, qr);
            const float4 k4 = values(load4_raw(k + 4 * lane), (const T *)nullptr);
            const float4 q4 = values(load4_raw(q + 4 * lane), (const T *)nullptr);
            if (on) v = values(load4_raw(static_cast<const T *>(A.v) + tok * A.v_stride + (long long)h * A.V + col), (const T *)nullptr);
            a = __ldg(A.a + tok * A.H + h);
            beta = __ldg(A.beta + tok * A.H + h);
            kk = warp_sum(dot4(k4, k4));
            qq = warp_sum(dot4(q4, q4));
            qk = warp_sum(dot4(q4, k4));
            if (!mbar_wait_bounded(&sm.full[st], ring.parity(st), A.wait_limit)) {
                atomicOr(A.status, SK_STATUS_DELTA_TIMEOUT);
                lost = !mbar_wait_bounded(&sm.full[st], ring.parity(st), DEFAULT_WAIT_CYCLES);
            }
            if (!lost) ring.landed(st);
            const float *src = states + (size_t)st * KDIM * V + r0 * V + 4 * lane;
            float4 d = zero4(), p = zero4();
            if (on) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float kf[4], qf[4];
                    row16_get(kr, j, kf);
                    row16_get(qr, j, qf);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[4 * j + e] = lds4(src + (4 * j + e) * V);
                        fma4(d, kf[e], s[4 * j + e]);
                        fma4(p, qf[e], s[4 * j + e]);
                    }
                }
                st4(&sm.part[pb][warp][0][4 * lane], d);
                st4(&sm.part[pb][warp][1][4 * lane], p);
            }
        }
        if (__syncthreads_or(lost)) {
            // given up: let the copies still on their way, the lost one among them, land (bounded)
            // before the CTA exits
            if (threadIdx.x == 0)
                for (int j = 0; j < DS_STAGES; ++j)
                    if (ring.pending(j)) mbar_wait_bounded(&sm.full[j], ring.parity(j), DEFAULT_WAIT_CYCLES);
            __syncthreads();
            return;
        }
        if (i + DS_STAGES < to) bring(i + DS_STAGES);
        if (sl >= 0 && on) {
            float4 d = zero4();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float4 x = lds4(&sm.part[pb][j][0][4 * lane]);
                d.x += x.x, d.y += x.y, d.z += x.z, d.w += x.w;
            }
            const float rk = A.normalize ? rsqrtf(kk + DELTA_QK_EPS) : 1.f;
            const float rq = A.scale * (A.normalize ? rsqrtf(qq + DELTA_QK_EPS) : 1.f);
            const float ar = a * rk;
            const float4 u = make_float4(beta * (v.x - ar * d.x), beta * (v.y - ar * d.y), beta * (v.z - ar * d.z),
                                         beta * (v.w - ar * d.w));
            float *Sg = A.S + (((long long)sl * A.H + h) * KDIM + r0) * A.V + col;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float kf[4];
                row16_get(kr, j, kf);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float f = rk * kf[e];
                    const float4 x = s[4 * j + e];
                    st4(Sg + (long long)(4 * j + e) * A.V, make_float4(fmaf(f, u.x, a * x.x), fmaf(f, u.y, a * x.y),
                                                                      fmaf(f, u.z, a * x.z), fmaf(f, u.w, a * x.w)));
                }
            }
            if (warp == (i & 7)) {
                float4 p = zero4();
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float4 x = lds4(&sm.part[pb][j][1][4 * lane]);
                    p.x += x.x, p.y += x.y, p.z += x.z, p.w += x.w;
                }
                const float f = rk * qk;
                store4(static_cast<T *>(A.y) + tok * A.y_stride + (long long)h * A.V + col,
                       make_float4(rq * fmaf(a, p.x, f * u.x), rq * fmaf(a, p.y, f * u.y), rq * fmaf(a, p.z, f * u.z),
                                   rq * fmaf(a, p.w, f * u.w)));
            }
        }
    }
}

template <class T>
cudaError_t launch_type(const DeltaArgs &a, int sms, cudaStream_t stream)
{
    const long long states = (long long)a.rows * a.H;
    // One token a row and states of 64 to 128 columns go through the stream of states, but for the
    // fewest.  First kernel / stream, us: 32 heads of 128, bf16: one row 4.4 / 4.9; 2: 4.6 / 4.9; 4: 6.9 /
    // 5.1; 128: 141 / 95; 512: 556 / 350.  400 rows of 32 heads, by columns: 16: 62 / 188; 32: 113 / 191;
    // 48: 161 / 197; 64: 220 / 210; 80: 314 / 225; 96: 315 / 242 (fp32 within 5%): below 64 columns half the
    // stream's lanes idle.  Wider states would be streamed by slabs, a copy for each of their rows: 320
    // states of 256 columns took 34 us that way, 28 by the first kernel.
    if (a.cu || a.V < DS_LEAST_V || a.V > DS_VW || 2 * states <= sms) {
        DeltaArgs A = a;
        A.sort = a.cu && a.rows > 1 && a.rows <= DELTA_SORT && states * (a.V / a.VS) > sms;
        delta_kernel<T><<<(unsigned)(states * (a.V / a.VS)), 2 * a.VS, 0, stream>>>(A);
    } else {
        const size_t head = (sizeof(DsSmem) + 127) / 128 * 128, column = (size_t)DS_STAGES * KDIM * 4;
        const size_t smem = head + column * a.V;
        // the limit belongs to the function, which other threads launch for other sizes: always the largest
        cudaError_t e = cudaFuncSetAttribute(delta_step_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)(head + column * DS_VW));
        if (e != cudaSuccess) return e;
        delta_step_kernel<T><<<(unsigned)(states < sms ? states : sms), DS_THREADS, smem, stream>>>(a);
    }
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta(const DeltaArgs &a, int sms, cudaStream_t stream)
{
    if (a.rows == 0) return cudaSuccess;
    switch (a.dtype) {
    case SKETCHSSM_BF16: return launch_type<__nv_bfloat16>(a, sms, stream);
    case SKETCHSSM_F16: return launch_type<__half>(a, sms, stream);
    default: return launch_type<float>(a, sms, stream);
    }
}

}  // namespace sk
