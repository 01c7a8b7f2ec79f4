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
// One CTA per (sequence, head, slice of 128 value columns), persistent, one per SM.  Everything
// on the chain is taken transposed: tensor-memory lane = value column.  A column's state (fp32)
// lives in the registers of two threads, its 64 token values pass through them, and the left
// operands S^T, R^T, U^T are written straight into tensor memory, with no shared memory, no
// transposition and no sum across threads.
//   warps 0-7   the chain: warps w and w + 4 share 32 lanes (columns), each half the tokens
//               (or key rows);
//   warps 8-11  one chunk ahead: q and k as operands, A, P and T;
//   warp 12     issues the chain's MMAs;
//   warp 13     writes the outputs, 14 forms the decays, 15 brings q, k and v (tensor copies).
//
// Precision.  The state is held in fp32, and after any prompt its error is 1e-7 to 3e-7 (2-norm of a head).
// Every operand x but q and k is split into two fp16 parts, x = 2^-e (hi + lo) (1 + 2^-22), e from the
// largest value of its row (or column), and products are taken hi hi + hi lo + lo hi in fp32; q and k, 8 or
// 11 bits wide, go into fp16 after a row's power of two (bf16 values below 2^-31 of the row's largest
// lose bits there).  Decays are off by 2^-22, products of two factors by twice that.  (fp16 pairs hold
// 22 bits where bf16 pairs hold 16, and bf16 triples hold 24 for half as many products again.)  y is
// rounded once.
//
// What bounds it.  A chunk takes 9,400 SM cycles (of them 2,560 of MMAs), 10,300 with all SMs at work.
// The preparation sets that pace: it waits 600 of them, the chain waits 1,250 for it.  Both wait for
// instructions more than for anything else: 2.4 of 6 stall cycles an issued instruction.  A chunk runs
// some 60 KB of straight code in six roles, where straight code beyond 32 KB came at 5.7 cycles an
// instruction and SM in a loop of nothing else.  Loops in its place (re-reading tensor memory, or the
// triangular products in one loop) traded that for latency and were slower at one sequence.  One sequence
// of 8192 tokens, 32 heads of 128, bf16: 638 us (32 of 148 SMs have work); 16 sequences of 8192 in all:
// 259 us; 48 of 32768: 931 us, 4.7 times what HBM needs for the bytes.  Token by token: 4705, 1193
// and 4339 us.  Slower were: 16 chain warps with half the work each (1044 us for the one sequence),
// T by a warp group of its own (758), rows of q, k and v by bulk copies of 128 and 256 bytes (the copy
// engine takes some 60 cycles a copy).
#include <cuda.h>

#include <cstddef>

#include "device_util.cuh"
#include "dtype_util.cuh"
#include "internal.cuh"
#include "ptx_util.cuh"
#include "wait_rule.cuh"

namespace sk {
namespace {

constexpr int DC_C = 64;        // tokens of a chunk
constexpr int DC_VW = 128;      // value columns of a slice
constexpr int DC_CHAIN = 256, DC_PREP = 128;
constexpr int DC_THREADS = DC_CHAIN + DC_PREP + 128;
// registers a thread after the split: 256 x 168 + 128 x 120 + 128 x 56 = 512 x 128
constexpr int DC_REG_CHAIN = 168, DC_REG_PREP = 120, DC_REG_HELP = 56;
constexpr int DC_KV = 3;        // stages of q and k; everything else has two
constexpr int DC_MOST_POLLS = 50000;  // about a second
constexpr float DC_STRONG = 100.f;  // exponents of a chunk's decays within which 2^(G_i - G_j) factors

// tensor memory columns
constexpr uint32_t TM_A = 0;     // K S^T, then U^T (64); with the next 64: the state's increment
constexpr uint32_t TM_Q = 128;   // Q S^T (64)
constexpr uint32_t TM_PU = 192;  // P U (64)
constexpr uint32_t TM_S = 256;   // S hi, lo (64 each); then U~ hi, lo (32 each)
constexpr uint32_t TM_R = 384;   // R hi, lo (32 each); then U hi, lo
constexpr uint32_t TM_KK = 448;  // [K; Q] K^T (64)

struct DcMaps {
    CUtensorMap q, k, v, y;
};

struct DcSmem {
    // 1024-byte aligned operand tiles, rows of 128 bytes, 128-byte swizzle
    uint8_t kq[DC_KV][2][128 * 128];  // k dims 0-63 | 64-127; rows 0-63 k, 64-127 q
    uint8_t tp[2][4][64 * 128];       // T hi, T lo, P hi, P lo
    float m[64][68];                  // A, then T, in fp32
    uint16_t v[2][DC_C][DC_VW];       // values, then outputs
    // per token: factors of v and K S in R; of U; of U for the state; of Q S; of P U
    float fv[2][DC_C], fks[2][DC_C], fu[2][DC_C], fw[2][DC_C], fqs[2][DC_C], fp[2][DC_C];
    // per token: beta; 2^G; 2^(G_63 - G); 2^(G - G_31) and its inverse; G, high and low part
    float beta[2][DC_C], dec[2][DC_C], rest[2][DC_C], er[2][DC_C], ec[2][DC_C], gh[2][DC_C], gl[2][DC_C];
    float col[DC_C];                  // factor of k_j in A and P
    float x[32][36];                  // products on the way to T
    uint32_t mx[2][2][DC_VW];         // column maxima of the two chain halves, two upper halves of fp32
    float gC[2];                      // the whole chunk's decay
    int strong[2];
    uint64_t b_ld[DC_KV], b_free[DC_KV], b_kq[DC_KV], b_v[2], b_vfree[2], b_sc[2], b_tp[2], b_out[2];
    uint64_t b_S, b_KS, b_QS, b_R, b_U, b_W, b_D, b_PU, b_KK, b_end;
    uint32_t taddr;
    int polls, late;                  // polls until a wait is late (negative: one has been given up); whether one was
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

// The whole warp runs the code around an MMA and one lane (`leads`) issues it: addresses and
// descriptors then stay in uniform registers (an MMA every 32 cycles at N = 64; 47 from a branch
// that one lane takes).
__device__ __forceinline__ uint32_t elect_lane()
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(r));
    return r;
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

// 16 columns
__device__ __forceinline__ void tmem_ld16n(uint32_t addr, float *x)
{
    uint32_t *r = reinterpret_cast<uint32_t *>(x);
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(addr)
                 : "memory");
}

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

// hi and lo fp16 parts of two scaled values: four instructions, the differences in fp32 straight
// from the halves
__device__ __forceinline__ void split2(float2 v, uint32_t &hi, uint32_t &lo)
{
    hi = h2_bits(__float22half2_rn(v));
    float2 d;
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tsub.rn.f32.f16 %0, l, %3;\n\tsub.rn.f32.f16 %1, u, %4;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "r"(hi), "f"(v.x), "f"(v.y));
    lo = h2_bits(__float22half2_rn(make_float2(-d.x, -d.y)));
}

// s + sum of the squares of two packed values
__device__ __forceinline__ float add_squares(uint32_t v, float s, const __nv_bfloat16 *)
{
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tfma.rn.f32.bf16 %0, l, l, %0;\n\tfma.rn.f32.bf16 %0, u, u, %0;\n\t}"
        : "+f"(s)
        : "r"(v));
    return s;
}
__device__ __forceinline__ float add_squares(uint32_t v, float s, const __half *)
{
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tfma.rn.f32.f16 %0, l, l, %0;\n\tfma.rn.f32.f16 %0, u, u, %0;\n\t}"
        : "+f"(s)
        : "r"(v));
    return s;
}

// two packed bf16 values times a power of two, as fp16
__device__ __forceinline__ uint32_t scale_to_half(uint32_t v, uint32_t mul)
{
    float2 d;
    asm("{\n\t.reg .b16 l, u, m, n;\n\tmov.b32 {l, u}, %2;\n\tmov.b32 {n, m}, %3;\n\t"
        "fma.rn.f32.bf16 %0, l, m, 0f00000000;\n\tfma.rn.f32.bf16 %1, u, m, 0f00000000;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "r"(v), "r"(mul));
    return h2_bits(__float22half2_rn(d));
}

// max(m, |v.x|, |v.y|), m not negative
__device__ __forceinline__ float max3(float m, float2 v)
{
    float r;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(v.x), "f"(v.y));
    return r;
}

__device__ __forceinline__ float2 two(float x) { return make_float2(x, x); }

// two neighbouring values of a per-token array in shared memory, four at a time
struct Four {
    float2 a, b;
};
__device__ __forceinline__ Four lds_four(const float *p)
{
    const float4 v = lds4(p);
    return {make_float2(v.x, v.y), make_float2(v.z, v.w)};
}

__device__ __forceinline__ float ex2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ---- which chunk comes next ----

static_assert(sizeof(DcSmem) <= 232448, "shared memory of one CTA");
static_assert(offsetof(DcSmem, kq) % 1024 == 0 && offsetof(DcSmem, tp) % 1024 == 0 &&
                  offsetof(DcSmem, m) == offsetof(DcSmem, tp) + sizeof(DcSmem::tp), "swizzled tiles");
static_assert(offsetof(DcSmem, m) % 16 == 0 && offsetof(DcSmem, v) % 16 == 0 && offsetof(DcSmem, fv) % 16 == 0 &&
                  offsetof(DcSmem, beta) % 16 == 0 && offsetof(DcSmem, col) % 16 == 0 && offsetof(DcSmem, b_ld) % 8 == 0,
              "vector accesses");

struct DcWalk {
    int item;           // in this CTA's order
    int chunk;          // of the item
    int h, slice, len, first, slot;
    bool there;
};

__device__ __forceinline__ void dc_fetch(const DeltaArgs &A, const DcSmem &sm, DcWalk &w)
{
    const unsigned nslice = (unsigned)(A.V + DC_VW - 1) / DC_VW, per = A.H * nslice;
    const unsigned items = A.rows * per, G = gridDim.x;
    w.chunk = 0;
    w.there = false;
#pragma unroll 1
    for (;; ++w.item) {
        // items go round back and forth, so that a CTA that gets a longer one gets a shorter
        // one next
        const unsigned base = w.item * G;
        if (base >= items) return;
        const unsigned k = base + ((w.item & 1) ? G - 1 - blockIdx.x : blockIdx.x);
        if (k >= items) continue;
        const int row = sm.order[k / per], rest = (int)(k % per);
        w.first = __ldg(A.cu + row);
        const int end = __ldg(A.cu + row + 1);
        w.slot = A.slot ? __ldg(A.slot + row) : A.before + row;
        if (w.first < 0 || end <= w.first || end > A.tokens || w.slot < 0 || w.slot >= A.slots ||
            (sm.dup[row >> 5] >> (row & 31) & 1))
            continue;
        w.len = end - w.first;
        w.h = rest / nslice;
        w.slice = rest - w.h * nslice;
        w.there = true;
        return;
    }
}

__device__ __forceinline__ void dc_start(DcWalk &w)
{
    w.item = -1;
    w.chunk = w.len = 0;
    w.there = true;
}

// the next chunk of this CTA (the first one after dc_start)
__device__ __forceinline__ void dc_next(const DeltaArgs &A, const DcSmem &sm, DcWalk &w)
{
    if (!w.there || ++w.chunk * DC_C < w.len) return;
    ++w.item;
    dc_fetch(A, sm, w);
}

// ---- waits: a number of polls of up to 20 us each; past the plan's limit recorded, past the
// default limit given up.  Then no wait that begins polls any more (wait_rule.cuh): the roles go
// through their chunks without waiting, no copies in or out are started and nothing is written to memory.
// Before the CTA ends, its copies and products under way are waited for, with a limit again.  The limit
// and the record lie in shared memory, and the plan's status word is told at the end: 48 prompts take
// 922 us so, 939 with the word told in each wait, whose code counts; a look at a flag by every wait
// costs 1% to 2% more. ----
__device__ __forceinline__ bool dc_poll(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity), "r"(20000)
        : "memory");
    return ok != 0;
}

struct DcWaitOps {
    const DeltaArgs &A;
    DcSmem &sm;
    uint64_t *bar;
    uint32_t parity;
    __device__ __forceinline__ int limit() const { return *(volatile int *)&sm.polls; }
    __device__ __forceinline__ bool test() const { return mbar_test_wait(bar, parity); }
    __device__ __forceinline__ bool poll() const { return dc_poll(bar, parity); }
    __device__ __forceinline__ void late() const { *(volatile int *)&sm.late = 1; }
    __device__ __forceinline__ void stop() const { *(volatile int *)&sm.polls = -1; }
    __device__ __forceinline__ bool stopped() const { return limit() < 0; }
};

__device__ __forceinline__ void dc_wait(const DeltaArgs &A, DcSmem &sm, uint64_t *bar, uint32_t parity)
{
    wait_by_rule(DcWaitOps{A, sm, bar, parity}, DC_MOST_POLLS);
}

// Whether a wait has been given up, the same for all lanes of the warp.
__device__ __forceinline__ bool dc_stopped(const DcSmem &sm)
{
    return __any_sync(0xffffffffu, *(const volatile int *)&sm.polls < 0);
}

// one arrival for a warp whose lanes have all done their part
__device__ __forceinline__ void warp_arrive(uint64_t *bar)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// ---- q, k, v of one chunk after the other, by tensor copies of 64 rows.  Rows past the
// sequence's end bring what lies there (or zeros): the readers leave them out ----

__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, int x, int y, uint64_t *bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void dc_bring(const DeltaArgs &A, DcSmem &sm, const DcMaps &maps)
{
    const uint32_t leads = elect_lane();
    DcWalk w, ahead;
    int nk = 0, nv = 0;  // chunks whose q and k, whose v were asked for
    dc_start(ahead);
    // q and k go one chunk before v: they are needed earlier, and v's place is free later
#pragma unroll 1
    for (int n = -1;; ++n) {
        w = ahead;
        dc_next(A, sm, ahead);
        if (ahead.there) {
            const int st = (n + 1) % DC_KV;
            if (n + 1 >= DC_KV) dc_wait(A, sm, &sm.b_free[st], ((n + 1) / DC_KV - 1) & 1);
            if (dc_stopped(sm)) break;
            ++nk;
            if (leads) {
                const int x = ahead.h / A.hpq * KDIM, y = ahead.first + ahead.chunk * DC_C;
                const uint32_t dst = smem_addr(sm.kq[st][0]);
                mbar_arrive_expect_tx(&sm.b_ld[st], 4 * 64 * 128);
#pragma unroll 1
                for (int i = 0; i < 2; ++i) {
                    tma_load(dst + i * 128 * 128, &maps.k, x + 64 * i, y, &sm.b_ld[st]);
                    tma_load(dst + i * 128 * 128 + 64 * 128, &maps.q, x + 64 * i, y, &sm.b_ld[st]);
                }
            }
            __syncwarp();
        }
        if (n < 0) continue;
        if (!w.there) break;
        const int sv = n & 1;
        if (n >= 2) dc_wait(A, sm, &sm.b_vfree[sv], (n / 2 - 1) & 1);
        if (dc_stopped(sm)) break;
        ++nv;
        if (leads) {
            mbar_arrive_expect_tx(&sm.b_v[sv], 64 * 256);
            tma_load(smem_addr(sm.v[sv]), &maps.v, w.h * A.V + w.slice * DC_VW, w.first + w.chunk * DC_C, &sm.b_v[sv]);
        }
        __syncwarp();
    }
    // each stage's last copies have landed before the CTA ends, read or not
#pragma unroll 1
    for (int c = max(nk - DC_KV, 0); c < nk; ++c) mbar_wait_bounded(&sm.b_ld[c % DC_KV], (c / DC_KV) & 1, DEFAULT_WAIT_CYCLES);
#pragma unroll 1
    for (int c = max(nv - 2, 0); c < nv; ++c) mbar_wait_bounded(&sm.b_v[c & 1], (c / 2) & 1, DEFAULT_WAIT_CYCLES);
}

// ---- outputs, from the place of their chunk's values ----

template <class T>
__device__ __forceinline__ void dc_store(const DeltaArgs &A, DcSmem &sm, const DcMaps &maps)
{
    const int lane = threadIdx.x & 31, c = lane & 15, r0 = lane >> 4;
    const uint32_t leads = elect_lane();
    DcWalk w;
    dc_start(w);
#pragma unroll 1
    for (int n = 0;; ++n) {
        dc_next(A, sm, w);
        if (!w.there) break;
        const int sv = n & 1, t0 = w.first + w.chunk * DC_C;
        const int left = w.len - w.chunk * DC_C, cols = A.V - w.slice * DC_VW;
        dc_wait(A, sm, &sm.b_out[sv], (n / 2) & 1);
        if (dc_stopped(sm)) break;
        if (left >= DC_C && cols >= DC_VW) {
            if (leads) {
                asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];" ::"l"(&maps.y),
                             "r"(w.h * A.V + w.slice * DC_VW), "r"(t0), "r"(smem_addr(sm.v[sv]))
                             : "memory");
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            }
        } else if (c * 8 < cols) {
            T *y = static_cast<T *>(A.y) + (long long)(t0 + r0) * A.y_stride + (long long)w.h * A.V + w.slice * DC_VW + c * 8;
#pragma unroll 1
            for (int t = r0; t < min(left, DC_C); t += 2, y += 2 * A.y_stride)
                *reinterpret_cast<uint4 *>(y) = *reinterpret_cast<const uint4 *>(&sm.v[sv][t][c * 8]);
        }
        warp_arrive(&sm.b_vfree[sv]);
    }
    if (leads) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    __syncwarp();
}

// ---- the decays of a chunk's tokens, two tokens a lane ----

// 2^(d / 2^40), off by 2^-22 whatever the size of d: the whole part goes into the exponent as it is, and
// the rest, of half a unit at most, through ex2.  (d rounded to fp32 as a whole is off by 2^-18 near
// 100, and two tokens' factors of opposite exponents then make a decay off by up to 2^-17.5.)  Below
// 2^-126: 0.
__device__ __forceinline__ float pow2_of(long long d)
{
    const int whole = (int)((d + (1LL << 39)) >> 40), rest = (int)(d >> 8);  // rest / 2^32 in [-1/2, 1/2)
    return ex2((float)rest * 0x1p-32f) * __uint_as_float((uint32_t)(min(max(whole, -127), 127) + 127) << 23);
}

__device__ __forceinline__ void dc_scalars(const DeltaArgs &A, DcSmem &sm)
{
    const int lane = threadIdx.x & 31;
    DcWalk w;
    dc_start(w);
    float a[2], beta[2];
    auto load = [&]() {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int t = 2 * lane + i;
            const bool there = w.there && w.chunk * DC_C + t < w.len;
            const long long at = (long long)(w.first + w.chunk * DC_C + t) * A.H + w.h;
            a[i] = there ? __ldg(A.a + at) : 1.f;
            beta[i] = there ? __ldg(A.beta + at) : 0.f;
        }
    };
    long long G[2], mid, end, top;
    float be[2];
    unsigned bad = 0;
    for (int n = -1;; ++n) {
        const int b = n & 1;
        const bool any = w.there;  // chunk n, whose a and beta are here
        if (n >= 0) {
            if (!any) break;
            // log2 a in steps of 2^-40: sums and differences are exact.  A decay of 0 counts as
            // 2^-150, which no fp32 product tells from it; a decay that is no number stays one.
            long long l[2];
            bool nan[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float x = log2f(a[i]);
                nan[i] = !(x == x);
                l[i] = (long long)(fminf(fmaxf(x, -150.f), 150.f) * 0x1p40f);
            }
            be[0] = beta[0], be[1] = beta[1];
            bad = __ballot_sync(0xffffffffu, nan[0] || nan[1]);
            long long s = l[0] + l[1];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long up = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += up;
            }
            G[0] = s - l[1], G[1] = s;
            mid = __shfl_sync(0xffffffffu, G[1], 15);
            end = __shfl_sync(0xffffffffu, G[1], 31);
            top = __shfl_sync(0xffffffffu, G[0], 0);
        }
        dc_next(A, sm, w);
        load();  // those of chunk n + 1, on their way while chunk n's are written down
        if (n < 0) continue;
        if (n >= 2) dc_wait(A, sm, &sm.b_tp[b], (n / 2 - 1) & 1);  // chunk n - 2 has been prepared
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
            const int t = 2 * lane + i;
            const long long Gi = i ? G[1] : G[0];
            const bool lost = bad & (0xffffffffu >> (31 - lane));  // from that token on
            const float g = (float)Gi * 0x1p-40f;
            sm.beta[b][t] = i ? be[1] : be[0];
            sm.dec[b][t] = lost ? __int_as_float(0x7fc00000) : pow2_of(Gi);
            sm.rest[b][t] = pow2_of(end - Gi);
            sm.er[b][t] = pow2_of(Gi - mid);
            sm.ec[b][t] = pow2_of(mid - Gi);
            sm.gh[b][t] = g;
            sm.gl[b][t] = (float)(Gi - (long long)(g * 0x1p40f)) * 0x1p-40f;
        }
        if (lane == 0) {
            const float span = fmaxf((float)(top - mid), (float)(mid - end)) * 0x1p-40f;
            sm.strong[b] = !(span < DC_STRONG) || (float)(end - top) * 0x1p-40f > DC_STRONG;
        }
        warp_arrive(&sm.b_sc[b]);
    }
}

// ---- A, P, T of one chunk ahead ----

// the part of x that tf32 holds (13 low mantissa bits cleared); the rest, x - tf32_part(x), is exact
// in fp32 and loses what is below 2^-23 of x in tf32
__device__ __forceinline__ float tf32_part(float x) { return __uint_as_float(__float_as_uint(x) & 0xFFFFE000u); }

__device__ __forceinline__ void mma_tf32(float (&d)[4], const float (&a)[4], const float (&b)[2])
{
    asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(__float_as_uint(a[0])), "r"(__float_as_uint(a[1])), "r"(__float_as_uint(a[2])),
                   "r"(__float_as_uint(a[3])), "r"(__float_as_uint(b[0])), "r"(__float_as_uint(b[1])));
}

// L[16 MT x 8 KT] B[8 KT x 8] as MT tiles of 16 rows x 8 columns, three tf32 products each (in
// accumulators of their own, so that none waits for another): fp32 accuracy.  l(m, i, k): L at
// row i + lane / 4, column k + lane % 4; b(k): B at row k + lane % 4, column lane / 4; LOWER: L is
// lower triangular; the first 8 `from` rows of B are zeros.
template <int MT, int KT, bool LOWER = false, class FL, class FB>
__device__ __forceinline__ void mul_tri(float (&d)[MT][4], int from, FL l, FB b)
{
    float d1[MT][4] = {}, d2[MT][4] = {};
#pragma unroll
    for (int ks = 0; ks < KT; ++ks) {
        if (ks < from) continue;
        float bh[2], bl[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float x = b(8 * ks + 4 * e);
            bh[e] = tf32_part(x);
            bl[e] = x - bh[e];
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            if (LOWER && 8 * ks >= 16 * (m + 1)) continue;
            float ah[4], al[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float x = l(m, 16 * m + 8 * (e & 1), 8 * ks + 4 * (e >> 1));
                ah[e] = tf32_part(x);
                al[e] = x - ah[e];
            }
            mma_tf32(d1[m], al, bh);
            mma_tf32(d2[m], ah, bl);
            mma_tf32(d[m], ah, bh);
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 4; ++e) d[m][e] += d1[m][e] + d2[m][e];
}

// T = (I + A)^-1 in place, A strictly lower triangular (zeros elsewhere): the 16 x 16 blocks on the
// diagonal by substitution (a column a lane, two blocks a warp: rows 32 half .. + 31), then
// T21 = -T22 A21 T11 for blocks of 16 and of 32 by all four warps of the group.  Substitution in
// blocks is as stable as substitution; the powers of A that a product form needs would not be.
__device__ __forceinline__ void invert_blocks(float (&M)[64][68], int half)
{
    const int lane = threadIdx.x & 31;
    const int o = 32 * half + (lane & 16), j = lane & 15;
    const float *L = &M[o][o];
    float x[16];
    x[0] = j == 0 ? 1.f : 0.f;
#pragma unroll
    for (int i = 1; i < 16; ++i) {
        // the newest value last: it is the one to wait for
        float s0 = i == j ? 1.f : 0.f, s1 = 0.f;
#pragma unroll
        for (int k4 = 0; k4 < i; k4 += 4) {
            const float4 a = lds4(L + i * 68 + k4);
            s0 = fmaf(-a.x, x[k4], s0);
            if (k4 + 1 < i) s1 = fmaf(-a.y, x[k4 + 1], s1);
            if (k4 + 2 < i) s0 = fmaf(-a.z, x[k4 + 2], s0);
            if (k4 + 3 < i) s1 = fmaf(-a.w, x[k4 + 3], s1);
        }
        x[i] = s0 + s1;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 16; ++i) M[o + i][o + j] = x[i];
}

__device__ __forceinline__ void invert_merge(float (&M)[64][68], float (&X)[32][36], int r)
{
    const int wq = r >> 5, lane = r & 31, g = lane >> 2, t = lane & 3;
    {
        const int o = 32 * (wq >> 1), n0 = 8 * (wq & 1), xr = 16 * (wq >> 1);
        const float *L21 = &M[o + 16 + g][o + t], *L22 = &M[o + 16 + g][o + 16 + t], *T11 = &M[o + t][o + n0 + g];
        float d[1][4] = {};
        mul_tri<1, 2>(d, wq & 1, [&](int, int i, int k) { return L21[i * 68 + k]; }, [&](int k) { return T11[k * 68]; });
        float *x = &X[xr][n0];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[(g + 8 * (e >> 1)) * 36 + 2 * t + (e & 1)] = d[0][e];
        __syncwarp();
        float f[1][4] = {};
        mul_tri<1, 2>(f, 0, [&](int, int i, int k) { return L22[i * 68 + k]; }, [&](int k) { return x[(k + t) * 36 + g]; });
        named_sync(5, DC_PREP);  // A21 has been read
#pragma unroll
        for (int e = 0; e < 4; ++e) M[o + 16 + g + 8 * (e >> 1)][o + n0 + 2 * t + (e & 1)] = -f[0][e];
    }
    named_sync(5, DC_PREP);
    {
        const int n0 = 8 * wq;
        const float *L21 = &M[32 + g][t], *L22 = &M[32 + g][32 + t], *T11 = &M[t][n0 + g];
        float d[2][4] = {};
        mul_tri<2, 4>(d, wq, [&](int, int i, int k) { return L21[i * 68 + k]; }, [&](int k) { return T11[k * 68]; });
        float *x = &X[0][n0];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[(16 * m + g + 8 * (e >> 1)) * 36 + 2 * t + (e & 1)] = d[m][e];
        __syncwarp();
        float f[2][4] = {};
        mul_tri<2, 4, true>(f, 0, [&](int, int i, int k) { return L22[i * 68 + k]; }, [&](int k) { return x[(k + t) * 36 + g]; });
        named_sync(5, DC_PREP);
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int e = 0; e < 4; ++e) M[32 + 16 * m + g + 8 * (e >> 1)][n0 + 2 * t + (e & 1)] = -f[m][e];
    }
    named_sync(5, DC_PREP);
}

// largest magnitude of 8 packed values
__device__ __forceinline__ float max_of(uint4 v, const __nv_bfloat16 *)
{
    auto a = [](uint32_t w) { return __habs2(*reinterpret_cast<__nv_bfloat162 *>(&w)); };
    const __nv_bfloat162 m = __hmax2(__hmax2(a(v.x), a(v.y)), __hmax2(a(v.z), a(v.w)));
    return fmaxf(__low2float(m), __high2float(m));
}

// 8 scaled values as fp16 parts, 16 bytes each
__device__ __forceinline__ void put8(uint8_t *hi, uint8_t *lo, const float2 *x, float mul)
{
    uint32_t h[4], l[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) split2(__fmul2_rn(x[e], two(mul)), h[e], l[e]);
    *reinterpret_cast<uint4 *>(hi) = make_uint4(h[0], h[1], h[2], h[3]);
    *reinterpret_cast<uint4 *>(lo) = make_uint4(l[0], l[1], l[2], l[3]);
}

template <class T>
__device__ __forceinline__ void dc_prep(const DeltaArgs &A, DcSmem &sm, uint32_t tmem)
{
    const int r = threadIdx.x - DC_CHAIN, wq = r >> 5;
    const int t = r & 63;        // token of this thread's row
    const bool is_q = r >= 64;
    const int half = wq & 1;     // rows 32 half .. of k or q: the warp's
    const uint32_t kk = tmem + TM_KK + ((uint32_t)(wq * 32) << 16);
    const uint32_t leads = elect_lane();
    DcWalk w;
    dc_start(w);
    for (int n = 0;; ++n) {
        dc_next(A, sm, w);
        if (!w.there) break;
        const int st = n % DC_KV, tp = n & 1;
        const bool there = t < w.len - w.chunk * DC_C;
        dc_wait(A, sm, &sm.b_ld[st], (n / DC_KV) & 1);

        // this thread's row of k or q: its norm, and (bf16) fp16 values at a power of two of their
        // own, in place.  The 16-byte pieces go in an order that keeps the row's lanes on
        // different banks.  fp16 rows are operands as they are.
        float f_own = 1.f;
        {
            constexpr bool CONVERT = sizeof(T) == 2 && !__is_same(T, __half);
            uint8_t *row = sm.kq[st][0] + r * 128;
            const int sw = (r & 7) << 4;
            float ss[4] = {};
            float m = 0.f, mul = 1.f;
            if (!there) {  // a row past the sequence's end: whatever lies there counts as zeros
#pragma unroll 1
                for (int i = 0; i < 256; i += 16)
                    *reinterpret_cast<uint4 *>(row + (i >> 7) * (128 * 128) + (i & 127)) = make_uint4(0, 0, 0, 0);
            }
            if (CONVERT || A.normalize) {
#pragma unroll 1
                for (int hf = 0; hf < 2; ++hf) {
                    uint4 raw[8];
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        raw[c] = *reinterpret_cast<const uint4 *>(row + hf * (128 * 128) + ((c << 4) ^ sw));
                    if constexpr (CONVERT) {
#pragma unroll
                        for (int c = 0; c < 8; ++c) m = fmaxf(m, max_of(raw[c], (const T *)nullptr));
                    }
                    if (A.normalize) {
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            const uint32_t v[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                ss[e] = add_squares(v[e], ss[e], (const T *)nullptr);
                            }
                        }
                    }
                }
            }
            if constexpr (CONVERT) {
                pow2_scale(m, mul, f_own);
#pragma unroll 1
                for (int hf = 0; hf < 2; ++hf) {
                    uint4 raw[8];
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        raw[c] = *reinterpret_cast<const uint4 *>(row + hf * (128 * 128) + ((c << 4) ^ sw));
#pragma unroll
                    for (int c = 0; c < 8; ++c) {
                        const uint32_t v[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
                        uint32_t o[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            o[e] = scale_to_half(v[e], __float_as_uint(mul));
                        *reinterpret_cast<uint4 *>(row + hf * (128 * 128) + ((c << 4) ^ sw)) =
                            make_uint4(o[0], o[1], o[2], o[3]);
                    }
                }
            }
            if (A.normalize) {
                f_own *= rsqrtf((ss[0] + ss[1]) + (ss[2] + ss[3]) + DELTA_QK_EPS);
            }
            if (is_q) f_own *= A.scale;
        }
        dc_wait(A, sm, &sm.b_sc[tp], (n / 2) & 1);
        const bool strong = sm.strong[tp];
        if (!is_q) sm.col[t] = strong ? f_own : f_own * sm.ec[tp][t];
        fence_async_smem();
        tc_fence_before();
        named_sync(5, DC_PREP);
        warp_arrive(&sm.b_kq[st]);
        if (wq == 0) {
            tc_fence_after();
            if (leads) {
                constexpr uint32_t idesc = idesc_f16(128, 64, false);
                const uint64_t d = sdesc_sw128(smem_addr(sm.kq[st][0]), 16, 1024);
#pragma unroll 4
                for (int i = 0; i < 8; ++i) {
                    const uint64_t at = d + (i >> 2) * 1024 + (i & 3) * 2;
                    mma_ss(tmem + TM_KK, at, at, idesc, i > 0);
                }
                umma_commit(&sm.b_KK);
            }
            __syncwarp();
        }
        const float beta = sm.beta[tp][t], dec = sm.dec[tp][t];
        float f = is_q ? f_own : f_own * beta;
        if (!strong) f *= sm.er[tp][t];
        const int last = is_q ? t : t - 1;
        dc_wait(A, sm, &sm.b_KK, n & 1);
        tc_fence_after();
        if (strong) {
            // the chunk forgets so much that the factors of its decays leave fp32's range: the
            // decays themselves, in place
            const float gh = sm.gh[tp][t], gl = sm.gl[tp][t];
#pragma unroll 1
            for (int c = 0; c < 64; c += 16) {
                float x[16];
                tmem_ld16n(kk + c, x);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    x[e] = c + e <= last ? x[e] * ex2((gh - sm.gh[tp][c + e]) + (gl - sm.gl[tp][c + e])) : 0.f;
                tmem_st16(kk + c, reinterpret_cast<const uint32_t (&)[16]>(x));
            }
            tmem_st_wait();
        }
        // this row of A or P; rows below 32 have zeros right of column 32, which stay from the start
        float2 x[32];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            if (c < 2 * half + 2) {
                tmem_ld16n(kk + 16 * c, reinterpret_cast<float *>(x + 8 * c));
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const Four cf = lds_four(sm.col + 16 * c + 4 * e);
                    x[8 * c + 2 * e] = __fmul2_rn(__fmul2_rn(x[8 * c + 2 * e], cf.a), two(f));
                    x[8 * c + 2 * e + 1] = __fmul2_rn(__fmul2_rn(x[8 * c + 2 * e + 1], cf.b), two(f));
                }
                if (c >= 2 * half) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        if (16 * c + 2 * e > last) x[8 * c + e].x = 0.f;
                        if (16 * c + 2 * e + 1 > last) x[8 * c + e].y = 0.f;
                    }
                }
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[8 * c + e] = two(0.f);
            }
        }
        if (!is_q) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
                if (e < 8 * half + 8) st4(&sm.m[t][4 * e], make_float4(x[2 * e].x, x[2 * e].y, x[2 * e + 1].x, x[2 * e + 1].y));
        }
        named_sync(5, DC_PREP);
        // this stage of T, P and their factors is free once the chunk two before has given its outputs
        if (n >= 2) dc_wait(A, sm, &sm.b_out[tp], (n / 2 - 1) & 1);
        const int sw = (t & 7) << 4;
        if (is_q) {
            float m = 0.f, mul, inv;
#pragma unroll
            for (int e = 0; e < 32; ++e) m = max3(m, x[e]);
            pow2_scale(m, mul, inv);
            uint8_t *hi = sm.tp[tp][2] + t * 128, *lo = hi + 64 * 128;
#pragma unroll
            for (int c = 0; c < 8; ++c)
                if (c < 4 * half + 4) put8(hi + ((c << 4) ^ sw), lo + ((c << 4) ^ sw), x + 4 * c, mul);
            sm.fp[tp][t] = inv;
            sm.fqs[tp][t] = dec * f_own;
        } else {
            invert_blocks(sm.m, half);
            sm.fv[tp][t] = beta;
            sm.fks[tp][t] = beta * dec * f_own;
            sm.fw[tp][t] = sm.rest[tp][t] * f_own;
            if (t == 63) sm.gC[tp] = dec;
        }
        named_sync(5, DC_PREP);
        invert_merge(sm.m, sm.x, r);
        {
            // rows of T, two threads each: every other piece of 8 columns (left of column 32 in
            // rows below it)
            const int row = r >> 1;
            float m = 0.f, mul, inv;
            Four v[4][2];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < 2 || row >= 32) {
                    v[i][0] = lds_four(&sm.m[row][16 * i + 8 * (r & 1)]);
                    v[i][1] = lds_four(&sm.m[row][16 * i + 8 * (r & 1) + 4]);
                    m = max3(max3(max3(max3(m, v[i][0].a), v[i][0].b), v[i][1].a), v[i][1].b);
                }
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
            pow2_scale(m, mul, inv);
            uint8_t *hi = sm.tp[tp][0] + row * 128, *lo = hi + 64 * 128;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < 2 || row >= 32) {
                    const float2 y[4] = {v[i][0].a, v[i][0].b, v[i][1].a, v[i][1].b};
                    const int at = ((2 * i + (r & 1)) << 4) ^ ((row & 7) << 4);
                    put8(hi + at, lo + at, y, mul);
                }
            if (!(r & 1)) sm.fu[tp][row] = inv;
        }
        fence_async_smem();
        tc_fence_before();
        warp_arrive(&sm.b_tp[tp]);
        named_sync(5, DC_PREP);  // T in fp32 has been read
    }
    if (wq == 0 && leads) umma_commit(&sm.b_end);
}

// ---- the chain's products ----

__device__ __forceinline__ void dc_issue(const DeltaArgs &A, DcSmem &sm, uint32_t tmem)
{
    const uint32_t leads = elect_lane();
    DcWalk w;
    dc_start(w);
    constexpr uint32_t i64 = idesc_f16(128, 64, false), i128 = idesc_f16(128, 128, true);
    // descriptors move by bytes / 16: 2 a step of 16 along K, 1024 a half of the key dimensions
    for (int n = 0;; ++n) {
        dc_next(A, sm, w);
        if (!w.there) break;
        const int st = n % DC_KV, tp = n & 1;
        const uint64_t k0 = sdesc_sw128(smem_addr(sm.kq[st][0]), 16, 1024);
        const uint64_t kn = sdesc_sw128(smem_addr(sm.kq[st][0]), 128 * 128, 1024);
        const uint64_t t0 = sdesc_sw128(smem_addr(sm.tp[tp][0]), 16, 1024);
        // K S: lo, then hi
        dc_wait(A, sm, &sm.b_kq[st], (n / DC_KV) & 1);
        dc_wait(A, sm, &sm.b_S, n & 1);
        tc_fence_after();
        if (leads) {
#pragma unroll 4
            for (int i = 0; i < 16; ++i)
                mma_ts(tmem + TM_A, tmem + TM_S + 8 * (i ^ 8), k0 + ((i >> 2) & 1) * 1024 + (i & 3) * 2, i64, i > 0);
            umma_commit(&sm.b_KS);
        }
        __syncwarp();
        // U = T R: (R lo, T hi), (R hi, T lo), (R hi, T hi)
        dc_wait(A, sm, &sm.b_R, n & 1);
        tc_fence_after();
        if (leads) {
#pragma unroll 4
            for (int i = 0; i < 12; ++i)
                mma_ts(tmem + TM_A, tmem + TM_R + (i < 4 ? 32 : 0) + 8 * (i & 3), t0 + ((i >> 2) == 1 ? 512 : 0) + (i & 3) * 2, i64,
                       i > 0);
            umma_commit(&sm.b_U);
        }
        __syncwarp();
        // Q S, in the shadow of what U goes through next, once the chunk before has read its own
        if (n >= 1) dc_wait(A, sm, &sm.b_out[(n - 1) & 1], ((n - 1) / 2) & 1);
        tc_fence_after();
        if (leads) {
#pragma unroll 4
            for (int i = 0; i < 16; ++i)
                mma_ts(tmem + TM_Q, tmem + TM_S + 8 * (i ^ 8), k0 + 512 + ((i >> 2) & 1) * 1024 + (i & 3) * 2, i64, i > 0);
            umma_commit(&sm.b_QS);
        }
        __syncwarp();
        // the state's increment: k as the right operand, tokens along K
        dc_wait(A, sm, &sm.b_W, n & 1);
        tc_fence_after();
        if (leads) {
#pragma unroll 4
            for (int i = 0; i < 8; ++i)
                mma_ts(tmem + TM_A, tmem + TM_S + 8 * (i ^ 4), kn + (i & 3) * 128, i128, i > 0);
            umma_commit(&sm.b_D);
            umma_commit(&sm.b_free[st]);
        }
        __syncwarp();
        // P U: (U lo, P hi), (U hi, P lo), (U hi, P hi)
        if (leads) {
#pragma unroll 4
            for (int i = 0; i < 12; ++i)
                mma_ts(tmem + TM_PU, tmem + TM_R + (i < 4 ? 32 : 0) + 8 * (i & 3),
                       t0 + 1024 + ((i >> 2) == 1 ? 512 : 0) + (i & 3) * 2, i64, i > 0);
            umma_commit(&sm.b_PU);
        }
        __syncwarp();
    }
    if (leads) umma_commit(&sm.b_end);
}

// ---- the chain ----

template <class T>
__device__ __forceinline__ void dc_chain(const DeltaArgs &A, DcSmem &sm, uint32_t tmem)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quad = warp & 3, g = warp >> 2;  // lanes 32 quad .. + 31; tokens 32 g .., key rows 64 g ..
    const int col = quad * 32 + lane;
    const uint32_t tm = tmem + ((uint32_t)(quad * 32) << 16);
    int flip = 0;  // which of the two exchange buffers comes next
    // maxima over both halves of this lane's column (upper halves: the exponents are what is needed)
    auto both = [&](float &a, float &b) {
        uint32_t m = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
        sm.mx[flip][g][col] = m;
        named_sync(1 + quad, 64);
        m = __vmaxu2(m, sm.mx[flip][g ^ 1][col]);
        flip ^= 1;
        a = __uint_as_float(m << 16);
        b = __uint_as_float(m & 0xffff0000u);
    };
    // 32 values (16 pairs) times mul: hi parts to 16 columns at `hi`, lo parts at `lo`
    auto put = [&](const float2 *x, float mul, uint32_t hi, uint32_t lo) {
        uint32_t h[16], l[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) split2(__fmul2_rn(x[i], two(mul)), h[i], l[i]);
        tmem_st16(hi, h);
        tmem_st16(lo, l);
    };
    DcWalk w;
    dc_start(w);
    float2 S[32];
    float *Sg = nullptr;
    bool own = false, pending = false;
    float sS = 0.f, sU = 0.f, sW = 0.f, s_old = 0.f;  // values of a unit of the parts of S, U, U~; of S a chunk ago
    for (int n = 0;; ++n) {
        const int tp = n & 1, tq = tp ^ 1;  // stages of this chunk and of the one before
        if (pending) {
            // the state after the chunk before
            const float2 gC = two(sm.gC[tq]);
            dc_wait(A, sm, &sm.b_D, (n - 1) & 1);
            tc_fence_after();
#pragma unroll
            for (int b = 0; b < 2; ++b) {
                float2 x[16];
                tmem_ld32(tm + TM_A + 64 * g + 32 * b, reinterpret_cast<float *>(x));
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    S[16 * b + i] = __ffma2_rn(two(sW), x[i], __fmul2_rn(gC, S[16 * b + i]));
            }
            if (w.chunk * DC_C + DC_C >= w.len) {
                if (*(volatile int *)&sm.polls < 0) own = false;  // (in the store's condition: spills)
                if (own) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        Sg[(long long)(2 * i) * A.V] = S[i].x;
                        Sg[(long long)(2 * i + 1) * A.V] = S[i].y;
                    }
                }
            }
        }
        dc_next(A, sm, w);
        if (w.there && w.chunk == 0) {
            own = col < A.V - w.slice * DC_VW;
            Sg = A.S + (((long long)w.slot * A.H + w.h) * KDIM + 64 * g) * A.V + w.slice * DC_VW + col;
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                S[i].x = own ? Sg[(long long)(2 * i) * A.V] : 0.f;
                S[i].y = own ? Sg[(long long)(2 * i + 1) * A.V] : 0.f;
            }
        }
        s_old = sS;
        if (w.there) {
            float m = 0.f, unused = 0.f, mul;
#pragma unroll
            for (int i = 0; i < 32; ++i) m = max3(m, S[i]);
            both(m, unused);
            pow2_scale(m, mul, sS);
            tc_fence_after();
            put(S, mul, tm + TM_S + 32 * g, tm + TM_S + 64 + 32 * g);
            put(S + 16, mul, tm + TM_S + 32 * g + 16, tm + TM_S + 64 + 32 * g + 16);
            tmem_st_wait();
            tc_fence_before();
            warp_arrive(&sm.b_S);
        }
        if (pending) {
            // the outputs of the chunk before, while this one's K S runs: into the place of its values
            dc_wait(A, sm, &sm.b_PU, (n - 1) & 1);
            tc_fence_after();
            float2 q[16], x[16];
            tmem_ld32(tm + TM_Q + 32 * g, reinterpret_cast<float *>(q));
            tmem_ld32(tm + TM_PU + 32 * g, reinterpret_cast<float *>(x));
            tmem_ld_wait();
            uint16_t *yp = &sm.v[tq][32 * g][col];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const Four fq = lds_four(sm.fqs[tq] + 32 * g + 4 * i), fp = lds_four(sm.fp[tq] + 32 * g + 4 * i);
                const float2 y0 = __ffma2_rn(__fmul2_rn(fq.a, two(s_old)), q[2 * i], __fmul2_rn(__fmul2_rn(fp.a, two(sU)), x[2 * i]));
                const float2 y1 = __ffma2_rn(__fmul2_rn(fq.b, two(s_old)), q[2 * i + 1],
                                             __fmul2_rn(__fmul2_rn(fp.b, two(sU)), x[2 * i + 1]));
                const uint32_t p0 = pack2(y0.x, y0.y, (const T *)nullptr), p1 = pack2(y1.x, y1.y, (const T *)nullptr);
                yp[(4 * i) * DC_VW] = (uint16_t)p0;
                yp[(4 * i + 1) * DC_VW] = (uint16_t)(p0 >> 16);
                yp[(4 * i + 2) * DC_VW] = (uint16_t)p1;
                yp[(4 * i + 3) * DC_VW] = (uint16_t)(p1 >> 16);
            }
            fence_async_smem();
            tc_fence_before();
            warp_arrive(&sm.b_out[tq]);
        }
        if (!w.there) break;
        pending = true;
        float2 x[16];
        float mul;
        // R
        {
            float m = 0.f, unused = 0.f, sR;
            dc_wait(A, sm, &sm.b_v[tp], (n / 2) & 1);
            dc_wait(A, sm, &sm.b_tp[tp], (n / 2) & 1);
            dc_wait(A, sm, &sm.b_KS, n & 1);
            tc_fence_after();
            tmem_ld32(tm + TM_A + 32 * g, reinterpret_cast<float *>(x));
            tmem_ld_wait();
            const uint16_t *vp = &sm.v[tp][32 * g][col];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const Four fk = lds_four(sm.fks[tp] + 32 * g + 4 * i), fv = lds_four(sm.fv[tp] + 32 * g + 4 * i);
                float2 v0 = make_float2(unpack2(vp[(4 * i) * DC_VW], (const T *)nullptr).x,
                                        unpack2(vp[(4 * i + 1) * DC_VW], (const T *)nullptr).x);
                float2 v1 = make_float2(unpack2(vp[(4 * i + 2) * DC_VW], (const T *)nullptr).x,
                                        unpack2(vp[(4 * i + 3) * DC_VW], (const T *)nullptr).x);
                x[2 * i] = __ffma2_rn(__fmul2_rn(x[2 * i], two(-sS)), fk.a, __fmul2_rn(fv.a, v0));
                x[2 * i + 1] = __ffma2_rn(__fmul2_rn(x[2 * i + 1], two(-sS)), fk.b, __fmul2_rn(fv.b, v1));
                m = max3(max3(m, x[2 * i]), x[2 * i + 1]);
            }
            const int left = own ? w.len - w.chunk * DC_C - 32 * g : 0;
            if (left < 32) {  // past the sequence's end or the value dimension: nobody's values
                m = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    if (2 * i >= left) x[i].x = 0.f;
                    if (2 * i + 1 >= left) x[i].y = 0.f;
                    m = max3(m, x[i]);
                }
            }
            both(m, unused);
            pow2_scale(m, mul, sR);
            put(x, mul, tm + TM_R + 16 * g, tm + TM_R + 32 + 16 * g);
            tmem_st_wait();
            tc_fence_before();
            warp_arrive(&sm.b_R);
            sU = sR;
        }
        // U, and U as the state takes it (U~)
        {
            float mu = 0.f, mw = 0.f, mulw;
            const float sR = sU;
            dc_wait(A, sm, &sm.b_U, n & 1);
            tc_fence_after();
            tmem_ld32(tm + TM_A + 32 * g, reinterpret_cast<float *>(x));
            tmem_ld_wait();
            float2 y[16];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const Four fu = lds_four(sm.fu[tp] + 32 * g + 4 * i), fw = lds_four(sm.fw[tp] + 32 * g + 4 * i);
                x[2 * i] = __fmul2_rn(x[2 * i], fu.a);  // in units of sR
                x[2 * i + 1] = __fmul2_rn(x[2 * i + 1], fu.b);
                y[2 * i] = __fmul2_rn(x[2 * i], fw.a);
                y[2 * i + 1] = __fmul2_rn(x[2 * i + 1], fw.b);
                mu = max3(max3(mu, x[2 * i]), x[2 * i + 1]);
                mw = max3(max3(mw, y[2 * i]), y[2 * i + 1]);
            }
            both(mu, mw);
            pow2_scale(mu, mul, sU);
            pow2_scale(mw, mulw, sW);
            sU *= sR;
            sW *= sR;
            put(x, mul, tm + TM_R + 16 * g, tm + TM_R + 32 + 16 * g);
            dc_wait(A, sm, &sm.b_QS, n & 1);  // S's parts have been read
            tc_fence_after();
            put(y, mulw, tm + TM_S + 16 * g, tm + TM_S + 32 + 16 * g);
            tmem_st_wait();
            tc_fence_before();
            warp_arrive(&sm.b_W);
        }
    }
}

// A launch takes DC_MAX_SEQS sequences, which each CTA sorts by itself; 768 sequences of 64 tokens, 8
// heads of 128: 452 us in two launches (token by token 1857 us).
//
// The order in which the launch's sequences are taken (longest first) and those whose slot an
// earlier one names; block 0 reports bad ones.
__device__ __forceinline__ void dc_order(const DeltaArgs &A, DcSmem &sm)
{
    for (int i = threadIdx.x; i < (A.rows + 31) / 32; i += DC_THREADS) sm.dup[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < A.rows; i += DC_THREADS) {
        const int c0 = __ldg(A.cu + i), c1 = __ldg(A.cu + i + 1), slot = A.slot ? __ldg(A.slot + i) : A.before + i;
        const int len = (int)((unsigned)c1 - (unsigned)c0);  // (bad bounds may be any numbers)
        int rank = 0;
        bool dup = false;
        int d0 = __ldg(A.cu);
        for (int j = 0; j < A.rows; ++j) {
            const int d1 = __ldg(A.cu + j + 1), other = (int)((unsigned)d1 - (unsigned)d0);
            d0 = d1;
            rank += other > len || (other == len && j < i);
            if (A.slot && j < i) dup = dup || __ldg(A.slot + j) == slot;
        }
        if (A.slot)
            for (int j = -A.before; j < 0; ++j) dup = dup || __ldg(A.slot + j) == slot;
        dup = dup && slot >= 0;
        sm.order[rank] = (uint16_t)i;
        if (dup) atomicOr(&sm.dup[i >> 5], 1u << (i & 31));
        const bool bad = c0 < 0 || c1 < c0 || c1 > A.tokens;
        if (blockIdx.x == 0 && slot >= 0 && (bad || (len > 0 && (dup || slot >= A.slots))))
            atomicOr(A.status, SK_STATUS_BAD_ROW);
    }
}

template <class T>
__global__ void __launch_bounds__(DC_THREADS, 1) delta_chunk_kernel(const DeltaArgs A, const __grid_constant__ DcMaps maps)
{
    extern __shared__ __align__(1024) unsigned char raw_smem[];
    DcSmem &sm = *reinterpret_cast<DcSmem *>(raw_smem);
    const int warp = threadIdx.x >> 5;
    if (warp == 0) {
        tmem_alloc(&sm.taddr, 512);
        tmem_relinquish();
    }
    if (threadIdx.x == 0) {
        sm.polls = A.polls;
        sm.late = 0;
        for (int i = 0; i < DC_KV; ++i) {
            mbar_init(&sm.b_ld[i], 1);
            mbar_init(&sm.b_free[i], 1);
            mbar_init(&sm.b_kq[i], DC_PREP / 32);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.b_v[i], 1);
            mbar_init(&sm.b_vfree[i], 1);
            mbar_init(&sm.b_sc[i], 1);
            mbar_init(&sm.b_tp[i], DC_PREP / 32);
            mbar_init(&sm.b_out[i], DC_CHAIN / 32);
        }
        mbar_init(&sm.b_S, DC_CHAIN / 32);
        mbar_init(&sm.b_R, DC_CHAIN / 32);
        mbar_init(&sm.b_W, DC_CHAIN / 32);
        for (uint64_t *b : {&sm.b_KS, &sm.b_QS, &sm.b_U, &sm.b_D, &sm.b_PU, &sm.b_KK}) mbar_init(b, 1);
        mbar_init(&sm.b_end, 2);  // both warps that issue products, when their last ones are done
        mbar_fence_init();
    }
    // what stays zero: T and P right of column 32 in rows below 32, A there
    for (int i = threadIdx.x; i < (int)(sizeof(sm.tp) + sizeof(sm.m)) / 16; i += DC_THREADS)
        reinterpret_cast<uint4 *>(sm.tp)[i] = make_uint4(0, 0, 0, 0);
    fence_async_smem();
    dc_order(A, sm);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    constexpr uint32_t tmem = 0;  // all columns of the SM's tensor memory: they start at 0
    constexpr int WP = DC_CHAIN / 32, WH = WP + DC_PREP / 32;  // first warps of the other groups
    if (warp < WP) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(DC_REG_CHAIN));
        dc_chain<T>(A, sm, tmem);
    } else if (warp < WH) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(DC_REG_PREP));
        dc_prep<T>(A, sm, tmem);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(DC_REG_HELP));
        if (warp == WH) {
            dc_issue(A, sm, tmem);
        } else if (warp == WH + 1)
            dc_store<T>(A, sm, maps);
        else if (warp == WH + 2)
            dc_scalars(A, sm);
        else
            dc_bring(A, sm, maps);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x == 0 && sm.late) atomicOr(A.status, SK_STATUS_DELTA_TIMEOUT);
    if (warp == 0) {
        mbar_wait_bounded(&sm.b_end, 0, DEFAULT_WAIT_CYCLES);
        __syncwarp();
        tmem_dealloc(sm.taddr, 512);
    }
}

// a map of a token tensor's 64-row, `box`-column tiles
bool dc_map(CUtensorMap *m, int dtype, const void *p, long long cols, long long tokens, long long stride, int box, bool swizzle)
{
    typedef CUresult (*Encode)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *, const cuuint64_t *,
                               const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                               CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
    static const Encode encode = [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return (Encode) nullptr;
        }
        return (Encode)f;
    }();
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)tokens}, strides[1] = {(cuuint64_t)stride * 2};
    const cuuint32_t boxes[2] = {(cuuint32_t)box, DC_C}, ones[2] = {1, 1};
    return encode && encode(m, dtype == SKETCHSSM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                            const_cast<void *>(p), dims, strides, boxes, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class T>
cudaError_t launch_type(const DeltaArgs &a, int sms, cudaStream_t stream)
{
    const long long qk = (long long)a.Hqk * KDIM, hv = (long long)a.H * a.V;
    DcMaps maps;
    if (!dc_map(&maps.q, a.dtype, a.q, qk, a.tokens, a.q_stride, 64, true) ||
        !dc_map(&maps.k, a.dtype, a.k, qk, a.tokens, a.k_stride, 64, true) ||
        !dc_map(&maps.v, a.dtype, a.v, hv, a.tokens, a.v_stride, DC_VW, false) ||
        !dc_map(&maps.y, a.dtype, a.y, hv, a.tokens, a.y_stride, DC_VW, false))
        return cudaErrorInvalidValue;
    DeltaArgs A = a;
    A.polls = (int)(a.wait_limit / 40000 < DC_MOST_POLLS ? a.wait_limit / 40000 : DC_MOST_POLLS);
    cudaError_t e = cudaFuncSetAttribute(delta_chunk_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)sizeof(DcSmem));
    if (e != cudaSuccess) return e;
    for (A.before = 0; A.before < a.rows; A.before += DC_MAX_SEQS) {
        A.rows = a.rows - A.before < DC_MAX_SEQS ? a.rows - A.before : DC_MAX_SEQS;
        A.cu = a.cu + A.before;
        if (a.slot) A.slot = a.slot + A.before;
        const long long items = (long long)A.rows * A.H * ((A.V + DC_VW - 1) / DC_VW);
        delta_chunk_kernel<T><<<(unsigned)(items < sms ? items : sms), DC_THREADS, sizeof(DcSmem), stream>>>(A, maps);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

bool delta_chunk_fits(const DeltaArgs &a)
{
    // Sequences of up to 10 tokens on average, and a single one of up to 20, go token by token (empty and
    // padded ones count, since the host knows the bounds and slots of none; one prompt of 8192 tokens takes
    // 639 us alone, 893 among 500 padded rows, 4810 among 1000): 32
    // heads of 128 columns, bf16, take (tokens a sequence: token by token / here) 10: 39 / 43 us for
    // 16 sequences, 563 / 553 for 256; 12: 43 / 43, 625 / 552; one sequence 10: 8.8 / 13.9, 20: 13.5 / 14.1,
    // 24: 15.1 / 14.1.
    return a.cu && a.dtype != SKETCHSSM_F32 && a.tokens > (a.rows == 1 ? 20LL : 10LL * a.rows);
}

cudaError_t launch_delta_chunk(const DeltaArgs &a, int sms, cudaStream_t stream)
{
    return a.dtype == SKETCHSSM_BF16 ? launch_type<__nv_bfloat16>(a, sms, stream)
                                     : launch_type<__half>(a, sms, stream);
}

}  // namespace sk
