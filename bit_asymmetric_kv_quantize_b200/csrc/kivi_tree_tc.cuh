// kivi_tree_tc.cuh -- attention of drafted tokens over an fp16 cache on the
// 5th-generation tensor cores (tcgen05), accumulators and the cache's numbers
// in tensor memory.
//
// The work is split as kivi_tree.cuh says, in tiles of 128 tokens; a row is a
// (query head of the group, node) pair, `nr` rows (a multiple of 16, at most
// 64) at a time.  Both products are taken transposed, so that the cache's side
// fills the 128 rows of the matrix instruction whatever the tree's size is:
//   S^T [128 tokens x nr]  = K^ [128 x D]      . Q^T   (A = K^, B = Q)
//   O^T [128 (D) x nr]    += V^^T [D x 128]    . P^T   (A = V^^T, B = P)
// A comes from tensor memory: lane = token for keys, whose packed words run
// along a token's channels, and lane = channel for values, whose words run
// along a channel's tokens.  So one thread unpacks whole words into its own
// lane, a warp's 32 lanes are one key group (or one value group) and share its
// scales, and the numbers never pass through shared memory.
//
// Numbers.  A stored key is c s + z.  Rounded to binary16 it would move a score
// by |q||K| 2^-12, more than everything else here together (key channels with
// large values have large z), so it is carried exactly to about 2^-18:
//   c s = c s_hi + c s_lo, s_hi the leading 7 bits of s: c s_hi is exact in
//   binary16 for c < 16, c s_lo is rounded at 2^-18 of c s; two products;
//   sum_d q_d z_d, the same for the 32 tokens of a group, is formed apart (z is
//   one of the cache's fp16 inputs, so it is exact in binary16) by mma.sync and
//   joins the score in binary32.
// Values alike: sum_t p_t z_t of each value group apart.  With them, as one
// more column of ones, the sum of the weights.  s is halved (a binary16 s_hi of
// a 1-bit group of the widest range would overflow), so raw keys and values
// are halved too and the results doubled in binary32.  The weights p are
// rounded to binary16 once, relative 2^-12 on average like the output's own
// rounding.  Scores, maxima, sums and accumulators are binary32.
//
// Running maximum: a row's reference m is raised only when a score of a tile
// exceeds it by more than 14 (in units of log2): weights up to 2^14 lose nothing
// in binary16 or in the binary32 sums.  The weights of a tile are formed with the
// references as they are while the excess is watched; one vote tells whether
// that held, and the rare tile where it did not raises the references, rescales
// O^T in tensor memory and forms its weights again.
//
// Warps: 4 unpack keys and 4 values (one code), 2 groups of 4 softmax, 4 the
// scales and zeros of keys and the zeros' products with the queries, 4 the
// scales and zeros of values and the sums over tokens, one issues the score
// products, one the value products, one the copies (cp.async.bulk of each
// tile's ranges into a ring).  The two softmax groups take every other tile,
// each with its own S^T, O^T and references (two streams, joined at the end of
// a segment), so that one's latencies hide behind the other.  Operands are
// handed over by halves, so that one half is unpacked while the products of the
// other run.  A role's code is a small loop: together they have to fit the
// instruction cache (with the roles unrolled, 369 KB of code, the kernel took
// four times as long).  All waits are bounded: one that runs out marks the block
// dead, whose further waits return at once and whose results are NaN.
#pragma once

#include <type_traits>

#include "kivi_tree.cuh"

namespace kivi {
namespace {

constexpr int kTcTile = 128;        // tokens
constexpr int kTcWarps = 27;
constexpr int kTcThreads = kTcWarps * 32;
constexpr float kTcSlack = 14.0f;   // log2 units a score may exceed m by
constexpr float kTcNone = -1.0e30f; // reference of a row that has seen nothing

// ---- layouts ---------------------------------------------------------------
template <int D, int BITS, int MB>
struct TcGeo {
  using Lt = Layout<D, BITS>;
  static constexpr int E = Lt::E, WB = Lt::WB, WK = Lt::WK, NJ = Lt::NJ;
  // a stage of the ring: 4 subtiles of 32 tokens, array after array
  static constexpr int KC = kTile * WK * 4;              // bytes of a subtile
  static constexpr int KM = D * MB;
  static constexpr int VC = kTile / E * WB * D * 4;
  static constexpr int VM = kTile * NJ * MB;
  static constexpr int O_KC = 0;
  static constexpr int O_KS = O_KC + 4 * KC;
  static constexpr int O_KZ = O_KS + 4 * KM;
  static constexpr int O_VC = O_KZ + 4 * KM;
  static constexpr int O_VS = O_VC + 4 * VC;
  static constexpr int O_VZ = O_VS + 4 * VM;
  static constexpr int STAGE = O_VZ + 4 * VM;
  static constexpr int NST = 3;
  // shared memory
  static constexpr int S_RING = 0;
  static constexpr int S_Q = S_RING + NST * STAGE;       // B operand, [64 rows][D]
  static constexpr int S_P = S_Q + 64 * D * 2;           // 2 x [64 rows][128 tokens]
  static constexpr int P_B = 64 * 128 * 2;
  static constexpr int S_RAW = S_P + 2 * P_B;            // raw values [128 tokens][D]
  static constexpr int S_KSC = S_RAW + 128 * D * 2;      // 2 x 4 groups x D x (hi, lo) halves
  static constexpr int S_VSC = S_KSC + 2 * 4 * D * 4;    // 2 x 4 groups x 128 x (hi, lo)
  static constexpr int S_ZK = S_VSC + 2 * 4 * 128 * 4;   // 2 x [4 groups][64 rows] float
  static constexpr int S_OFF = S_ZK + 2 * 4 * 64 * 4;    // [2 streams][4 warps][64 rows] float
  static constexpr int S_WMAX = S_OFF + 2 * 4 * 64 * 4;  // the same
  static constexpr int S_M = S_WMAX + 2 * 4 * 64 * 4;    // [2 streams][64 rows]
  static constexpr int S_F = S_M + 2 * 64 * 4;           // the same
  static constexpr int S_LZ = S_F + 2 * 64 * 4;          // [2 streams][64 rows][8]
  static constexpr int S_MASK = S_LZ + 2 * 64 * 8 * 4;   // [256][8] words
  // zeros as binary16 in operand order, rows padded against bank conflicts:
  // keys 4 groups x D, values 8 rows x 128 tokens (4 groups, ones, nothing)
  static constexpr int ZLD = 136;
  static constexpr int S_ZH = S_MASK + 256 * 8 * 4;
  static constexpr int S_ZV = S_ZH + 2 * 4 * ZLD * 2;    // 2 x (both tables)
  static constexpr int BYTES = S_ZV + 2 * 8 * ZLD * 2;
};

// Position of code i of a block of E in the order of the operands: the pair
// (i, i + E/2) of a block is one 32-bit register.
template <int E>
__host__ __device__ constexpr int tc_pos(int i) {
  return i / E * E + 2 * (i % (E / 2)) + (i % E >= E / 2 ? 1 : 0);
}
template <int E>
__host__ __device__ constexpr int tc_elem(int k) {
  return k / E * E + (k % E >> 1) + (k & 1) * (E / 2);
}

// ---- PTX ---------------------------------------------------------------------
__device__ __forceinline__ uint32_t tc_smem(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}
// Barriers go by their 32-bit shared address.
__device__ __forceinline__ void tc_bar_init(uint32_t b, int n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(b), "r"(n) : "memory");
}
__device__ __forceinline__ void tc_arrive(uint32_t b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(b) : "memory");
}
__device__ __forceinline__ void tc_expect(uint32_t b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(b), "r"(bytes)
               : "memory");
}
// Waits for phase `n` (counted from 0) of a barrier; bounded: rounds of 4096 tries,
// between which a dead block gives up, and some seconds of them in all.  (Tries
// without a time limit: with one they sleep, and wake late.)
__device__ __forceinline__ void tc_wait(uint32_t b, int n, volatile int* dead) {
#pragma unroll 1
  for (int rounds = 0; rounds < (1 << 15); ++rounds) {
    uint32_t left;  // tries left, 0: none of them saw the phase end
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .u32 k;\n\t"
        "mov.u32 k, 4096;\n\t"
        "TRY:\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra DONE;\n\t"
        "sub.u32 k, k, 1;\n\t"
        "setp.ne.u32 p, k, 0;\n\t"
        "@p bra TRY;\n\t"
        "DONE:\n\t"
        "mov.u32 %0, k;\n\t}"
        : "=r"(left)
        : "r"(b), "r"(n & 1)
        : "memory");
    if (left != 0 || *dead) return;
  }
  *dead = 1;
}
__device__ __forceinline__ void tc_copy(uint32_t dst, const void* src, uint32_t bytes, uint32_t b) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          dst),
      "l"(src), "r"(bytes), "r"(b)
      : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// 8 / 16 columns of the warp's 32 lanes.
__device__ __forceinline__ void tc_st8(uint32_t t, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(t),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]));
}
__device__ __forceinline__ void tc_ld16(uint32_t t, float (&r)[16]) {
  uint32_t u[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]),
        "=r"(u[7]), "=r"(u[8]), "=r"(u[9]), "=r"(u[10]), "=r"(u[11]), "=r"(u[12]), "=r"(u[13]),
        "=r"(u[14]), "=r"(u[15])
      : "r"(t));
  tc_wait_ld();
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __uint_as_float(u[i]);
}
__device__ __forceinline__ void tc_st16(uint32_t t, const float (&r)[16]) {
  uint32_t u[8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(r[8 * h + i]);
    tc_st8(t + 8 * h, u);
  }
}
// Four columns, for the loops that run seldom.
__device__ __forceinline__ void tc_ld4(uint32_t t, float (&r)[4]) {
  uint32_t u[4];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3])
               : "r"(t));
  tc_wait_ld();
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = __uint_as_float(u[i]);
}
// Instruction descriptor of kind::f16: D binary32, A and B binary16, A K-major.
__device__ __forceinline__ uint32_t tc_idesc(int n, bool b_mn) {
  return (1u << 4) | (b_mn ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}
// Shared-memory descriptor without swizzle: 8 x 16-byte core matrices.
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | ((uint64_t)(lbo >> 4) << 16) |
         ((uint64_t)(sbo >> 4) << 32) | (1ULL << 46);
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                       bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
      : "memory");
}
__device__ __forceinline__ void tc_commit(uint32_t b) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(b)
               : "memory");
}
// A row of K-slices of one product: 8 columns of A and 256 bytes of B each.
template <int KS>
__device__ __forceinline__ void tc_mma_row(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                           bool add) {
#pragma unroll 2
  for (int ks = 0; ks < KS; ++ks) tc_mma(d, a + 8 * ks, b + 16 * ks, idesc, add || ks > 0);
}
// One lane of the warp, the same each time.
__device__ __forceinline__ bool tc_elect() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ float tc_warp_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float tc_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void tc_mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                            uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool TRANS>
__device__ __forceinline__ void tc_ldm(uint32_t (&a)[4], uint32_t addr) {
  if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
                 : "r"(addr)
                 : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(a[0]), "=r"(a[1]), "=r"(a[2]), "=r"(a[3])
                 : "r"(addr)
                 : "memory");
}
// All warps but the copying one, which runs ahead over the segments.
__device__ __forceinline__ void tc_sync_segment() {
  tc_fence_before();
  asm volatile("bar.sync 3, %0;" ::"n"(kTcThreads - 32) : "memory");
  tc_fence_after();
}
// Barrier of softmax group `sg` (barriers 1 and 2).
__device__ __forceinline__ void tc_group(int sg) {
  if (sg == 0)
    asm volatile("bar.sync 1, 128;" ::: "memory");
  else
    asm volatile("bar.sync 2, 128;" ::: "memory");
}
// Barriers of the four warps of the zeros' products, of those that unpack values
// and of those of the sums.
__device__ __forceinline__ void tc_zeros_sync() { asm volatile("bar.sync 4, 128;" ::: "memory"); }
__device__ __forceinline__ void tc_values_sync() { asm volatile("bar.sync 6, 128;" ::: "memory"); }
__device__ __forceinline__ void tc_sums_sync() { asm volatile("bar.sync 5, 128;" ::: "memory"); }
// Barrier of the group that tells whether any of its threads has `x`.
__device__ __forceinline__ bool tc_group_any(int sg, bool x) {
  uint32_t r;
  if (sg == 0)
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred.aligned q, 1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
        "barrier.cta.red.or.pred.aligned q, 2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"((uint32_t)x)
        : "memory");
  return r != 0;
}

// ---- codes as binary16 ---------------------------------------------------------
// The eight pairs of registers 8 q .. 8 q + 7 of a lane (16 codes in operand
// order) as exact binary16 integers.  A pair (i, i + E/2) of a word has its
// codes in the two 16-bit halves, at bit BITS * i of each; a mask leaves it at
// bit e < 10 of the half, 0x6400 | (c << e) is 1024 + c 2^e, and one fused
// multiply-add by 2^-e gives c.
__device__ __forceinline__ uint32_t tc_hfma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t tc_hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
template <int E_BIT>
__device__ __forceinline__ uint32_t tc_code(uint32_t masked) {
  if constexpr (E_BIT == 0) {
    uint32_t d;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(masked | 0x64006400u), "r"(0xE400E400u));
    return d;
  } else {
    constexpr uint32_t inv = (uint32_t)(15 - E_BIT) << 10;            // 2^-e
    constexpr uint32_t off = 0x8000u | ((uint32_t)(25 - E_BIT) << 10);  // -2^(10 - e)
    return tc_hfma2(masked | 0x64006400u, inv | (inv << 16), off | (off << 16));
  }
}
// Pair I of a block whose words are w[0 .. WB).
template <int BITS, int I>
__device__ __forceinline__ uint32_t tc_pair(const uint32_t* w) {
  if constexpr (BITS == 3) {
    constexpr int e = I & 7, sh = I < 8 ? 0 : 8;
    constexpr uint32_t m = 0x00010001u << e;
    const uint32_t p = ((w[0] >> sh) & m) | (((w[1] >> sh) << 1) & (m << 1)) |
                       (((w[2] >> sh) << 2) & (m << 2));
    return tc_code<e>(p);
  } else {
    constexpr int per = 10 / BITS;  // pairs whose codes end below bit 10 of the half
    constexpr int sh = I / per * per * BITS, e = I % per * BITS;
    constexpr uint32_t m = ((1u << BITS) - 1u) * 0x00010001u << e;
    return tc_code<e>((sh ? w[0] >> sh : w[0]) & m);
  }
}
// What a loop over a lane's words takes at a time: kUnit codes in kUnitW words.
template <int BITS>
struct TcUnit {
  static constexpr int E = BITS == 3 ? 32 : 32 / BITS, WB = BITS == 3 ? 3 : 1;
  static constexpr int kUnit = E < 16 ? 16 : E;
  static constexpr int kUnitW = kUnit / E * WB;
};
// 16 of a unit's codes, registers 8 HALF .. of its part of the operand row.
template <int BITS, int HALF>
__device__ __forceinline__ void tc_codes16(const uint32_t* w, uint32_t (&c)[8]) {
  if constexpr (BITS == 4) {
    c[0] = tc_pair<4, 0>(w);
    c[1] = tc_pair<4, 1>(w);
    c[2] = tc_pair<4, 2>(w);
    c[3] = tc_pair<4, 3>(w);
    c[4] = tc_pair<4, 0>(w + 1);
    c[5] = tc_pair<4, 1>(w + 1);
    c[6] = tc_pair<4, 2>(w + 1);
    c[7] = tc_pair<4, 3>(w + 1);
  } else {
    c[0] = tc_pair<BITS, 8 * HALF + 0>(w);
    c[1] = tc_pair<BITS, 8 * HALF + 1>(w);
    c[2] = tc_pair<BITS, 8 * HALF + 2>(w);
    c[3] = tc_pair<BITS, 8 * HALF + 3>(w);
    c[4] = tc_pair<BITS, 8 * HALF + 4>(w);
    c[5] = tc_pair<BITS, 8 * HALF + 5>(w);
    c[6] = tc_pair<BITS, 8 * HALF + 6>(w);
    c[7] = tc_pair<BITS, 8 * HALF + 7>(w);
  }
}
// Half of s in two binary16 parts: its leading 7 bits, and the rest.
__device__ __forceinline__ void tc_split(float s, __half* hi, __half* lo) {
  s *= 0.5f;
  const float h = __uint_as_float(__float_as_uint(s) & 0xFFFE0000u);
  *hi = __float2half_rn(h);
  *lo = __float2half_rn(s - __half2float(*hi));
}
// 16 codes times their scales (8 pairs of s_hi and of s_lo from shared memory, one
// address for the whole warp) into the two planes.
__device__ __forceinline__ void tc_put16(uint32_t t_hi, uint32_t t_lo, const uint32_t (&c)[8],
                                         const uint4* hi, const uint4* lo) {
  uint32_t r[8];
  const uint4 a = hi[0], b = hi[1];
  r[0] = tc_hmul2(c[0], a.x);
  r[1] = tc_hmul2(c[1], a.y);
  r[2] = tc_hmul2(c[2], a.z);
  r[3] = tc_hmul2(c[3], a.w);
  r[4] = tc_hmul2(c[4], b.x);
  r[5] = tc_hmul2(c[5], b.y);
  r[6] = tc_hmul2(c[6], b.z);
  r[7] = tc_hmul2(c[7], b.w);
  tc_st8(t_hi, r);
  const uint4 e = lo[0], f = lo[1];
  r[0] = tc_hmul2(c[0], e.x);
  r[1] = tc_hmul2(c[1], e.y);
  r[2] = tc_hmul2(c[2], e.z);
  r[3] = tc_hmul2(c[3], e.w);
  r[4] = tc_hmul2(c[4], f.x);
  r[5] = tc_hmul2(c[5], f.y);
  r[6] = tc_hmul2(c[6], f.z);
  r[7] = tc_hmul2(c[7], f.w);
  tc_st8(t_lo, r);
}
// Some units of a lane's words (`stride` words apart) into its row of the two planes;
// hi, lo: the parts of their scales.  The loop stays a loop: the kernel's roles share
// the instruction cache.
template <int BITS>
__device__ __forceinline__ void tc_unpack(uint32_t t_hi, const uint32_t* words, int stride,
                                          const uint4* hi, const uint4* lo, int units) {
  using U = TcUnit<BITS>;
  constexpr int H = U::kUnit / 16;
#pragma unroll(H == 2 ? 1 : 2)
  for (int u = 0; u < units; ++u) {
    uint32_t w[U::kUnitW], c[8];
#pragma unroll
    for (int i = 0; i < U::kUnitW; ++i) w[i] = words[i * stride];
    words += U::kUnitW * stride;
    tc_codes16<BITS, 0>(w, c);
    tc_put16(t_hi, t_hi + 64, c, hi, lo);
    if constexpr (H == 2) {
      tc_codes16<BITS, 1>(w, c);
      tc_put16(t_hi + 8, t_hi + 72, c, hi + 2, lo + 2);
    }
    hi += 2 * H;
    lo += 2 * H;
    t_hi += 8 * H;
  }
}
// Eight adjacent raw elements; aligned: by one 16-byte load.
__device__ __forceinline__ uint4 tc_raw8(const __half* p, bool aligned) {
  if (aligned) return *reinterpret_cast<const uint4*>(p);
  uint16_t v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __half_as_ushort(p[i]);
  return make_uint4(v[0] | (uint32_t)v[1] << 16, v[2] | (uint32_t)v[3] << 16,
                    v[4] | (uint32_t)v[5] << 16, v[6] | (uint32_t)v[7] << 16);
}

// Two runs of eight raw elements, halved, in operand order: pairs (x_j, y_j), or
// for blocks of 8 (x_j, x_j+4), then y.  (Halving keeps infinities and NaN.)
template <int E>
__device__ __forceinline__ void tc_raw_pairs(const uint4& x, const uint4& y, uint32_t (&r)[8]) {
  if constexpr (E >= 16) {
    r[0] = __byte_perm(x.x, y.x, 0x5410);
    r[1] = __byte_perm(x.x, y.x, 0x7632);
    r[2] = __byte_perm(x.y, y.y, 0x5410);
    r[3] = __byte_perm(x.y, y.y, 0x7632);
    r[4] = __byte_perm(x.z, y.z, 0x5410);
    r[5] = __byte_perm(x.z, y.z, 0x7632);
    r[6] = __byte_perm(x.w, y.w, 0x5410);
    r[7] = __byte_perm(x.w, y.w, 0x7632);
  } else {
    r[0] = __byte_perm(x.x, x.z, 0x5410);
    r[1] = __byte_perm(x.x, x.z, 0x7632);
    r[2] = __byte_perm(x.y, x.w, 0x5410);
    r[3] = __byte_perm(x.y, x.w, 0x7632);
    r[4] = __byte_perm(y.x, y.z, 0x5410);
    r[5] = __byte_perm(y.x, y.z, 0x7632);
    r[6] = __byte_perm(y.y, y.w, 0x5410);
    r[7] = __byte_perm(y.y, y.w, 0x7632);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) r[j] = tc_hmul2(r[j], 0x38003800u);
}
// 128 raw tokens from `first` on (the window's r tokens at wp, then the drafted ones
// at dp up to n) into rows of D in shared memory, by the 128 threads of the values'
// warps.
template <int D>
__device__ __forceinline__ void tc_stage_raw(uint4* dst, int th, const __half* wp, const __half* dp,
                                             int first, int r, int n) {
  const bool al = ((uintptr_t)dp & 15) == 0;
#pragma unroll 4
  for (int j = 0; j < D / 8; ++j) {
    const int k = th + 128 * j, i = first + k / (D / 8), c = k % (D / 8) * 8;
    uint4 x = make_uint4(0, 0, 0, 0);
    if (i < r)
      x = *reinterpret_cast<const uint4*>(wp + i * D + c);
    else if (i < n)
      x = tc_raw8(dp + (i - r) * D + c, al);
    dst[k] = x;
  }
  tc_values_sync();
}
// C0 .. C1 of a lane's raw key row, halved, into its operand row: 16 places are two
// runs of 8 channels E / 2 apart (or two blocks of 8 channels).  src null: zeros.
template <int E>
__device__ __forceinline__ void tc_raw_keys(uint32_t t_hi, const __half* src, int c0, int c1) {
  const bool al = ((uintptr_t)src & 15) == 0;
#pragma unroll 2
  for (int c = c0; c < c1; ++c) {
    const int e0 = E >= 16 ? 16 * c / E * E + 16 * c % E / 2 : 16 * c;
    uint4 x = make_uint4(0, 0, 0, 0), y = x;
    if (src != nullptr) {
      x = tc_raw8(src + e0, al);
      y = tc_raw8(src + e0 + (E >= 16 ? E / 2 : 8), al);
    }
    uint32_t r[8];
    tc_raw_pairs<E>(x, y, r);
    tc_st8(t_hi + 8 * c, r);
  }
}
// Places 16 c0 .. 16 c1 - 1 of a lane's channel of 128 raw tokens (`v`, rows of D
// in shared memory), halved, into its operand row.  Infinities and NaN are left out
// (they join at the segment's end, for the rows that attend to them); returns
// whether there were any.
template <int D, int E>
__device__ __forceinline__ bool tc_raw_values(uint32_t t_hi, const __half* v, int c0, int c1) {
  uint32_t odd = 0;
#pragma unroll 1
  for (int c = c0; c < c1; ++c) {
    const __half* s0 = v + (E >= 16 ? 16 * c / E * E + 16 * c % E / 2 : 16 * c) * D;
    const __half* s1 = s0 + (E >= 16 ? E / 2 : 8) * D;
    uint32_t a[8], b[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      a[k] = __half_as_ushort(s0[k * D]);
      b[k] = __half_as_ushort(s1[k * D]);
    }
    const uint4 x = make_uint4(a[0] | a[1] << 16, a[2] | a[3] << 16, a[4] | a[5] << 16, a[6] | a[7] << 16);
    const uint4 y = make_uint4(b[0] | b[1] << 16, b[2] | b[3] << 16, b[4] | b[5] << 16, b[6] | b[7] << 16);
    uint32_t q[8];
    tc_raw_pairs<E>(x, y, q);
#pragma unroll
    for (int j = 0; j < 8; ++j) {  // exponent bits all set
      const uint32_t f = ((q[j] & 0x7C007C00u) + 0x04000400u) & 0x80008000u;
      odd |= f;
      q[j] &= ~((f >> 15) * 0xFFFFu);
    }
    tc_st8(t_hi + 8 * c, q);
  }
  return odd != 0;
}

// Whether rows row0 .. row0 + 15 see drafted token `node`, one bit each.
__device__ __forceinline__ uint32_t tc_seen(const uint32_t* mask_s, int node, int row0, int N) {
  uint32_t bits = 0;
  int q = row0 % N;
#pragma unroll 1
  for (int e = 0; e < 16; ++e) {
    bits |= ((mask_s[q * 8 + (node >> 5)] >> (node & 31)) & 1u) << e;
    if (++q == N) q = 0;
  }
  return bits;
}

// Tensor-memory columns.
constexpr uint32_t kTKhi = 0, kTKlo = 64, kTVhi = 128, kTVlo = 192, kTO = 256, kTS = 384;

// Barriers, 8 bytes each, by their number.
struct TcBar {
  static constexpr int raw_full = 0, raw_empty = 3;  // [stage]
  // scales' parts set out for the unpacking warps: [keys, values][tile parity]
  static constexpr int sc_full = 6, sc_free = 10;
  // halves of the operands in tensor memory: [keys, values][half]
  static constexpr int a_full = 14, a_free = 18;
  static constexpr int s_full = 22, s_empty = 24;  // [stream], and those that follow
  static constexpr int p_full = 26, pv_done = 28, h_done = 30, z_full = 32, z_empty = 34;
  static constexpr int N = 36;
};

// One segment: tiles [t0, t0 + nt) of a group.
struct TcSeg {
  long long b, unit, n_q;
  int t0, nt, tq;      // first tile, tiles, tiles of quantized tokens
  int r, row0, nrows;  // nrows: rows of this block that exist
  bool whole, ok;
};
// A block's walk over its range: sequence, KV head, row block, tile, tiles left.
struct TcWalk {
  long long b, left;
  int h, rb, t;
};

template <int D, int BITS, typename M>
__global__ void __launch_bounds__(kTcThreads, 1) tree_tc_kernel(TreeArgs a, TreePlan p) {
  using Ge = TcGeo<D, BITS, (int)sizeof(M)>;
  constexpr int E = Ge::E, WK = Ge::WK, NJ = Ge::NJ;
  constexpr int KS = D / 16;  // k-slices of the scores
  extern __shared__ __align__(128) unsigned char sm[];
  __shared__ uint64_t s_bars[TcBar::N];
  __shared__ TcWalk s_walk;
  __shared__ uint32_t s_tmem;
  __shared__ int s_dead, s_odd;
  __shared__ int s_poison[2];   // [segment parity]
  __shared__ int s_resc[2];     // [stream]: the tile's rows were rescaled
  volatile int* dead = &s_dead;
  const uint32_t bar0 = tc_smem(s_bars), sm0 = tc_smem(sm);
  auto bar = [&](int k) -> uint32_t { return bar0 + 8u * (uint32_t)k; };
  // what a whole warp shares is broadcast, so that it lives in uniform registers
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int rows = a.gq * a.N, mw = (a.N + 31) / 32;
  const int nr = p.rb, nch = nr / 16;

  // ---- set-up
  if (warp == 24) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     tc_smem(&s_tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 0) {
    TreeAt at = tree_find(a, p, 0);
    const long long total = at.total, W = tree_range(p, total), x = blockIdx.x * W;
    at = tree_find(a, p, x);
    if (lane == 0) {
      s_walk.left = x < total ? min(W, total - x) : 0;
      s_walk.b = at.b;
      if (x < total) {
        const long long ut = tree_seq(a, p, at.b).ut, grp = at.rem / ut;
        s_walk.t = (int)(at.rem - grp * ut);
        s_walk.h = (int)(grp / p.n_rb);
        s_walk.rb = (int)(grp - (long long)s_walk.h * p.n_rb);
      }
    }
  }
  if (tid == 32) {
    s_dead = 0;
    for (int i = 0; i < 2; ++i) s_poison[i] = 0;
    for (int i = 0; i < 3; ++i) {
      tc_bar_init(bar(TcBar::raw_full + i), 1);
      tc_bar_init(bar(TcBar::raw_empty + i), 16);
    }
    for (int i = 0; i < 2; ++i) {
      for (int k = 0; k < 2; ++k) {
        tc_bar_init(bar(TcBar::sc_full + 2 * k + i), 4);
        tc_bar_init(bar(TcBar::sc_free + 2 * k + i), 4);
        tc_bar_init(bar(TcBar::a_full + 2 * k + i), 4);
        tc_bar_init(bar(TcBar::a_free + 2 * k + i), 1);
      }
      tc_bar_init(bar(TcBar::s_full + i), 1);
      tc_bar_init(bar(TcBar::s_empty + i), 4);
      tc_bar_init(bar(TcBar::p_full + i), 4);
      tc_bar_init(bar(TcBar::pv_done + i), 1);
      tc_bar_init(bar(TcBar::h_done + i), 4);
      tc_bar_init(bar(TcBar::z_full + i), 4);
      tc_bar_init(bar(TcBar::z_empty + i), 4);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  for (int i = tid; i < 2 * 8 * Ge::ZLD; i += kTcThreads)
    reinterpret_cast<__half*>(sm + Ge::S_ZV)[i] = __float2half_rn(i / Ge::ZLD % 8 == 4 ? 1.0f : 0.0f);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
  TcWalk walk = s_walk;

  // streams: tiles of even and of odd count
  float* m_s = reinterpret_cast<float*>(sm + Ge::S_M);    // [stream][64]
  float* f_s = reinterpret_cast<float*>(sm + Ge::S_F);    // [stream][64]
  float* zk_s = reinterpret_cast<float*>(sm + Ge::S_ZK);  // [stream][group][64]
  float* lz_s = reinterpret_cast<float*>(sm + Ge::S_LZ);  // [stream][64][8]
  uint32_t* mask_s = reinterpret_cast<uint32_t*>(sm + Ge::S_MASK);

  // A range ends within a group at most at its own end: segments after the first
  // begin with a group.
  auto next_seg = [&](TcWalk& w) -> TcSeg {
    const TreeSeq q = tree_seq(a, p, w.b);
    TcSeg g;
    g.t0 = w.t;
    g.nt = (int)min(q.ut - w.t, w.left);
    g.b = w.b;
    g.unit = w.b * a.Hkv + w.h;
    g.row0 = w.rb * nr;
    g.nrows = min(rows - g.row0, nr);
    g.n_q = q.n_q;
    g.r = q.r;
    g.ok = q.ok;
    g.tq = q.ok ? (int)((q.n_q + kTcTile - 1) / kTcTile) : 0;
    g.whole = w.t == 0 && g.nt == q.ut;
    w.left -= g.nt;
    w.t = 0;
    if (++w.rb == p.n_rb) {
      w.rb = 0;
      if (++w.h == a.Hkv) {
        w.h = 0;
        ++w.b;
      }
    }
    return g;
  };

  if (warp == 26) {
    // ==== copies: runs ahead over all segments; the ring alone holds it back.
    // Lane i < 4 copies subtile i.
    int st = 0;
    const long long Ts = store_tokens(a.c);
    while (walk.left > 0) {
      const TcSeg g = next_seg(walk);
      for (int t = g.t0; t < min(g.t0 + g.nt, g.tq); ++t, ++st) {
        const int s = st % Ge::NST;
        if (st >= Ge::NST) tc_wait(bar(TcBar::raw_empty + s), st / Ge::NST - 1, dead);
        const long long tile = t * 4LL + lane;
        long long su = 0, stl = 0;
        const bool have = lane < 4 && tile < g.n_q / kTile && store_tile(a.c, g.unit, tile, &su, &stl);
        const int n = __popc(__ballot_sync(0xffffffffu, have));
        const uint32_t fb = bar(TcBar::raw_full + s);
        if (lane == 0) tc_expect(fb, n * (Ge::KC + 2 * Ge::KM + Ge::VC + 2 * Ge::VM));
        __syncwarp();
        if (have && !*dead) {
          using Lt = Layout<D, BITS>;
          const uint32_t dst = sm0 + Ge::S_RING + s * Ge::STAGE;
          const long long km = su * Lt::k_meta_unit(Ts) * (int)sizeof(M) + stl * Ge::KM;
          const long long vm = su * Lt::v_meta_unit(Ts) * (int)sizeof(M) + stl * Ge::VM;
          tc_copy(dst + Ge::O_KC + lane * Ge::KC,
                  (const char*)(a.c.k_codes + su * Lt::k_codes_unit(Ts)) + stl * Ge::KC, Ge::KC, fb);
          tc_copy(dst + Ge::O_KS + lane * Ge::KM, (const char*)a.c.k_scale + km, Ge::KM, fb);
          tc_copy(dst + Ge::O_KZ + lane * Ge::KM, (const char*)a.c.k_zero + km, Ge::KM, fb);
          tc_copy(dst + Ge::O_VC + lane * Ge::VC,
                  (const char*)(a.c.v_codes + su * Lt::v_codes_unit(Ts)) + stl * Ge::VC, Ge::VC, fb);
          tc_copy(dst + Ge::O_VS + lane * Ge::VM, (const char*)a.c.v_scale + vm, Ge::VM, fb);
          tc_copy(dst + Ge::O_VZ + lane * Ge::VM, (const char*)a.c.v_zero + vm, Ge::VM, fb);
        }
      }
    }
    // no copy may still be under way when the block ends (bounded again; a dead
    // block has stages without copies, whose waits run out)
    int never = 0;
    for (int i = max(st - Ge::NST, 0); i < st; ++i)
      tc_wait(bar(TcBar::raw_full + (i % Ge::NST)), i / Ge::NST, &never);
    __syncwarp();
  }

  // ==== segments
  // counters of this block: tiles, and tiles that went through the ring
  int it0 = 0, st0 = 0;
  for (int seg = 0; warp < 26 && walk.left > 0; ++seg) {
    const TcSeg g = next_seg(walk);
    const int t1 = g.t0 + g.nt;
    // ---- start of a segment: queries, mask, references, pages
    if (tid == 0) s_odd = 0;
    if (!g.ok) s_poison[seg & 1] = 1;
    if (a.c.bt != nullptr && g.ok) {  // a page outside the pool poisons the group
      const long long i1 = min(t1 * 4LL, g.n_q / kTile);
#pragma unroll 1
      for (long long i = g.t0 * 4LL + tid; i < i1; i += kTcThreads - 32) {
        long long su, stl;
        if (!store_tile(a.c, g.unit, i, &su, &stl)) s_poison[seg & 1] = 1;
      }
    }
    {
      const __half* qp = static_cast<const __half*>(a.q) + (g.unit * rows + g.row0) * D;
      const bool al = ((uintptr_t)qp & 15) == 0;
      // operand order along channels; rows that do not exist are 0
#pragma unroll 1
      for (int i = tid; i < nr * (D / 8); i += kTcThreads - 32) {
        const int row = i / (D / 8), c0 = i % (D / 8) * 8;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (row < g.nrows) x = tc_raw8(qp + row * D + c0, al);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
        unsigned char* q = sm + Ge::S_Q + row / 8 * (D * 16) + row % 8 * 16;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int k = tc_pos<E>(c0 + e);
          *reinterpret_cast<uint16_t*>(q + k / 8 * 128 + k % 8 * 2) = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
        }
      }
#pragma unroll 1
      for (int i = tid; i < a.N * mw; i += kTcThreads - 32)
        mask_s[i / mw * 8 + i % mw] = a.mask[g.b * a.N * mw + i];
      if (tid < 128) m_s[tid] = kTcNone;
    }
    tc_fence_smem();
    tc_sync_segment();

    if (!g.ok) {
    } else if (warp < 8) {
      // ==== keys (lane = token of subtile w) and values (lane = channel of group w),
      // by one code, in halves (keys of 32 channels in one piece)
      using U = TcUnit<BITS>;
      const int vals = warp >> 2, w = warp & 3;
      const int n_codes = vals ? 128 : D, halves = vals || D > 32 ? 2 : 1;
      const int units = n_codes / halves / U::kUnit, cols = n_codes / halves / 2;
      const uint32_t t_hi = tmem + ((uint32_t)(w * 32) << 16) + (vals ? kTVhi : kTKhi);
      const __half* sc0 = reinterpret_cast<const __half*>(sm + (vals ? Ge::S_VSC : Ge::S_KSC)) + w * 2 * n_codes;
      const int o_w = vals ? Ge::O_VC + (w * 32 + lane) * 4 : Ge::O_KC + w * Ge::KC + lane * WK * 4;
      const int w_str = vals ? D : 1;
      const bool act = !vals || w < NJ;
      int it = it0, st = st0;
      for (int t = g.t0; t < t1; ++t, ++it) {
        const int s = st % Ge::NST;
        const bool raw = t >= g.tq;
        const unsigned char* stg = sm + Ge::S_RING + s * Ge::STAGE;
        const int first = (t - g.tq) * kTcTile;  // of the raw tokens
        const __half* src = nullptr;
        if (!raw) {
          // (the scales' writers have waited for the copies)
          tc_wait(bar(TcBar::raw_full + s), st / Ge::NST, dead);
          tc_wait(bar(TcBar::sc_full + 2 * vals + (st & 1)), st >> 1, dead);
        } else if (!vals) {
          // raw tokens: the window, then the drafted ones; halved like s
          const int i = first + w * 32 + lane;
          if (i < g.r)
            src = static_cast<const __half*>(a.c.k_res) + (g.unit * a.c.R + i) * D;
          else if (i < g.r + a.N)
            src = static_cast<const __half*>(a.k) + (g.unit * a.N + (i - g.r)) * D;
        } else {
          tc_stage_raw<D>(reinterpret_cast<uint4*>(sm + Ge::S_RAW), w * 32 + lane,
                          static_cast<const __half*>(a.c.v_res) + g.unit * a.c.R * D,
                          static_cast<const __half*>(a.v) + g.unit * a.N * D, first, g.r, g.r + a.N);
        }
        const __half* sc = sc0 + (st & 1) * 8 * n_codes;
#pragma unroll 1
        for (int h = 0; h < halves; ++h) {
          if (it > 0) tc_wait(bar(TcBar::a_free + 2 * vals + h), it - 1, dead);
          tc_fence_after();
          if (!act) {
          } else if (!raw) {
            tc_unpack<BITS>(t_hi + h * cols, reinterpret_cast<const uint32_t*>(stg + o_w) + h * units * U::kUnitW * w_str,
                            w_str, reinterpret_cast<const uint4*>(sc) + h * (cols / 4),
                            reinterpret_cast<const uint4*>(sc + n_codes) + h * (cols / 4), units);
          } else if (!vals) {
            tc_raw_keys<E>(t_hi, src, h * cols / 8, (h + 1) * cols / 8);
          } else {
            if (tc_raw_values<D, E>(t_hi, reinterpret_cast<const __half*>(sm + Ge::S_RAW) + w * 32 + lane,
                                    h * cols / 8, (h + 1) * cols / 8))
              s_odd = 1;
          }
          tc_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) tc_arrive(bar(TcBar::a_full + 2 * vals + h));
        }
        if (!raw) {
          if (lane == 0) {
            tc_arrive(bar(TcBar::raw_empty + s));
            tc_arrive(bar(TcBar::sc_free + 2 * vals + (st & 1)));
          }
          ++st;
        } else if (vals) {
          tc_values_sync();  // the raw values may be written again
        }
      }
    } else if (warp < 16) {
      // ==== softmax: lane = token; stream sg takes the tiles of its parity
      const int sg = (warp - 8) >> 2, sw = warp & 3;
      const uint32_t t_lane = tmem + ((uint32_t)(sw * 32) << 16) + 64 * sg;
      float* off_s = reinterpret_cast<float*>(sm + Ge::S_OFF) + (sg * 4 + sw) * 64;
      float* wmax_s = reinterpret_cast<float*>(sm + Ge::S_WMAX) + sg * 256;  // + 64 warp
      float* mr_s = m_s + 64 * sg;
      const float* zk = zk_s + (sg * 4 + sw) * 64;
      const float c1 = 2.0f * a.qscale;
      const int pk = tc_pos<E>(sw * 32 + lane);  // the token's place in the second product
      unsigned char* pb = sm + Ge::S_P + sg * Ge::P_B + pk / 8 * 128 + pk % 8 * 16;
      for (int t = g.t0 + ((it0 + sg) & 1); t < t1; t += 2) {
        const int it = it0 + t - g.t0;
        const bool raw = t >= g.tq;
        // the token of this lane: in the cache (all rows see it), drafted, or none
        const long long i = (long long)(raw ? t - g.tq : t) * kTcTile + sw * 32 + lane;
        const bool in = raw ? i < g.r : i < g.n_q;
        const int node = raw && i >= g.r && i < g.r + a.N ? (int)(i - g.r) : -1;
        auto seen = [&](int ch) -> uint32_t {  // 16 bits, one for each row of chunk ch
          return in ? 0xFFFFu : (node < 0 ? 0u : tc_seen(mask_s, node, g.row0 + ch * 16, a.N));
        };
        // what the products of the stream's last tile read may be written again
        if (it >= 2) {
          tc_wait(bar(TcBar::pv_done + sg), (it >> 1) - 1, dead);
          tc_wait(bar(TcBar::h_done + sg), (it >> 1) - 1, dead);
        }
        tc_wait(bar(TcBar::z_full + sg), it >> 1, dead);
        tc_wait(bar(TcBar::s_full + sg), it >> 1, dead);
        tc_fence_after();
        bool resc = false;
#pragma unroll 1
        for (int tries = 0; tries < 2; ++tries) {
          for (int e = lane; e < nr; e += 32) off_s[e] = mr_s[e] - zk[e];
          __syncwarp();
          // ---- weights against the references, and by how much a score exceeds its own
          float over = -__builtin_huge_valf();
#pragma unroll 1
          for (int ch = 0; ch < nch; ++ch) {
            float v[16];
            tc_ld16(t_lane + kTS + ch * 16, v);
            const uint32_t sees = seen(ch);
#pragma unroll
            for (int e4 = 0; e4 < 4; ++e4) {
              const float4 o = *reinterpret_cast<const float4*>(off_s + ch * 16 + 4 * e4);
              v[4 * e4] = fmaf(v[4 * e4], c1, -o.x);
              v[4 * e4 + 1] = fmaf(v[4 * e4 + 1], c1, -o.y);
              v[4 * e4 + 2] = fmaf(v[4 * e4 + 2], c1, -o.z);
              v[4 * e4 + 3] = fmaf(v[4 * e4 + 3], c1, -o.w);
            }
            if (__any_sync(0xffffffffu, sees != 0xFFFFu)) {  // raw tokens, or the end
#pragma unroll
              for (int e = 0; e < 16; ++e)
                if (!((sees >> e) & 1u)) v[e] = -__builtin_huge_valf();
            }
            uint32_t w[8];
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              over = fmaxf(over, fmaxf(v[e], v[e + 1]));
              const __half2 h = __floats2half2_rn(tc_ex2(v[e]), tc_ex2(v[e + 1]));
              w[e / 2] = *reinterpret_cast<const uint32_t*>(&h);
            }
            *reinterpret_cast<uint4*>(pb + (2 * ch) * 2048) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(pb + (2 * ch + 1) * 2048) = make_uint4(w[4], w[5], w[6], w[7]);
          }
          if (!tc_group_any(sg, over > kTcSlack) || tries == 1) break;
          // ---- new references: each warp's maxima, joined
          resc = true;
#pragma unroll 1
          for (int ch = 0; ch < nch; ++ch) {
            float v[16];
            tc_ld16(t_lane + kTS + ch * 16, v);
            const uint32_t sees = seen(ch);
            float mine = kTcNone;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float d = tc_warp_max((sees >> e) & 1u ? fmaf(v[e], c1, zk[ch * 16 + e]) : kTcNone);
              if (lane == e) mine = d;
            }
            if (lane < 16) wmax_s[sw * 64 + ch * 16 + lane] = mine;
          }
          tc_group(sg);
          const int e = sw * 32 + lane;  // a row of each thread
          if (e < nr) {
            const float old = mr_s[e];
            const float mn = fmaxf(fmaxf(fmaxf(wmax_s[e], wmax_s[64 + e]),
                                         fmaxf(wmax_s[128 + e], wmax_s[192 + e])),
                                   old);
            f_s[64 * sg + e] = old == kTcNone ? 0.0f : tc_ex2(old - mn);
            mr_s[e] = mn;
          }
          tc_group(sg);
          if (t - g.t0 >= 2) {  // accumulators so far (their product was waited for above)
#pragma unroll 1
            for (int ch = 0; ch < nch; ++ch) {
              float v[16];
              tc_ld16(t_lane + kTO + ch * 16, v);
#pragma unroll
              for (int k = 0; k < 16; ++k) v[k] *= f_s[64 * sg + ch * 16 + k];
              tc_st16(t_lane + kTO + ch * 16, v);
            }
            tc_wait_st();
          }
        }
        if (lane == 0 && sw == 0) s_resc[sg] = resc;
        tc_fence_before();
        tc_fence_smem();
        __syncwarp();
        if (lane == 0) {
          tc_arrive(bar(TcBar::p_full + sg));
          tc_arrive(bar(TcBar::s_empty + sg));
          tc_arrive(bar(TcBar::z_empty + sg));
        }
      }
    } else if (warp < 20) {
      // ==== keys' scales in two parts, and sum_d q_d z_gd of the tile's four groups for
      // 16-row chunk zw
      const int zw = warp - 16, zt = zw * 32 + lane, n8 = lane >> 2, kq = (lane & 3) * 2;
      int it = it0, st = st0;
      for (int t = g.t0; t < t1; ++t, ++it) {
        const int par = it & 1;
        const bool raw = t >= g.tq;
        __half* zh = reinterpret_cast<__half*>(sm + Ge::S_ZH) + par * 4 * Ge::ZLD;
        if (!raw) {
          const int s = st % Ge::NST;
          const unsigned char* stg = sm + Ge::S_RING + s * Ge::STAGE;
          const M* kz = reinterpret_cast<const M*>(stg + Ge::O_KZ);
          const M* ks = reinterpret_cast<const M*>(stg + Ge::O_KS);
          __half* sc = reinterpret_cast<__half*>(sm + Ge::S_KSC) + (st & 1) * 8 * D;
          tc_wait(bar(TcBar::raw_full + s), st / Ge::NST, dead);
          if (st >= 2) tc_wait(bar(TcBar::sc_free + (st & 1)), (st >> 1) - 1, dead);
#pragma unroll 2
          for (int j = 0; j < 4 * D / 128; ++j) {
            const int i = zt + 128 * j, gr = i / D, c = tc_pos<E>(i % D);
            zh[gr * Ge::ZLD + c] = __float2half_rn(to_f32(kz[i]));
            tc_split(to_f32(ks[i]), &sc[gr * 2 * D + c], &sc[gr * 2 * D + D + c]);
          }
          tc_zeros_sync();
          if (lane == 0) {
            tc_arrive(bar(TcBar::raw_empty + s));
            tc_arrive(bar(TcBar::sc_full + (st & 1)));
          }
          ++st;
        }
        if (it >= 2) tc_wait(bar(TcBar::z_empty + par), (it >> 1) - 1, dead);
        // lane n8 of a column reads group n8's row; columns 4 .. 7 are read by nobody
        const __half* zr = zh + (n8 & 3) * Ge::ZLD + kq;
        if (zw < nch) {
          const int ch = zw;
          float zc[4] = {0.f, 0.f, 0.f, 0.f};
          if (!raw) {
            // rows 16 ch + (lane % 16), channels 16 ks + 8 (lane / 16)
            const int row = 16 * ch + (lane & 15);
            const uint32_t qa =
                (sm0 + Ge::S_Q) + row / 8 * (D * 16) + (lane >> 4) * 128 + row % 8 * 16;
#pragma unroll 4
            for (int ks = 0; ks < KS; ++ks) {
              uint32_t av[4];
              tc_ldm<false>(av, qa + 256 * ks);
              tc_mma16816(zc, av, *reinterpret_cast<const uint32_t*>(zr + 16 * ks),
                          *reinterpret_cast<const uint32_t*>(zr + 16 * ks + 8));
            }
          }
          if (kq < 4) {  // lane: rows n8, n8 + 8; groups kq, kq + 1
            float* z = zk_s + (par * 4 + kq) * 64 + 16 * ch + n8;
            z[0] = zc[0] * a.qscale;
            z[64] = zc[1] * a.qscale;
            z[8] = zc[2] * a.qscale;
            z[72] = zc[3] * a.qscale;
          }
        }
        __syncwarp();
        if (lane == 0) tc_arrive(bar(TcBar::z_full + par));
      }
    } else if (warp < 24) {
      // ==== values' scales in two parts, and the sums over tokens of the weights and of the
      // values' zeros: chunk uw of each stream.  A tile is prepared before the sums of
      // the one before it.
      const int uw = warp - 20, ut = uw * 32 + lane, n8 = lane >> 2, kq = (lane & 3) * 2;
      float acc[2][4];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[k][e] = 0.f;
      int st = st0;
#pragma unroll 1
      for (int t = g.t0; t <= t1; ++t) {
        if (t < t1) {
          const int par = (it0 + t - g.t0) & 1;
          __half* zv = reinterpret_cast<__half*>(sm + Ge::S_ZV) + par * 8 * Ge::ZLD;
          if (t < g.tq) {
            const int s = st % Ge::NST;
            const unsigned char* stg = sm + Ge::S_RING + s * Ge::STAGE;
            const M* vz = reinterpret_cast<const M*>(stg + Ge::O_VZ) + ut * NJ;
            const M* vs = reinterpret_cast<const M*>(stg + Ge::O_VS) + ut * NJ;
            __half* sc = reinterpret_cast<__half*>(sm + Ge::S_VSC) + (st & 1) * 8 * 128 + tc_pos<E>(ut);
            // tokens that do not exist: 0 (their weight 0 times NaN would not be)
            const bool have = ut < g.n_q - (long long)t * kTcTile;
            tc_wait(bar(TcBar::raw_full + s), st / Ge::NST, dead);
            if (st >= 2) tc_wait(bar(TcBar::sc_free + 2 + (st & 1)), (st >> 1) - 1, dead);
#pragma unroll 2
            for (int j = 0; j < NJ; ++j) {
              zv[j * Ge::ZLD + tc_pos<E>(ut)] = __float2half_rn(have ? to_f32(vz[j]) : 0.f);
              tc_split(have ? to_f32(vs[j]) : 0.f, &sc[j * 256], &sc[j * 256 + 128]);
            }
            tc_sums_sync();
            if (lane == 0) {
              tc_arrive(bar(TcBar::raw_empty + s));
              tc_arrive(bar(TcBar::sc_full + 2 + (st & 1)));
            }
            ++st;
          } else {
#pragma unroll
            for (int j = 0; j < NJ; ++j) zv[j * Ge::ZLD + ut] = __ushort_as_half(0);
            tc_sums_sync();
          }
        }
        if (t == g.t0) continue;
        const int it = it0 + t - 1 - g.t0, par = it & 1;
        const __half* zr = reinterpret_cast<const __half*>(sm + Ge::S_ZV) + (par * 8 + n8) * Ge::ZLD + kq;
        // 8 x 8 blocks (tokens x rows) of weights, transposed on the way: rows 16 uw + 0 / 8,
        // tokens 16 ks + 0 / 8
        const int blk = lane >> 3;
        const uint32_t pbase = (sm0 + Ge::S_P + par * Ge::P_B) + uw * 4096 + (blk & 1) * 2048 +
                               (blk >> 1) * 128 + (lane & 7) * 16;
        tc_wait(bar(TcBar::p_full + par), it >> 1, dead);
        if (uw < nch) {
          float x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = par ? acc[1][e] : acc[0][e];
          if (s_resc[par]) {
            const float f0 = f_s[par * 64 + 16 * uw + n8], f1 = f_s[par * 64 + 16 * uw + n8 + 8];
            x[0] *= f0;
            x[1] *= f0;
            x[2] *= f1;
            x[3] *= f1;
          }
#pragma unroll 4
          for (int ks = 0; ks < 8; ++ks) {
            uint32_t av[4];
            tc_ldm<true>(av, pbase + ks * 256);
            tc_mma16816(x, av, *reinterpret_cast<const uint32_t*>(zr + 16 * ks),
                        *reinterpret_cast<const uint32_t*>(zr + 16 * ks + 8));
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            acc[0][e] = par ? acc[0][e] : x[e];
            acc[1][e] = par ? x[e] : acc[1][e];
          }
        }
        __syncwarp();
        if (lane == 0) tc_arrive(bar(TcBar::h_done + par));
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (uw < nch) {
          float* z = lz_s + (64 * k + 16 * uw + n8) * 8 + kq;
          z[0] = acc[k][0];
          z[1] = acc[k][1];
          z[64] = acc[k][2];
          z[65] = acc[k][3];
        }
      }
    } else {
      // ==== score products (warp 24) and value products (25), by halves of the operand
      const int vals = warp - 24;
      const bool one = tc_elect();
      const uint32_t id = tc_idesc(nr, vals);
      const uint64_t desc = vals ? tc_desc((sm0 + Ge::S_P), 128, 2048)
                                 : tc_desc((sm0 + Ge::S_Q), 128, D * 16);
      const int halves = vals || D > 32 ? 2 : 1, ksh = (vals ? 8 : KS) / halves;
      const uint32_t t_a = tmem + (vals ? kTVhi : kTKhi), t_d = tmem + (vals ? kTO : kTS);
      int it = it0;
#pragma unroll 1
      for (int t = g.t0; t < t1; ++t, ++it) {
        const int par = __shfl_sync(0xffffffffu, it & 1, 0);
        const bool lo = t < g.tq;
        bool add = vals && t - g.t0 >= 2;
        if (vals)
          tc_wait(bar(TcBar::p_full + par), it >> 1, dead);
        else if (it >= 2)
          tc_wait(bar(TcBar::s_empty + par), (it >> 1) - 1, dead);
#pragma unroll 1
        for (int h = 0; h < halves; ++h) {
          tc_wait(bar(TcBar::a_full + 2 * vals + h), it, dead);
          tc_fence_after();
          if (one) {
            const uint64_t b = desc + (vals ? par * (Ge::P_B / 16) : 0) + h * ksh * 16;
            const uint32_t aa = t_a + h * ksh * 8;
#pragma unroll 1
            for (int pl = 0; pl < (lo ? 2 : 1); ++pl)
#pragma unroll 2
              for (int ks = 0; ks < ksh; ++ks) {
                tc_mma(t_d + 64 * par, aa + 64 * pl + 8 * ks, b + 16 * ks, id, add);
                add = true;
              }
            tc_commit(bar(TcBar::a_free + 2 * vals + h));
            if (h == halves - 1) tc_commit(vals ? bar(TcBar::pv_done + par) : bar(TcBar::s_full + par));
          }
          add = true;
          __syncwarp();
        }
      }
      --it;
      if (vals) tc_wait(bar(TcBar::pv_done + (it & 1)), it >> 1, dead);  // and all before it
    }
    tc_sync_segment();

    // ---- end of a segment: lane = channel, 4 rows at a time
    if (warp >= 8 && warp < 16) {
      const int sg = (warp - 8) >> 2, sw = warp & 3;
      const int ch_d = sw * 32 + lane;
      const uint32_t t_lane = tmem + kTO + ((uint32_t)(sw * 32) << 16);
      const bool poison = s_poison[seg & 1] != 0 || *dead != 0;
      // streams that took a tile: by the parity of the block's count
      const bool u0 = g.nt > 1 || (it0 & 1) == 0, u1 = g.nt > 1 || (it0 & 1) == 1;
      const int i1 = s_odd ? min((t1 - g.tq) * kTcTile, g.r + a.N) : 0;
      float* part = a.part + (2 * (long long)blockIdx.x + (g.t0 == 0)) * tree_part(p, D);
      __half* out = static_cast<__half*>(a.out) + (g.unit * rows + g.row0) * (long long)D + ch_d;
#pragma unroll 1
      for (int e4 = 4 * sg; e4 < g.nrows && sw < NJ; e4 += 8) {
        float v0[4] = {0.f, 0.f, 0.f, 0.f}, v1[4] = {0.f, 0.f, 0.f, 0.f};
        if (g.ok && u0) tc_ld4(t_lane + e4, v0);
        if (g.ok && u1) tc_ld4(t_lane + 64 + e4, v1);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int row = e4 + e;
          if (row >= g.nrows) break;
          // the streams' parts, against the larger reference
          float m = m_s[row], o = fmaf(2.0f, v0[e], lz_s[8 * row + sw]), l = lz_s[8 * row + 4];
          if (!u0) o = l = 0.f;
          if (u1) {
            const float m1 = m_s[64 + row], mx = fmaxf(m, m1);
            const float w0 = tc_ex2(m - mx), w1 = tc_ex2(m1 - mx);
            o = w0 * o + w1 * fmaf(2.0f, v1[e], lz_s[8 * (64 + row) + sw]);
            l = w0 * l + w1 * lz_s[8 * (64 + row) + 4];
            m = mx;
          }
          // infinite or NaN raw values, of the tokens that the row attends to
#pragma unroll 1
          for (int i = max(g.t0 - g.tq, 0) * kTcTile; i < i1; ++i) {
            const __half w = i < g.r
                                 ? static_cast<const __half*>(a.c.v_res)[(g.unit * a.c.R + i) * D + ch_d]
                                 : static_cast<const __half*>(a.v)[(g.unit * a.N + i - g.r) * D + ch_d];
            if ((__half_as_ushort(w) & 0x7C00u) == 0x7C00u &&
                (i < g.r || (tc_seen(mask_s, i - g.r, g.row0 + row, a.N) & 1u)))
              o += __half2float(w);
          }
          if (poison) {
            o = m = 0.f;
            l = kNaN;
          }
          if (g.whole) {
            out[row * D] = __float2half_rn(l == 0.f ? 0.f : __fdividef(o, l));
          } else {
            part[2 * nr + row * D + ch_d] = o;
            if (ch_d == 0) {
              part[2 * row] = m;
              part[2 * row + 1] = l;
            }
          }
        }
      }
    }
    if (tid == 0) s_poison[(seg & 1) ^ 1] = 0;  // the next segment's
    if (g.ok) {
      it0 += g.nt;
      st0 += max(min(t1, g.tq) - g.t0, 0);
    }
    tc_sync_segment();
  }

  __syncthreads();
  if (warp == 24) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

}  // namespace
}  // namespace kivi
