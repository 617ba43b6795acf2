// kivi_tree_tc.cuh -- attention of drafted tokens over an fp16 cache on the
// 5th-generation tensor cores (tcgen05), accumulators and the cache's numbers
// in tensor memory.
//
// The work is split as kivi_tree.cuh says, in tiles of 128 tokens; a row is a
// (query head of the group, node) pair, `nr` rows (a multiple of 16, at most
// 128) at a time.  Both products are taken transposed, so that the cache's side
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
// exceeds it by more than 8 (in units of log2), since weights up to 2^8 lose
// nothing; that is checked for all rows by one vote, and the rare tile that
// needs it rescales O^T in tensor memory.
//
// Warps: 4 unpack keys, 4 unpack values, 8 softmax (two groups of four, 16
// rows at a time in turn), 4 for the zeros' products and the sums, one issues
// the matrix instructions, one the copies (cp.async.bulk of each tile's six
// ranges into a ring).  All waits are bounded: one that runs out marks the
// block dead, whose further waits return at once and whose results are NaN.
#pragma once

#include <type_traits>

#include "kivi_tree.cuh"

namespace kivi {
namespace {

constexpr int kTcTile = 128;        // tokens
constexpr int kTcWarps = 22;
constexpr int kTcThreads = kTcWarps * 32;
constexpr float kTcSlack = 8.0f;    // log2 units a score may exceed m by
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
  static constexpr int S_Q = S_RING + NST * STAGE;        // B operand, 128 rows
  static constexpr int S_P = S_Q + 128 * D * 2;           // 2 x [128 rows x 128 tokens]
  static constexpr int S_KSC = S_P + 2 * 128 * 128 * 2;   // 4 warps x D x (hi, lo) halves
  static constexpr int S_VSC = S_KSC + 4 * D * 4;         // 4 warps x 128 x (hi, lo)
  static constexpr int S_ZK = S_VSC + 4 * 128 * 4;        // 2 x [4 groups][128 rows] float
  static constexpr int S_OFF = S_ZK + 2 * 4 * 128 * 4;    // [4 warps][128 rows] float
  static constexpr int S_WMAX = S_OFF + 4 * 128 * 4;      // [4 warps][128 rows]
  static constexpr int S_M = S_WMAX + 4 * 128 * 4;        // [128 rows]
  static constexpr int S_F = S_M + 128 * 4;               // 2 x [128 rows]
  static constexpr int S_LZ = S_F + 2 * 128 * 4;          // [128 rows][8]
  static constexpr int S_MASK = S_LZ + 128 * 8 * 4;       // [256][8] words
  // zeros as binary16 in operand order, rows padded against bank conflicts:
  // keys 4 groups x D, values 8 rows x 128 tokens (4 groups, ones, nothing)
  static constexpr int ZLD = 136;
  static constexpr int S_ZH = S_MASK + 256 * 8 * 4;
  static constexpr int S_ZV = S_ZH + 8 * ZLD * 2;         // 2 x
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
__device__ __forceinline__ void tc_bar_init(uint64_t* b, int n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(tc_smem(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void tc_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(tc_smem(b)) : "memory");
}
__device__ __forceinline__ void tc_expect(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(tc_smem(b)),
               "r"(bytes)
               : "memory");
}
// Waits for phase `n` (counted from 0) of a barrier; bounded: each try suspends
// for up to a microsecond, so some seconds at most.
__device__ __forceinline__ void tc_wait(uint64_t* b, int n, volatile int* dead) {
  const uint32_t addr = tc_smem(b), par = (uint32_t)(n & 1);
#pragma unroll 1
  for (int tries = 0; tries < (1 << 21); ++tries) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 1000;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(addr), "r"(par)
        : "memory");
    if (ok || *dead) return;
  }
  *dead = 1;
}
__device__ __forceinline__ void tc_copy(void* dst, const void* src, uint32_t bytes, uint64_t* b) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          tc_smem(dst)),
      "l"(src), "r"(bytes), "r"(tc_smem(b))
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
__device__ __forceinline__ void tc_commit(uint64_t* b) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   tc_smem(b))
               : "memory");
}
// A row of K-slices of one product: 8 columns of A and 256 bytes of B each.
template <int KS>
__device__ __forceinline__ void tc_mma_row(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                           bool add) {
#pragma unroll
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
template <int ID>
__device__ __forceinline__ void tc_named() {
  asm volatile("bar.sync %0, 128;" ::"n"(ID) : "memory");
}
// The same for group `sg` of two (barriers 1 and 2).
__device__ __forceinline__ void tc_group(int sg) {
  if (sg == 0)
    tc_named<1>();
  else
    tc_named<2>();
}
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
// A lane's words (`stride` words apart) into its row of the two planes, N codes; sc:
// their scales' parts, hi[N] and lo[N].  The loop stays a loop: the kernel's roles
// share the instruction cache.
template <int BITS, int N>
__device__ __forceinline__ void tc_unpack(uint32_t t_hi, uint32_t t_lo, const uint32_t* words,
                                          int stride, const __half* sc) {
  using U = TcUnit<BITS>;
  const uint4* hi = reinterpret_cast<const uint4*>(sc);
  const uint4* lo = reinterpret_cast<const uint4*>(sc + N);
#pragma unroll(N / U::kUnit >= 4 ? 2 : 1)
  for (int u = 0; u < N / U::kUnit; ++u) {
    uint32_t w[U::kUnitW], c[8];
#pragma unroll
    for (int i = 0; i < U::kUnitW; ++i) w[i] = words[(u * U::kUnitW + i) * stride];
    constexpr int H = U::kUnit / 16;
    tc_codes16<BITS, 0>(w, c);
    tc_put16(t_hi + 8 * H * u, t_lo + 8 * H * u, c, hi + 2 * H * u, lo + 2 * H * u);
    if constexpr (H == 2) {
      tc_codes16<BITS, 1>(w, c);
      tc_put16(t_hi + 16 * u + 8, t_lo + 16 * u + 8, c, hi + 4 * u + 2, lo + 4 * u + 2);
    }
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

struct TcBars {
  uint64_t raw_full[3], raw_empty[3];
  uint64_t k_full, v_full;
  uint64_t s_full[2], s_empty[2];
  uint64_t p_full[2], pv_done[2], h_done[2];
  uint64_t z_full[2], z_empty[2];
};

// One segment: tiles [t0, t0 + nt) of a group.
struct TcSeg {
  long long b, unit, n_q;
  int t0, nt, tq;      // first tile, tiles, tiles of quantized tokens
  int r, row0, nrows;  // nrows: rows of this block that exist
  bool whole, ok;
};

template <int D, int BITS, typename M>
__global__ void __launch_bounds__(kTcThreads, 1) tree_tc_kernel(TreeArgs a, TreePlan p) {
  using Ge = TcGeo<D, BITS, (int)sizeof(M)>;
  constexpr int E = Ge::E, WK = Ge::WK, NJ = Ge::NJ;
  constexpr int KS = D / 16;  // k-slices of the scores
  extern __shared__ __align__(128) unsigned char sm[];
  __shared__ TcBars bars;
  __shared__ TreeAt s_at;
  __shared__ uint32_t s_tmem;
  __shared__ int s_dead, s_odd;
  __shared__ int s_poison[2];   // [segment parity]
  __shared__ int s_resc[2][8];  // [tile parity][16 rows]: rows were rescaled
  volatile int* dead = &s_dead;
  // what a whole warp shares is broadcast, so that it lives in uniform registers
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;

  // ---- set-up
  if (warp == 20) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     tc_smem(&s_tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 0) {
    TreeAt at = tree_find(a, p, 0);
    const long long total = at.total;
    at = tree_find(a, p, blockIdx.x * tree_range(p, total));
    at.total = total;
    if (lane == 0) s_at = at;
  }
  if (tid == 32) {
    s_dead = 0;
    for (int i = 0; i < 2; ++i) s_poison[i] = 0;
    for (int i = 0; i < 3; ++i) {
      tc_bar_init(&bars.raw_full[i], 1);
      tc_bar_init(&bars.raw_empty[i], 12);
    }
    tc_bar_init(&bars.k_full, 4);
    tc_bar_init(&bars.v_full, 4);
    for (int i = 0; i < 2; ++i) {
      tc_bar_init(&bars.s_full[i], 1);
      tc_bar_init(&bars.s_empty[i], 8);
      tc_bar_init(&bars.p_full[i], 8);
      tc_bar_init(&bars.pv_done[i], 1);
      tc_bar_init(&bars.h_done[i], 4);
      tc_bar_init(&bars.z_full[i], 4);
      tc_bar_init(&bars.z_empty[i], 8);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  for (int i = tid; i < 2 * 8 * Ge::ZLD; i += kTcThreads)
    reinterpret_cast<__half*>(sm + Ge::S_ZV)[i] = __float2half_rn(i / Ge::ZLD % 8 == 4 ? 1.0f : 0.0f);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
  const long long total = s_at.total, W = tree_range(p, total);
  long long x = blockIdx.x * W;
  const long long end = x + W < total ? x + W : total;
  long long sb = s_at.b, rem = s_at.rem;
  const int rows = a.gq * a.N, mw = (a.N + 31) / 32;
  const int nr = p.rb, nch = nr / 16;
  const bool s2 = nr <= 64;  // two S buffers

  float* m_s = reinterpret_cast<float*>(sm + Ge::S_M);
  float* f_s = reinterpret_cast<float*>(sm + Ge::S_F);
  float* zk_s = reinterpret_cast<float*>(sm + Ge::S_ZK);
  float* lz_s = reinterpret_cast<float*>(sm + Ge::S_LZ);
  uint32_t* mask_s = reinterpret_cast<uint32_t*>(sm + Ge::S_MASK);

  // counters of this block: tiles, and tiles that went through the ring; the
  // copying warp runs ahead of the others, over its own walk of the segments
  int it0 = 0, st0 = 0;

  auto next_seg = [&](long long& xx, long long& bb, long long& rr, TcSeg& g) {
    TreeSeq q = tree_seq(a, p, bb);
    const long long gpb = (long long)a.Hkv * p.n_rb;
    while (rr >= gpb * q.ut) {
      rr -= gpb * q.ut;
      ++bb;
      q = tree_seq(a, p, bb);
    }
    const int ut = (int)q.ut, grp = (int)(rr / ut), left = (int)min(end - xx, 1LL << 30);
    g.t0 = (int)(rr - (long long)grp * ut);
    g.nt = ut - g.t0 < left ? ut - g.t0 : left;
    g.b = bb;
    g.unit = bb * a.Hkv + grp / p.n_rb;
    g.row0 = grp % p.n_rb * p.rb;
    g.nrows = rows - g.row0 < nr ? rows - g.row0 : nr;
    g.n_q = q.n_q;
    g.r = q.r;
    g.ok = q.ok;
    g.tq = q.ok ? (int)((q.n_q + kTcTile - 1) / kTcTile) : 0;
    g.whole = g.t0 == 0 && g.nt == ut;
    xx += g.nt;
    rr += g.nt;
  };

  if (warp == 21) {
    // ==== copies: runs ahead over all segments; the ring alone holds it back
    long long xx = x, bb = sb, rr = rem;
    int st = 0;
    if (lane == 0) {
      while (xx < end) {
        TcSeg g;
        next_seg(xx, bb, rr, g);
        if (!g.ok) continue;
        for (int t = g.t0; t < g.t0 + g.nt && t < g.tq; ++t, ++st) {
          const int s = st % Ge::NST;
          if (st >= Ge::NST) tc_wait(&bars.raw_empty[s], st / Ge::NST - 1, dead);
          if (*dead) break;
          unsigned char* dst = sm + Ge::S_RING + s * Ge::STAGE;
          const long long left = (g.n_q - (long long)t * kTcTile) / kTile;
          const int ns = left < 4 ? (int)left : 4;
          const long long Ts = store_tokens(a.c);
          uint32_t bytes = 0;
          for (int pass = 0; pass < 2; ++pass) {
            // contiguous stores: all subtiles at once; paged: one by one
            const int step = a.c.bt ? 1 : ns;
            for (int i = 0; i < ns; i += step) {
              long long su, stl;
              if (!store_tile(a.c, g.unit, t * 4LL + i, &su, &stl)) continue;
              if (pass == 0) {
                bytes += step * (Ge::KC + 2 * Ge::KM + Ge::VC + 2 * Ge::VM);
                continue;
              }
              using Lt = Layout<D, BITS>;
              const unsigned char* kc = (const unsigned char*)(a.c.k_codes + su * Lt::k_codes_unit(Ts)) + stl * Ge::KC;
              const unsigned char* ks = (const unsigned char*)a.c.k_scale + su * Lt::k_meta_unit(Ts) * sizeof(M) + stl * Ge::KM;
              const unsigned char* kz = (const unsigned char*)a.c.k_zero + su * Lt::k_meta_unit(Ts) * sizeof(M) + stl * Ge::KM;
              const unsigned char* vc = (const unsigned char*)(a.c.v_codes + su * Lt::v_codes_unit(Ts)) + stl * Ge::VC;
              const unsigned char* vs = (const unsigned char*)a.c.v_scale + su * Lt::v_meta_unit(Ts) * sizeof(M) + stl * Ge::VM;
              const unsigned char* vz = (const unsigned char*)a.c.v_zero + su * Lt::v_meta_unit(Ts) * sizeof(M) + stl * Ge::VM;
              uint64_t* fb = &bars.raw_full[s];
              tc_copy(dst + Ge::O_KC + i * Ge::KC, kc, step * Ge::KC, fb);
              tc_copy(dst + Ge::O_KS + i * Ge::KM, ks, step * Ge::KM, fb);
              tc_copy(dst + Ge::O_KZ + i * Ge::KM, kz, step * Ge::KM, fb);
              tc_copy(dst + Ge::O_VC + i * Ge::VC, vc, step * Ge::VC, fb);
              tc_copy(dst + Ge::O_VS + i * Ge::VM, vs, step * Ge::VM, fb);
              tc_copy(dst + Ge::O_VZ + i * Ge::VM, vz, step * Ge::VM, fb);
            }
            if (pass == 0) tc_expect(&bars.raw_full[s], bytes);
          }
        }
      }
      // no copy may still be under way when the block ends (bounded again)
      int never = 0;
      for (int i = st > Ge::NST ? st - Ge::NST : 0; i < st; ++i)
        tc_wait(&bars.raw_full[i % Ge::NST], i / Ge::NST, &never);
    }
    __syncwarp();
  }

  // ==== segments
  for (int seg = 0; warp < 21 && x < end; ++seg) {
    TcSeg g;
    next_seg(x, sb, rem, g);
    // ---- start of a segment: queries, mask, references, pages
    if (tid == 0) s_odd = 0;
    if (!g.ok) s_poison[seg & 1] = 1;
    if (a.c.bt != nullptr && g.ok) {  // a page outside the pool poisons the group
      const long long i1 =
          (g.t0 + g.nt) * 4LL < g.n_q / kTile ? (g.t0 + g.nt) * 4LL : g.n_q / kTile;
      for (long long i = g.t0 * 4LL + tid; i < i1; i += kTcThreads - 32) {
        long long su, stl;
        if (!store_tile(a.c, g.unit, i, &su, &stl)) s_poison[seg & 1] = 1;
      }
    }
    {
      const __half* qp = static_cast<const __half*>(a.q) + (g.unit * rows + g.row0) * D;
      // operand order along channels; rows that do not exist are 0
      for (int i = tid; i < nr * D; i += kTcThreads - 32) {
        const int row = i / D, ch = i % D, k = tc_pos<E>(ch);
        const __half v = row < g.nrows ? qp[(long long)row * D + ch] : __ushort_as_half(0);
        *reinterpret_cast<__half*>(sm + Ge::S_Q + row / 8 * (D * 16) + k / 8 * 128 + row % 8 * 16 +
                                   k % 8 * 2) = v;
      }
      for (int i = tid; i < a.N * mw; i += kTcThreads - 32)
        mask_s[i / mw * 8 + i % mw] = a.mask[(g.b * a.N) * mw + i];
      for (int i = tid; i < 128; i += kTcThreads - 32) m_s[i] = kTcNone;
    }
    tc_fence_smem();
    tc_sync_segment();

    if (g.ok) {
      if (warp < 4) {
        // ==== keys: lane = token of subtile `warp`
        const uint32_t t_lane = tmem + ((uint32_t)(warp * 32) << 16);
        __half* sc = reinterpret_cast<__half*>(sm + Ge::S_KSC + warp * D * 4);  // hi[D], lo[D]
        int it = it0, st = st0;
        for (int t = g.t0; t < g.t0 + g.nt; ++t, ++it) {
          if (t < g.tq) {
            const int s = st % Ge::NST;
            tc_wait(&bars.raw_full[s], st / Ge::NST, dead);
            const unsigned char* stg = sm + Ge::S_RING + s * Ge::STAGE;
            const M* ks = reinterpret_cast<const M*>(stg + Ge::O_KS + warp * Ge::KM);
            __syncwarp();
#pragma unroll
            for (int c = lane; c < D; c += 32) {
              __half hi, lo;
              tc_split(to_f32(ks[c]), &hi, &lo);
              sc[tc_pos<E>(c)] = hi;
              sc[D + tc_pos<E>(c)] = lo;
            }
            __syncwarp();
            if (it > 0) tc_wait(&bars.s_full[(it - 1) & 1], (it - 1) >> 1, dead);
            tc_fence_after();
            tc_unpack<BITS, D>(
                t_lane + kTKhi, t_lane + kTKlo,
                reinterpret_cast<const uint32_t*>(stg + Ge::O_KC + warp * Ge::KC) + lane * WK, 1, sc);
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              tc_arrive(&bars.raw_empty[s]);
              tc_arrive(&bars.k_full);
            }
            ++st;
          } else {
            // raw tokens: the window, then the drafted ones; halved like s
            const int i = (t - g.tq) * kTcTile + warp * 32 + lane;
            const __half* src = nullptr;
            if (i < g.r)
              src = static_cast<const __half*>(a.c.k_res) + (g.unit * a.c.R + i) * D;
            else if (i < g.r + a.N)
              src = static_cast<const __half*>(a.k) + (g.unit * a.N + (i - g.r)) * D;
            const bool al = ((uintptr_t)src & 15) == 0;
            if (it > 0) tc_wait(&bars.s_full[(it - 1) & 1], (it - 1) >> 1, dead);
            tc_fence_after();
            // 16 places of the operand order: two runs of 8 channels, E / 2 apart (or
            // two blocks of 8 channels)
#pragma unroll 2
            for (int c = 0; c < D / 16; ++c) {
              const int e0 = E >= 16 ? 16 * c / E * E + 16 * c % E / 2 : 16 * c;
              uint4 x = make_uint4(0, 0, 0, 0), y = x;
              if (src != nullptr) {
                x = tc_raw8(src + e0, al);
                y = tc_raw8(src + e0 + (E >= 16 ? E / 2 : 8), al);
              }
              uint32_t r[8];
              if constexpr (E >= 16) {  // (x_j, y_j)
                r[0] = __byte_perm(x.x, y.x, 0x5410);
                r[1] = __byte_perm(x.x, y.x, 0x7632);
                r[2] = __byte_perm(x.y, y.y, 0x5410);
                r[3] = __byte_perm(x.y, y.y, 0x7632);
                r[4] = __byte_perm(x.z, y.z, 0x5410);
                r[5] = __byte_perm(x.z, y.z, 0x7632);
                r[6] = __byte_perm(x.w, y.w, 0x5410);
                r[7] = __byte_perm(x.w, y.w, 0x7632);
              } else {  // (x_j, x_j+4), then y
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
              tc_st8(t_lane + kTKhi + 8 * c, r);
            }
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) tc_arrive(&bars.k_full);
          }
        }
      } else if (warp < 8) {
        // ==== values: lane = channel of group `vw`
        const int vw = warp - 4;
        const int ch = vw * 32 + lane;
        const uint32_t t_lane = tmem + ((uint32_t)(vw * 32) << 16);
        __half* sc = reinterpret_cast<__half*>(sm + Ge::S_VSC + vw * 128 * 4);  // hi[128], lo[128]
        int it = it0, st = st0;
        for (int t = g.t0; t < g.t0 + g.nt; ++t, ++it) {
          if (t < g.tq) {
            const int s = st % Ge::NST;
            tc_wait(&bars.raw_full[s], st / Ge::NST, dead);
            if (vw < NJ) {
              const unsigned char* stg = sm + Ge::S_RING + s * Ge::STAGE;
              const M* vs = reinterpret_cast<const M*>(stg + Ge::O_VS);
              const long long n = g.n_q - (long long)t * kTcTile;  // tokens that exist
              __syncwarp();
#pragma unroll
              for (int k = lane; k < 128; k += 32) {
                __half hi = __ushort_as_half(0), lo = hi;
                if (k < n) tc_split(to_f32(vs[k * NJ + vw]), &hi, &lo);
                sc[tc_pos<E>(k)] = hi;
                sc[128 + tc_pos<E>(k)] = lo;
              }
              __syncwarp();
              if (it > 0) tc_wait(&bars.pv_done[(it - 1) & 1], (it - 1) >> 1, dead);
              tc_fence_after();
              tc_unpack<BITS, 128>(t_lane + kTVhi, t_lane + kTVlo,
                                   reinterpret_cast<const uint32_t*>(stg + Ge::O_VC) + ch, D, sc);
              tc_wait_st();
              tc_fence_before();
            } else if (it > 0) {
              tc_wait(&bars.pv_done[(it - 1) & 1], (it - 1) >> 1, dead);
            }
            __syncwarp();
            if (lane == 0) {
              tc_arrive(&bars.raw_empty[s]);
              tc_arrive(&bars.v_full);
            }
            ++st;
          } else {
            if (it > 0) tc_wait(&bars.pv_done[(it - 1) & 1], (it - 1) >> 1, dead);
            tc_fence_after();
            if (vw < NJ) {
              const int first = (t - g.tq) * kTcTile, n = g.r + a.N;
              const __half* wp = static_cast<const __half*>(a.c.v_res) + g.unit * a.c.R * D + ch;
              const __half* dp = static_cast<const __half*>(a.v) + g.unit * a.N * D + ch;
              uint32_t odd = 0;
#pragma unroll 1
              for (int c0 = 0; c0 < 128; c0 += 16) {
                uint16_t v[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                  const int i = first + tc_elem<E>(c0 + k);
                  v[k] = i < n ? __half_as_ushort(i < g.r ? wp[i * D] : dp[(i - g.r) * D]) : 0;
                }
                uint32_t r[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  uint32_t u = v[2 * j] | (uint32_t)v[2 * j + 1] << 16;
                  // infinities and NaN join at the segment's end, for the rows that
                  // attend to them
                  const uint32_t x = (((u & 0x7C007C00u) + 0x04000400u) & 0x80008000u);
                  odd |= x;
                  u &= ~((x >> 15) * 0xFFFFu);
                  r[j] = tc_hmul2(u, 0x38003800u);
                }
                tc_st8(t_lane + kTVhi + c0 / 2, r);
              }
              if (odd) s_odd = 1;
              tc_wait_st();
              tc_fence_before();
            }
            __syncwarp();
            if (lane == 0) tc_arrive(&bars.v_full);
          }
        }
      } else if (warp < 16) {
        // ==== softmax: group sg takes the 16-row chunks sg, sg + 2, ..; lane = token
        const int sg = (warp - 8) >> 2, sw = warp & 3;
        const uint32_t t_lane = tmem + ((uint32_t)(sw * 32) << 16);
        float* off_s = reinterpret_cast<float*>(sm + Ge::S_OFF) + sw * 128;
        float* wmax_s = reinterpret_cast<float*>(sm + Ge::S_WMAX) + sw * 128;
        const float c1 = 2.0f * a.qscale;
        const int pk = tc_pos<E>(sw * 32 + lane);  // the token's place in the second product
        int it = it0;
        for (int t = g.t0; t < g.t0 + g.nt; ++t, ++it) {
          const int par = it & 1;
          const bool raw = t >= g.tq;
          const uint32_t t_s = t_lane + kTS + (s2 ? 64 * par : 0);
          // the token of this lane: in the cache (all rows see it), drafted, or none
          const long long i = (long long)(raw ? t - g.tq : t) * kTcTile + sw * 32 + lane;
          bool in = raw ? i < g.r : i < g.n_q;
          const int node = raw && i >= g.r && i < g.r + a.N ? (int)(i - g.r) : -1;
          auto seen = [&](int ch) -> uint32_t {  // 16 bits, one for each row of chunk ch
            return in ? 0xFFFFu : (node < 0 ? 0u : tc_seen(mask_s, node, g.row0 + ch * 16, a.N));
          };
          // what the products two tiles ago read (weights, factors) may be written again
          if (it >= 2) {
            tc_wait(&bars.pv_done[par], (it >> 1) - 1, dead);
            tc_wait(&bars.h_done[par], (it >> 1) - 1, dead);
          }
          tc_wait(&bars.z_full[par], it >> 1, dead);
          for (int e = lane; e < nr; e += 32)
            if (((e >> 4) & 1) == sg) off_s[e] = m_s[e] - zk_s[(par * 4 + sw) * 128 + e];
          __syncwarp();
          tc_wait(&bars.s_full[par], it >> 1, dead);
          tc_fence_after();
          // ---- does any score exceed its row's reference by too much?
          float over = -__builtin_huge_valf();
          for (int ch = sg; ch < nch; ch += 2) {
            float v[16];
            tc_ld16(t_s + ch * 16, v);
            const uint32_t sees = seen(ch);
#pragma unroll
            for (int e4 = 0; e4 < 4; ++e4) {
              const float4 o = *reinterpret_cast<const float4*>(off_s + ch * 16 + 4 * e4);
              const float oo[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float d = fmaf(v[4 * e4 + e], c1, -oo[e]);
                over = fmaxf(over, (sees >> (4 * e4 + e)) & 1u ? d : over);
              }
            }
          }
          const bool need = tc_group_any(sg, over > kTcSlack);
          if (need) {
            // ---- new references: each warp's maxima, joined
            for (int ch = sg; ch < nch; ch += 2) {
              float v[16];
              tc_ld16(t_s + ch * 16, v);
              const uint32_t sees = seen(ch);
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const int row = ch * 16 + e;
                float d = (sees >> e) & 1u ? fmaf(v[e], c1, zk_s[(par * 4 + sw) * 128 + row]) : kTcNone;
                d = warp_max(d);
                if (lane == e) wmax_s[row] = d;
              }
            }
            tc_group(sg);
            const float* wm = reinterpret_cast<const float*>(sm + Ge::S_WMAX);
            for (int e = (sw * 32 + lane); e < nr; e += 128) {
              if (((e >> 4) & 1) != sg) continue;
              const float old = m_s[e];
              const float mn = fmaxf(fmaxf(fmaxf(wm[e], wm[128 + e]), fmaxf(wm[256 + e], wm[384 + e])), old);
              f_s[par * 128 + e] = old == kTcNone ? 0.0f : tc_ex2(old - mn);
              m_s[e] = mn;
            }
            tc_group(sg);
            for (int e = lane; e < nr; e += 32)
              if (((e >> 4) & 1) == sg) off_s[e] = m_s[e] - zk_s[(par * 4 + sw) * 128 + e];
            if (t > g.t0) {
              // ---- accumulators so far, once the product before this one is done
              tc_wait(&bars.pv_done[(it - 1) & 1], (it - 1) >> 1, dead);
              tc_fence_after();
              for (int ch = sg; ch < nch; ch += 2) {
                float v[16];
                tc_ld16(t_lane + kTO + ch * 16, v);
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] *= f_s[par * 128 + ch * 16 + e];
                tc_st16(t_lane + kTO + ch * 16, v);
              }
              tc_wait_st();
            }
            __syncwarp();
          }
          if (lane == 0 && sw == 0)
            for (int ch = sg; ch < nch; ch += 2) s_resc[par][ch] = need;
          // ---- weights
          unsigned char* pb = sm + Ge::S_P + par * 128 * 128 * 2 + pk / 8 * 128 + pk % 8 * 16;
          for (int ch = sg; ch < nch; ch += 2) {
            float v[16];
            tc_ld16(t_s + ch * 16, v);
            const uint32_t sees = seen(ch);
            uint32_t w[8];
#pragma unroll
            for (int e4 = 0; e4 < 4; ++e4) {
              const float4 o = *reinterpret_cast<const float4*>(off_s + ch * 16 + 4 * e4);
              const float oo[4] = {o.x, o.y, o.z, o.w};
              float e[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                e[k] = tc_ex2(fmaf(v[4 * e4 + k], c1, -oo[k]));
                if (!((sees >> (4 * e4 + k)) & 1u)) e[k] = 0.0f;
              }
              const __half2 h0 = __floats2half2_rn(e[0], e[1]), h1 = __floats2half2_rn(e[2], e[3]);
              w[2 * e4] = *reinterpret_cast<const uint32_t*>(&h0);
              w[2 * e4 + 1] = *reinterpret_cast<const uint32_t*>(&h1);
            }
            *reinterpret_cast<uint4*>(pb + (2 * ch) * 2048) = make_uint4(w[0], w[1], w[2], w[3]);
            *reinterpret_cast<uint4*>(pb + (2 * ch + 1) * 2048) = make_uint4(w[4], w[5], w[6], w[7]);
          }
          tc_fence_before();
          tc_fence_smem();
          __syncwarp();
          if (lane == 0) {
            tc_arrive(&bars.s_empty[par]);
            tc_arrive(&bars.z_empty[par]);
            tc_arrive(&bars.p_full[par]);
          }
        }
      } else if (warp < 20) {
        // ==== zeros' products and the sums: chunks hw, hw + 4 of 16 rows
        const int hw = warp - 16;
        float acc[2][4];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[k][e] = 0.f;
        const int n8 = lane >> 2, kq = (lane & 3) * 2, ht = hw * 32 + lane;
        __half* zh = reinterpret_cast<__half*>(sm + Ge::S_ZH);
        int st = st0;
        // the zeros' part of tile t: their products with the queries for its scores,
        // and the values' zeros set out for its sums
        auto zeros = [&](int t, int it) {
          const int par = it & 1;
          __half* zv = reinterpret_cast<__half*>(sm + Ge::S_ZV) + par * 8 * Ge::ZLD;
          const bool raw = t >= g.tq;
          if (!raw) {
            const int s = st % Ge::NST;
            const unsigned char* stg = sm + Ge::S_RING + s * Ge::STAGE;
            const long long n = g.n_q - (long long)t * kTcTile;
            tc_wait(&bars.raw_full[s], st / Ge::NST, dead);
            const M* kz = reinterpret_cast<const M*>(stg + Ge::O_KZ);
            const M* vz = reinterpret_cast<const M*>(stg + Ge::O_VZ);
#pragma unroll 2
            for (int i = ht; i < 4 * D; i += 128)
              zh[i / D * Ge::ZLD + tc_pos<E>(i % D)] = __float2half_rn(to_f32(kz[i]));
#pragma unroll
            for (int j = 0; j < NJ; ++j)
              zv[j * Ge::ZLD + tc_pos<E>(ht)] =
                  ht < n ? __float2half_rn(to_f32(vz[ht * NJ + j])) : __ushort_as_half(0);
            tc_named<4>();
            if (lane == 0) tc_arrive(&bars.raw_empty[s]);
            ++st;
          } else {
#pragma unroll
            for (int j = 0; j < NJ; ++j) zv[j * Ge::ZLD + ht] = __ushort_as_half(0);
            tc_named<4>();
          }
          if (it >= 2) tc_wait(&bars.z_empty[par], (it >> 1) - 1, dead);
          float zc[2][4];
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int e = 0; e < 4; ++e) zc[k][e] = 0.f;
          if (!raw && hw < nch) {
#pragma unroll 2
            for (int ks = 0; ks < KS; ++ks) {
              // rows 4 .. 7 of the table are not there: columns that nothing reads
              const __half* zr = zh + (n8 & 3) * Ge::ZLD + 16 * ks + kq;
              const uint32_t b0 = *reinterpret_cast<const uint32_t*>(zr);
              const uint32_t b1 = *reinterpret_cast<const uint32_t*>(zr + 8);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int ch = hw + 4 * k;
                if (ch < nch) {
                  // rows 16 ch + (lane % 16), channels 16 ks + 8 (lane / 16)
                  uint32_t av[4];
                  const int row = 16 * ch + (lane & 15);
                  tc_ldm<false>(av, tc_smem(sm + Ge::S_Q) + row / 8 * (D * 16) +
                                        (2 * ks + (lane >> 4)) * 128 + row % 8 * 16);
                  tc_mma16816(zc[k], av, b0, b1);
                }
              }
            }
          }
          // lane (row n8, n8 + 8; groups kq, kq + 1)
          if (kq < 4) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int ch = hw + 4 * k;
              if (ch < nch) {
                float* z = zk_s + par * 4 * 128 + 16 * ch + n8;
                z[kq * 128] = zc[k][0] * a.qscale;
                z[(kq + 1) * 128] = zc[k][1] * a.qscale;
                z[kq * 128 + 8] = zc[k][2] * a.qscale;
                z[(kq + 1) * 128 + 8] = zc[k][3] * a.qscale;
              }
            }
          }
          __syncwarp();
          if (lane == 0) tc_arrive(&bars.z_full[par]);
          tc_named<4>();  // the keys' table may be written again
        };
        int it = it0;
        zeros(g.t0, it);
        for (int t = g.t0; t < g.t0 + g.nt; ++t, ++it) {
          const int par = it & 1;
          if (t + 1 < g.t0 + g.nt) zeros(t + 1, it + 1);
          // ---- sums over the tile's tokens
          tc_wait(&bars.p_full[par], it >> 1, dead);
          const __half* zv = reinterpret_cast<const __half*>(sm + Ge::S_ZV) + (par * 8 + n8) * Ge::ZLD + kq;
          const uint32_t pbase = tc_smem(sm + Ge::S_P + par * 128 * 128 * 2);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int ch = hw + 4 * k;
            if (ch < nch) {
              if (s_resc[par][ch]) {
                const float f0 = f_s[par * 128 + 16 * ch + n8], f1 = f_s[par * 128 + 16 * ch + n8 + 8];
                acc[k][0] *= f0;
                acc[k][1] *= f0;
                acc[k][2] *= f1;
                acc[k][3] *= f1;
              }
#pragma unroll 2
              for (int ks = 0; ks < 8; ++ks) {
                // 8 x 8 blocks (tokens x rows), transposed on the way: rows 16 ch + 0 / 8,
                // tokens 16 ks + 0 / 8
                const int blk = lane >> 3;
                uint32_t av[4];
                tc_ldm<true>(av, pbase + (2 * ch + (blk & 1)) * 2048 + (2 * ks + (blk >> 1)) * 128 +
                                     (lane & 7) * 16);
                tc_mma16816(acc[k], av, *reinterpret_cast<const uint32_t*>(zv + 16 * ks),
                            *reinterpret_cast<const uint32_t*>(zv + 16 * ks + 8));
              }
            }
          }
          __syncwarp();
          if (lane == 0) tc_arrive(&bars.h_done[par]);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int ch = hw + 4 * k;
          if (ch < nch) {
            float* z = lz_s + (16 * ch + n8) * 8 + kq;
            z[0] = acc[k][0];
            z[1] = acc[k][1];
            z[64] = acc[k][2];
            z[65] = acc[k][3];
          }
        }
      } else if (warp == 20) {
        // ==== matrix instructions
        const uint32_t id_s = tc_idesc(nr, false), id_o = tc_idesc(nr, true);
        const uint64_t q_desc = tc_desc(tc_smem(sm + Ge::S_Q), 128, D * 16);
        const uint64_t p_desc = tc_desc(tc_smem(sm + Ge::S_P), 128, 2048);
        const bool one = tc_elect();
        auto scores = [&](int t, int it) {
          const int par = __shfl_sync(0xffffffffu, it & 1, 0);
          tc_wait(&bars.k_full, it, dead);
          if (s2) {
            if (it >= 2) tc_wait(&bars.s_empty[par], (it >> 1) - 1, dead);
          } else if (it >= 1) {
            tc_wait(&bars.s_empty[par ^ 1], (it - 1) >> 1, dead);
          }
          tc_fence_after();
          const uint32_t d = tmem + kTS + (s2 ? 64 * par : 0);
          const bool lo = t < g.tq;
          if (one) {
            tc_mma_row<KS>(d, tmem + kTKhi, q_desc, id_s, false);
            if (lo) tc_mma_row<KS>(d, tmem + kTKlo, q_desc, id_s, true);
            tc_commit(&bars.s_full[par]);
          }
          __syncwarp();
        };
        int it = it0;
        scores(g.t0, it);
        for (int t = g.t0; t < g.t0 + g.nt; ++t, ++it) {
          const int par = __shfl_sync(0xffffffffu, it & 1, 0);
          if (t + 1 < g.t0 + g.nt) scores(t + 1, it + 1);
          tc_wait(&bars.v_full, it, dead);
          tc_wait(&bars.p_full[par], it >> 1, dead);
          tc_fence_after();
          const uint64_t pd = p_desc + (par ? 128 * 128 * 2 / 16 : 0);
          const bool lo = t < g.tq, add = t > g.t0;
          if (one) {
            tc_mma_row<8>(tmem + kTO, tmem + kTVhi, pd, id_o, add);
            if (lo) tc_mma_row<8>(tmem + kTO, tmem + kTVlo, pd, id_o, true);
            tc_commit(&bars.pv_done[par]);
          }
          __syncwarp();
        }
        it = it0 + g.nt - 1;
        tc_wait(&bars.pv_done[it & 1], it >> 1, dead);
      }
    }
    tc_sync_segment();

    // ---- end of a segment: lane = channel, 16 rows at a time
    if (warp >= 8 && warp < 16) {
      const int sg = (warp - 8) >> 2, sw = warp & 3;
      const int ch_d = sw * 32 + lane;
      const uint32_t t_lane = tmem + ((uint32_t)(sw * 32) << 16);
      const bool poison = s_poison[seg & 1] != 0 || *dead != 0;
      float* part = a.part + (2 * (long long)blockIdx.x + (g.t0 == 0)) * tree_part(p, D);
      for (int ch = sg; ch < nch; ch += 2) {
        float v[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) v[e] = 0.f;
        if (g.ok) tc_ld16(t_lane + kTO + ch * 16, v);
        if (ch_d >= D) continue;
        // infinite or NaN raw values, of the tokens that a row attends to
        const int i1 = s_odd ? min((g.t0 + g.nt - g.tq) * kTcTile, g.r + a.N) : 0;
#pragma unroll 1
        for (int i = max(g.t0 - g.tq, 0) * kTcTile; i < i1; ++i) {
          const __half w = i < g.r ? static_cast<const __half*>(a.c.v_res)[(g.unit * a.c.R + i) * D + ch_d]
                                   : static_cast<const __half*>(a.v)[(g.unit * a.N + i - g.r) * D + ch_d];
          if ((__half_as_ushort(w) & 0x7C00u) != 0x7C00u) continue;
          const uint32_t sees = i < g.r ? 0xFFFFu : tc_seen(mask_s, i - g.r, g.row0 + ch * 16, a.N);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if ((sees >> e) & 1u) v[e] += __half2float(w);
        }
        __half* out = static_cast<__half*>(a.out) + (g.unit * rows + g.row0 + ch * 16) * (long long)D + ch_d;
        const float* lz = lz_s + ch * 128;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int row = ch * 16 + e;
          const float l = poison ? kNaN : lz[8 * e + 4];
          const float o = fmaf(2.0f, v[e], lz[8 * e + sw]);
          if (row >= g.nrows) continue;
          if (g.whole) {
            out[e * D] = __float2half_rn(l == 0.f ? 0.f : __fdividef(poison ? 0.f : o, l));
          } else {
            part[2 * nr + row * D + ch_d] = poison ? 0.f : o;
            if (ch_d == 0) {
              part[2 * row] = poison ? 0.f : m_s[row];
              part[2 * row + 1] = l;
            }
          }
        }
      }
    }
    if (tid == 0) s_poison[(seg & 1) ^ 1] = 0;  // the next segment's
    if (g.ok) {
      it0 += g.nt;
      const int q1 = min(g.t0 + g.nt, g.tq);
      if (q1 > g.t0) st0 += q1 - g.t0;
    }
    tc_sync_segment();
  }

  __syncthreads();
  if (warp == 20) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

}  // namespace
}  // namespace kivi
