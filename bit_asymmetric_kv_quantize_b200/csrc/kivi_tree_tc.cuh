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
// large values have large z), so it is carried to about 2^-18:
//   c s + z = c' s + z', c' = c - (2^bits - 1) / 2, z' = z + (2^bits - 1) / 2 s;
//   c' s = c' s_hi + c' s_lo, s_hi the leading 7 bits of s: c' s_hi is exact in
//   binary16, c' s_lo is rounded at 2^-18 of c' s; two products;
//   sum_d q_d z'_d, the same for the 32 tokens of a group, is formed apart (z'
//   as the sum of two binary16 numbers, off by 2^-22 of it at most) by mma.sync and
//   joins the score in binary32.
// Values alike: sum_t p_t z'_t of each value group apart.  With them, as one
// more column of ones, the sum of the weights.
// Why the codes are centered: the tensor cores cut each accumulation off toward
// zero.  With c itself all addends of a sum over tokens are positive, and the cuts
// add up (the results of a 16384-token GQA layer were off by 1.3e-4 on average, as
// much as a binary16 output's rounding); the sums of c' stay near zero, unless a
// channel's codes are mostly on one side.  Then, and for the sums of z' and of the weights,
// each of the n / 16 additions cuts off up to 2^-23 of the sum so far: 2^20 tokens of one
// sign in one range came out 6.4e-3 too small.  So a range takes a group in segments of
// kTcMost tiles at most, 1024 additions a plane, whose partials are joined in binary32 in
// the range's slot (131072 tokens a group: 0.9 % more time with 3 rows, 3.4 % with 64).
// A scale below binary16's normal range keeps fewer bits: c' s is off by at most
// 15 * 2^-25 < 2^-21 there.
// s is halved (a binary16 s_hi of a 1-bit group of the widest range would
// overflow), so raw keys and values are halved too and the results doubled in
// binary32.  The weights p are rounded to binary16 once, relative 2^-12 on
// average like the output's own rounding.  Scores, maxima, sums and accumulators
// are binary32.
//
// Running maximum: a row's reference m is raised only when a score of a tile
// exceeds it by more than 15 (in units of log2), and then to 4 below the tile's
// maximum.  Weights up to 2^15 lose nothing in binary16 or in the binary32 sums.
// Binary16 takes a weight below 2^-25 for 0, so what is lost lies below 2^-29 of the
// largest: 2^-15 of it for all tokens of a segment, a sixteenth of the output's own
// rounding (with the maximum itself for reference it was 2^-25, and 2^-11).  A lower
// reference leaves less room: with 8 below, more tiles raise theirs (16384-token GQA
// layer of 8 sequences 273 us, against 263 with 4 and 259 with none).
// The weights of a tile are formed with the references as they are while the excess
// is watched; one vote tells whether that held, and the tile where it did not raises
// the references, rescales O^T in tensor memory and forms its weights again.
//
// A block's warps walk through a tile together; warp w has lanes 32 (w % 4) .. + 31
// of tensor memory and a share of the columns.  For each tile:
//   keys unpacked, and their zeros' products
//   (a further warp issues the score products)
//   the next tile's scales and zeros set out; weights; values unpacked
//   (it issues the value products)
//   sums over the tile's tokens
// One more warp issues the copies (cp.async.bulk of each tile's ranges into a ring).
// With a role to each warp and mbarriers between them, the same work took twice as
// long: the waiting warps' polling and their different code filled the issue slots and
// the instruction cache.  Waits on copies and matrix instructions are bounded: one
// that runs out marks the block dead, whose further waits return soon and whose
// results are NaN.
//
// Two forms (PARTS: groups of four warps).  Up to 64 rows: two blocks of 8 workers on
// an SM, so that one computes while the other waits for its matrix instructions or for
// tensor memory's store port (unpacking writes 128 KB a tile, about 1000 cycles of
// it); a block has 256 columns of tensor memory, values take the keys' place.  From 65
// rows on: one block of 16 workers and up to 128 rows, which unpacks the cache once
// where two row blocks would do it twice; the values have planes of their own and
// are unpacked while the score products run.  Measured on 8 sequences x 32 heads of 4096
// tokens at 2 bits, two blocks against one of 16 workers: 8 rows 119 and 174 us, 32
// rows 139 and 185, 64 rows 180 and 217; 80 rows (2 x 48) 295 and 249, 128 rows (2 x 64)
// 338 and 293, 160 rows (3 x 64, 2 x 80) 507 and 498.  (Both have since got faster, wider
// loads and stores and a shorter segment's end: 114, 130, 167, 240, 283 and 484 us for those
// row counts in the form that is taken.)
//
// What bounds it: neither DRAM (6 to 16 % of its rate) nor the matrix instructions (8
// to 27 % of their pipe), but instructions and the barriers between a tile's steps, half
// each: 50 to 53 % of the issue slots are used (7.4 K warp instructions a tile with 16 rows,
// 13.9 K with 96), and most stalls are waits at barriers (1.8 to 2.7 of the 8 to 9 warps
// a scheduler's issue waits for).
// A 4096-token layer of 8 x 32 heads with 16 nodes takes 116 us (1.3 TB/s of the cache,
// 74 TFLOP/s of the products), a 16384-token GQA layer of 16 x 8 heads, 96 rows,
// 427 us (241 TFLOP/s), a paged batch of 24 x 8 heads to 6000 tokens at 4 bits, 244
// rows, 485 us (192 TFLOP/s).
#pragma once

#include <type_traits>

#include "kivi_tree.cuh"

namespace kivi {
namespace {

constexpr int kTcTile = 128;        // tokens
// Threads of a block of PARTS x 4 workers, one warp for the matrix instructions and one
// for the copies.
template <int PARTS>
constexpr int kTcThreads = (4 * PARTS + 2) * 32;
constexpr float kTcSlack = 15.0f;   // log2 units a score may exceed m by
constexpr float kTcBelow = 4.0f;    // and those by which a rise leaves m below the maximum
constexpr float kTcNone = -1.0e30f; // reference of a row that has seen nothing
constexpr int kTcMost = 128;        // tiles of a segment at most

// ---- layouts ---------------------------------------------------------------
template <int D, int BITS, int MB, int PARTS>
struct TcGeo {
  static constexpr int ROWS = 32 * PARTS;                // rows of a block at most
  static constexpr int WARPS = 4 * PARTS, WORKERS = 32 * WARPS;
  static constexpr int RT = 16 * PARTS;                  // raw tokens staged at a time
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
  static constexpr int RING = PARTS == 2 ? 49152 : 98304;
  static constexpr int NST = RING / STAGE < 5 ? RING / STAGE : 5;
  // shared memory
  static constexpr int S_RING = 0;
  static constexpr int S_Q = S_RING + NST * STAGE;       // B operand, [ROWS][D]
  static constexpr int S_P = S_Q + ROWS * D * 2;         // [ROWS][128 tokens]
  // raw values [RT tokens][D]; at the end of a segment the sums, [PARTS][ROWS][8]
  static constexpr int S_RAW = S_P + ROWS * 128 * 2;
  static constexpr int S_LZ = S_RAW;
  static constexpr int LZ = PARTS * ROWS * 8 * 4;
  static constexpr int S_KSC = S_RAW + (RT * D * 2 > LZ ? RT * D * 2 : LZ);
                                                         // 4 groups x D x (hi, lo) halves
  static constexpr int S_VSC = S_KSC + 4 * D * 4;        // 2 x 4 groups x 128 x (hi, lo)
  // (a group's row is padded: a warp's stores of one token's groups meet other banks)
  static constexpr int VLD = 272;
  static constexpr int S_ZK = S_VSC + 2 * 4 * VLD * 2;   // [PARTS][4 groups][ROWS] float
  static constexpr int S_OFF = S_ZK + PARTS * 4 * ROWS * 4;  // [WARPS][16 rows]
  static constexpr int S_WMAX = S_OFF + WARPS * 16 * 4;  // [4 groups][ROWS]
  static constexpr int S_M = S_WMAX + 4 * ROWS * 4;      // [ROWS]
  static constexpr int S_F = S_M + ROWS * 4;             // [ROWS]
  // zeros as binary16 in operand order, rows padded against bank conflicts:
  // (high parts, low parts): keys 2 x 4 groups x D, values 9 rows x 128 tokens (high
  // parts of 4 groups, ones, low parts of 4 groups)
  static constexpr int ZLD = 136;
  static constexpr int S_ZH = S_F + ROWS * 4;
  static constexpr int S_ZV = S_ZH + 8 * ZLD * 2;        // 2 x
  static constexpr int S_MASK = S_ZV + 2 * 9 * ZLD * 2;  // [N][ceil(N / 32)] words
  static constexpr int BYTES = S_MASK;                   // and the mask
  // of two blocks on an SM, or of one
  static constexpr int MOST = PARTS == 2 ? (227 * 1024 + 1024) / 2 - 1024 : 227 * 1024 - 1024;
  // (up to 64 rows are up to 64 nodes)
  static constexpr int MASK = PARTS == 2 ? 64 * 2 * 4 : 256 * 8 * 4;
  static_assert(NST >= 2 && BYTES + MASK + 256 <= MOST, "the blocks of an SM share it");
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
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(b), "r"(bytes)
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
// Barriers: of the workers (1), of them and the warp of the matrix instructions (3),
// and of the block with a vote (2: a thread's `x`).
template <int PARTS>
__device__ __forceinline__ void tc_sync_workers() {
  tc_fence_before();
  asm volatile("bar.sync 1, %0;" ::"n"(kTcThreads<PARTS> - 64) : "memory");
  tc_fence_after();
}
template <int PARTS>
__device__ __forceinline__ void tc_sync_scores() {
  tc_fence_before();
  asm volatile("bar.sync 3, %0;" ::"n"(kTcThreads<PARTS> - 32) : "memory");
  tc_fence_after();
}
template <int PARTS>
__device__ __forceinline__ bool tc_sync_any(bool x) {
  uint32_t r;
  tc_fence_before();
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred.aligned q, 2, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "n"(kTcThreads<PARTS>)
      : "memory");
  tc_fence_after();
  return r != 0;
}

// ---- codes as binary16 ---------------------------------------------------------
// The eight pairs of registers 8 q .. 8 q + 7 of a lane (16 codes in operand
// order) as exact binary16 numbers c' = c - (2^BITS - 1) / 2.  A pair (i, i + E/2)
// of a word has its codes in the two 16-bit halves, at bit BITS * i of each; a shift
// and a mask leave it at bit e of the half, 1 <= e, e + BITS <= 10; 0x6400 | (c << e) is
// 1024 + c 2^e, and one fused multiply-add by 2^-e gives c' (2^(10 - e) plus the
// center is a binary16 number from e = 1 on).
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
// The constants stand in registers that the compiler does not see through: it would
// form them again for each pair, an instruction each.
struct TcConst {
  uint32_t magic;             // 1024 in both halves
  uint32_t inv[10], off[10];  // 2^-e and -(2^(10 - e) + center)
};
template <int BITS>
__device__ __forceinline__ TcConst tc_const() {
  TcConst k;
  asm volatile("mov.b32 %0, 0x64006400;" : "=r"(k.magic));
#pragma unroll
  for (int e = 1; e < 10; ++e) {
    k.inv[e] = ((15u - e) << 10) * 0x00010001u;
    k.off[e] = (0x8000u | (25u - e) << 10 | ((1u << BITS) - 1u) << (e - 1)) * 0x00010001u;
    asm volatile("" : "+r"(k.inv[e]), "+r"(k.off[e]));
  }
  return k;
}
// (x & m) | magic, then 1024 + c 2^e to c'.
template <int BITS, int E_BIT>
__device__ __forceinline__ uint32_t tc_code(uint32_t x, uint32_t m, const TcConst& k) {
  uint32_t d, y;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(x), "r"(m), "r"(k.magic));
  if constexpr (E_BIT == 0) {  // 3 bits only: -1024, -3.5
    static_assert(BITS == 3, "the other formats begin at bit 1");
    asm("{\n\t.reg .b32 z;\n\tadd.rn.f16x2 z, %1, %2;\n\tadd.rn.f16x2 %0, z, %3;\n\t}"
        : "=r"(d)
        : "r"(y), "r"(0xE400E400u), "r"(0xC300C300u));
  } else {
    d = tc_hfma2(y, k.inv[E_BIT], k.off[E_BIT]);
  }
  return d;
}
// Pair I of a block whose words are w[0 .. WB).
template <int BITS, int I>
__device__ __forceinline__ uint32_t tc_pair(const uint32_t* w, const TcConst& k) {
  if constexpr (BITS == 3) {
    constexpr int e = I & 7, sh = I < 8 ? 0 : 8;
    constexpr uint32_t m = 0x00010001u << e;
    const uint32_t p = ((w[0] >> sh) & m) | (((w[1] >> sh) << 1) & (m << 1)) |
                       (((w[2] >> sh) << 2) & (m << 2));
    return tc_code<3, e>(p, 0xFFFFFFFFu, k);
  } else {
    constexpr int per = 9 / BITS;  // pairs of one shift
    constexpr int at = I / per * per * BITS, e = 1 + I % per * BITS;
    constexpr uint32_t m = ((1u << BITS) - 1u) * 0x00010001u << e;
    if constexpr (at == 0)
      return tc_code<BITS, e>(w[0] << 1, m, k);
    else
      return tc_code<BITS, e>(w[0] >> (at - 1), m, k);
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
__device__ __forceinline__ void tc_codes16(const uint32_t* w, uint32_t (&c)[8], const TcConst& k) {
  if constexpr (BITS == 4) {
    c[0] = tc_pair<4, 0>(w, k);
    c[1] = tc_pair<4, 1>(w, k);
    c[2] = tc_pair<4, 2>(w, k);
    c[3] = tc_pair<4, 3>(w, k);
    c[4] = tc_pair<4, 0>(w + 1, k);
    c[5] = tc_pair<4, 1>(w + 1, k);
    c[6] = tc_pair<4, 2>(w + 1, k);
    c[7] = tc_pair<4, 3>(w + 1, k);
  } else {
    c[0] = tc_pair<BITS, 8 * HALF + 0>(w, k);
    c[1] = tc_pair<BITS, 8 * HALF + 1>(w, k);
    c[2] = tc_pair<BITS, 8 * HALF + 2>(w, k);
    c[3] = tc_pair<BITS, 8 * HALF + 3>(w, k);
    c[4] = tc_pair<BITS, 8 * HALF + 4>(w, k);
    c[5] = tc_pair<BITS, 8 * HALF + 5>(w, k);
    c[6] = tc_pair<BITS, 8 * HALF + 6>(w, k);
    c[7] = tc_pair<BITS, 8 * HALF + 7>(w, k);
  }
}
// Two scales, halved, in two binary16 parts each (the leading 7 bits, and the rest), and
// their z' = z + s * center in two parts: operand pairs at c of four rows.
template <int BITS>
__device__ __forceinline__ void tc_scales(float2 s, float2 z, __half* s_hi, __half* s_lo,
                                          __half* z_hi, __half* z_lo) {
  constexpr float kCenter = 0.5f * ((1 << BITS) - 1);
  const float2 x = make_float2(fmaf(s.x, kCenter, z.x), fmaf(s.y, kCenter, z.y));
  const __half2 zh = __floats2half2_rn(x.x, x.y);
  const float2 zf = __half22float2(zh);
  *reinterpret_cast<__half2*>(z_hi) = zh;
  *reinterpret_cast<__half2*>(z_lo) = __floats2half2_rn(x.x - zf.x, x.y - zf.y);
  s.x *= 0.5f;
  s.y *= 0.5f;
  const __half2 sh = __floats2half2_rn(__uint_as_float(__float_as_uint(s.x) & 0xFFFE0000u),
                                       __uint_as_float(__float_as_uint(s.y) & 0xFFFE0000u));
  const float2 sf = __half22float2(sh);
  *reinterpret_cast<__half2*>(s_hi) = sh;
  *reinterpret_cast<__half2*>(s_lo) = __floats2half2_rn(s.x - sf.x, s.y - sf.y);
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
// Units `part`, part + PARTS, .. (of n) of a lane's words (`stride` words apart) into its
// row of the two planes; hi, lo: the parts of the row's scales.
template <int BITS, int PARTS>
__device__ __forceinline__ void tc_unpack(uint32_t t_hi, const uint32_t* words, int stride,
                                          const uint4* hi, const uint4* lo, int part, int n,
                                          const TcConst& k) {
  using U = TcUnit<BITS>;
  constexpr int H = U::kUnit / 16;
#pragma unroll(H == 2 ? 1 : 2)
  for (int u = part; u < n; u += PARTS) {
    uint32_t w[U::kUnitW], c[8];
#pragma unroll
    for (int i = 0; i < U::kUnitW; ++i) w[i] = words[(u * U::kUnitW + i) * stride];
    tc_codes16<BITS, 0>(w, c, k);
    tc_put16(t_hi + 8 * H * u, t_hi + 8 * H * u + 64, c, hi + 2 * H * u, lo + 2 * H * u);
    if constexpr (H == 2) {
      tc_codes16<BITS, 1>(w, c, k);
      tc_put16(t_hi + 16 * u + 8, t_hi + 16 * u + 72, c, hi + 4 * u + 2, lo + 4 * u + 2);
    }
  }
}
// The same for a token's key words, which are adjacent: a part takes adjacent units and
// loads their words in pieces as wide as they are aligned (word by word, the lanes' rows
// of WK words would meet in a few banks).
template <int D, int BITS, int PARTS>
__device__ __forceinline__ void tc_unpack_keys(uint32_t t_hi, const uint32_t* row, const uint4* hi,
                                               const uint4* lo, int part, const TcConst& k) {
  using U = TcUnit<BITS>;
  constexpr int H = U::kUnit / 16, n = D / U::kUnit, per = n < PARTS ? 1 : n / PARTS;
  constexpr int NW = per * U::kUnitW;
  if (part * per >= n) return;
  uint32_t w[NW];
  const uint32_t* src = row + part * NW;
  if constexpr (NW % 4 == 0) {
#pragma unroll
    for (int i = 0; i < NW; i += 4) {
      const uint4 x = *reinterpret_cast<const uint4*>(src + i);
      w[i] = x.x;
      w[i + 1] = x.y;
      w[i + 2] = x.z;
      w[i + 3] = x.w;
    }
  } else if constexpr (NW % 2 == 0) {
#pragma unroll
    for (int i = 0; i < NW; i += 2) {
      const uint2 x = *reinterpret_cast<const uint2*>(src + i);
      w[i] = x.x;
      w[i + 1] = x.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NW; ++i) w[i] = src[i];
  }
#pragma unroll
  for (int j = 0; j < per; ++j) {
    const int u = part * per + j;
    uint32_t c[8];
    tc_codes16<BITS, 0>(w + j * U::kUnitW, c, k);
    tc_put16(t_hi + 8 * H * u, t_hi + 8 * H * u + 64, c, hi + 2 * H * u, lo + 2 * H * u);
    if constexpr (H == 2) {
      tc_codes16<BITS, 1>(w + j * U::kUnitW, c, k);
      tc_put16(t_hi + 16 * u + 8, t_hi + 16 * u + 72, c, hi + 4 * u + 2, lo + 4 * u + 2);
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
// RT raw tokens from `first` on (the window's r tokens at wp, then the drafted ones
// at dp up to n) into rows of D in shared memory, by all workers.  Loads without
// branches, so that they are under way together; a token that does not exist reads
// the window's first row.
template <int D, int RT, int WORKERS>
__device__ __forceinline__ void tc_stage_raw(uint4* dst, const __half* wp, const __half* dp,
                                             int first, int r, int n) {
  constexpr int J = (RT * (D / 8) + WORKERS - 1) / WORKERS;
  const bool al = ((uintptr_t)dp & 15) == 0;
  uint4 x[J];
#pragma unroll
  for (int j = 0; j < J; ++j) {
    const int k = (threadIdx.x + WORKERS * j) % (RT * (D / 8)), i = first + k / (D / 8);
    const int c = k % (D / 8) * 8;
    x[j] = *reinterpret_cast<const uint4*>(al && i >= r && i < n ? dp + (i - r) * D + c
                                                                 : wp + (i < r ? i * D + c : c));
    if (i >= n) x[j] = make_uint4(0, 0, 0, 0);
    if (!al && i >= r && i < n) x[j] = tc_raw8(dp + (i - r) * D + c, false);
  }
#pragma unroll
  for (int j = 0; j < J; ++j) dst[(threadIdx.x + WORKERS * j) % (RT * (D / 8))] = x[j];
}
// A lane's raw key row, halved, into its operand row, 16-place pieces c0 .. c0 + N - 1:
// two runs of 8 channels E / 2 apart each (or two blocks of 8 channels).  Loads as
// above; row: a readable row, have: whether its numbers count.
template <int E, int N>
__device__ __forceinline__ void tc_raw_keys(uint32_t t_hi, const __half* row, bool have, int c0) {
  const bool al = ((uintptr_t)row & 15) == 0;
  uint4 x[N], y[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int c = c0 + j, e0 = E >= 16 ? 16 * c / E * E + 16 * c % E / 2 : 16 * c;
    x[j] = tc_raw8(row + e0, al);
    y[j] = tc_raw8(row + e0 + (E >= 16 ? E / 2 : 8), al);
  }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    uint32_t r[8];
    tc_raw_pairs<E>(x[j], y[j], r);
#pragma unroll
    for (int k = 0; k < 8; ++k) r[k] = have ? r[k] : 0u;
    tc_st8(t_hi + 8 * (c0 + j), r);
  }
}
// 16 places of a lane's channel of the staged raw tokens (`v`, rows of D in shared memory),
// halved, into its operand row.  Infinities and NaN are left out (they join at the
// segment's end, for the rows that attend to them); returns whether there were any.
template <int D, int E>
__device__ __forceinline__ bool tc_raw_values(uint32_t t_hi, const __half* v, int piece) {
  uint32_t odd = 0;
  {
    const __half* s0 = v + (E >= 16 ? 16 * piece / E * E + 16 * piece % E / 2 : 16 * piece) * D;
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
    tc_st8(t_hi, q);
  }
  return odd != 0;
}

// A warp's common truth value, in a uniform register.
__device__ __forceinline__ bool tc_uniform(bool x) {
  return __shfl_sync(0xffffffffu, (int)x, 0) != 0;
}
// Whether rows row0 .. row0 + 15 see drafted token `node`, one bit each.
__device__ __forceinline__ uint32_t tc_seen(const uint32_t* mask_s, int node, int row0, int N) {
  uint32_t bits = 0;
  const int mw = (N + 31) / 32;
  int q = row0 % N;
#pragma unroll 1
  for (int e = 0; e < 16; ++e) {
    bits |= ((mask_s[q * mw + (node >> 5)] >> (node & 31)) & 1u) << e;
    if (++q == N) q = 0;
  }
  return bits;
}

// An accumulator at its weight; an infinite or NaN one is kept where that comes to 0 (as in
// tree_merge_kernel).
__device__ __forceinline__ float tc_part(float f, float x) {
  return f != 0.f || isfinite(x) ? f * x : x;
}
// The infinite and NaN values of raw tokens i0 .. i1 - 1 that row `row` of the KV head attends to,
// added up (w, d: one channel of the window and of the drafted tokens).
template <int D>
__device__ __noinline__ float tc_odd(const __half* w, const __half* d, const uint32_t* mask_s, int i0,
                                     int i1, int r, int row, int N) {
  float o = 0.f;
  for (int i = i0; i < i1; ++i) {
    const __half x = i < r ? w[i * D] : d[(i - r) * D];
    if ((__half_as_ushort(x) & 0x7C00u) == 0x7C00u &&
        (i < r || (tc_seen(mask_s, i - r, row, N) & 1u)))
      o += __half2float(x);
  }
  return o;
}

// Tensor-memory columns: two planes of keys; two of values (the same ones where two
// blocks share tensor memory); S^T; O^T.
template <int PARTS>
struct TcCols {
  static constexpr bool APART = PARTS == 4;
  static constexpr uint32_t A = 0, V = APART ? 128 : 0, S = V + 128, O = S + 32 * PARTS,
                            N = O + 32 * PARTS;
};

// Barriers for what is asynchronous, 8 bytes each, by their number.
struct TcBar {
  static constexpr int raw = 0, scores = 5, values = 6, N = 7;  // raw: [stage]
};

// One segment of a group: what of it falls into the block's range, or kTcMost tiles of that.
struct TcSeg {
  long long b, unit, n_q;
  int t0, t1, tq;      // tiles [t0, t1); of the group, tq of quantized tokens
  int t1s;             // the segment's end of those
  int r, row0, nrows;  // nrows: rows of this block that exist
  bool ends, ok;       // ends: with the group
};
// A block's walk over its range: sequence, KV head, row block, tile, tiles left.
struct TcWalk {
  long long b, left;
  int h, rb, t;
};

template <int D, int BITS, typename M, int PARTS>
__global__ void __launch_bounds__(kTcThreads<PARTS>, PARTS == 2 ? 2 : 1)
    tree_tc_kernel(TreeArgs a, TreePlan p) {
  using Ge = TcGeo<D, BITS, (int)sizeof(M), PARTS>;
  using Col = TcCols<PARTS>;
  constexpr int ROWS = Ge::ROWS, WORKERS = Ge::WORKERS, RT = Ge::RT;
  constexpr int RC = ROWS / 64;  // 16-row chunks of a warp in the products of the zeros
  constexpr int E = Ge::E, WK = Ge::WK, NJ = Ge::NJ;
  constexpr int KS = D / 16;  // k-slices of the scores
  extern __shared__ __align__(128) unsigned char sm[];
  __shared__ uint64_t s_bars[TcBar::N];
  __shared__ TcWalk s_walk;
  __shared__ uint32_t s_tmem;
  __shared__ int s_dead, s_odd;
  __shared__ int s_first;       // the tile of the group at which the range meets it
  __shared__ int s_poison[2];   // [segment parity]
  volatile int* dead = &s_dead;
  const uint32_t bar0 = tc_smem(s_bars), sm0 = tc_smem(sm);
  auto bar = [&](int k) -> uint32_t { return bar0 + 8u * (uint32_t)k; };
  // what a whole warp shares is broadcast, so that it lives in uniform registers
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int rows = a.gq * a.N, mw = (a.N + 31) / 32;
  const int nr = p.rb, nch = nr / 16;

  // ---- set-up
  asm volatile("griddepcontrol.launch_dependents;");
  if (warp == Ge::WARPS) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     tc_smem(&s_tmem)),
                 "n"(Col::N)
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
    for (int i = 0; i < TcBar::N; ++i) tc_bar_init(bar(i), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  for (int i = tid; i < 2 * 9 * Ge::ZLD; i += kTcThreads<PARTS>)
    reinterpret_cast<__half*>(sm + Ge::S_ZV)[i] = __float2half_rn(i / Ge::ZLD % 9 == 4 ? 1.0f : 0.0f);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
  TcWalk walk = s_walk;

  float* m_s = reinterpret_cast<float*>(sm + Ge::S_M);    // references
  float* f_s = reinterpret_cast<float*>(sm + Ge::S_F);    // factors of a rise
  float* zk_s = reinterpret_cast<float*>(sm + Ge::S_ZK);  // [part][group][ROWS]
  float* lz_s = reinterpret_cast<float*>(sm + Ge::S_LZ);  // [part][ROWS][8]
  uint32_t* mask_s = reinterpret_cast<uint32_t*>(sm + Ge::S_MASK);

  // A range ends within a group at most at its own end: the first segment of a group after
  // the range's first group begins with it.
  auto next_seg = [&](TcWalk& w) -> TcSeg {
    // what steers the warp is broadcast: without that the compiler takes it for
    // divergent and guards each tensor-memory access (some 50 instructions each)
    const TreeSeq q = tree_seq(a, p, w.b);
    TcSeg g;
    g.t0 = w.t;
    const int end = w.t + (int)min(q.ut - w.t, w.left);
    g.t1 = min(end, w.t + kTcMost);
    g.b = w.b;
    g.unit = w.b * a.Hkv + w.h;
    g.row0 = w.rb * nr;
    g.nrows = min(rows - g.row0, nr);
    g.n_q = q.n_q;
    g.r = q.r;
    g.ok = q.ok;
    g.tq = q.ok ? (int)((q.n_q + kTcTile - 1) / kTcTile) : 0;
    g.t1s = min(g.t1, g.tq);
    g.ends = g.t1 == q.ut;
    const bool more = g.t1 < end;
    w.left -= g.t1 - g.t0;
    g.t0 = __shfl_sync(0xffffffffu, g.t0, 0);
    g.t1 = __shfl_sync(0xffffffffu, g.t1, 0);
    g.tq = __shfl_sync(0xffffffffu, g.tq, 0);
    g.t1s = __shfl_sync(0xffffffffu, g.t1s, 0);
    g.r = __shfl_sync(0xffffffffu, g.r, 0);
    g.nrows = __shfl_sync(0xffffffffu, g.nrows, 0);
    g.ok = __shfl_sync(0xffffffffu, (int)g.ok, 0) != 0;
    g.ends = __shfl_sync(0xffffffffu, (int)g.ends, 0) != 0;
    w.t = g.t1;
    if (!more) {
      w.t = 0;
      if (++w.rb == p.n_rb) {
        w.rb = 0;
        if (++w.h == a.Hkv) {
          w.h = 0;
          ++w.b;
        }
      }
    }
    return g;
  };

  if (warp == Ge::WARPS + 1) {
    // ==== copies: lane k < 6 copies a tile's part of array k, in one piece, or one for
    // each page that it touches; a tile's stage is free once the block has passed the
    // barrier of the tile NST before it
    TcWalk ahead = walk;
    TcSeg n{};
    int nt = 0, issued = 0, done = 0;  // the next tile of n, tiles copied and used up
    const long long Ts = store_tokens(a.c);
    // array k: codes, scales, zeros of keys, then of values
    const int k = lane % 3;
    const bool val = lane >= 3;
    const char* src = static_cast<const char*>(
        val ? (k == 0 ? (const void*)a.c.v_codes : k == 1 ? a.c.v_scale : a.c.v_zero)
            : (k == 0 ? (const void*)a.c.k_codes : k == 1 ? a.c.k_scale : a.c.k_zero));
    const int size = val ? (k == 0 ? Ge::VC : Ge::VM) : (k == 0 ? Ge::KC : Ge::KM);
    const long long unit_bytes = Ts / kTile * size;
    const uint32_t o_dst = val ? (k == 0 ? Ge::O_VC : k == 1 ? Ge::O_VS : Ge::O_VZ)
                               : (k == 0 ? Ge::O_KC : k == 1 ? Ge::O_KS : Ge::O_KZ);
    auto fill = [&]() {
      while (issued < done + Ge::NST) {
        while (nt >= n.t1s) {  // the next segment with quantized tiles
          if (ahead.left <= 0) return;
          n = next_seg(ahead);
          nt = n.t0;
        }
        const int s = issued % Ge::NST;
        const uint32_t fb = bar(TcBar::raw + s), dst = sm0 + Ge::S_RING + s * Ge::STAGE;
        const int subs = (int)min(n.n_q / kTile - nt * 4LL, 4LL), page = a.c.R / kTile;
        for (int i = 0, run; i < subs; i += run) {
          const long long tile = nt * 4LL + i;
          run = a.c.bt == nullptr ? subs : min(subs - i, page - (int)(tile % page));
          long long su, stl;
          if (!store_tile(a.c, n.unit, tile, &su, &stl)) continue;
          if (lane == 0) tc_expect(fb, run * (2 * Ge::KM + Ge::KC + Ge::VC + 2 * Ge::VM));
          __syncwarp();
          if (lane < 6)
            tc_copy(dst + o_dst + i * size, src + su * unit_bytes + stl * size, run * size, fb);
        }
        if (lane == 0) tc_arrive(fb);
        ++nt;
        ++issued;
      }
    };
    fill();
    while (tc_uniform(walk.left > 0)) {
      const TcSeg g = next_seg(walk);
      for (int t = g.t0; t < g.t1 && g.ok; ++t) {  // the block's barriers
        if (tc_sync_any<PARTS>(false)) tc_sync_any<PARTS>(false);
        if (t < g.t1s) {
          ++done;
          fill();
        }
      }
    }
    for (int i = max(issued - Ge::NST, 0); i < issued; ++i)  // none is under way at the end
      tc_wait(bar(TcBar::raw + i % Ge::NST), i / Ge::NST, dead);
  } else if (warp == Ge::WARPS) {
    // ==== matrix instructions
    const bool one = tc_elect();
    const uint32_t id_s = tc_idesc(nr, false), id_o = tc_idesc(nr, true);
    const uint64_t q_desc = tc_desc(sm0 + Ge::S_Q, 128, D * 16), p_desc = tc_desc(sm0 + Ge::S_P, 128, 2048);
    while (tc_uniform(walk.left > 0)) {
      const TcSeg g = next_seg(walk);
      if (!g.ok) continue;
      for (int t = g.t0; t < g.t1; ++t) {
        const bool lo = t < g.t1s;
        tc_sync_scores<PARTS>();
        if (one) {
          tc_mma_row<KS>(tmem + Col::S, tmem + Col::A, q_desc, id_s, false);
          if (lo) tc_mma_row<KS>(tmem + Col::S, tmem + Col::A + 64, q_desc, id_s, true);
          tc_commit(bar(TcBar::scores));
        }
        __syncwarp();
        if (tc_sync_any<PARTS>(false)) tc_sync_any<PARTS>(false);
        if (one) {
          tc_mma_row<8>(tmem + Col::O, tmem + Col::V, p_desc, id_o, t > g.t0);
          if (lo) tc_mma_row<8>(tmem + Col::O, tmem + Col::V + 64, p_desc, id_o, true);
          tc_commit(bar(TcBar::values));
        }
        __syncwarp();
      }
    }
  } else {
    // ==== workers
    const int q = warp & 3, part = warp >> 2;  // lanes of tensor memory, share of the columns
    const uint32_t t_q = tmem + ((uint32_t)(q * 32) << 16);
    const int n8 = lane >> 2, kq = (lane & 3) * 2;  // fragments of mma.sync
    const int pk = tc_pos<E>(q * 32 + lane);        // this lane's token in the second product
    const float c1 = 2.0f * a.qscale;
    const TcConst konst = tc_const<BITS>();
    __half* ksc = reinterpret_cast<__half*>(sm + Ge::S_KSC);
    __half* vsc0 = reinterpret_cast<__half*>(sm + Ge::S_VSC);
    __half* zh = reinterpret_cast<__half*>(sm + Ge::S_ZH);
    __half* zv0 = reinterpret_cast<__half*>(sm + Ge::S_ZV);
    float* off_s = reinterpret_cast<float*>(sm + Ge::S_OFF) + warp * 16;
    float* wmax_s = reinterpret_cast<float*>(sm + Ge::S_WMAX);
    int it0 = 0, st0 = 0;  // tiles of the segments before, and those of the ring
    for (int seg = 0; tc_uniform(walk.left > 0); ++seg) {
      const TcSeg g = next_seg(walk);
      const __half* wk = static_cast<const __half*>(a.c.k_res) + g.unit * a.c.R * D;
      const __half* wv = static_cast<const __half*>(a.c.v_res) + g.unit * a.c.R * D;
      const __half* dk = static_cast<const __half*>(a.k) + g.unit * a.N * D;
      const __half* dv = static_cast<const __half*>(a.v) + g.unit * a.N * D;
      const int n_raw = g.r + a.N;
      // ---- start of a segment: queries, mask, references, pages
      if (tid == 0) {
        s_odd = 0;
        if (seg == 0 || g.t0 == 0) s_first = g.t0;
      }
      if (!g.ok) s_poison[seg & 1] = 1;
      if (a.c.bt != nullptr && g.ok) {  // a page outside the pool poisons the group
        const long long i1 = min(g.t1 * 4LL, g.n_q / kTile);
#pragma unroll 1
        for (long long i = g.t0 * 4LL + tid; i < i1; i += WORKERS) {
          long long su, stl;
          if (!store_tile(a.c, g.unit, i, &su, &stl)) s_poison[seg & 1] = 1;
        }
      }
      {
        const __half* qp = static_cast<const __half*>(a.q) + (g.unit * rows + g.row0) * D;
        const bool al = ((uintptr_t)qp & 15) == 0;
        // operand order along channels; rows that do not exist are 0
#pragma unroll 2
        for (int i = tid; i < nr * (D / 8); i += WORKERS) {
          const int row = i / (D / 8), c0 = i % (D / 8) * 8;
          uint4 x = make_uint4(0, 0, 0, 0);
          if (row < g.nrows) x = tc_raw8(qp + row * D + c0, al);
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
          unsigned char* d = sm + Ge::S_Q + row / 8 * (D * 16) + row % 8 * 16;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int k = tc_pos<E>(c0 + e);
            *reinterpret_cast<uint16_t*>(d + k / 8 * 128 + k % 8 * 2) = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
          }
        }
#pragma unroll 1
        for (int i = tid; i < a.N * mw; i += WORKERS)
          mask_s[i] = a.mask[g.b * a.N * mw + i];
        if (tid < ROWS) m_s[tid] = kTcNone;
      }
      tc_fence_smem();

      // scales and zeros of tile t's keys (2 D pairs of channels, of 4 groups) and values
      // (64 NJ pairs of tokens)
      auto set_out = [&](int t) {
        __half* zv = zv0 + (t & 1) * 9 * Ge::ZLD;
        __half* vsc = vsc0 + (t & 1) * 4 * Ge::VLD;
        const bool raw = t >= g.t1s;
        const unsigned char* stg = sm + Ge::S_RING + (st0 + t - g.t0) % Ge::NST * Ge::STAGE;
        if (!raw) tc_wait(bar(TcBar::raw + (st0 + t - g.t0) % Ge::NST), (st0 + t - g.t0) / Ge::NST, dead);
        const long long left = g.n_q - (long long)t * kTcTile;
#pragma unroll
        for (int j = 0; j < (4 * D + WORKERS - 1) / WORKERS; ++j) {
          const int i = tid + WORKERS * j;
          if (i < 2 * D) {
            const int gr = i / (D / 2), p = i % (D / 2);
            const int c = 2 * p, d = p / (E / 2) * E + p % (E / 2);  // the pair (d, d + E / 2)
            const M* sp = reinterpret_cast<const M*>(stg + Ge::O_KS) + gr * D + d;
            const M* zp = reinterpret_cast<const M*>(stg + Ge::O_KZ) + gr * D + d;
            if (!raw)
              tc_scales<BITS>(make_float2(to_f32(sp[0]), to_f32(sp[E / 2])),
                              make_float2(to_f32(zp[0]), to_f32(zp[E / 2])), &ksc[gr * 2 * D + c],
                              &ksc[gr * 2 * D + D + c], &zh[gr * Ge::ZLD + c], &zh[(4 + gr) * Ge::ZLD + c]);
          } else if (i < 4 * D) {
            const int m = i - 2 * D, gr = m % NJ, p = m / NJ;
            const int c = 2 * p, tok = p / (E / 2) * E + p % (E / 2);
            const M* sp = reinterpret_cast<const M*>(stg + Ge::O_VS) + tok * NJ + gr;
            const M* zp = reinterpret_cast<const M*>(stg + Ge::O_VZ) + tok * NJ + gr;
            // tokens that do not exist: 0 (their weight 0 times NaN would not be)
            const bool h0 = !raw && tok < left, h1 = !raw && tok + E / 2 < left;
            tc_scales<BITS>(make_float2(h0 ? to_f32(sp[0]) : 0.f, h1 ? to_f32(sp[E / 2 * NJ]) : 0.f),
                            make_float2(h0 ? to_f32(zp[0]) : 0.f, h1 ? to_f32(zp[E / 2 * NJ]) : 0.f),
                            &vsc[gr * Ge::VLD + c], &vsc[gr * Ge::VLD + 128 + c], &zv[gr * Ge::ZLD + c],
                            &zv[(5 + gr) * Ge::ZLD + c]);
          }
        }
      };
      // keys of tile t into tensor memory, and their zeros' products
      auto put_keys = [&](int t) {
        float zc[RC][4] = {};
        if (t < g.t1s) {
          const unsigned char* stg = sm + Ge::S_RING + (st0 + t - g.t0) % Ge::NST * Ge::STAGE;
          const __half* sc = ksc + q * 2 * D;
          tc_unpack_keys<D, BITS, PARTS>(
              t_q + Col::A, reinterpret_cast<const uint32_t*>(stg + Ge::O_KC + q * Ge::KC) + lane * WK,
              reinterpret_cast<const uint4*>(sc), reinterpret_cast<const uint4*>(sc + D), part, konst);
          // sum_d q_d z'_gd for rows 16 q .. (and 64 further on), over this part's channels
          // (the warp's q counts rows here); columns: the groups' high parts, their low parts
          const __half* zr = zh + n8 * Ge::ZLD + kq;
#pragma unroll
          for (int c = 0; c < RC; ++c) {
            if (q + 4 * c >= nch) break;
            const int row = 16 * (q + 4 * c) + (lane & 15);
            const uint32_t qa = sm0 + Ge::S_Q + row / 8 * (D * 16) + (lane >> 4) * 128 + row % 8 * 16;
#pragma unroll
            for (int j = 0; j < (KS + PARTS - 1) / PARTS; ++j) {
              const int ks = part + PARTS * j;
              if (KS < PARTS && ks >= KS) break;
              uint32_t av[4];
              tc_ldm<false>(av, qa + 256 * ks);
              tc_mma16816(zc[c], av, *reinterpret_cast<const uint32_t*>(zr + 16 * ks),
                          *reinterpret_cast<const uint32_t*>(zr + 16 * ks + 8));
            }
          }
        } else {
          // raw tokens: the window, then the drafted ones; halved like s
          const int i = (t - g.tq) * kTcTile + q * 32 + lane;
          const __half* src = i < g.r ? wk + i * D : (i < n_raw ? dk + (i - g.r) * D : wk);
          constexpr int N = D / 16 < PARTS ? 1 : D / 16 / PARTS;
          if (part * N < D / 16) tc_raw_keys<E, N>(t_q + Col::A, src, i < n_raw, part * N);
        }
#pragma unroll
        for (int c = 0; c < RC; ++c) {
          if (q + 4 * c >= nch) break;
#pragma unroll
          for (int e = 0; e < 4; ++e) zc[c][e] += __shfl_xor_sync(0xffffffffu, zc[c][e], 2);
          // (all lanes go through all chunks: shuffles above)
          if (kq < 4) {  // lane: rows n8, n8 + 8; groups kq, kq + 1
            float* z = zk_s + (part * 4 + kq) * ROWS + 16 * (q + 4 * c) + n8;
            z[0] = zc[c][0] * a.qscale;
            z[ROWS] = zc[c][1] * a.qscale;
            z[8] = zc[c][2] * a.qscale;
            z[ROWS + 8] = zc[c][3] * a.qscale;
          }
        }
      };
      float acc[RC][4] = {};
      // sums over tile t's tokens, of the weights and of the values' zeros: rows 16 q .. (and
      // 64 further on), this part's tokens
      auto sums = [&](int t) {
        // (columns 5 .. 7 are read by nobody); a second product adds the low parts
        const __half* zr = zv0 + ((t & 1) * 9 + (n8 < 4 ? n8 : 4)) * Ge::ZLD + kq;
        const __half* zl = zv0 + ((t & 1) * 9 + 5 + (n8 & 3)) * Ge::ZLD + kq;
        const uint32_t keep = n8 < 4 ? 0xFFFFFFFFu : 0u;
        // 8 x 8 blocks (tokens x rows) of weights, transposed on the way
        const int blk = lane >> 3;
        const uint32_t pa = sm0 + Ge::S_P + q * 4096 + (blk & 1) * 2048 + (blk >> 1) * 128 + (lane & 7) * 16;
#pragma unroll
        for (int c = 0; c < RC; ++c) {
          if (q + 4 * c >= nch) break;
#pragma unroll
          for (int j = 0; j < 8 / PARTS; ++j) {
            const int ks = 8 / PARTS * part + j;
            uint32_t av[4];
            tc_ldm<true>(av, pa + c * 4 * 4096 + ks * 256);
            tc_mma16816(acc[c], av, *reinterpret_cast<const uint32_t*>(zr + 16 * ks),
                        *reinterpret_cast<const uint32_t*>(zr + 16 * ks + 8));
            tc_mma16816(acc[c], av, *reinterpret_cast<const uint32_t*>(zl + 16 * ks) & keep,
                        *reinterpret_cast<const uint32_t*>(zl + 16 * ks + 8) & keep);
          }
        }
      };
      // values of tile t into tensor memory
      auto put_values = [&](int t) {
        if (t >= g.t1s) {
#pragma unroll 1
          for (int n = 0; n < kTcTile / RT; ++n) {
            tc_sync_workers<PARTS>();
            tc_stage_raw<D, RT, WORKERS>(reinterpret_cast<uint4*>(sm + Ge::S_RAW), wv, dv,
                                         (t - g.tq) * kTcTile + RT * n, g.r, n_raw);
            tc_sync_workers<PARTS>();
            if (q < NJ && tc_raw_values<D, E>(t_q + Col::V + RT / 2 * n + 8 * part,
                                              reinterpret_cast<const __half*>(sm + Ge::S_RAW) + q * 32 + lane, part))
              s_odd = 1;
          }
        } else if (q < NJ) {
          const unsigned char* stg = sm + Ge::S_RING + (st0 + t - g.t0) % Ge::NST * Ge::STAGE;
          const __half* sc = vsc0 + (t & 1) * 4 * Ge::VLD + q * Ge::VLD;
          tc_unpack<BITS, PARTS>(t_q + Col::V, reinterpret_cast<const uint32_t*>(stg + Ge::O_VC) + q * 32 + lane, D,
                                 reinterpret_cast<const uint4*>(sc), reinterpret_cast<const uint4*>(sc + 128), part,
                                 128 / TcUnit<BITS>::kUnit, konst);
        }
      };
      auto zeros = [&](const float* zk, int row) -> float {  // zk: of a group; over the parts
        float z = zk[row];
#pragma unroll
        for (int e = 1; e < PARTS; ++e) z += zk[e * 4 * ROWS + row];
        return z;
      };

      if (g.ok) {
        set_out(g.t0);
        tc_sync_workers<PARTS>();
#pragma unroll 1
        for (int t = g.t0; t < g.t1; ++t) {
          const int it = it0 + t - g.t0;
          const bool raw = t >= g.t1s;
          // ---- keys
          auto done_values = [&]() {  // the planes were read, and so were the weights
            if (t == g.t0) return;
            tc_wait(bar(TcBar::values), it - 1, dead);
            tc_fence_after();
          };
          if (!Col::APART) done_values();
          put_keys(t);
          tc_wait_st();
          tc_sync_scores<PARTS>();
          if (t + 1 < g.t1) set_out(t + 1);
          if (Col::APART) {
            done_values();
            put_values(t);
          }
          // ---- weights of 16-row chunks part, part + PARTS, against the references; `over`: by
          // how much a score exceeds its own.  The lane's token: in the cache (all rows see
          // it), drafted, or none
          const long long i = (long long)(raw ? t - g.tq : t) * kTcTile + q * 32 + lane;
          const bool in = raw ? i < g.r : i < g.n_q;
          const int node = raw && i >= g.r && i < n_raw ? (int)(i - g.r) : -1;
          auto seen = [&](int ch) -> uint32_t {  // one bit for each row
            return in ? 0xFFFFu : node < 0 ? 0u : tc_seen(mask_s, node, g.row0 + 16 * ch, a.N);
          };
          unsigned char* pb = sm + Ge::S_P + pk / 8 * 128 + pk % 8 * 16;
          const float* zk = zk_s + q * ROWS;  // the zeros' products of the lane's group
          auto weights = [&]() -> float {
            float over = -__builtin_huge_valf();
#pragma unroll 1
            for (int ch = part; ch < nch; ch += PARTS) {
              if (lane < 16) {
                const int row = 16 * ch + lane;
                off_s[lane] = m_s[row] - zeros(zk, row);
              }
              __syncwarp();
              float v[16];
              tc_ld16(t_q + Col::S + 16 * ch, v);
#pragma unroll
              for (int e4 = 0; e4 < 4; ++e4) {
                const float4 o = *reinterpret_cast<const float4*>(off_s + 4 * e4);
                v[4 * e4] = fmaf(v[4 * e4], c1, -o.x);
                v[4 * e4 + 1] = fmaf(v[4 * e4 + 1], c1, -o.y);
                v[4 * e4 + 2] = fmaf(v[4 * e4 + 2], c1, -o.z);
                v[4 * e4 + 3] = fmaf(v[4 * e4 + 3], c1, -o.w);
              }
              __syncwarp();
              const uint32_t sees = seen(ch);
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
              *reinterpret_cast<uint4*>(pb + ch * 4096) = make_uint4(w[0], w[1], w[2], w[3]);
              *reinterpret_cast<uint4*>(pb + ch * 4096 + 2048) = make_uint4(w[4], w[5], w[6], w[7]);
            }
            return over;
          };
          tc_wait(bar(TcBar::scores), it, dead);
          tc_fence_after();
          const float over = weights();
          if (!Col::APART) put_values(t);
          tc_wait_st();
          tc_fence_smem();
          const bool rise = tc_uniform(tc_sync_any<PARTS>(over > kTcSlack));
          if (rise) {
            // ---- new references: the maxima of the tile, joined over its groups
#pragma unroll 1
            for (int ch = part; ch < nch; ch += PARTS) {
              float v[16];
              tc_ld16(t_q + Col::S + 16 * ch, v);
              const uint32_t sees = seen(ch);
              const float z = lane < 16 ? zeros(zk, 16 * ch + lane) : 0.f;
              float mine = kTcNone;
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float d = fmaf(v[e], c1, __shfl_sync(0xffffffffu, z, e));
                const float m = tc_warp_max((sees >> e) & 1u ? d : kTcNone);
                if (lane == e) mine = m;
              }
              if (lane < 16) wmax_s[q * ROWS + 16 * ch + lane] = mine;
            }
            tc_sync_workers<PARTS>();
            if (tid < nr) {
              const float old = m_s[tid];
              const float mn = fmaxf(fmaxf(fmaxf(wmax_s[tid], wmax_s[ROWS + tid]),
                                           fmaxf(wmax_s[2 * ROWS + tid], wmax_s[3 * ROWS + tid])) - kTcBelow,
                                     old);
              f_s[tid] = old == kTcNone ? 0.0f : tc_ex2(old - mn);
              m_s[tid] = mn;
            }
            tc_sync_workers<PARTS>();
            weights();
            if (t > g.t0) {  // the accumulators so far (their products are done)
#pragma unroll 1
              for (int ch = part; ch < nch; ch += PARTS) {
                float v[16];
                tc_ld16(t_q + Col::O + 16 * ch, v);
#pragma unroll
                for (int k = 0; k < 16; ++k) v[k] *= f_s[16 * ch + k];
                tc_st16(t_q + Col::O + 16 * ch, v);
              }
              tc_wait_st();
            }
#pragma unroll
            for (int c = 0; c < RC; ++c) {
              if (q + 4 * c >= nch) break;
              const float* f = f_s + 16 * (q + 4 * c) + n8;
              acc[c][0] *= f[0];
              acc[c][1] *= f[0];
              acc[c][2] *= f[8];
              acc[c][3] *= f[8];
            }
            tc_fence_smem();
            tc_sync_any<PARTS>(false);
          }
          sums(t);
        }
#pragma unroll
        for (int c = 0; c < RC; ++c) {
          if (q + 4 * c >= nch) break;
          float* z = lz_s + (part * ROWS + 16 * (q + 4 * c) + n8) * 8 + kq;
          z[0] = acc[c][0];
          z[1] = acc[c][1];
          z[64] = acc[c][2];
          z[65] = acc[c][3];
        }
        tc_wait(bar(TcBar::values), it0 + g.t1 - 1 - g.t0, dead);
      }
      tc_sync_workers<PARTS>();

      // ---- end of a segment: rows first (reference and sum joined with those of the segments
      // before it, and the weights of both), then lane = channel, rows 4 part .. of each 4 PARTS
      {
        const int ch_d = q * 32 + lane;
        const bool odd = s_odd != 0;  // infinite or NaN raw values
        const int i1 = odd ? min((g.t1 - g.tq) * kTcTile, n_raw) : 0;
        const int first = s_first;
        const bool whole = first == 0 && g.ends, cont = g.t0 != first;
        float* pt = a.part + (2 * (long long)blockIdx.x + (first == 0)) * tree_part(p, D);
        __half* out = static_cast<__half*>(a.out) + (g.unit * rows + g.row0) * (long long)D + ch_d;
        if (tid < g.nrows) {
          float l = s_poison[seg & 1] != 0 || *dead != 0 ? kNaN : 0.f, m = m_s[tid];
#pragma unroll
          for (int i = 0; i < PARTS; ++i) l += lz_s[(i * ROWS + tid) * 8 + 4];
          bool mark = odd;
          if (cont) {
            const float m0 = pt[2 * tid], l0 = pt[2 * tid + 1], top = fmaxf(m0, m);
            const float f0 = tc_ex2(m0 - top), f = tc_ex2(m - top);
            mark |= __float_as_int(l0) < 0;
            l = fmaf(f0, fabsf(l0), f * l);
            m = top;
            wmax_s[tid] = f;
            wmax_s[ROWS + tid] = f0;
          }
          f_s[tid] = l;
          if (!whole) {
            pt[2 * tid] = m;
            pt[2 * tid + 1] = mark ? -l : l;
          }
        }
        tc_sync_workers<PARTS>();
#pragma unroll 1
        for (int e4 = 4 * part; e4 < g.nrows && q < NJ; e4 += 4 * PARTS) {
          float v[4] = {0.f, 0.f, 0.f, 0.f};
          if (g.ok) tc_ld4(t_q + Col::O + e4, v);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int row = e4 + e;
            if (row >= g.nrows) break;
            float zs = 0.f;
#pragma unroll
            for (int i = 0; i < PARTS; ++i) zs += lz_s[(i * ROWS + row) * 8 + q];
            float o = fmaf(2.0f, v[e], zs);
            float* po = pt + 2 * nr + row * D + ch_d;
            if (odd)
              o += tc_odd<D>(wv + ch_d, dv + ch_d, mask_s, max(g.t0 - g.tq, 0) * kTcTile, i1, g.r, g.row0 + row, a.N);
            if (cont) o = tc_part(wmax_s[row], o) + tc_part(wmax_s[ROWS + row], *po);
            if (whole) {
              const float l = f_s[row];
              out[row * D] = __float2half_rn(l == 0.f ? 0.f : __fdividef(o, l));
            } else {
              *po = o;
            }
          }
        }
      }
      if (tid == 0) s_poison[(seg & 1) ^ 1] = 0;  // the next segment's
      if (g.ok) {
        it0 += g.t1 - g.t0;
        st0 += max(g.t1s - g.t0, 0);
      }
      tc_sync_workers<PARTS>();
    }
  }

  __syncthreads();
  if (warp == Ge::WARPS) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(Col::N)
                 : "memory");
  }
}

}  // namespace
}  // namespace kivi
