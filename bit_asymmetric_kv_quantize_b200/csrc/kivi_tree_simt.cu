// kivi_tree_simt.cu -- attention of drafted tokens over a binary32 cache on
// CUDA cores, everything in binary32.
//
// For row (query head, node i) of a KV head, over the cache's tokens t and
// the drafted tokens j whose bit is set in the node's mask:
//   s = softmax_scale * <q, K^>,  out = sum exp(s - max) V^ / sum exp(s - max).
// One pass, tile by tile: running maximum and sum of each row, accumulators
// rescaled when the maximum rises.  A tile of 32 tokens is turned into
// numbers in shared memory once for all rows of the block; scores and
// accumulators are register tiles of a matrix product, in packed binary32 pairs.
// There is no binary32 matrix instruction, and binary16 operands would lose what a
// binary32 cache is kept for.
// What bounds it: latency.  6 x 4 heads of up to 2999 tokens at 3 bits, 39 rows,
// take 43 us; the arithmetic alone (39 rows in a block of 64) would take 11 us at 75
// TFLOP/s, but a block has four warps, three blocks an SM (168 registers a thread hold
// the tiles; at D 128 some 240, two blocks), and 39 % of the issue slots are used:
// each waits for its tile's words (0.9 warps a scheduler's issue) and for shared memory
// (1.2).
#include "kivi_dequant.cuh"
#include "kivi_tree.cuh"

namespace kivi {
namespace {

constexpr int kThreads = 128;

// Two binary32 lanes in one instruction (the packed .f32x2 arithmetic of sm_100),
// each rounded like its scalar counterpart.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n\t.reg .b64 x, y, z, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\t"
      "mov.b64 {%0, %1}, w;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
constexpr int kTT = 32;  // = one key group
// Tiles of a segment at most.  A sum that grows by equal steps is off by as much as half a
// unit of its last place at each of them, always to the same side: 16384 equal values in one
// range came out 4.7e-5 off, 2^20 of them 3e-3.  So a range takes a group in segments of
// 512 tokens, whose partials are joined in the range's slot (2e-6 and 6e-6; 3 to 5 % more
// time where ranges are that long).
constexpr int kSimtMost = 16;

// An accumulator at its weight; an infinite or NaN one is kept where that comes to 0 (as in
// tree_merge_kernel).
__device__ __forceinline__ float simt_part(float f, float x) {
  return f != 0.f || isfinite(x) ? f * x : x;
}

template <int D, int RB>
struct SimtSmem {
  static constexpr int LD = D + 4;  // row stride of K: 8 rows on different banks
  static constexpr int Q = 0;
  static constexpr int K = Q + RB * D;
  static constexpr int V = K + kTT * LD;
  static constexpr int P = V + kTT * D;         // [token][row]
  static constexpr int PL = RB + 4;
  static constexpr int SCL = P + kTT * PL;
  static constexpr int FLOATS = SCL + RB;
};

template <int D, int BITS, int RB>
__global__ void __launch_bounds__(kThreads) tree_simt_kernel(TreeArgs a, TreePlan p) {
  using SM = SimtSmem<D, RB>;
  constexpr int TCN = RB == 64 ? 8 : 16;         // column groups of the scores
  constexpr int SR = RB / (kThreads / TCN), SC = kTT / TCN;
  constexpr int PCN = RB == 64 ? 16 : 32;        // column groups of the accumulators
  constexpr int OR = RB / (kThreads / PCN), OC = D / PCN;
  constexpr int OV = OC >= 4 ? 4 : OC;           // adjacent channels of a thread
  constexpr int ON = OC / OV;
  static_assert(kTT == kTile && kTT == kG, "a tile is a key group");
  asm volatile("griddepcontrol.launch_dependents;");
  extern __shared__ __align__(16) float sm[];
  __shared__ TreeAt s_at;
  __shared__ int s_odd;  // the segment has infinite or NaN raw values
  const int tid = threadIdx.x;
  const long long W0 = blockIdx.x;
  if (tid < 32) {
    TreeAt at = tree_find(a, p, 0);
    const long long W = tree_range(p, at.total);
    const long long total = at.total;
    at = tree_find(a, p, W0 * W);
    at.total = total;
    if (tid == 0) s_at = at;
  }
  __syncthreads();
  const long long total = s_at.total, W = tree_range(p, total);
  long long x = W0 * W;
  const long long end = x + W < total ? x + W : total;
  if (x >= end) return;
  long long b = s_at.b, rem = s_at.rem;
  const int rows = a.gq * a.N, mw = (a.N + 31) / 32;
  const float kInf = __builtin_huge_valf();

  bool begins = false;  // the range has the group's first tile
  while (x < end) {
    const TreeSeq q = tree_seq(a, p, b);
    const long long gpb = (long long)a.Hkv * p.n_rb;
    if (rem >= gpb * q.ut) {  // next sequence
      rem -= gpb * q.ut;
      ++b;
      continue;
    }
    const long long grp = rem / q.ut, tile0 = rem % q.ut;
    const long long left = end - x;
    const long long most = left < kSimtMost ? left : kSimtMost;
    const long long nt = q.ut - tile0 < most ? q.ut - tile0 : most;
    const bool cont = x != W0 * W && tile0 != 0;  // joins the segment before
    if (!cont) begins = tile0 == 0;
    const int h = (int)(grp / p.n_rb), row0 = (int)(grp % p.n_rb) * RB;
    const long long unit = b * a.Hkv + h;
    const long long tq = (q.n_q + kTT - 1) / kTT;

    __syncthreads();  // the segment before has read its last tile
    if (tid == 0) s_odd = 0;
    const float* qp = static_cast<const float*>(a.q) + (unit * rows + row0) * D;
    for (int i = tid; i < RB * D; i += kThreads)
      sm[SM::Q + i] = row0 + i / D < rows ? qp[i] * a.qscale : 0.f;

    float m[SR], l[SR], acc[OR][OC];
#pragma unroll
    for (int i = 0; i < SR; ++i) {
      m[i] = -kInf;
      l[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < OR; ++i)
#pragma unroll
      for (int j = 0; j < OC; ++j) acc[i][j] = 0.f;
    bool poison = !q.ok;
    const int sr0 = tid / TCN * SR, sc0 = tid % TCN;
    const int or0 = tid / PCN * OR, oc0 = tid % PCN * OV;

    for (long long t = tile0; t < tile0 + nt && !poison; ++t) {
      const bool raw = t >= tq;  // window and drafted tokens, as they are
      // ---- the tile as numbers
      constexpr int COLS = D / 4, TPT = kTT / (kThreads / COLS);  // tokens of a thread
      const int ch = tid % COLS * 4, tk = tid / COLS * TPT;
      __syncthreads();  // the tile before is read
      if (!raw) {
        long long su, stl;
        if (!store_tile(a.c, unit, t, &su, &stl)) {
          poison = true;  // the same for the whole block
          break;
        }
        using Lt = Layout<D, BITS>;
        const long long row = stl * kTT + tk, Ts = store_tokens(a.c);
        const uint32_t* ku = a.c.k_codes + su * Lt::k_codes_unit(Ts);
        const uint32_t* vu = a.c.v_codes + su * Lt::v_codes_unit(Ts);
        const long long mo = su * Lt::v_meta_unit(Ts) + row * Lt::NJ + ch / kGv;
        float s[4], z[4];
        key_meta<D, BITS, float, 4>(a.c, su, row, ch, s, z);
#pragma unroll
        for (int i = 0; i < TPT; ++i) {
          uint32_t kw[Lt::WB], vw[Lt::WB][4];
          int c[4];
          key_words<D, BITS, 4>(ku, row + i, ch, kw);
          key_codes<D, BITS, 4>(kw, ch, c);
          *reinterpret_cast<float4*>(sm + SM::K + (tk + i) * SM::LD + ch) =
              make_float4(fmaf((float)c[0], s[0], z[0]), fmaf((float)c[1], s[1], z[1]),
                          fmaf((float)c[2], s[2], z[2]), fmaf((float)c[3], s[3], z[3]));
          const float vs = a.c.v_scale_f()[mo + i * Lt::NJ], vz = a.c.v_zero_f()[mo + i * Lt::NJ];
          value_words<D, BITS, 4>(vu, row + i, ch, vw);
          value_codes<D, BITS, 4>(vw, row + i, c);
          *reinterpret_cast<float4*>(sm + SM::V + (tk + i) * D + ch) =
              make_float4(fmaf((float)c[0], vs, vz), fmaf((float)c[1], vs, vz),
                          fmaf((float)c[2], vs, vz), fmaf((float)c[3], vs, vz));
        }
      } else {
        const long long first = (t - tq) * kTT;
#pragma unroll
        for (int i = 0; i < TPT; ++i) {
          const long long tok = first + tk + i;
          const float* kp = nullptr;
          const float* vp = nullptr;
          if (tok < q.r) {
            kp = static_cast<const float*>(a.c.k_res) + (unit * a.c.R + tok) * D + ch;
            vp = static_cast<const float*>(a.c.v_res) + (unit * a.c.R + tok) * D + ch;
          } else if (tok < q.r + a.N) {
            kp = static_cast<const float*>(a.k) + (unit * a.N + tok - q.r) * D + ch;
            vp = static_cast<const float*>(a.v) + (unit * a.N + tok - q.r) * D + ch;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            sm[SM::K + (tk + i) * SM::LD + ch + e] = kp ? kp[e] : 0.f;
            // an infinity or a NaN is left out: it joins at the segment's end, for the rows
            // that attend to it (0 times it would spoil the others, and a later rescaling
            // by 0 itself)
            const float x = vp ? vp[e] : 0.f;
            const bool fin = isfinite(x);
            if (!fin) s_odd = 1;
            sm[SM::V + (tk + i) * D + ch + e] = fin ? x : 0.f;
          }
        }
      }
      __syncthreads();
      // ---- scores
      // (each as two sums, over the even and the odd channels)
      float2 s2[SR][SC];
#pragma unroll
      for (int i = 0; i < SR; ++i)
#pragma unroll
        for (int j = 0; j < SC; ++j) s2[i][j] = make_float2(0.f, 0.f);
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        float4 qv[SR], kv[SC];
#pragma unroll
        for (int i = 0; i < SR; ++i)
          qv[i] = *reinterpret_cast<const float4*>(sm + SM::Q + (sr0 + i) * D + d);
#pragma unroll
        for (int j = 0; j < SC; ++j)
          kv[j] = *reinterpret_cast<const float4*>(sm + SM::K + (sc0 + j * TCN) * SM::LD + d);
#pragma unroll
        for (int i = 0; i < SR; ++i)
#pragma unroll
          for (int j = 0; j < SC; ++j) {
            s2[i][j] = fma2(make_float2(qv[i].x, qv[i].y), make_float2(kv[j].x, kv[j].y), s2[i][j]);
            s2[i][j] = fma2(make_float2(qv[i].z, qv[i].w), make_float2(kv[j].z, kv[j].w), s2[i][j]);
          }
      }
      float sc[SR][SC];
#pragma unroll
      for (int i = 0; i < SR; ++i)
#pragma unroll
        for (int j = 0; j < SC; ++j) sc[i][j] = s2[i][j].x + s2[i][j].y;
      // ---- masks: drafted tokens that a node does not see, and the end
      if (raw) {
#pragma unroll
        for (int i = 0; i < SR; ++i) {
          const int row = row0 + sr0 + i;
          const uint32_t* mk = a.mask + (b * a.N + row % a.N) * mw;
#pragma unroll
          for (int j = 0; j < SC; ++j) {
            const long long tok = (t - tq) * kTT + sc0 + j * TCN;
            bool in = tok < q.r;
            if (!in && tok < q.r + a.N && row < rows) {
              const int node = (int)(tok - q.r);
              in = (mk[node / 32] >> (node % 32)) & 1u;
            }
            if (!in) sc[i][j] = -kInf;
          }
        }
      }
      // ---- running maximum and sum (the TCN threads of a row are neighbours)
#pragma unroll
      for (int i = 0; i < SR; ++i) {
        float mx = sc[i][0];
#pragma unroll
        for (int j = 1; j < SC; ++j) mx = fmaxf(mx, sc[i][j]);
#pragma unroll
        for (int o = 1; o < TCN; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float mn = fmaxf(m[i], mx);
        const float base = mn == -kInf ? 0.f : mn;  // nothing seen so far
        const float f = exp2f(m[i] - base);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < SC; ++j) {
          const float e = exp2f(sc[i][j] - base);
          sm[SM::P + (sc0 + j * TCN) * SM::PL + sr0 + i] = e;
          sum += e;
        }
#pragma unroll
        for (int o = 1; o < TCN; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l[i] = l[i] * f + sum;
        m[i] = mn;
        if (sc0 == 0) sm[SM::SCL + sr0 + i] = f;
      }
      __syncthreads();
      // ---- accumulators
#pragma unroll
      for (int i = 0; i < OR; ++i) {
        const float f = sm[SM::SCL + or0 + i];
#pragma unroll
        for (int j = 0; j < OC; ++j) acc[i][j] *= f;
      }
#pragma unroll 4
      for (int tk2 = 0; tk2 < kTT; ++tk2) {
        float pv[OR], vv[OC];
#pragma unroll
        for (int i = 0; i < OR; i += 4)
          *reinterpret_cast<float4*>(pv + i) =
              *reinterpret_cast<const float4*>(sm + SM::P + tk2 * SM::PL + or0 + i);
#pragma unroll
        for (int g = 0; g < ON; ++g)
#pragma unroll
          for (int e = 0; e < OV; ++e)
            vv[g * OV + e] = sm[SM::V + tk2 * D + g * (D / ON) + oc0 + e];
#pragma unroll
        for (int i = 0; i < OR; ++i) {
          if constexpr (OC % 2 == 0) {
#pragma unroll
            for (int j = 0; j < OC; j += 2) {
              const float2 r = fma2(make_float2(pv[i], pv[i]), make_float2(vv[j], vv[j + 1]),
                                    make_float2(acc[i][j], acc[i][j + 1]));
              acc[i][j] = r.x;
              acc[i][j + 1] = r.y;
            }
          } else {
#pragma unroll
            for (int j = 0; j < OC; ++j) acc[i][j] = fmaf(pv[i], vv[j], acc[i][j]);
          }
        }
      }
    }

    // ---- the segment's end
    const bool whole = begins && tile0 + nt == q.ut;
    float* pp = a.part + (2 * W0 + begins) * tree_part(p, D);
    if (poison) {  // refused sequence, or a page outside the pool
#pragma unroll
      for (int i = 0; i < SR; ++i) {
        l[i] = kNaN;
        m[i] = 0.f;
      }
    }
    __syncthreads();
    if (sc0 == 0) {
#pragma unroll
      for (int i = 0; i < SR; ++i) {
        sm[SM::P + 2 * (sr0 + i)] = m[i];
        sm[SM::P + 2 * (sr0 + i) + 1] = l[i];
      }
    }
    __syncthreads();
    if (cont) {
      // joined with the segments so far: rows first (a sum's sign only marks partials with
      // infinite or NaN raw values), then the accumulators at the weights of both
      float* f_s = sm + SM::P + 2 * RB;
      if (tid < RB) {
        const float m0 = pp[2 * tid], l0 = pp[2 * tid + 1], m1 = sm[SM::P + 2 * tid];
        const float top = fmaxf(m0, m1), base = top == -kInf ? 0.f : top;
        const float f0 = exp2f(m0 - base), f1 = exp2f(m1 - base);
        const float lr = fmaf(f0, fabsf(l0), f1 * sm[SM::P + 2 * tid + 1]);
        sm[SM::P + 2 * tid] = top;
        sm[SM::P + 2 * tid + 1] = __float_as_int(l0) < 0 ? -lr : lr;
        f_s[tid] = f0;
        f_s[RB + tid] = f1;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < OR; ++i) {
        const float f0 = f_s[or0 + i], f1 = f_s[RB + or0 + i];
#pragma unroll
        for (int g = 0; g < ON; ++g)
#pragma unroll
          for (int e = 0; e < OV; ++e)
            acc[i][g * OV + e] =
                simt_part(f0, pp[2 * RB + (or0 + i) * D + g * (D / ON) + oc0 + e]) +
                simt_part(f1, acc[i][g * OV + e]);
      }
    }
    float* dst;  // the block's rows of the output, or the accumulators of its partial
    if (whole) {
      dst = static_cast<float*>(a.out) + (unit * rows + row0) * D;
#pragma unroll
      for (int i = 0; i < OR; ++i) {
        if (row0 + or0 + i >= rows) continue;
        const float lr = fabsf(sm[SM::P + 2 * (or0 + i) + 1]);
        const float inv = 1.f / lr;
#pragma unroll
        for (int g = 0; g < ON; ++g)
#pragma unroll
          for (int e = 0; e < OV; ++e)
            dst[(or0 + i) * D + g * (D / ON) + oc0 + e] =
                lr == 0.f ? 0.f : acc[i][g * OV + e] * inv;
      }
    } else {
      for (int i = tid; i < 2 * RB; i += kThreads)
        pp[i] = s_odd && (i & 1) ? -fabsf(sm[SM::P + i]) : sm[SM::P + i];
      dst = pp + 2 * RB;
#pragma unroll
      for (int i = 0; i < OR; ++i)
#pragma unroll
        for (int g = 0; g < ON; ++g)
#pragma unroll
          for (int e = 0; e < OV; ++e)
            dst[(or0 + i) * D + g * (D / ON) + oc0 + e] = acc[i][g * OV + e];
    }
    if (s_odd && !poison) {  // infinite or NaN raw values, of the tokens that a row attends to
      __syncthreads();       // (added to what the block's threads just wrote)
      const long long i1 = min((tile0 + nt - tq) * kTT, (long long)q.r + a.N);
#pragma unroll 1
      for (int i = tid; i < min(RB, rows - row0) * D; i += kThreads) {
        const int row = i / D;
        if (whole && sm[SM::P + 2 * row + 1] == 0.f) continue;  // no weight: stays 0
        const uint32_t* mk = a.mask + (b * a.N + (row0 + row) % a.N) * mw;
#pragma unroll 1
        for (long long tok = max(tile0 - tq, 0LL) * kTT; tok < i1; ++tok) {
          const int node = (int)(tok - q.r);
          const float v =
              node < 0 ? static_cast<const float*>(a.c.v_res)[(unit * a.c.R + tok) * D + i % D]
                       : static_cast<const float*>(a.v)[(unit * a.N + node) * D + i % D];
          if (!isfinite(v) && (node < 0 || ((mk[node / 32] >> (node % 32)) & 1u))) dst[i] += v;
        }
      }
    }
    x += nt;
    rem += nt;
  }
}

template <int D, int BITS, int RB>
cudaError_t tree_r(const TreeArgs& a, const TreePlan& p, cudaStream_t s) {
  constexpr int bytes = SimtSmem<D, RB>::FLOATS * 4;
  static std::atomic<bool> done[kTreeDevices];
  const cudaError_t e = tree_smem(tree_simt_kernel<D, BITS, RB>, bytes, done);
  if (e != cudaSuccess) return e;
  tree_simt_kernel<D, BITS, RB><<<p.ctas, kThreads, bytes, s>>>(a, p);
  return cudaGetLastError();
}
template <int D, int BITS>
cudaError_t tree_t(const TreeArgs& a, const TreePlan& p, cudaStream_t s) {
  return p.rb == 16 ? tree_r<D, BITS, 16>(a, p, s) : tree_r<D, BITS, 64>(a, p, s);
}
template <int BITS>
cudaError_t tree_d(const TreeArgs& a, const TreePlan& p, cudaStream_t s) {
  switch (a.D) {
    case 32: return tree_t<32, BITS>(a, p, s);
    case 64: return tree_t<64, BITS>(a, p, s);
    case 128: return tree_t<128, BITS>(a, p, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t tree_simt(const TreeArgs& a, const TreePlan& p, cudaStream_t s) {
  switch (a.bits) {
    case 1: return tree_d<1>(a, p, s);
    case 2: return tree_d<2>(a, p, s);
    case 3: return tree_d<3>(a, p, s);
    case 4: return tree_d<4>(a, p, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace kivi
