// kivi_tree_merge.cu -- the join of the partials of attention of drafted
// tokens, and the choice of its kernel.
#include "kivi_tree.cuh"

namespace kivi {
namespace {

constexpr int kMergeRows = 8;
constexpr int kMergeThreads = 32 * kMergeRows;

// The sum of a lane's share of the partials (P: the first one's piece were it a slot 0) where
// some may not be finite: one with a weight of 0 is added as it is.
__device__ __noinline__ float4 merge_odd(const float* P, long long stride, const float* w, int s,
                                         int n, int step) {
  auto join = [](float e, float x, float sum) {
    return e != 0.f || isfinite(x) ? fmaf(e, x, sum) : sum + x;
  };
  float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
  for (; s < n; s += step) {
    const float e = w[s];
    const float4 v = __ldcg(reinterpret_cast<const float4*>(P + (s == 0 ? 1 : 2LL * s) * stride));
    num.x = join(e, v.x, num.x);
    num.y = join(e, v.y, num.y);
    num.z = join(e, v.z, num.z);
    num.w = join(e, v.w, num.w);
  }
  return num;
}

// Block (group, 8 rows of it), a warp for each row: of the segments' partials (m_s,
// l_s, acc_s), M = max m_s and weights 2^(m_s - M) first, then
// out = sum 2^(m_s - M) acc_s / sum 2^(m_s - M) l_s with all loads independent of each
// other: bound by their latency (a long cache of few heads has a partial of every CTA;
// 9 rows of one binary32 head of 20011 tokens, 313 partials, take 30 us in all at D 64 and
// 48 at D 128; with each partial weighed as it came the first took 41).  A row that
// attended to nothing (all l_s = 0) is 0.  An infinite or NaN accumulator keeps its part
// where the weight of its segment comes to 0: what a row attends to may not vanish with
// the way in which the work is split.  The split kernels say by the sign of l_s where
// there may be any (asking each accumulator here took the 48 us to 107, and a second
// walk behind the first, by its registers, to 54).
template <int D, typename T>
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(TreeArgs a, TreePlan p) {
  const long long gpb = (long long)a.Hkv * p.n_rb;
  const long long grp = blockIdx.x;
  const long long b = grp / gpb;
  const int h = (int)(grp % gpb / p.n_rb), rb = (int)(grp % p.n_rb);
  const TreeSeq q = tree_seq(a, p, b);
  __shared__ long long s_total, s_first;
  if (threadIdx.x < 32) {
    // the group's first tile: those of the sequences before it, then its own
    long long total, first;
    if (a.st == nullptr) {
      total = a.B * gpb * q.ut;
      first = b * gpb * q.ut;
    } else {
      long long t = 0, f = 0;
      for (long long i = threadIdx.x; i < a.B; i += 32) {
        const long long n = gpb * tree_seq(a, p, i).ut;
        t += n;
        f += i < b ? n : 0;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        t += __shfl_xor_sync(0xffffffffu, t, o);
        f += __shfl_xor_sync(0xffffffffu, f, o);
      }
      total = t;
      first = f;
    }
    if (threadIdx.x == 0) {
      s_total = total;
      s_first = first + (grp % gpb) * q.ut;
    }
  }
  __syncthreads();
  const long long W = tree_range(p, s_total);
  const long long c0 = s_first / W, c1 = (s_first + q.ut - 1) / W;
  // launched while the split kernel runs, which every block waits for (a grid that
  // ended before it would let the stream's next kernel overtake it)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (c0 == c1) return;  // written by its only CTA
  const int rows = a.gq * a.N, n = (int)(c1 - c0 + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.y * kMergeRows + warp;
  if (row >= p.rb || rb * p.rb + row >= rows) return;
  const long long stride = tree_part(p, D);
  // partial s: slot 1 of the first CTA, slot 0 of the others
  const float* P = a.part + 2 * c0 * stride;
  auto at = [&](int s) { return P + (s == 0 ? stride : 2LL * s * stride); };
  extern __shared__ float w_s[];  // [8 rows][partials]
  float* w = w_s + warp * n;
  float M = -__builtin_huge_valf();
  bool odd = false;
  for (int s = lane; s < n; s += 32) {
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(at(s)) + row);
    if (ml.y != 0.f) M = fmaxf(M, ml.x);
    odd |= __float_as_int(ml.y) < 0;
  }
  M = warp_max(M);
  odd = __any_sync(0xffffffffu, odd);
  float den = 0.f;
  for (int s = lane; s < n; s += 32) {
    const float2 ml = __ldcg(reinterpret_cast<const float2*>(at(s)) + row);
    const float e = ml.y == 0.f ? 0.f : exp2f(ml.x - M);
    w[s] = e;
    den = fmaf(e, fabsf(ml.y), den);
  }
  den = warp_sum(den);
  __syncwarp();
  constexpr int LPR = D / 4, SPL = 32 / LPR;  // lanes of a row, and how many share the partials
  const int d = lane % LPR * 4;
  float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
  if (odd) {
    num = merge_odd(P + 2 * p.rb + (long long)row * D + d, stride, w, lane / LPR, n, SPL);
  } else {
#pragma unroll 8
    for (int s = lane / LPR; s < n; s += SPL) {
      const float e = w[s];
      const float4 v = __ldcg(reinterpret_cast<const float4*>(at(s) + 2 * p.rb + (long long)row * D + d));
      num.x = fmaf(e, v.x, num.x);
      num.y = fmaf(e, v.y, num.y);
      num.z = fmaf(e, v.z, num.z);
      num.w = fmaf(e, v.w, num.w);
    }
  }
#pragma unroll
  for (int o = LPR; o < 32; o <<= 1) {
    num.x += __shfl_xor_sync(0xffffffffu, num.x, o);
    num.y += __shfl_xor_sync(0xffffffffu, num.y, o);
    num.z += __shfl_xor_sync(0xffffffffu, num.z, o);
    num.w += __shfl_xor_sync(0xffffffffu, num.w, o);
  }
  if (lane >= LPR) return;
  T* o = static_cast<T*>(a.out) + ((b * a.Hkv + h) * (long long)rows + (long long)rb * p.rb + row) * D + d;
  const float inv = 1.f / den;
  o[0] = from_f32<T>(den == 0.f ? 0.f : num.x * inv);
  o[1] = from_f32<T>(den == 0.f ? 0.f : num.y * inv);
  o[2] = from_f32<T>(den == 0.f ? 0.f : num.z * inv);
  o[3] = from_f32<T>(den == 0.f ? 0.f : num.w * inv);
}

template <int D, typename T>
cudaError_t merge_t(const TreeArgs& a, const TreePlan& p, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)a.B * a.Hkv * p.n_rb), (unsigned)((p.rb + kMergeRows - 1) / kMergeRows));
  cfg.blockDim = dim3(kMergeThreads);
  cfg.dynamicSmemBytes = (size_t)kMergeRows * p.ctas * sizeof(float);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, tree_merge_kernel<D, T>, a, p);
}
template <typename T>
cudaError_t merge_d(const TreeArgs& a, const TreePlan& p, cudaStream_t s) {
  switch (a.D) {
    case 32: return merge_t<32, T>(a, p, s);
    case 64: return merge_t<64, T>(a, p, s);
    case 128: return merge_t<128, T>(a, p, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

// The plan of a call.  CUDA cores (binary32): 64 rows a block, or 16 where all fit
// (four blocks on an SM instead of three; at D 128 of two, whose ranges are cut for
// three).  Tensor cores: up to 64 rows two blocks of threads on an SM, more in row blocks
// of equal size up to 128 rows, one block on an SM (both sides measured:
// kivi_tree_tc.cuh).
static TreePlan tree_plan(int gq, int N, int dtype, int sms) {
  const int rows = gq * N;
  TreePlan p;
  if (dtype == 1) {
    p.rb = rows <= 16 ? 16 : 64;
    p.n_rb = (rows + p.rb - 1) / p.rb;
    p.tt = 32;
    p.ctas = sms * (p.rb == 16 ? 4 : 3);
    p.parts = 0;
  } else {
    p.parts = rows <= 64 ? 2 : 4;
    const int most = 32 * p.parts;
    p.n_rb = (rows + most - 1) / most;
    p.rb = ((rows + p.n_rb - 1) / p.n_rb + 15) / 16 * 16;
    p.n_rb = (rows + p.rb - 1) / p.rb;
    p.tt = 128;
    p.ctas = p.parts == 2 ? 2 * sms : sms;
  }
  return p;
}

size_t tree_workspace_bytes(int gq, int D, int dtype, int N, int sms) {
  const TreePlan p = tree_plan(gq, N, dtype, sms);
  return (size_t)(tree_slots(p) * tree_part(p, D)) * sizeof(float);
}

cudaError_t launch_tree(const TreeArgs& a, cudaStream_t s) {
  const TreePlan p = tree_plan(a.gq, a.N, a.dtype, a.sms);
  const cudaError_t e = a.dtype == 1    ? tree_simt(a, p, s)
                        : a.meta == 1 ? tree_tc_meta16(a, p, s)
                                      : tree_tc_f32(a, p, s);
  if (e != cudaSuccess) return e;
  return a.dtype == 1 ? merge_d<float>(a, p, s) : merge_d<__half>(a, p, s);
}

}  // namespace kivi
