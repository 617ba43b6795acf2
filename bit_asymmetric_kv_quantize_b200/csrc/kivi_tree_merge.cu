// kivi_tree_merge.cu -- the join of the partials of attention of drafted
// tokens, and the choice of its kernel.
#include "kivi_tree.cuh"

namespace kivi {
namespace {

constexpr int kMergeRows = 8;
constexpr int kMergeThreads = 128;

// Block (group, 8 rows of it): for each row the segments' partials
// (m_s, l_s, acc_s), M = max m_s: out = sum 2^(m_s - M) acc_s / sum 2^(m_s - M) l_s;
// a row that attended to nothing (all l_s = 0) is 0.
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
  const int rows = a.gq * a.N;
  const long long stride = tree_part(p, D);
  T* out = static_cast<T*>(a.out) + ((b * a.Hkv + h) * (long long)rows + (long long)rb * p.rb) * D;
  constexpr int C4 = D / 4;
  for (int i = threadIdx.x; i < kMergeRows * C4; i += kMergeThreads) {
    const int row = blockIdx.y * kMergeRows + i / C4, d = i % C4 * 4;
    if (row >= p.rb || rb * p.rb + row >= rows) continue;
    float M = -__builtin_huge_valf(), den = 0.f;
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
    for (long long c = c0; c <= c1; ++c) {
      const float* P = a.part + (2 * c + (c == c0)) * stride;
      const float m = __ldcg(P + 2 * row), l = __ldcg(P + 2 * row + 1);
      const float4 v = __ldcg(reinterpret_cast<const float4*>(P + 2 * p.rb + (long long)row * D + d));
      if (l == 0.f) continue;
      const float Mn = fmaxf(M, m);
      const float e0 = M == Mn ? 1.f : exp2f(M - Mn), e1 = m == Mn ? 1.f : exp2f(m - Mn);
      den = den * e0 + l * e1;
      num.x = num.x * e0 + v.x * e1;
      num.y = num.y * e0 + v.y * e1;
      num.z = num.z * e0 + v.z * e1;
      num.w = num.w * e0 + v.w * e1;
      M = Mn;
    }
    const float inv = 1.f / den;
    T* o = out + (long long)row * D + d;
    o[0] = from_f32<T>(den == 0.f ? 0.f : num.x * inv);
    o[1] = from_f32<T>(den == 0.f ? 0.f : num.y * inv);
    o[2] = from_f32<T>(den == 0.f ? 0.f : num.z * inv);
    o[3] = from_f32<T>(den == 0.f ? 0.f : num.w * inv);
  }
}

template <int D, typename T>
cudaError_t merge_t(const TreeArgs& a, const TreePlan& p, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)a.B * a.Hkv * p.n_rb), (unsigned)((p.rb + kMergeRows - 1) / kMergeRows));
  cfg.blockDim = dim3(kMergeThreads);
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

// The plan of a call.  CUDA cores (binary32): 64 rows a block, or 16 where all
// fit.  Tensor cores: up to 64 rows a block, more in blocks of equal size (each
// unpacks the cache again); two blocks of threads per SM.
static TreePlan tree_plan(int gq, int N, int dtype, int sms) {
  const int rows = gq * N;
  TreePlan p;
  if (dtype == 1) {
    p.rb = rows <= 16 ? 16 : 64;
    p.n_rb = (rows + p.rb - 1) / p.rb;
    p.tt = 32;
    p.ctas = sms * (p.rb == 16 ? 4 : 3);
    p.min_w = 2;
  } else {
    p.n_rb = (rows + 63) / 64;
    p.rb = ((rows + p.n_rb - 1) / p.n_rb + 15) / 16 * 16;
    p.n_rb = (rows + p.rb - 1) / p.rb;
    p.tt = 128;
    p.ctas = 2 * sms;
    p.min_w = 1;
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
