// kivi_tree_tc.cu -- instances of the tensor-core attention of drafted tokens
// for caches with binary32 scales and zeros.
#include "kivi_tree_tc.cuh"

namespace kivi {
namespace {

template <int D, int BITS, int PARTS>
cudaError_t tc_p(const TreeArgs& a, const TreePlan& p, cudaStream_t s) {
  using Ge = TcGeo<D, BITS, (int)sizeof(float), PARTS>;
  const int bytes = a.N * ((a.N + 31) / 32) * 4 + Ge::BYTES;
  static std::atomic<bool> done[kTreeDevices];
  const cudaError_t e = tree_smem(tree_tc_kernel<D, BITS, float, PARTS>, Ge::MOST, done);
  if (e != cudaSuccess) return e;
  tree_tc_kernel<D, BITS, float, PARTS><<<p.ctas, kTcThreads<PARTS>, bytes, s>>>(a, p);
  return cudaGetLastError();
}
template <int D, int BITS>
cudaError_t tc_t(const TreeArgs& a, const TreePlan& p, cudaStream_t s) {
  return p.parts == 2 ? tc_p<D, BITS, 2>(a, p, s) : tc_p<D, BITS, 4>(a, p, s);
}
template <int BITS>
cudaError_t tc_d(const TreeArgs& a, const TreePlan& p, cudaStream_t s) {
  switch (a.D) {
    case 32: return tc_t<32, BITS>(a, p, s);
    case 64: return tc_t<64, BITS>(a, p, s);
    case 128: return tc_t<128, BITS>(a, p, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t tree_tc_f32(const TreeArgs& a, const TreePlan& p, cudaStream_t s) {
  switch (a.bits) {
    case 1: return tc_d<1>(a, p, s);
    case 2: return tc_d<2>(a, p, s);
    case 3: return tc_d<3>(a, p, s);
    case 4: return tc_d<4>(a, p, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace kivi
