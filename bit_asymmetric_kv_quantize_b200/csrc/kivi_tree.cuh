// kivi_tree.cuh -- the split of the work of attention of drafted tokens, and
// the merge of its partials; shared by its kernels.
//
// The query heads of one KV head and the N nodes are rows of one product
// (row = query head within the group * N + node), so the cache is read once
// for all of them.  RB rows make a row block.  A (sequence, KV head, row
// block) is a group; its tiles are those of the sequence's quantized tokens,
// then of its raw ones (the window and, straight behind it, the drafted
// tokens), TT tokens each.  All groups'
// tiles, end to end, are cut into equal ranges of W, one per CTA, whatever the
// lengths are, so a ragged batch keeps all CTAs busy.  A group that falls into
// one range is written out at once; of any other, each CTA leaves a partial
// (max, sum, accumulators of RB rows; the sums negative where raw values of the
// segment are infinite or NaN) in one of its two slots -- slot 1: the segment
// begins the group, slot 0: it does not -- and tree_merge_kernel joins them.
// Nothing is counted or kept between calls, so calls may be captured and replayed
// in any order on one workspace.
#pragma once

#include <atomic>

#include "kivi_draft.cuh"

namespace kivi {

struct TreePlan {
  int rb;      // rows of a block
  int tt;      // tokens of a tile
  int n_rb;    // row blocks of a KV head
  int ctas;    // CTAs of the split kernel
  int parts;   // tensor cores: groups of four warps in a block
};

__host__ __device__ inline long long tree_slots(const TreePlan& p) { return 2LL * p.ctas; }
// Floats of one partial: rb pairs (max, sum), then [rb][D] accumulators.
__host__ __device__ inline long long tree_part(const TreePlan& p, int D) {
  return (long long)p.rb * (D + 2);
}

struct TreeSeq {
  long long n_q;
  int r;
  bool ok;
  long long ut;  // tiles of each of its groups
};
__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& a, const TreePlan& p, long long b) {
  TreeSeq o;
  if (a.st != nullptr) {
    const SeqLen L = seq_len(a.st[b], false, a.c.Tq, a.c.R);
    o.n_q = L.n_q;
    o.r = L.r;
    o.ok = L.ok;
  } else {
    o.n_q = a.n_q;
    o.r = a.r;
    o.ok = true;
  }
  // a refused sequence keeps one tile, which writes its NaNs
  o.ut = o.ok ? (o.n_q + p.tt - 1) / p.tt + (o.r + a.N + p.tt - 1) / p.tt : 1;
  return o;
}

// Where tile x of all lies: sequence b, tile rem of its groups' tiles; and the
// tiles in all.  Called by one whole warp; x may lie past the end (b = B).
struct TreeAt {
  long long total;
  long long b;
  long long rem;
};
__device__ __forceinline__ TreeAt tree_find(const TreeArgs& a, const TreePlan& p, long long x) {
  const long long gpb = (long long)a.Hkv * p.n_rb;
  TreeAt o;
  if (a.st == nullptr) {
    const long long per = gpb * tree_seq(a, p, 0).ut;
    o.total = a.B * per;
    o.b = x / per;
    o.rem = x % per;
    return o;
  }
  const int lane = threadIdx.x & 31;
  long long sum = 0;
  o.b = a.B;
  o.rem = 0;
  for (long long b0 = 0; b0 < a.B; b0 += 32) {
    const long long b = b0 + lane;
    long long n = b < a.B ? gpb * tree_seq(a, p, b).ut : 0;
    long long incl = n;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long t = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += t;
    }
    const long long first = sum + incl - n;
    const unsigned here = __ballot_sync(0xffffffffu, x >= first && x < first + n);
    if (here) {
      const int l = __ffs(here) - 1;
      o.b = b0 + l;
      o.rem = x - __shfl_sync(0xffffffffu, first, l);
    }
    sum += __shfl_sync(0xffffffffu, incl, 31);
  }
  o.total = sum;
  return o;
}
// Tiles of a CTA's range: one at least (every group has a tile); longer ones leave SMs
// idle where a cache is short.
__device__ __forceinline__ long long tree_range(const TreePlan& p, long long total) {
  return (total + p.ctas - 1) / p.ctas;
}

// Lets `kernel` have `bytes` of dynamic shared memory on the current device; asked for
// once per device (`done`, one flag for each).
constexpr int kTreeDevices = 128;
template <typename K>
cudaError_t tree_smem(K kernel, int bytes, std::atomic<bool>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool known = dev >= 0 && dev < kTreeDevices;
  if (known && done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && known) done[dev].store(true, std::memory_order_relaxed);
  return e;
}

// The kernels: binary32 caches on CUDA cores, fp16 ones on the tensor cores
// (binary32 or binary16 scales and zeros).
cudaError_t tree_simt(const TreeArgs& a, const TreePlan& p, cudaStream_t s);
cudaError_t tree_tc_f32(const TreeArgs& a, const TreePlan& p, cudaStream_t s);
cudaError_t tree_tc_meta16(const TreeArgs& a, const TreePlan& p, cudaStream_t s);

}  // namespace kivi
