// kivi_draft.cuh -- launchers of the operators around drafted tokens
// (kivi_tree_*.cu, kivi_read.cu, kivi_rope.cu, the commit in
// kivi_quantize.cu), and the split of the tree attention's work.
#pragma once

#include "kivi_internal.cuh"

namespace kivi {

// ---- attention of drafted tokens over the cache --------------------------
struct TreeArgs {
  CacheView c;
  const void* q;         // [B][Hq][N][D]
  const void* k;         // [B][Hkv][N][D]
  const void* v;
  const uint32_t* mask;  // [B][N][ceil(N / 32)]
  void* out;             // [B][Hq][N][D]
  float* part;           // partials, tree_workspace_bytes()
  int B, Hkv, gq, D, bits, dtype, meta, N;
  long long n_q;         // host-counted caches (st null)
  int r;
  const DevState* st;    // ragged caches: one state per sequence
  float qscale;          // softmax_scale * log2(e)
  int sms;
};
size_t tree_workspace_bytes(int gq, int D, int dtype, int N, int sms);
cudaError_t launch_tree(const TreeArgs& a, cudaStream_t s);

// ---- read-back ------------------------------------------------------------
// K, V [units][T][D]: tokens t0 .. t0+T-1 of every unit; tokens behind a
// sequence's last one, and those of a page outside the pool, are not written.
cudaError_t launch_read(const CacheView& c, int units, int Hkv, int D, int bits, int dtype,
                        long long n_q, int r, const DevState* st, long long t0, long long T,
                        void* K, void* V, cudaStream_t s);

// ---- commit of an accepted path -------------------------------------------
cudaError_t launch_commit(const CacheView& c, int B, int Hkv, int D, int bits, int dtype,
                          const void* k, const void* v, const int* path, const int* count, int N,
                          int P, DevState* st, cudaStream_t s);

// ---- norms and rotary positions of a step's projections --------------------
constexpr int kRopeMaxAxes = 4;
struct RopeArgs {
  const void* qkv;          // [B][N] rows of (Hq + 2 Hkv) * D, `stride` elements apart
  long long stride;
  const long long* pos;     // [axes][B][N]
  const double* inv_freq;   // [rot / 2]
  const void* qw;           // [D] or null
  const void* kw;
  void* q;                  // [B][Hq][N][D]
  void* k;                  // [B][Hkv][N][D]
  void* v;
  int B, N, Hq, Hkv, D, rot, axes, interleaved, dtype;
  int section_end[kRopeMaxAxes];  // pair i turns by axis a: i < section_end[a]
  float eps;
};
// sms: of the device
cudaError_t launch_rope(const RopeArgs& a, int sms, cudaStream_t s);

}  // namespace kivi
