// kivi_rope.cu -- a step's projections made ready for the cache: each head of
// queries and keys normed and turned by its token's positions, and all heads
// laid out as the cache and its attention take them ([B][H][N][D]), in one
// pass over [B][N][(Hq + 2 Hkv) D].
//
// For a head x of D channels, in binary32 and rounded once at the end:
//   y = x * rsqrt(mean(x^2) + eps) * w          (no weight: y = x)
//   pair i < rot/2, angle a = pos[axis(i)] * f_i:
//     (y1, y2) -> (y1 cos a - y2 sin a, y2 cos a + y1 sin a)
// Channels from rot on are not turned; values are only laid out.  The angle is
// formed in binary64 and reduced to a fraction of a turn there, since at a
// position of 10^6 a binary32 product would be off by 0.06 radians.
// (KIVI quantizes keys after their rotation: mlsanity.com abstract, keys as
// the attention reads them.)
#include "kivi_draft.cuh"

namespace kivi {
namespace {

constexpr int kRopeThreads = 256;

// Block: tokens blockIdx.x * TB ..; the table of its cosines and sines is made
// once and used by all heads.  D / CH lanes hold a row, 16 bytes each.
template <int D, typename T>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeArgs a, int TB) {
  constexpr int CH = 16 / (int)sizeof(T);
  constexpr int LPR = D / CH;  // lanes of a row
  extern __shared__ float2 cs[];  // [TB][rot / 2]
  const long long tokens = (long long)a.B * a.N;
  const long long tok0 = (long long)blockIdx.x * TB;
  const int half = a.rot / 2;
  for (int i = threadIdx.x; i < TB * half; i += kRopeThreads) {
    const int p = i % half;
    const long long tok = tok0 + i / half;
    if (tok >= tokens) break;
    int ax = 0;
    while (ax + 1 < a.axes && p >= a.section_end[ax]) ++ax;
    constexpr double kTurn = 0.15915494309189533577;  // 1 / (2 pi)
    const double turns = (double)a.pos[ax * tokens + tok] * a.inv_freq[p] * kTurn;
    float sn, cn;
    sincospif((float)(2.0 * (turns - rint(turns))), &sn, &cn);
    cs[i] = make_float2(cn, sn);
  }
  __syncthreads();
  const int H = a.Hq + 2 * a.Hkv;
  const int lane = threadIdx.x % LPR, ch0 = lane * CH;
  const T* in = static_cast<const T*>(a.qkv);
  float wq[CH], wk[CH];
#pragma unroll
  for (int e = 0; e < CH; ++e) {
    wq[e] = a.qw ? to_f32(static_cast<const T*>(a.qw)[ch0 + e]) : 1.0f;
    wk[e] = a.kw ? to_f32(static_cast<const T*>(a.kw)[ch0 + e]) : 1.0f;
  }
  // every thread of a warp runs the same number of rounds (shuffles inside)
  const int rows = TB * H;
  constexpr int RPB = kRopeThreads / LPR;
  for (int i0 = 0; i0 < rows; i0 += RPB) {
    const int i = i0 + threadIdx.x / LPR;
    const int tl = i / H, h = i % H;
    const long long tok = tok0 + tl;
    const bool live = i < rows && tok < tokens;
    uint4 raw = make_uint4(0, 0, 0, 0);
    if (live) raw = *reinterpret_cast<const uint4*>(in + tok * a.stride + (long long)h * D + ch0);
    const long long b = tok / a.N, n = tok % a.N;
    float x[CH];
#pragma unroll
    for (int e = 0; e < CH; ++e) x[e] = to_f32(reinterpret_cast<const T*>(&raw)[e]);
    const bool isq = h < a.Hq, isk = !isq && h < a.Hq + a.Hkv;
    if (a.qw || a.kw) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < CH; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if ((isq && a.qw) || (isk && a.kw)) {
        const float rs = rsqrtf(ss / (float)D + a.eps);
#pragma unroll
        for (int e = 0; e < CH; ++e) x[e] = x[e] * rs * (isq ? wq[e] : wk[e]);
      }
    }
    const float2* t = cs + tl * half;
    float y[CH];
    if (a.interleaved) {
#pragma unroll
      for (int e = 0; e < CH; e += 2) {
        const int p = (ch0 + e) / 2;
        const float2 f = (live && ch0 < a.rot) ? t[p] : make_float2(1.f, 0.f);
        y[e] = x[e] * f.x - x[e + 1] * f.y;
        y[e + 1] = x[e + 1] * f.x + x[e] * f.y;
      }
      if (ch0 >= a.rot) {  // not turned (a zero times an infinity would spoil it)
#pragma unroll
        for (int e = 0; e < CH; ++e) y[e] = x[e];
      }
    } else {
      // pair (p, p + half): half is a multiple of CH, so the partner channels
      // are those of one other lane
      const bool lo = ch0 < half, in_rot = ch0 < a.rot;
      const int other = !in_rot ? lane : (lo ? lane + half / CH : lane - half / CH);
#pragma unroll
      for (int e = 0; e < CH; ++e) {
        const float o = __shfl_sync(0xffffffffu, x[e], other, LPR);
        const float2 f = (live && in_rot) ? t[(lo ? ch0 : ch0 - half) + e] : make_float2(1.f, 0.f);
        y[e] = lo ? x[e] * f.x - o * f.y : x[e] * f.x + o * f.y;
        if (!in_rot) y[e] = x[e];
      }
    }
    if (!live) continue;
    T* dst;
    if (isq)
      dst = static_cast<T*>(a.q) + ((b * a.Hq + h) * a.N + n) * D;
    else if (isk)
      dst = static_cast<T*>(a.k) + ((b * a.Hkv + (h - a.Hq)) * a.N + n) * D;
    else
      dst = static_cast<T*>(a.v) + ((b * a.Hkv + (h - a.Hq - a.Hkv)) * a.N + n) * D;
    if (isq || isk) {
      T o[CH];
#pragma unroll
      for (int e = 0; e < CH; ++e) o[e] = from_f32<T>(y[e]);
      raw = *reinterpret_cast<const uint4*>(o);
    }
    *reinterpret_cast<uint4*>(dst + ch0) = raw;
  }
}

template <int D, typename T>
cudaError_t rope_t(const RopeArgs& a, cudaStream_t s) {
  const long long tokens = (long long)a.B * a.N;
  const int TB = 2;
  const long long blocks = (tokens + TB - 1) / TB;
  rope_kernel<D, T><<<(unsigned)blocks, kRopeThreads, TB * (a.rot / 2) * sizeof(float2), s>>>(a, TB);
  return cudaGetLastError();
}

template <typename T>
cudaError_t rope_d(const RopeArgs& a, cudaStream_t s) {
  switch (a.D) {
    case 32: return rope_t<32, T>(a, s);
    case 64: return rope_t<64, T>(a, s);
    case 128: return rope_t<128, T>(a, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, cudaStream_t s) {
  return a.dtype == 1 ? rope_d<float>(a, s) : rope_d<__half>(a, s);
}

}  // namespace kivi
