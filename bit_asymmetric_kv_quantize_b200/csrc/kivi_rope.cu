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
constexpr int kRopeRows = 4;  // rows of a thread under way at a time

// Block: tokens blockIdx.x * TB .., head rows blockIdx.y, + gridDim.y, .. of them in
// rounds.  The table of the tokens' cosines and sines is made once and used by all
// heads.  D / CH lanes hold a row, 16 bytes each; four rows' loads are issued
// before any is worked on.
template <int D, typename T>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeArgs a, int TB) {
  constexpr int CH = 16 / (int)sizeof(T);
  constexpr int LPR = D / CH;                // lanes of a row
  constexpr int RPB = kRopeThreads / LPR;    // rows of a round
  extern __shared__ float2 cs[];             // [TB][rot / 2]
  const int tokens = a.B * a.N;
  const int tok0 = blockIdx.x * TB;
  const int half = a.rot / 2;
  const int H = a.Hq + 2 * a.Hkv;
  const int lane = threadIdx.x % LPR, ch0 = lane * CH;
  const int rows = min(TB, tokens - tok0) * H;
  const T* in = static_cast<const T*>(a.qkv);
  // this thread's rows: i, i + step, ..; as token tl and head h
  const int step = RPB * gridDim.y;
  const int i0 = blockIdx.y * RPB + threadIdx.x / LPR;
  int tl = i0 / H, h = i0 % H;
  auto next = [&](int& t, int& x) {
    x += step;
    while (x >= H) {
      x -= H;
      ++t;
    }
  };
  uint4 raw[kRopeRows];
  auto load = [&](int i, int t, int x) {
    int ti = i;
#pragma unroll
    for (int r = 0; r < kRopeRows; ++r) {
      raw[r] = make_uint4(0, 0, 0, 0);
      if (ti < rows)
        raw[r] = *reinterpret_cast<const uint4*>(in + (long long)(tok0 + t) * a.stride + x * D + ch0);
      ti += step;
      next(t, x);
    }
  };
  load(i0, tl, h);
  for (int i = threadIdx.x; i < TB * half; i += kRopeThreads) {
    const int p = i % half, tok = tok0 + i / half;
    if (tok >= tokens) break;
    // (ends behind the last section are rot / 2, beyond every pair)
    const int ax = (p >= a.section_end[0]) + (p >= a.section_end[1]) + (p >= a.section_end[2]);
    constexpr double kTurn = 0.15915494309189533577;  // 1 / (2 pi)
    const double turns = (double)a.pos[(long long)ax * tokens + tok] * a.inv_freq[p] * kTurn;
    float sn, cn;
    sincospif((float)(2.0 * (turns - rint(turns))), &sn, &cn);
    cs[i] = make_float2(cn, sn);
  }
  float wq[CH], wk[CH];
#pragma unroll
  for (int e = 0; e < CH; ++e) {
    wq[e] = a.qw ? to_f32(static_cast<const T*>(a.qw)[ch0 + e]) : 1.0f;
    wk[e] = a.kw ? to_f32(static_cast<const T*>(a.kw)[ch0 + e]) : 1.0f;
  }
  const bool lo = ch0 < half, in_rot = ch0 < a.rot;
  // pair (p, p + half): half is a multiple of CH, so the partner channels are those
  // of one other lane
  const int other = a.interleaved || !in_rot ? lane : (lo ? lane + half / CH : lane - half / CH);
  const int t0 = a.interleaved ? ch0 / 2 : (lo ? ch0 : ch0 - half);  // in the table
  const int tok_b = tok0 / a.N, tok_n = tok0 % a.N;
  __syncthreads();

  // every thread of a warp runs the same number of rounds (shuffles inside)
  for (int base = blockIdx.y * RPB; base < rows; base += kRopeRows * step) {
    int ti = base + threadIdx.x / LPR;
#pragma unroll
    for (int r = 0; r < kRopeRows; ++r) {
      const bool live = ti < rows;
      float x[CH];
#pragma unroll
      for (int e = 0; e < CH; ++e) x[e] = to_f32(reinterpret_cast<const T*>(&raw[r])[e]);
      const bool isq = h < a.Hq, isk = !isq && h < a.Hq + a.Hkv;
      if (a.qw || a.kw) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < CH; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if ((isq && a.qw) || (isk && a.kw)) {
          const float rs = rsqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
          for (int e = 0; e < CH; ++e) x[e] = x[e] * rs * (isq ? wq[e] : wk[e]);
        }
      }
      const float2* t = cs + (live ? tl : 0) * half + t0;
      float y[CH];
      if (a.interleaved) {
#pragma unroll
        for (int e = 0; e < CH; e += 2) {
          const float2 f = in_rot ? t[e / 2] : make_float2(1.f, 0.f);
          y[e] = x[e] * f.x - x[e + 1] * f.y;
          y[e + 1] = x[e + 1] * f.x + x[e] * f.y;
        }
      } else {
#pragma unroll
        for (int e = 0; e < CH; ++e) {
          const float o = __shfl_sync(0xffffffffu, x[e], other, LPR);
          const float2 f = in_rot ? t[e] : make_float2(1.f, 0.f);
          y[e] = fmaf(lo ? -o : o, f.y, x[e] * f.x);
        }
      }
      if (live) {
        uint4 res = raw[r];  // values are laid out as they are
        if (isq || isk) {
          T o[CH];
#pragma unroll
          for (int e = 0; e < CH; ++e) o[e] = from_f32<T>(in_rot ? y[e] : x[e]);
          res = *reinterpret_cast<const uint4*>(o);
        }
        int b = tok_b, n = tok_n + tl;
        while (n >= a.N) {
          n -= a.N;
          ++b;
        }
        T* dst = isq ? static_cast<T*>(a.q) + (((long long)b * a.Hq + h) * a.N + n) * D
                     : (isk ? static_cast<T*>(a.k) + (((long long)b * a.Hkv + h - a.Hq) * a.N + n) * D
                            : static_cast<T*>(a.v) + (((long long)b * a.Hkv + h - a.Hq - a.Hkv) * a.N + n) * D);
        *reinterpret_cast<uint4*>(dst + ch0) = res;
      }
      ti += step;
      next(tl, h);
    }
    if (base + kRopeRows * step < rows) load(ti, tl, h);
  }
}

template <int D, typename T>
cudaError_t rope_t(const RopeArgs& a, cudaStream_t s) {
  const int tokens = a.B * a.N;
  constexpr int RPB = kRopeThreads * 16 / (int)sizeof(T) / D;
  // enough tokens: four a block; few: one, its heads spread over blocks that take one
  // round each (each makes the token's table again)
  const int TB = tokens >= 2048 ? 4 : 1;
  const int H = a.Hq + 2 * a.Hkv, spread = (H + RPB - 1) / RPB;
  const dim3 grid((unsigned)((tokens + TB - 1) / TB), TB == 4 ? 1 : (unsigned)min(spread, 65535));
  rope_kernel<D, T><<<grid, kRopeThreads, TB * (a.rot / 2) * sizeof(float2), s>>>(a, TB);
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
