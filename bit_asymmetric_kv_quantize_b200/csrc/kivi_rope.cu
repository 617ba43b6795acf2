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

// Four adjacent elements, loaded and stored as one piece.
template <typename T>
struct Four;
template <>
struct Four<__half> {
  uint2 v;
  __device__ __forceinline__ void widen(float* x) const {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&v.x));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&v.y));
    x[0] = a.x;
    x[1] = a.y;
    x[2] = b.x;
    x[3] = b.y;
  }
  __device__ __forceinline__ void round(const float* x) {
    const __half2 a = __floats2half2_rn(x[0], x[1]), b = __floats2half2_rn(x[2], x[3]);
    v.x = *reinterpret_cast<const uint32_t*>(&a);
    v.y = *reinterpret_cast<const uint32_t*>(&b);
  }
};
template <>
struct Four<float> {
  float4 v;
  __device__ __forceinline__ void widen(float* x) const {
    x[0] = v.x;
    x[1] = v.y;
    x[2] = v.z;
    x[3] = v.w;
  }
  __device__ __forceinline__ void round(const float* x) {
    v = make_float4(x[0], x[1], x[2], x[3]);
  }
};

// The rows of one kind (queries, keys or values): nh heads of each of the block's
// tokens, D / 8 lanes a row.  A lane holds two pieces of four channels at ca and cb: both
// halves of its four pairs, so that no value has to cross lanes for the turn.  Four
// rows' loads are issued before any is worked on.  w: the norm's weight, or null.
template <int D, typename T, bool INTER, bool TURN>
__device__ __forceinline__ void rope_rows(const RopeArgs& a, const T* in, T* out,
                                          const T* __restrict__ w, int nh, int tok0, int ntok,
                                          int ca, int cb, bool turns, const float4* cs) {
  constexpr int LPR = D / 8, RPB = kRopeThreads / LPR;
  const int rows = ntok * nh, step = RPB * gridDim.y, half = a.rot / 2;
  float wa[4], wb[4];
  if (TURN && w != nullptr) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      wa[e] = to_f32(w[ca + e]);
      wb[e] = to_f32(w[cb + e]);
    }
  }
  // a row as token tl of the block and head h
  int i = blockIdx.y * RPB + threadIdx.x / LPR;
  int tl = i / nh, h = i % nh;
  const int dt = step / nh, dh = step % nh;
  // every thread of a warp runs the same number of rounds (shuffles inside)
  for (int base = blockIdx.y * RPB; base < rows; base += kRopeRows * step) {
    Four<T> xa[kRopeRows], xb[kRopeRows];
    int rt[kRopeRows], rh[kRopeRows];
#pragma unroll
    for (int r = 0; r < kRopeRows; ++r) {
      rt[r] = i < rows ? tl : -1;
      rh[r] = h;
      if (i < rows) {
        const T* src = in + (long long)(tok0 + tl) * a.stride + h * D;
        xa[r] = *reinterpret_cast<const Four<T>*>(src + ca);
        xb[r] = *reinterpret_cast<const Four<T>*>(src + cb);
      } else {
        xa[r].v = xb[r].v = {};
      }
      i += step;
      h += dh;
      tl += dt + (h >= nh);
      if (h >= nh) h -= nh;
    }
#pragma unroll
    for (int r = 0; r < kRopeRows; ++r) {
      const int t = max(rt[r], 0);
      if (TURN) {  // values are laid out as they are
        float x[4], y[4];
        xa[r].widen(x);
        xb[r].widen(y);
        if (w != nullptr) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) ss = fmaf(y[e], y[e], fmaf(x[e], x[e], ss));
#pragma unroll
          for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float rs = rsqrtf(ss * (1.0f / D) + a.eps);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            x[e] = x[e] * rs * wa[e];
            y[e] = y[e] * rs * wb[e];
          }
        }
        if (turns) {
          const float4* f = cs + t * (half / 2);
          const float4 f0 = f[0], f1 = f[1];
          const float c[4] = {f0.x, f0.z, f1.x, f1.z}, sn[4] = {f0.y, f0.w, f1.y, f1.w};
          if (INTER) {  // pairs (0, 1), (2, 3) of each piece
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float* p = e < 2 ? x + 2 * e : y + 2 * (e - 2);
              const float u = p[0], v = p[1];
              p[0] = fmaf(-v, sn[e], u * c[e]);
              p[1] = fmaf(u, sn[e], v * c[e]);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float u = x[e], v = y[e];
              x[e] = fmaf(-v, sn[e], u * c[e]);
              y[e] = fmaf(u, sn[e], v * c[e]);
            }
          }
        }
        xa[r].round(x);
        xb[r].round(y);
      }
      if (rt[r] >= 0) {
        const int tok = tok0 + t, b = tok / a.N, n = tok - b * a.N;
        T* dst = out + (((long long)b * nh + rh[r]) * a.N + n) * D;
        *reinterpret_cast<Four<T>*>(dst + ca) = xa[r];
        *reinterpret_cast<Four<T>*>(dst + cb) = xb[r];
      }
    }
  }
}

// Block: tokens blockIdx.x * TB ..; gridDim.y blocks share their rows.  The table of
// the tokens' cosines and sines is made once and used by all heads.
// Bound by issue (64 % of the slots) and DRAM together: 4 x 8191 tokens of 48 heads
// (32 + 2 x 8, D 128, binary16, three axes) take 183 us, 4.4 TB/s of a copy's 6.5.  Both
// halves of a pair in one lane took it from 288 us (a shuffle for each value), four
// rows' loads in flight from 345.  A decode step's 16 tokens take 5 us, which is a
// launch, the binary64 angles and one round of loads.
template <int D, typename T, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(RopeArgs a, int TB) {
  extern __shared__ float4 cs[];  // [TB][rot / 2] (cosine, sine)
  const int tokens = a.B * a.N, tok0 = blockIdx.x * TB, ntok = min(TB, tokens - tok0);
  const int half = a.rot / 2;
  for (int i = threadIdx.x; i < ntok * half; i += kRopeThreads) {
    const int p = i % half, tok = tok0 + i / half;
    // (ends behind the last section are rot / 2, beyond every pair)
    const int ax = (p >= a.section_end[0]) + (p >= a.section_end[1]) + (p >= a.section_end[2]);
    constexpr double kTurn = 0.15915494309189533577;  // 1 / (2 pi)
    const double turns = (double)a.pos[(long long)ax * tokens + tok] * a.inv_freq[p] * kTurn;
    float sn, cn;
    sincospif((float)(2.0 * (turns - rint(turns))), &sn, &cn);
    reinterpret_cast<float2*>(cs)[i] = make_float2(cn, sn);
  }
  __syncthreads();
  // rot is a multiple of 16: a lane's channels turn all or not at all
  const int lane = threadIdx.x % (D / 8);
  const bool turns = lane < a.rot / 8;
  const bool split = turns && !INTER;
  const int ca = split ? 4 * lane : 8 * lane, cb = split ? half + 4 * lane : 8 * lane + 4;
  const float4* f = cs + 2 * lane;  // pairs 4 lane .. 4 lane + 3
  const T* in = static_cast<const T*>(a.qkv);
  rope_rows<D, T, INTER, true>(a, in, static_cast<T*>(a.q), static_cast<const T*>(a.qw), a.Hq, tok0,
                               ntok, ca, cb, turns, f);
  rope_rows<D, T, INTER, true>(a, in + a.Hq * D, static_cast<T*>(a.k), static_cast<const T*>(a.kw),
                               a.Hkv, tok0, ntok, ca, cb, turns, f);
  rope_rows<D, T, INTER, false>(a, in + (a.Hq + a.Hkv) * D, static_cast<T*>(a.v), (const T*)nullptr,
                                a.Hkv, tok0, ntok, 8 * lane, 8 * lane + 4, false, f);
}

template <int D, typename T>
cudaError_t rope_t(const RopeArgs& a, int sms, cudaStream_t s) {
  const int tokens = a.B * a.N;
  constexpr int RPB = kRopeThreads * 8 / D;
  // As many tokens a block (of 8, 4, 2) as leave every SM a block, since a block's table
  // and its rounds of rows (RPB * kRopeRows at a time) serve all of them; else one token,
  // its heads spread over blocks that take one round each (each makes the table again).  With
  // 1 / 2 / 4 / 8 tokens a block (148 SMs, warm, us): 3102 tokens of 20 heads (binary32,
  // D 64) 37 / 21 / 13 / 8.5; 8191 of 48 heads (binary16, D 128) 174 / 74 / 58 / 53; 420 of
  // those 10.2 / 6.8 / 7.8 / 12.0; 16 of them 4.8 / 5.3 / 7.5 / 11.7.  At a step itself wide
  // rows would do a little better with the number before (592 tokens of 48 heads: 6.9 with
  // two, 7.9 with four), narrow ones with the one after.
  const int TB = tokens >= 8 * sms ? 8 : tokens >= 4 * sms ? 4 : tokens >= 2 * sms ? 2 : 1;
  const int spread = (a.Hq + RPB - 1) / RPB;
  const dim3 grid((unsigned)((tokens + TB - 1) / TB), TB > 1 ? 1 : (unsigned)min(spread, 65535));
  const size_t bytes = TB * (a.rot / 2) * sizeof(float2);
  if (a.interleaved)
    rope_kernel<D, T, true><<<grid, kRopeThreads, bytes, s>>>(a, TB);
  else
    rope_kernel<D, T, false><<<grid, kRopeThreads, bytes, s>>>(a, TB);
  return cudaGetLastError();
}

template <typename T>
cudaError_t rope_d(const RopeArgs& a, int sms, cudaStream_t s) {
  switch (a.D) {
    case 32: return rope_t<32, T>(a, sms, s);
    case 64: return rope_t<64, T>(a, sms, s);
    case 128: return rope_t<128, T>(a, sms, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int sms, cudaStream_t s) {
  return a.dtype == 1 ? rope_d<float>(a, sms, s) : rope_d<__half>(a, sms, s);
}

}  // namespace kivi
