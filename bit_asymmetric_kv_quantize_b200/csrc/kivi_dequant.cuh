// kivi_dequant.cuh -- stored codes as numbers: c * s + z of a few adjacent
// channels of one token, shared by the read-back and by the attention of
// drafted tokens over the cache.
#pragma once

#include "kivi_internal.cuh"

namespace kivi {
namespace {

// The words that hold CH codes (CH in {4, 8}) of token t, channels ch0 ..
// ch0+CH-1 (ch0 a multiple of CH), in a key array [.][T][WK]: a token's codes
// are adjacent bits, CH * BITS of one word, or CH bits of each of three planes.
template <int D, int BITS, int CH>
__device__ __forceinline__ void key_words(const uint32_t* __restrict__ unit, long long t, int ch0,
                                          uint32_t (&w)[Layout<D, BITS>::WB]) {
  using Lt = Layout<D, BITS>;
  static_assert(CH <= Lt::E, "the codes of a call stand in one block");
  const uint32_t* row = unit + t * Lt::WK + ch0 / Lt::E * Lt::WB;
#pragma unroll
  for (int p = 0; p < Lt::WB; ++p) w[p] = row[p];
}
// Those codes.
template <int D, int BITS, int CH>
__device__ __forceinline__ void key_codes(const uint32_t (&w)[Layout<D, BITS>::WB], int ch0,
                                          int (&c)[CH]) {
  using Lt = Layout<D, BITS>;
  if constexpr (BITS == 3) {
    const int sh = ch0 % 32;
    const uint32_t a = w[0] >> sh, b = w[1] >> sh, e = w[2] >> sh;
#pragma unroll
    for (int i = 0; i < CH; ++i)
      c[i] = (int)(((a >> i) & 1u) | (((b >> i) & 1u) << 1) | (((e >> i) & 1u) << 2));
  } else {
    const uint32_t x = w[0] >> (ch0 % Lt::E * BITS);
#pragma unroll
    for (int i = 0; i < CH; ++i) c[i] = (int)((x >> (i * BITS)) & Lt::MASK);
  }
}

// The same of a value array [.][T/E * WB][D], whose words run along tokens: CH
// adjacent words of each plane (a 16-byte load for each four), which hold the codes of
// E tokens; then those of token t.
template <int D, int BITS, int CH>
__device__ __forceinline__ void value_words(const uint32_t* __restrict__ unit, long long t,
                                            int ch0, uint32_t (&w)[Layout<D, BITS>::WB][CH]) {
  using Lt = Layout<D, BITS>;
  const uint32_t* row = unit + t / Lt::E * Lt::WB * D + ch0;
#pragma unroll
  for (int p = 0; p < Lt::WB; ++p)
#pragma unroll
    for (int k = 0; k < CH; k += 4) {
      const uint4 a = *reinterpret_cast<const uint4*>(row + p * D + k);
      w[p][k] = a.x;
      w[p][k + 1] = a.y;
      w[p][k + 2] = a.z;
      w[p][k + 3] = a.w;
    }
}
template <int D, int BITS, int CH>
__device__ __forceinline__ void value_codes(const uint32_t (&w)[Layout<D, BITS>::WB][CH],
                                            long long t, int (&c)[CH]) {
  using Lt = Layout<D, BITS>;
  const int i0 = (int)(t % Lt::E);
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    if constexpr (BITS == 3)
      c[k] = (int)(((w[0][k] >> i0) & 1u) | (((w[1][k] >> i0) & 1u) << 1) |
                   (((w[2][k] >> i0) & 1u) << 2));
    else
      c[k] = (int)((w[0][k] >> (i0 * BITS)) & Lt::MASK);
  }
}

// CH adjacent scales or zeros widened to float; p aligned to CH elements of 2 bytes.
template <int CH, typename M>
__device__ __forceinline__ void load_meta_row(const M* p, float (&o)[CH]) {
#pragma unroll
  for (int k = 0; k < CH; k += 4) {
    float v[4];
    load_meta<4>(p + k, v);
    o[k] = v[0];
    o[k + 1] = v[1];
    o[k + 2] = v[2];
    o[k + 3] = v[3];
  }
}

// A stored number, c * s + z by one fused multiply-add: the product is not
// rounded, the sum once to 24 bits.  Kept entries (dense-and-sparse caches)
// replace it by their value: of key channels ch0.. of token t of store array
// unit su, and of value channels.
template <int D, int CH>
__device__ __forceinline__ void key_kept(const CacheView& c, long long su, long long t, int ch0,
                                         float (&o)[CH]) {
  if (c.k_out == 0) return;
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const long long lo = ((su * (store_tokens(c) / kG) + t / kG) * D + ch0 + i) * c.k_out;
    for (int m = 0; m < c.k_out; ++m)
      if (c.k_oi[lo + m] == (int)(t % kG)) o[i] = c.k_ov[lo + m];
  }
}
template <int D, int CH>
__device__ __forceinline__ void value_kept(const CacheView& c, long long su, long long t, int ch0,
                                           float (&o)[CH]) {
  if (c.v_out == 0) return;
  const long long lo = ((su * store_tokens(c) + t) * (D / kGv) + ch0 / kGv) * c.v_out;
  for (int m = 0; m < c.v_out; ++m) {
    const int e = c.v_oi[lo + m] - ch0 % kGv;
    const float x = c.v_ov[lo + m];
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (e == i) o[i] = x;
  }
}
// Scales and zeros of key channels ch0.. in the group of token t.
template <int D, int BITS, typename M, int CH>
__device__ __forceinline__ void key_meta(const CacheView& c, long long su, long long t, int ch0,
                                         float (&s)[CH], float (&z)[CH]) {
  using Lt = Layout<D, BITS>;
  const long long o = su * Lt::k_meta_unit(store_tokens(c)) + t / kG * D + ch0;
  load_meta_row<CH, M>(static_cast<const M*>(c.k_scale) + o, s);
  load_meta_row<CH, M>(static_cast<const M*>(c.k_zero) + o, z);
}

}  // namespace
}  // namespace kivi
