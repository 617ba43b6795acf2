// kivi_dequant.cuh -- stored codes as numbers: c * s + z of a few adjacent
// channels of one token, shared by the read-back and by the attention of
// drafted tokens over the cache.
#pragma once

#include "kivi_internal.cuh"

namespace kivi {
namespace {

// CH codes (CH in {4, 8}) of token t, channels ch0 .. ch0+CH-1 (ch0 a multiple
// of CH) of a key array [.][T][WK]: a token's codes are adjacent bits, CH * BITS
// of one word, or CH bits of each of three planes.
template <int D, int BITS, int CH>
__device__ __forceinline__ void key_codes(const uint32_t* __restrict__ unit, long long t, int ch0,
                                          int (&c)[CH]) {
  using Lt = Layout<D, BITS>;
  const uint32_t* row = unit + t * Lt::WK;
  if constexpr (BITS == 3) {
    const uint32_t* p = row + ch0 / 32 * 3;
    const int sh = ch0 % 32;
    const uint32_t a = p[0] >> sh, b = p[1] >> sh, e = p[2] >> sh;
#pragma unroll
    for (int i = 0; i < CH; ++i)
      c[i] = (int)(((a >> i) & 1u) | (((b >> i) & 1u) << 1) | (((e >> i) & 1u) << 2));
  } else {
    static_assert(CH <= Lt::E, "the codes of a call stand in one word");
    const uint32_t w = row[ch0 / Lt::E] >> (ch0 % Lt::E * BITS);
#pragma unroll
    for (int i = 0; i < CH; ++i) c[i] = (int)((w >> (i * BITS)) & Lt::MASK);
  }
}

// The same of a value array [.][T/E * WB][D], whose words run along tokens:
// CH adjacent words (a 16-byte load for each four), one code of each.
template <int D, int BITS, int CH>
__device__ __forceinline__ void value_codes(const uint32_t* __restrict__ unit, long long t,
                                            int ch0, int (&c)[CH]) {
  using Lt = Layout<D, BITS>;
  const uint32_t* row = unit + t / Lt::E * Lt::WB * D + ch0;
  const int i0 = (int)(t % Lt::E);
#pragma unroll
  for (int k = 0; k < CH; k += 4) {
    if constexpr (BITS == 3) {
      const uint4 a = *reinterpret_cast<const uint4*>(row + k);
      const uint4 b = *reinterpret_cast<const uint4*>(row + D + k);
      const uint4 e = *reinterpret_cast<const uint4*>(row + 2 * D + k);
      auto code = [&](uint32_t x, uint32_t y, uint32_t z) {
        return (int)(((x >> i0) & 1u) | (((y >> i0) & 1u) << 1) | (((z >> i0) & 1u) << 2));
      };
      c[k] = code(a.x, b.x, e.x);
      c[k + 1] = code(a.y, b.y, e.y);
      c[k + 2] = code(a.z, b.z, e.z);
      c[k + 3] = code(a.w, b.w, e.w);
    } else {
      const uint4 a = *reinterpret_cast<const uint4*>(row + k);
      const int sh = i0 * BITS;
      c[k] = (int)((a.x >> sh) & Lt::MASK);
      c[k + 1] = (int)((a.y >> sh) & Lt::MASK);
      c[k + 2] = (int)((a.z >> sh) & Lt::MASK);
      c[k + 3] = (int)((a.w >> sh) & Lt::MASK);
    }
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

// Key channels ch0.. of token t of store array unit su as numbers.  c * s + z
// is one fused multiply-add: the product is not rounded, the sum once to 24
// bits.  Kept entries (dense-and-sparse caches) replace it by their value.
template <int D, int BITS, typename M, int CH>
__device__ __forceinline__ void key_values(const CacheView& c, long long su, long long t, int ch0,
                                           const float (&s)[CH], const float (&z)[CH],
                                           float (&o)[CH]) {
  using Lt = Layout<D, BITS>;
  const long long Ts = store_tokens(c);
  int code[CH];
  key_codes<D, BITS, CH>(c.k_codes + su * Lt::k_codes_unit(Ts), t, ch0, code);
#pragma unroll
  for (int i = 0; i < CH; ++i) o[i] = fmaf((float)code[i], s[i], z[i]);
  if (c.k_out > 0) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const long long lo = ((su * (Ts / kG) + t / kG) * D + ch0 + i) * c.k_out;
      for (int m = 0; m < c.k_out; ++m)
        if (c.k_oi[lo + m] == (int)(t % kG)) o[i] = c.k_ov[lo + m];
    }
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

// Value channels ch0.. of token t of store array unit su as numbers.
template <int D, int BITS, typename M, int CH>
__device__ __forceinline__ void value_values(const CacheView& c, long long su, long long t,
                                             int ch0, float (&o)[CH]) {
  using Lt = Layout<D, BITS>;
  const long long Ts = store_tokens(c);
  int code[CH];
  value_codes<D, BITS, CH>(c.v_codes + su * Lt::v_codes_unit(Ts), t, ch0, code);
  const int j = ch0 / kGv;
  const long long mo = su * Lt::v_meta_unit(Ts) + t * Lt::NJ + j;
  const float s = to_f32(static_cast<const M*>(c.v_scale)[mo]);
  const float z = to_f32(static_cast<const M*>(c.v_zero)[mo]);
#pragma unroll
  for (int i = 0; i < CH; ++i) o[i] = fmaf((float)code[i], s, z);
  if (c.v_out > 0) {
    const long long lo = mo * c.v_out;
    for (int m = 0; m < c.v_out; ++m) {
      const int e = c.v_oi[lo + m] - ch0 % kGv;
      const float x = c.v_ov[lo + m];
#pragma unroll
      for (int i = 0; i < CH; ++i)
        if (e == i) o[i] = x;
    }
  }
}

}  // namespace
}  // namespace kivi
