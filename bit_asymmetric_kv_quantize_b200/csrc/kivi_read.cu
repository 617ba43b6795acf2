// kivi_read.cu -- read-back: tokens t0 .. t0+T-1 of every unit of a cache as
// numbers, [unit][T][D].  A quantized token is c * s + z (one fused
// multiply-add in binary32, rounded once more to the output type), a window
// token its stored value.
//
// Method: "KIVI: A Tuning-Free Asymmetric 2bit Quantization for KV Cache",
// study.space summary: a grouped part and a full-precision residual part, one
// after the other along the token axis.
#include "kivi_dequant.cuh"
#include "kivi_draft.cuh"

namespace kivi {
namespace {

template <typename T, int CH>
__device__ __forceinline__ void store_row(T* p, const float (&x)[CH], bool wide) {
  if (wide) {
    T y[CH];
#pragma unroll
    for (int i = 0; i < CH; ++i) y[i] = from_f32<T>(x[i]);
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(y);
  } else {
#pragma unroll
    for (int i = 0; i < CH; ++i) p[i] = from_f32<T>(x[i]);
  }
}

// A block takes one 32-token tile of one unit (tiles count from the start of
// the sequence; n_q is a multiple of 32, so a tile lies in the store or in the
// window as a whole).  A thread takes CH adjacent channels (16 bytes of the
// output) of four adjacent tokens: the key group's scales and zeros and the
// value words (which run along tokens) are loaded once for the four.
// Bound by the stores' traffic to DRAM, next to the unpacking's integer work (64 % of
// its pipe): 8 x 32 heads of 4096 tokens at 2 bits take 93 us, 5.0 TB/s of codes read
// and numbers written (a copy reaches 6.5), 117 us when each row's loads waited for the
// stores before them; the last 401 of 5001 tokens of 2 sequences x 8 heads 3 us.
template <int D, int BITS, typename T, typename M>
__global__ void __launch_bounds__(D / (16 / (int)sizeof(T)) * 8)
    read_kernel(CacheView c, int Hkv, long long n_q, int r, const DevState* st, long long t0,
                long long T_len, T* __restrict__ K, T* __restrict__ V, int wide) {
  constexpr int CH = 16 / (int)sizeof(T);
  constexpr int COLS = D / CH;
  const long long unit = blockIdx.y;
  if (st != nullptr) {
    const SeqLen L = seq_len(st[unit / Hkv], false, c.Tq, c.R);
    if (!L.ok) return;
    n_q = L.n_q;
    r = L.r;
  }
  const long long tile = t0 / kTile + blockIdx.x;
  const long long base = tile * kTile;  // the tile's first token
  const int col = threadIdx.x % COLS, ch0 = col * CH;
  const int q0 = threadIdx.x / COLS * 4;  // first of the thread's four tokens
  const long long end = t0 + T_len < n_q + r ? t0 + T_len : n_q + r;
  if (base + q0 >= end || base + q0 + 4 <= t0) return;
  T* Ko = K + (unit * T_len - t0) * D + ch0;
  T* Vo = V + (unit * T_len - t0) * D + ch0;
  if (base < n_q) {
    long long su, stl;
    if (!store_tile(c, unit, tile, &su, &stl)) return;
    using Lt = Layout<D, BITS>;
    const long long row = stl * kTile + q0, Ts = store_tokens(c);
    // all loads before the first store, which the compiler would not move them across
    const uint32_t* ku = c.k_codes + su * Lt::k_codes_unit(Ts);
    const long long mo = su * Lt::v_meta_unit(Ts) + row * Lt::NJ + ch0 / kGv;
    float s[CH], z[CH], vs[4], vz[4];
    uint32_t kw[4][Lt::WB], vw[Lt::WB][CH];
    key_meta<D, BITS, M, CH>(c, su, row, ch0, s, z);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      key_words<D, BITS, CH>(ku, row + i, ch0, kw[i]);
      vs[i] = to_f32(static_cast<const M*>(c.v_scale)[mo + i * Lt::NJ]);
      vz[i] = to_f32(static_cast<const M*>(c.v_zero)[mo + i * Lt::NJ]);
    }
    value_words<D, BITS, CH>(c.v_codes + su * Lt::v_codes_unit(Ts), row, ch0, vw);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long t = base + q0 + i;
      if (t < t0 || t >= end) continue;
      int code[CH];
      float x[CH];
      key_codes<D, BITS, CH>(kw[i], ch0, code);
#pragma unroll
      for (int e = 0; e < CH; ++e) x[e] = fmaf((float)code[e], s[e], z[e]);
      key_kept<D, CH>(c, su, row + i, ch0, x);
      store_row<T, CH>(Ko + t * D, x, wide);
      value_codes<D, BITS, CH>(vw, row + i, code);
#pragma unroll
      for (int e = 0; e < CH; ++e) x[e] = fmaf((float)code[e], vs[i], vz[i]);
      value_kept<D, CH>(c, su, row + i, ch0, x);
      store_row<T, CH>(Vo + t * D, x, wide);
    }
  } else {
    const T* kr = static_cast<const T*>(c.k_res) + unit * c.R * D + ch0;
    const T* vr = static_cast<const T*>(c.v_res) + unit * c.R * D + ch0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const long long t = base + q0 + i;
      if (t >= t0 && t < end) {
        const uint4 a = *reinterpret_cast<const uint4*>(kr + (t - n_q) * D);
        const uint4 b = *reinterpret_cast<const uint4*>(vr + (t - n_q) * D);
        if (wide) {
          *reinterpret_cast<uint4*>(Ko + t * D) = a;
          *reinterpret_cast<uint4*>(Vo + t * D) = b;
        } else {
          const T* pa = reinterpret_cast<const T*>(&a);
          const T* pb = reinterpret_cast<const T*>(&b);
#pragma unroll
          for (int e = 0; e < CH; ++e) {
            Ko[t * D + e] = pa[e];
            Vo[t * D + e] = pb[e];
          }
        }
      }
    }
  }
}

template <int D, int BITS, typename T, typename M>
cudaError_t read_t(const CacheView& c, int units, int Hkv, long long n_q, int r,
                   const DevState* st, long long t0, long long T_len, void* K, void* V,
                   cudaStream_t s) {
  const long long tiles = (t0 + T_len - 1) / kTile - t0 / kTile + 1;
  const dim3 grid((unsigned)tiles, (unsigned)units);
  const int wide = (((uintptr_t)K | (uintptr_t)V) & 15u) == 0;
  read_kernel<D, BITS, T, M><<<grid, D / (16 / (int)sizeof(T)) * 8, 0, s>>>(
      c, Hkv, n_q, r, st, t0, T_len, (T*)K, (T*)V, wide);
  return cudaGetLastError();
}

template <int BITS, typename T, typename M>
cudaError_t read_d(int D, const CacheView& c, int units, int Hkv, long long n_q, int r,
                   const DevState* st, long long t0, long long T_len, void* K, void* V,
                   cudaStream_t s) {
  switch (D) {
    case 32: return read_t<32, BITS, T, M>(c, units, Hkv, n_q, r, st, t0, T_len, K, V, s);
    case 64: return read_t<64, BITS, T, M>(c, units, Hkv, n_q, r, st, t0, T_len, K, V, s);
    case 128: return read_t<128, BITS, T, M>(c, units, Hkv, n_q, r, st, t0, T_len, K, V, s);
  }
  return cudaErrorInvalidValue;
}

template <typename T, typename M>
cudaError_t read_b(int bits, int D, const CacheView& c, int units, int Hkv, long long n_q, int r,
                   const DevState* st, long long t0, long long T_len, void* K, void* V,
                   cudaStream_t s) {
  switch (bits) {
    case 1: return read_d<1, T, M>(D, c, units, Hkv, n_q, r, st, t0, T_len, K, V, s);
    case 2: return read_d<2, T, M>(D, c, units, Hkv, n_q, r, st, t0, T_len, K, V, s);
    case 3: return read_d<3, T, M>(D, c, units, Hkv, n_q, r, st, t0, T_len, K, V, s);
    case 4: return read_d<4, T, M>(D, c, units, Hkv, n_q, r, st, t0, T_len, K, V, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

cudaError_t launch_read(const CacheView& c, int units, int Hkv, int D, int bits, int dtype,
                        long long n_q, int r, const DevState* st, long long t0, long long T,
                        void* K, void* V, cudaStream_t s) {
  if (dtype == 1) return read_b<float, float>(bits, D, c, units, Hkv, n_q, r, st, t0, T, K, V, s);
  if (c.meta == 1)
    return read_b<__half, __half>(bits, D, c, units, Hkv, n_q, r, st, t0, T, K, V, s);
  return read_b<__half, float>(bits, D, c, units, Hkv, n_q, r, st, t0, T, K, V, s);
}

}  // namespace kivi
