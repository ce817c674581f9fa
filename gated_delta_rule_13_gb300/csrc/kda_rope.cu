// Rotary positions (kda_rope): pairs of channels turned by position x frequency.
//
//   (a, b) -> scale (a cos t - b sin t, b cos t + a sin t),  t = position * inv_freq[pair]
//
// and with `transpose` the transposed map, its gradient, t -> -t.
//
// The angle.  A position reaches 2^31 and an angle must be right to 2^-25 of a turn for
// fp32 results, so that position x frequency in fp32 would be off by whole radians.  A
// frequency is held as turns per position in 64-bit fixed point, 2^-64 of a turn: the
// product with an integer position, modulo 2^64, is the fraction of a turn itself, by one
// integer multiplication and without a reduction.  The frequency's own rounding, 2^-65,
// grows by the position to at most 2^-34 of a turn.  The upper 32 bits as a signed number
// give t / pi in [-1, 1).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kda_latent_tc.cuh"
#include "kda_rows.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kGroup = 4;          // pieces in flight per thread
constexpr int kMaxAngles = 2048;   // of a block

// Turns per position, 2^64 to the turn, of an angle per position in radians: the product
// with 1 / (2 pi), held as the sum of two doubles.
__device__ __forceinline__ uint64_t turns_of(double f) {
  constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;
  const double hi = f * kHi, lo = fma(f, kHi, -hi) + f * kLo;
  const double frac = hi - floor(hi);                    // exact
  return (uint64_t)(frac * 0x1p64) + (uint64_t)(int64_t)(lo * 0x1p64);
}

template <typename T>
struct Elems;
template <>
struct Elems<float> {
  static constexpr int kVec = 4;
  static __device__ __forceinline__ void unpack(const uint4 &v, float *x) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float *x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
};
template <>
struct Elems<__nv_bfloat16> {
  static constexpr int kVec = 8;
  static __device__ __forceinline__ void unpack(const uint4 &v, float *x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = sm100::unpack_bf16x2(w[i]);
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
  static __device__ __forceinline__ uint4 pack(const float *x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = sm100::pack_bf16x2(x[2 * i], x[2 * i + 1]);
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// A piece is what a thread turns at a time: with vectors, 16 bytes (interleaved pairs) or
// 16 bytes of either half; else one pair.
template <typename T, bool kInterleaved, bool kVector>
struct Piece {
  static constexpr int kE = kVector ? Elems<T>::kVec : 1;
  static constexpr int kPairs = kInterleaved ? (kVector ? kE / 2 : 1) : kE;
  static constexpr int kRegs = kVector ? (kInterleaved ? 1 : 2) : 1;   // 16-byte registers
  uint4 raw[kRegs];
  __device__ __forceinline__ void load(const T *row, int pair, int half) {
    if constexpr (kVector) {
      raw[0] = *reinterpret_cast<const uint4 *>(row + (kInterleaved ? 2 * pair : pair));
      if constexpr (!kInterleaved) raw[1] = *reinterpret_cast<const uint4 *>(row + half + pair);
    } else {
      raw[0].x = __float_as_uint(to_float(row[kInterleaved ? 2 * pair : pair]));
      raw[0].y = __float_as_uint(to_float(row[kInterleaved ? 2 * pair + 1 : half + pair]));
    }
  }
  __device__ __forceinline__ void turn_store(T *row, int pair, int half, const float2 *cs) const {
    if constexpr (!kVector) {
      const float a = __uint_as_float(raw[0].x), b = __uint_as_float(raw[0].y);
      row[kInterleaved ? 2 * pair : pair] = from_float<T>(a * cs[0].x - b * cs[0].y);
      row[kInterleaved ? 2 * pair + 1 : half + pair] = from_float<T>(b * cs[0].x + a * cs[0].y);
    } else if constexpr (kInterleaved) {
      float x[kE], y[kE];
      Elems<T>::unpack(raw[0], x);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const float2 r = cs[i];
        y[2 * i] = x[2 * i] * r.x - x[2 * i + 1] * r.y;
        y[2 * i + 1] = x[2 * i + 1] * r.x + x[2 * i] * r.y;
      }
      *reinterpret_cast<uint4 *>(row + 2 * pair) = Elems<T>::pack(y);
    } else {
      float a[kE], b[kE], u[kE], v[kE];
      Elems<T>::unpack(raw[0], a);
      Elems<T>::unpack(raw[1], b);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const float2 r = cs[i];
        u[i] = a[i] * r.x - b[i] * r.y;
        v[i] = b[i] * r.x + a[i] * r.y;
      }
      *reinterpret_cast<uint4 *>(row + pair) = Elems<T>::pack(u);
      *reinterpret_cast<uint4 *>(row + half + pair) = Elems<T>::pack(v);
    }
  }
};

struct Shape {
  int unit_bits, head_bits;   // lanes of a block: pieces of a row, heads, the rest tokens
  int tokens;                 // of a block
  int heads;                  // of a block (the key counts as head H)
};

// Block (x: tokens, y: heads).  Its angles' cosines and sines are worked out once, in
// shared memory, while its first pieces are on their way.
template <typename T, bool kInterleaved, bool kVector>
__global__ void __launch_bounds__(kThreads) kda_rope_kernel(const RopeArgs a, const Shape sh) {
  using P = Piece<T, kInterleaved, kVector>;
  extern __shared__ float2 cs[];                         // [tokens][pairs]
  __shared__ uint64_t step[kRopeMax / 2];
  const int half = a.dr / 2, tid = threadIdx.x;
  const int units = half / P::kPairs;
  const int unit = tid & ((1 << sh.unit_bits) - 1);
  const int hl = (tid >> sh.unit_bits) & ((1 << sh.head_bits) - 1);
  const int tl = tid >> (sh.unit_bits + sh.head_bits);
  const int hp = 1 << sh.head_bits, tp = kThreads >> (sh.unit_bits + sh.head_bits);
  const int64_t t0 = (int64_t)blockIdx.x * sh.tokens;
  const int nt = (int)min((int64_t)sh.tokens, a.n - t0);
  const int h0 = blockIdx.y * sh.heads;
  const int h1 = min(h0 + sh.heads, a.H + (a.k != nullptr));
  const int pair = unit * P::kPairs;
  // Pieces of this thread: heads h0 + hl + i hp of tokens tl + j tp, heads first.
  int t = unit < units && h0 + hl < h1 ? tl : nt, h = h0 + hl;
  P piece[kGroup];
  T *to[kGroup];
  int at[kGroup];                                        // token of the block, -1: none
  const auto load = [&] {
#pragma unroll
    for (int i = 0; i < kGroup; ++i) {
      at[i] = -1;
      if (t < nt) {
        const int64_t tok = t0 + t;
        const T *from;
        if (h < a.H) {
          from = static_cast<const T *>(a.x) + tok * a.x_ts + h * a.x_hs;
          to[i] = static_cast<T *>(a.out) + tok * a.o_ts + h * a.o_hs;
        } else {
          from = static_cast<const T *>(a.k) + tok * a.k_ts;
          to[i] = static_cast<T *>(a.k_out) + tok * a.ko_ts;
        }
        piece[i].load(from, pair, half);
        at[i] = t;
        h += hp;
        if (h >= h1) {
          h = h0 + hl;
          t += tp;
        }
      }
    }
  };
  load();
  for (int i = tid; i < half; i += kThreads) step[i] = turns_of(a.inv_freq[i]);
  __syncthreads();
  for (int i = tid; i < nt * half; i += kThreads) {
    const int tok = i / half, p = i - tok * half;
    const uint64_t turns = (uint64_t)(int64_t)a.positions[t0 + tok] * step[p];
    float s, c;
    sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &s, &c);
    cs[i] = make_float2(c * a.scale, (a.transpose ? -s : s) * a.scale);
  }
  __syncthreads();
  while (at[0] >= 0) {
#pragma unroll
    for (int i = 0; i < kGroup; ++i)
      if (at[i] >= 0) piece[i].turn_store(to[i], pair, half, cs + at[i] * half + pair);
    load();
  }
}

int bits_for(int n) {
  int b = 0;
  while ((1 << b) < n) ++b;
  return b;
}

template <typename T, bool kInterleaved, bool kVector>
cudaError_t launch(const RopeArgs &a, cudaStream_t stream) {
  using P = Piece<T, kInterleaved, kVector>;
  const int half = a.dr / 2, units = half / P::kPairs, heads = a.H + (a.k != nullptr);
  Shape sh;
  sh.unit_bits = bits_for(units);
  sh.head_bits = bits_for(heads);
  if (sh.unit_bits + sh.head_bits > 8) sh.head_bits = 8 - sh.unit_bits;
  // the key beside a full set of heads takes a turn of its own rather than twice the lanes
  if (sh.head_bits > 0 && (1 << (sh.head_bits - 1)) == a.H) --sh.head_bits;
  const int tp = kThreads >> (sh.unit_bits + sh.head_bits), hp = 1 << sh.head_bits;
  const int sms = latent::sm_count() > 0 ? latent::sm_count() : 1;
  // Tokens of a block: about 8 pieces a thread, as far as the grid keeps four blocks an SM.
  int turns = (heads + hp - 1) / hp;                     // of a thread, for one token
  sh.tokens = tp;
  while (turns * (sh.tokens / tp) < 8 && sh.tokens * 2 * half <= kMaxAngles &&
         (a.n + sh.tokens * 2 - 1) / (sh.tokens * 2) >= 4 * sms)
    sh.tokens *= 2;
  while (sh.tokens * half > kMaxAngles) sh.tokens /= 2;
  // Few tokens: their heads over several blocks.
  sh.heads = heads;
  const int64_t blocks = (a.n + sh.tokens - 1) / sh.tokens;
  while (sh.heads > hp && blocks * ((heads + sh.heads - 1) / sh.heads) < sms)
    sh.heads = (sh.heads / 2 + hp - 1) / hp * hp;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)blocks, (unsigned)((heads + sh.heads - 1) / sh.heads));
  kda_rope_kernel<T, kInterleaved, kVector>
      <<<grid, kThreads, (size_t)sh.tokens * half * sizeof(float2), stream>>>(a, sh);
  return cudaGetLastError();
}

template <typename T, bool kInterleaved>
cudaError_t pick(const RopeArgs &a, cudaStream_t stream) {
  using P = Piece<T, kInterleaved, true>;
  // 16-byte pieces where every row starts on 16 bytes and has whole ones.
  constexpr int kV = Elems<T>::kVec;
  uintptr_t bits = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.out) |
                   reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.k_out);
  const bool whole = bits % 16 == 0 && (a.dr / 2) % P::kPairs == 0 && a.x_ts % kV == 0 &&
                     a.x_hs % kV == 0 && a.o_ts % kV == 0 && a.o_hs % kV == 0 &&
                     a.k_ts % kV == 0 && a.ko_ts % kV == 0;
  return whole ? launch<T, kInterleaved, true>(a, stream)
               : launch<T, kInterleaved, false>(a, stream);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &a, cudaStream_t stream) {
  if (a.n == 0) return cudaSuccess;
  if (a.bf16)
    return a.interleaved ? pick<__nv_bfloat16, true>(a, stream)
                         : pick<__nv_bfloat16, false>(a, stream);
  return a.interleaved ? pick<float, true>(a, stream) : pick<float, false>(a, stream);
}

}  // namespace kda
