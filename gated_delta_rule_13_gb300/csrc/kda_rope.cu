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
// integer multiplication and without a reduction.  The frequency's own rounding, 2^-64,
// grows by the position to at most 2^-32 of a turn.  The upper 32 bits as a signed number
// give t / pi in [-1, 1), all of them: 24 go to sine and cosine, the others are added to what
// these give (rounded to 24 bits an angle near half a turn was off by 9e-8, and a sine of
// 1e-3 by 1e-4 of itself).
//
// Bound by HBM: a rotated channel is read and written once, 3 operations each.  96 bytes in
// flight a thread and 1024 threads an SM (64 and 128 bytes, 1280 threads: up to 10 % slower),
// rows of all heads of a token in one block so that its angles are worked out once.  Measured
// (cold inputs): 8192 tokens x 96 heads x 64 channels fp32, 403 MB both ways, 61.7 us, 6.5 TB/s;
// 16384 x 16 bf16 with the shared key, 71 MB, 16.1 us, of which a launch and one block's way are
// 2.5 (a plain copy of as many bytes: 12.5); 64 x 96 with the key 2.6 us.  Loads and stores
// past the caches made no difference.  Rows that start on 8, 4 or 2 bytes go in pieces of these,
// bound by instructions: 16384 x 16 of 74 channels bf16 40 us, of 72 in halves 19.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>

#include "kda_latent_tc.cuh"
#include "kda_rows.h"

namespace kda {
namespace {

constexpr int kThreads = 256, kSmThreads = 1024;   // of a block at most, of an SM
// Pieces in flight per thread: of 16 bytes 96 bytes of them.
template <bool kInterleaved, int kB>
constexpr int kGroup = kInterleaved || kB < 16 ? 6 : 3;
constexpr int kMaxAngles = 2048;   // of a block

// Whether a frequency has an angle here: a number of magnitude below 2^64, up to which turns_of
// has all its bits.
__device__ __forceinline__ bool has_angle(double f) {
  return ((uint64_t)__double_as_longlong(f) >> 52 & 2047) < 1023 + 64;
}
// Turns per position, 2^64 to the turn and modulo a turn, of such an angle per position in radians:
// the significand times 2^130 / (2 pi), shifted by what the exponent leaves.  In integers, because
// the 64-bit floating-point pipe is narrow here: off by two at most.
__device__ __forceinline__ uint64_t turns_of(double f) {
  constexpr uint64_t kHi = 0xa2f9836e4e441529ull, kLo = 0xfc2757d1f534ddc1ull;  // 2^130 / (2 pi)
  const uint64_t bits = (uint64_t)__double_as_longlong(f);
  const int exponent = (int)(bits >> 52 & 2047);
  const uint64_t m = (bits & 0xfffffffffffffull) | (exponent ? 1ull << 52 : 0);
  uint64_t w0 = m * kLo, w1 = __umul64hi(m, kLo), w2 = __umul64hi(m, kHi);
  const uint64_t mid = m * kHi;
  w1 += mid;
  w2 += w1 < mid;
  const int shift = 1141 - exponent, bit = shift & 63;
  if (shift >= 192) return 0;
  const uint64_t lo = shift < 64 ? w0 : shift < 128 ? w1 : w2;
  const uint64_t hi = shift < 64 ? w1 : shift < 128 ? w2 : 0;
  const uint64_t t = bit ? lo >> bit | hi << (64 - bit) : lo;
  return bits >> 63 ? 0 - t : t;
}

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

// kB bytes that lie on kB.
template <typename T, int kB>
struct Words {
  static constexpr int kE = kB / (int)sizeof(T);
  uint32_t w[kB / 4];
  __device__ __forceinline__ void load(const T *at) {
    if constexpr (kB == 16) {
      const uint4 v = *reinterpret_cast<const uint4 *>(at);
      w[0] = v.x;
      w[1] = v.y;
      w[2] = v.z;
      w[3] = v.w;
    } else if constexpr (kB == 8) {
      const uint2 v = *reinterpret_cast<const uint2 *>(at);
      w[0] = v.x;
      w[1] = v.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t *>(at);
    }
  }
  __device__ __forceinline__ void unpack(float (&x)[kE]) const {
#pragma unroll
    for (int i = 0; i < kB / 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        x[i] = __uint_as_float(w[i]);
      } else {
        const float2 f = sm100::unpack_bf16x2(w[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    }
  }
  static __device__ __forceinline__ void store(T *at, const float (&x)[kE]) {
    uint32_t w[kB / 4];
#pragma unroll
    for (int i = 0; i < kB / 4; ++i) {
      if constexpr (sizeof(T) == 4) w[i] = __float_as_uint(x[i]);
      else w[i] = sm100::pack_bf16x2(x[2 * i], x[2 * i + 1]);
    }
    if constexpr (kB == 16) *reinterpret_cast<uint4 *>(at) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (kB == 8) *reinterpret_cast<uint2 *>(at) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t *>(at) = w[0];
  }
};

// A piece is what a thread turns at a time: kB bytes of pairs (interleaved) or kB bytes of either
// half; with kB = 0 one pair, channel by channel.
template <typename T, bool kInterleaved, int kB>
struct Piece {
  using V = Words<T, kB>;
  static constexpr int kE = V::kE, kPairs = kInterleaved ? kE / 2 : kE;
  static_assert(kPairs >= 1, "a whole pair");
  V raw[kInterleaved ? 1 : 2];
  __device__ __forceinline__ void load(const T *row, int pair, int half) {
    raw[0].load(row + (kInterleaved ? 2 * pair : pair));
    if constexpr (!kInterleaved) raw[1].load(row + half + pair);
  }
  __device__ __forceinline__ void turn_store(T *row, int pair, int half, const float2 *cs) const {
    float a[kE];
    raw[0].unpack(a);
    if constexpr (kInterleaved) {
      float y[kE];
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const float2 r = cs[i];
        y[2 * i] = a[2 * i] * r.x - a[2 * i + 1] * r.y;
        y[2 * i + 1] = a[2 * i + 1] * r.x + a[2 * i] * r.y;
      }
      V::store(row + 2 * pair, y);
    } else {
      float b[kE], u[kE], v[kE];
      raw[1].unpack(b);
#pragma unroll
      for (int i = 0; i < kPairs; ++i) {
        const float2 r = cs[i];
        u[i] = a[i] * r.x - b[i] * r.y;
        v[i] = b[i] * r.x + a[i] * r.y;
      }
      V::store(row + pair, u);
      V::store(row + half + pair, v);
    }
  }
};
template <typename T, bool kInterleaved>
struct Piece<T, kInterleaved, 0> {
  static constexpr int kPairs = 1;
  T a, b;
  __device__ __forceinline__ void load(const T *row, int pair, int half) {
    a = row[kInterleaved ? 2 * pair : pair];
    b = row[kInterleaved ? 2 * pair + 1 : half + pair];
  }
  __device__ __forceinline__ void turn_store(T *row, int pair, int half, const float2 *cs) const {
    const float x = to_float(a), y = to_float(b);
    row[kInterleaved ? 2 * pair : pair] = from_float<T>(x * cs[0].x - y * cs[0].y);
    row[kInterleaved ? 2 * pair + 1 : half + pair] = from_float<T>(y * cs[0].x + x * cs[0].y);
  }
};

struct Shape {
  int units;        // pieces of a row: as many threads have one row, neighbours the next
  int tokens;       // of a block
  int heads;        // of a block (the key counts as head H)
  int step;         // rows a block takes at a time
  uint32_t magic, unit_magic;   // 2^32 / heads and / units, rounded up; 0 for one: not used
};
// x / by for x by < 2^32
__device__ __forceinline__ int quotient(int x, int by, uint32_t magic) {
  return by == 1 ? x : (int)__umulhi((uint32_t)x, magic);
}

// Block (x: tokens, y: heads); its rows, a token's heads beside one another, go over the lanes in
// turn.  The cosines and sines of its angles are worked out once, in shared memory, while its
// first pieces are on their way.
template <typename T, bool kInterleaved, int kB>
__global__ void __launch_bounds__(kThreads, kSmThreads / kThreads) kda_rope_kernel(const RopeArgs a, const Shape sh) {
  using P = Piece<T, kInterleaved, kB>;
  extern __shared__ float2 cs[];                         // [tokens][pairs]
  const int half = a.dr / 2, tid = threadIdx.x;
  const int step = sh.step;
  int r = quotient(tid, sh.units, sh.unit_magic);
  const int pair = (tid - r * sh.units) * P::kPairs;
  const int64_t t0 = (int64_t)blockIdx.x * sh.tokens;
  const int nt = (int)min((int64_t)sh.tokens, a.n - t0);
  const int h0 = blockIdx.y * sh.heads, heads = min(sh.heads, a.H + (a.k != nullptr) - h0);
  const int rows = r < step ? nt * sh.heads : 0;         // of the last heads some are none
  constexpr int G = kGroup<kInterleaved, kB>;
  P piece[G];
  T *to[G];
  int at[G];                                        // token of the block, -1: none
  const auto load = [&] {
#pragma unroll
    for (int i = 0; i < G; ++i) {
      at[i] = -1;
      const int t = quotient(r, sh.heads, sh.magic), h = r - t * sh.heads;
      if (r < rows && h < heads) {
        const int64_t tok = t0 + t;
        const T *from;
        if (h0 + h < a.H) {
          from = static_cast<const T *>(a.x) + tok * a.x_ts + (h0 + h) * a.x_hs;
          to[i] = static_cast<T *>(a.out) + tok * a.o_ts + (h0 + h) * a.o_hs;
        } else {
          from = static_cast<const T *>(a.k) + tok * a.k_ts;
          to[i] = static_cast<T *>(a.k_out) + tok * a.ko_ts;
        }
        piece[i].load(from, pair, half);
        at[i] = t;
      }
      r += step;
    }
  };
  load();
  for (int i = tid; i < nt * half; i += blockDim.x) {
    const int tok = i / half, p = i - tok * half;
    const double freq = a.inv_freq[p];
    const uint64_t turns = (uint64_t)(int64_t)a.positions[t0 + tok] * turns_of(freq);
    float s, c;
    // what fp32 holds of t / pi exactly, 24 bits of 32, and the rest d, below 2^-21: the sine of
    // the sum is s + c d, its cosine c - s d, but for d^2 / 2
    const uint32_t top = (uint32_t)(turns >> 32), low = top & 255;
    sincospif(has_angle(freq) ? (float)(int32_t)(top - low) * 0x1p-31f : CUDART_NAN_F, &s, &c);
    const float d = (float)low * (CUDART_PI_F * 0x1p-31f), u = fmaf(c, d, s), v = fmaf(-s, d, c);
    cs[i] = make_float2(v * a.scale, (a.transpose ? -u : u) * a.scale);
  }
  __syncthreads();
  for (;;) {
#pragma unroll
    for (int i = 0; i < G; ++i)
      if (at[i] >= 0) piece[i].turn_store(to[i], pair, half, cs + at[i] * half + pair);
    if (r >= rows) break;
    load();
  }
}

template <typename T, bool kInterleaved, int kB>
cudaError_t launch(const RopeArgs &a, cudaStream_t stream) {
  using P = Piece<T, kInterleaved, kB>;
  const int half = a.dr / 2, units = half / P::kPairs, heads = a.H + (a.k != nullptr);
  const int64_t sms = latent::sm_count() > 0 ? latent::sm_count() : 1;
  Shape sh;
  sh.units = units;
  // Blocks are small, 128 threads, unless a token's heads are more than these have in flight.
  constexpr int G = kGroup<kInterleaved, kB>;
  const int threads = kThreads / 2 / units * G >= heads ? kThreads / 2 : kThreads;
  const int64_t blocks_sm = kSmThreads / threads, lanes = threads / units;  // rows at a time
  // A block's rows: what its lanes have in flight, or all heads of a token, whose angles are then
  // worked out once, where tokens are enough to fill the SMs; fewer where SMs would have none.
  int64_t rows = lanes * G;
  if (heads > rows && a.n >= blocks_sm * sms) rows = heads < 16 * lanes ? heads : 16 * lanes;
  while (rows > lanes && a.n * heads < rows * blocks_sm * sms) rows /= 2;
  sh.heads = heads;
  if (heads > rows) {                                    // one token over several blocks
    const int64_t split = (heads + rows - 1) / rows;
    sh.heads = (int)((heads + split - 1) / split);
  }
  sh.tokens = (int)(rows / sh.heads);
  if (sh.tokens > kMaxAngles / half) sh.tokens = kMaxAngles / half;
  if (sh.tokens < 1) sh.tokens = 1;
  sh.step = (int)lanes;
  const auto magic = [](int by) { return (uint32_t)(((1ull << 32) + by - 1) / by); };
  sh.magic = magic(sh.heads);
  sh.unit_magic = magic(units);
  const int64_t blocks = (a.n + sh.tokens - 1) / sh.tokens;
  const dim3 grid((unsigned)blocks, (unsigned)((heads + sh.heads - 1) / sh.heads));
  kda_rope_kernel<T, kInterleaved, kB>
      <<<grid, threads, (size_t)sh.tokens * half * sizeof(float2), stream>>>(a, sh);
  return cudaGetLastError();
}

template <typename T, bool kInterleaved>
cudaError_t pick(const RopeArgs &a, cudaStream_t stream) {
  // Pieces of as many bytes as every row starts on and has whole ones of.
  constexpr int kEsz = sizeof(T);
  uintptr_t bits = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.out) |
                   reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.k_out);
  for (const int64_t v : {a.x_ts, a.x_hs, a.o_ts, a.o_hs, a.k_ts, a.ko_ts,
                          (int64_t)(kInterleaved ? a.dr : a.dr / 2)})
    bits |= (uintptr_t)v * kEsz;
  if (bits % 16 == 0) return launch<T, kInterleaved, 16>(a, stream);
  if (bits % 8 == 0) return launch<T, kInterleaved, 8>(a, stream);
  if constexpr (kEsz == 2)
    if (bits % 4 == 0) return launch<T, kInterleaved, 4>(a, stream);
  return launch<T, kInterleaved, 0>(a, stream);
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
