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
// grows by the position to at most 2^-33 of a turn.  The upper 32 bits as a signed number
// give t / pi in [-1, 1).
//
// Bound by HBM: a rotated channel is read and written once, 3 operations each.  96 bytes in
// flight a thread and 1024 threads an SM (64 and 128 bytes, 1280 threads: up to 10 % slower),
// rows of all heads of a token in one block so that its angles are worked out once.  Measured
// (cold inputs): 8192 tokens x 96 heads x 64 channels fp32, 403 MB both ways, 60.8 us, 6.6 TB/s;
// 16384 x 16 bf16 with the shared key, 71 MB, 16.0 us, of which a launch and one block's way are
// 2.5 (a plain copy of as many bytes: 12.5); 64 x 96 with the key 2.6 us.  Loads and stores
// past the caches made no difference.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kda_latent_tc.cuh"
#include "kda_rows.h"

namespace kda {
namespace {

constexpr int kThreads = 256, kSmThreads = 1024;   // of a block at most, of an SM
template <bool kInterleaved>
constexpr int kGroup = kInterleaved ? 6 : 3;   // pieces in flight per thread: 96 bytes
constexpr int kMaxAngles = 2048;   // of a block

// Turns per position, 2^64 to the turn and modulo a turn, of an angle per position in radians,
// |f| < 2^118: the significand times 2^130 / (2 pi), shifted by what the exponent leaves.  In
// integers, because the 64-bit floating-point pipe is narrow here: off by one at most.
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
  if (shift < 0 || shift >= 192) return 0;
  const uint64_t lo = shift < 64 ? w0 : shift < 128 ? w1 : w2;
  const uint64_t hi = shift < 64 ? w1 : shift < 128 ? w2 : 0;
  const uint64_t t = bit ? lo >> bit | hi << (64 - bit) : lo;
  return bits >> 63 ? 0 - t : t;
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
  int unit_bits;    // lanes of a block: pieces of a row, the rest rows
  int tokens;       // of a block
  int heads;        // of a block (the key counts as head H)
  uint32_t magic;   // 2^32 / heads, rounded up
};

// Block (x: tokens, y: heads); its rows, a token's heads beside one another, go over the lanes in
// turn.  The cosines and sines of its angles are worked out once, in shared memory, while its
// first pieces are on their way.
template <typename T, bool kInterleaved, bool kVector>
__global__ void __launch_bounds__(kThreads, kSmThreads / kThreads) kda_rope_kernel(const RopeArgs a, const Shape sh) {
  using P = Piece<T, kInterleaved, kVector>;
  extern __shared__ float2 cs[];                         // [tokens][pairs]
  const int half = a.dr / 2, tid = threadIdx.x;
  const int unit = tid & ((1 << sh.unit_bits) - 1), step = blockDim.x >> sh.unit_bits;
  const int pair = unit * P::kPairs;
  const int64_t t0 = (int64_t)blockIdx.x * sh.tokens;
  const int nt = (int)min((int64_t)sh.tokens, a.n - t0);
  const int h0 = blockIdx.y * sh.heads, heads = min(sh.heads, a.H + (a.k != nullptr) - h0);
  const int rows = pair < half ? nt * sh.heads : 0;      // of the last heads some are none
  int r = tid >> sh.unit_bits;
  constexpr int G = kGroup<kInterleaved>;
  P piece[G];
  T *to[G];
  int at[G];                                        // token of the block, -1: none
  const auto load = [&] {
#pragma unroll
    for (int i = 0; i < G; ++i) {
      at[i] = -1;
      const int t = sh.heads == 1 ? r : (int)__umulhi((uint32_t)r, sh.magic), h = r - t * sh.heads;
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
    const uint64_t turns = (uint64_t)(int64_t)a.positions[t0 + tok] * turns_of(a.inv_freq[p]);
    float s, c;
    sincospif((float)(int32_t)(turns >> 32) * 0x1p-31f, &s, &c);
    cs[i] = make_float2(c * a.scale, (a.transpose ? -s : s) * a.scale);
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

template <typename T, bool kInterleaved, bool kVector>
cudaError_t launch(const RopeArgs &a, cudaStream_t stream) {
  using P = Piece<T, kInterleaved, kVector>;
  const int half = a.dr / 2, units = half / P::kPairs, heads = a.H + (a.k != nullptr);
  const int64_t sms = latent::sm_count() > 0 ? latent::sm_count() : 1;
  Shape sh;
  sh.unit_bits = 0;
  while ((1 << sh.unit_bits) < units) ++sh.unit_bits;
  // Blocks are small, 128 threads, unless a token's heads are more than these have in flight.
  constexpr int G = kGroup<kInterleaved>;
  const int threads = (kThreads / 2 >> sh.unit_bits) * G >= heads && units <= kThreads / 2
                          ? kThreads / 2 : kThreads;
  const int64_t blocks_sm = kSmThreads / threads, lanes = threads >> sh.unit_bits;  // rows at a time
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
  sh.magic = (uint32_t)(((1ull << 32) + sh.heads - 1) / sh.heads);   // 0 for one head: not used
  const int64_t blocks = (a.n + sh.tokens - 1) / sh.tokens;
  const dim3 grid((unsigned)blocks, (unsigned)((heads + sh.heads - 1) / sh.heads));
  kda_rope_kernel<T, kInterleaved, kVector>
      <<<grid, threads, (size_t)sh.tokens * half * sizeof(float2), stream>>>(a, sh);
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
