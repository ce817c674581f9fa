// Norm over a row's channels, with or without its mean (kda_norm_fwd), and its gradient
// (kda_norm_bwd).
//
//   m = mean x (0 without), r = 1 / sqrt(mean (x - m)^2 + eps),  z = (x - m) r
//   y = z w + b
//   dx = r (w g - mean(w g) - z mean(w g z))   (without the mean: no second term)
//   dw = sum over rows of g z,  db = sum over rows of g
//
// Bound by HBM: two passes of bytes forward, three back.  A row is read once: by four to 512
// threads, into registers (few rows) or, many rows, some rows ahead into shared memory.
// The variance is the mean square of what the mean leaves, from the row on chip, so that a mean
// far from zero costs no more digits than its own rounding.  Statistics and sums are fp32; values are taken in pairs, which
// halves the instructions (with one at a time the gradient of 16384 x 7168 was bound by them:
// 167 us).  The gradient's blocks walk over the rows with the sums of dw and db in registers and
// leave one pair of rows each in the workspace; a second kernel adds these in the blocks' order,
// so that results do not vary between calls.
//
// Rows that start anywhere go through shared memory in 16-byte pieces all the same, put to their
// places there, and the results back to pieces; instructions and barriers then bind them (61 and
// 50 % of the issue slots at 8192 x 7169 bf16).
//
// Measured (cold): 16384 x 7168 bf16 forward 76 us (6.2 TB/s), gradient 110 us (6.4); gradient of
// 16384 x 512 fp32 21.6 us (4.6), of which the two sums are 4; 64 x 7168 2.9 us; 1 M x 128 bf16
// 90 us (5.9), 1 M x 64 46 (5.8; with half a warp a row 85).  Anywhere: 8192 x 7169 bf16 65 and
// 121 us (3.6 and 2.9 TB/s; by single channels 192 and 201), 60000 x 513 45 and 78 (2.7 and 2.4).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "kda_latent_tc.cuh"
#include "kda_rows.h"

namespace kda {
namespace {

constexpr int kShort = 256;              // channels of a short row: a warp's, or less than one's

// Two fp32 values at a time: the same roundings in half the instructions.
struct F2 {
  uint64_t v;
  __device__ __forceinline__ F2() {}
  __device__ __forceinline__ F2(float a, float b) {
    asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(a), "f"(b));
  }
  __device__ __forceinline__ float2 get() const {
    float2 x;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x.x), "=f"(x.y) : "l"(v));
    return x;
  }
  __device__ __forceinline__ float sum() const {
    const float2 x = get();
    return x.x + x.y;
  }
};
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
  F2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
  F2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return d;
}

// What a thread holds of a row, E channels: 16-byte vectors tid, tid + N, ..., or single
// channels.  A vector that the row ends in is put together from single channels.
template <typename T, int N, int E, bool kVector>
struct Row {
  static constexpr int kV = kVector ? 16 / (int)sizeof(T) : 1;
  static constexpr int kCount = E / kV;                  // vectors
  static constexpr int kRegs = E * (int)sizeof(T) / 4;
  uint32_t raw[kRegs];
  static __device__ __forceinline__ int channel(int i) { // of element i of this thread
    return (i / kV * N + threadIdx.x % N) * kV + i % kV;
  }
  __device__ __forceinline__ void set(int i, T v) {
    if constexpr (sizeof(T) == 4) raw[i] = __float_as_uint(v);
    else {
      const uint32_t w = __bfloat16_as_ushort(v);
      raw[i / 2] = i & 1 ? (raw[i / 2] & 0xffffu) | w << 16 : (raw[i / 2] & 0xffff0000u) | w;
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(raw[i]);
    else return __uint_as_float(i & 1 ? raw[i / 2] & 0xffff0000u : raw[i / 2] << 16);
  }
  __device__ __forceinline__ F2 two(int i) const { return F2(get(2 * i), get(2 * i + 1)); }
  __device__ __forceinline__ void load(const T *row, int W) {
#pragma unroll
    for (int i = 0; i < kRegs; ++i) raw[i] = 0;
#pragma unroll
    for (int j = 0; j < kCount; ++j) {
      const int c = channel(j * kV);
      if constexpr (kVector) {
        if (c + kV <= W) {
          const uint4 v = *reinterpret_cast<const uint4 *>(row + c);
          raw[4 * j] = v.x;
          raw[4 * j + 1] = v.y;
          raw[4 * j + 2] = v.z;
          raw[4 * j + 3] = v.w;
        } else if (c < W) {
#pragma unroll
          for (int e = 0; e < kV; ++e)
            if (c + e < W) set(j * kV + e, row[c + e]);
        }
      } else if (c < W) {
        set(j, row[c]);
      }
    }
  }
  // f: pair of elements -> values
  template <class F>
  static __device__ __forceinline__ void store(T *row, int W, F f) {
#pragma unroll
    for (int j = 0; j < kCount; ++j) {
      const int c = channel(j * kV);
      if (c >= W) continue;
      if constexpr (kVector) {
        float2 y[kV / 2];
#pragma unroll
        for (int k = 0; k < kV / 2; ++k) y[k] = f(j * kV / 2 + k);
        if (c + kV <= W) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (sizeof(T) == 4) w[k] = __float_as_uint(k & 1 ? y[k / 2].y : y[k / 2].x);
            else w[k] = sm100::pack_bf16x2(y[k].x, y[k].y);
          }
          *reinterpret_cast<uint4 *>(row + c) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
          for (int e = 0; e < kV; ++e)
            if (c + e < W) put(row + c + e, e & 1 ? y[e / 2].y : y[e / 2].x);
        }
      } else {
        const float2 y = f(j / 2);
        put(row + c, j & 1 ? y.y : y.x);
      }
    }
  }
  static __device__ __forceinline__ void put(T *to, float y) {
    if constexpr (sizeof(T) == 4) *to = y;
    else *to = __float2bfloat16_rn(y);
  }
  // The same channels of an fp32 vector (`none` without one, and past the row).
  static __device__ __forceinline__ void load_vector(const float *p, int W, float none, float (&v)[E]) {
#pragma unroll
    for (int j = 0; j < kCount; ++j) {
      const int c = channel(j * kV);
      if (kVector && p && c + kV <= W) {
#pragma unroll
        for (int e = 0; e < kV; e += 4) {
          const float4 x = __ldg(reinterpret_cast<const float4 *>(p + c + e));
          v[j * kV + e] = x.x;
          v[j * kV + e + 1] = x.y;
          v[j * kV + e + 2] = x.z;
          v[j * kV + e + 3] = x.w;
        }
      } else {
#pragma unroll
        for (int e = 0; e < kV; ++e) v[j * kV + e] = p && c + e < W ? __ldg(p + c + e) : none;
      }
    }
  }
};

// Sums over the N threads of a row, a group of a block of consecutive warps; `part` alternates
// between two places, so that one barrier a call is enough.
template <int N, int K>
__device__ __forceinline__ void row_sum(float (&x)[K], float *part) {  // [K][N / 32]
  constexpr int kLanes = N < 32 ? N : 32;
  const unsigned mask = N < 32 ? ((1u << kLanes) - 1) << (threadIdx.x & 31 & ~(kLanes - 1)) : ~0u;
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) x[k] += __shfl_xor_sync(mask, x[k], o);
  if constexpr (N > 32) {
    constexpr int kWarps = N / 32;
    const int warp = threadIdx.x % N >> 5, lane = threadIdx.x & 31;
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) part[k * kWarps + warp] = x[k];
    sm100::named_sync(1 + threadIdx.x / N, N);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float y = part[k * kWarps + lane % kWarps];
#pragma unroll
      for (int o = kWarps / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
      x[k] = y;
    }
  }
}
template <int N>
constexpr int kPart = N < 32 ? 1 : N / 32;               // floats of `part` for each sum

// Mean and reciprocal deviation of a row held in registers; part: two places of N / 32, `turn`
// alternates between calls.
template <int N, int E, class R>
__device__ __forceinline__ void statistics(const NormArgs &a, const R &x, float *part, int turn,
                                           float &m, float &r) {
  const float inv = 1.f / a.W;
  m = 0.f;
  if (a.center) {
    F2 t[2] = {F2(0.f, 0.f), F2(0.f, 0.f)};
#pragma unroll
    for (int i = 0; i < E / 2; ++i) t[i & 1] = t[i & 1] + x.two(i);
    float s[1] = {(t[0] + t[1]).sum()};
    row_sum<N, 1>(s, part);
    m = s[0] * inv;
  }
  F2 t[2] = {F2(0.f, 0.f), F2(0.f, 0.f)};
  const F2 m2(-m, -m);
#pragma unroll
  for (int j = 0; j < R::kCount; ++j)
    if (R::channel(j * R::kV) + R::kV <= a.W) {
      if constexpr (R::kV > 1)
#pragma unroll
        for (int k = 0; k < R::kV / 2; ++k) {
          const F2 d = x.two(j * R::kV / 2 + k) + m2;
          t[k & 1] = fma2(d, d, t[k & 1]);
        }
      else {
        const F2 d(x.get(j) - m, 0.f);
        t[j & 1] = fma2(d, d, t[j & 1]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < R::kV; ++k)
        if (R::channel(j * R::kV + k) < a.W) {
          const F2 d(x.get(j * R::kV + k) - m, 0.f);
          t[0] = fma2(d, d, t[0]);
        }
    }
  float v[1] = {(t[0] + t[1]).sum()};
  row_sum<N, 1>(v, part + (a.center || turn ? kPart<N> : 0));
  r = rsqrtf(fmaf(v[0], inv, a.eps));
}
// wb(i, w, b): weight and bias of this thread's pair i of channels.
template <int N, class R, class F, class T>
__device__ __forceinline__ void finish(const NormArgs &a, int64_t row, const R &x, float m, float r,
                                       F wb, T *out) {
  if (threadIdx.x % N == 0) {
    if (a.mean) a.mean[row] = m;
    if (a.rstd) a.rstd[row] = r;
  }
  const F2 m2(-m, -m), r2(r, r);
  R::store(out, a.W, [&](int i) {
    F2 w, b;
    wb(i, w, b);
    return fma2((x.two(i) + m2) * r2, w, b).get();
  });
}

// One row a group of N threads, straight from memory: for few rows.
template <int N>
constexpr int kBlock = N < 256 ? 256 : N;
template <typename T, int N, int E, bool kVector>
__global__ void __launch_bounds__(kBlock<N>, kVector ? 1 : 1024 / kBlock<N>) kda_norm_fwd_kernel(const NormArgs a) {
  using R = Row<T, N, E, kVector>;
  constexpr int kRows = kBlock<N> / N;
  __shared__ float part[kRows][2 * kPart<N>];
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / N;
  if (row >= a.n) return;                                // a whole group
  R x;
  x.load(static_cast<const T *>(a.x) + row * a.x_rs, a.W);
  float w[E], b[E], m, r;
  R::load_vector(a.weight, a.W, 1.f, w);
  R::load_vector(a.bias, a.W, 0.f, b);
  statistics<N, E>(a, x, part[threadIdx.x / N], 0, m, r);
  const auto wb = [&](int i, F2 &u, F2 &v) {
    u = F2(w[2 * i], w[2 * i + 1]);
    v = F2(b[2 * i], b[2 * i + 1]);
  };
  finish<N>(a, row, x, m, r, wb, static_cast<T *>(a.out) + row * a.out_rs);
}

// ------------------------------------------------------------------ many rows
// One block an SM; each group of N threads walks over rows of its own, with weight and bias
// in shared memory.  Every thread copies the channels it will read itself, some rows ahead,
// into shared memory (cp.async): no thread waits for another but in the row's sums.
// The gradient's threads have twice the registers, for the sums of dw and db.
template <int N, int E>
constexpr int kFwdThreads = N * E > 8192 ? 512 : 1024;   // (weight and bias of long rows take room)
constexpr int kBwdThreads = 512;
constexpr int kRingSpace = 230400;       // shared memory without what is declared
// Rows ahead, beside `vectors` bytes.
constexpr int stages(int row_bytes, int vectors) {
  return (kRingSpace - vectors) / row_bytes < 4 ? (kRingSpace - vectors) / row_bytes : 4;
}
// Bytes of a row's place: its vectors in order, one more where rows start anywhere.
template <typename T, int N, int E, bool kAny>
constexpr int kSlot = N * E * (int)sizeof(T) + (kAny ? 16 : 0);
template <typename T, int N, int E, bool kAny>
constexpr int kFwdStages = stages(kFwdThreads<N, E> / N * kSlot<T, N, E, kAny>, 2 * N *E * 4);
template <typename T, int N, int E, bool kAny>
constexpr int kBwdStages =
    stages(2 * (kBwdThreads / N) * kSlot<T, N, E, kAny>,
           kAny && N *E <= kShort ? kRingSpace / 2 + 2048 : N *E * 4);   // (two blocks an SM)

// An fp32 vector [W] into shared memory, laid out as threads read it: [E / 4][N] 16 bytes.
template <typename T, int N, int E, bool kAny>
__device__ __forceinline__ void keep_vector(uint32_t dst, const float *p, int W, float none) {
  if (threadIdx.x >= N) return;
  using R = Row<T, N, E, true>;
  float w[E];
  if constexpr (kAny) {
#pragma unroll
    for (int i = 0; i < E; ++i) w[i] = p && R::channel(i) < W ? __ldg(p + R::channel(i)) : none;
  } else {
    R::load_vector(p, W, none, w);
  }
#pragma unroll
  for (int q = 0; q < E / 4; ++q)
    sm100::st_shared_v4(dst + (q * N + threadIdx.x) * 16, __float_as_uint(w[4 * q]),
                        __float_as_uint(w[4 * q + 1]), __float_as_uint(w[4 * q + 2]),
                        __float_as_uint(w[4 * q + 3]));
}

// A vector in shared memory.
template <typename T>
struct Piece {
  uint4 v;
  __device__ __forceinline__ explicit Piece(uint32_t at) : v(sm100::ld_shared_v4(at)) {}
  __device__ __forceinline__ F2 two(int k) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (sizeof(T) == 4)
      return F2(__uint_as_float(w[2 * k & 3]), __uint_as_float(w[(2 * k + 1) & 3]));
    else return F2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
  }
};
template <typename T>
__device__ __forceinline__ uint4 pack16(const float2 *y) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (sizeof(T) == 4) w[k] = __float_as_uint(k & 1 ? y[k / 2].y : y[k / 2].x);
    else w[k] = sm100::pack_bf16x2(y[k].x, y[k].y);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void put16(uint32_t at, uint4 v) {
  sm100::st_shared_v4(at, v.x, v.y, v.z, v.w);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int kLeft>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
// This thread's vectors of a row, `live` of them, which starts at `row`, into its place.
template <typename T, int N, int E>
__device__ __forceinline__ void copy_row(uint32_t slot, const T *row, int live) {
  constexpr int kV = 16 / sizeof(T);
  const int lane = threadIdx.x % N;
#pragma unroll
  for (int j = 0; j < E / kV; ++j)
    if (j < live) copy16(slot + (j * N + lane) * 16, row + (j * N + lane) * kV);
}

// ---- rows that start anywhere, and rows that end inside 16 bytes
// Whole 16-byte pieces from the one that the row starts in go into its place; two neighbours
// make a vector.  Of the last piece only what is the row's is read, of the first what is before
// the row too, where that is still the tensor's (`first`: where that starts).
template <typename T, int N, int E>
__device__ __forceinline__ void copy_any(uint32_t slot, const T *row, int W, const void *first) {
  constexpr int kV = 16 / sizeof(T);
  const int lane = threadIdx.x % N;
  const uintptr_t at = reinterpret_cast<uintptr_t>(row);
  const int k = (int)(at & 15), bytes = k + W * (int)sizeof(T);
  const char *piece = reinterpret_cast<const char *>(at - k);
#pragma unroll
  for (int j = 0; j <= E / kV; ++j) {
    const int c = j * N + lane, left = bytes - 16 * c;
    if (left <= 0 || (j == E / kV && lane > 0)) continue;
    if (c == 0 && piece < static_cast<const char *>(first)) {
      for (int e = 0; e < kV && e < W && k + e * (int)sizeof(T) < 16; ++e) {
        const uint32_t to = slot + k + e * (int)sizeof(T);
        if constexpr (sizeof(T) == 4)
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(to), "f"(row[e]) : "memory");
        else
          asm volatile("st.shared.u16 [%0], %1;" ::"r"(to), "h"(__bfloat16_as_ushort(row[e])) : "memory");
      }
    } else {
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(slot + c * 16),
                   "l"(piece + (int64_t)c * 16), "r"(min(left, 16)) : "memory");
    }
  }
}
// All threads of a row.
template <int N>
__device__ __forceinline__ void group_sync() {
  if constexpr (N > 32) sm100::named_sync(1 + threadIdx.x / N, N);
  else if constexpr (N == 32) __syncwarp();
  else __syncwarp(((1u << N) - 1) << (threadIdx.x & 31 & ~(N - 1)));
}
// 16 bytes from `at` of shared memory on, a multiple of sizeof(T) with kWord words after the last
// multiple of 16 (-1: any number).
template <typename T, int kWord>
__device__ __forceinline__ uint4 load_any(uint32_t at) {
  const uint4 lo = sm100::ld_shared_v4(at & ~15u), hi = sm100::ld_shared_v4((at & ~15u) + 16);
  uint32_t w[9] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w, 0};
  if constexpr (kWord < 0) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = at & 8 ? w[i + 2] : w[i];
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = at & 4 ? w[i + 1] : w[i];
  }
  constexpr int k0 = kWord < 0 ? 0 : kWord;
  if constexpr (sizeof(T) == 2)
#pragma unroll
    for (int i = k0; i < k0 + 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], (at & 2) * 8);
  return make_uint4(w[k0], w[k0 + 1], w[k0 + 2], w[k0 + 3]);
}
// f(kWord) for what is read from `at` and multiples of 16 bytes from there.  A warp with one row
// has one of four ways to go.
template <int N, class F>
__device__ __forceinline__ void by_word(uint32_t at, F f) {
  using std::integral_constant;
  if constexpr (N < 32) return f(integral_constant<int, -1>{});
  switch (at >> 2 & 3) {
    case 0: return f(integral_constant<int, 0>{});
    case 1: return f(integral_constant<int, 1>{});
    case 2: return f(integral_constant<int, 2>{});
    default: return f(integral_constant<int, 3>{});
  }
}
// This thread's vectors, `live` of them, of a row that starts at `at`; zeros past the row.
template <typename T, int N, int kCount>
__device__ __forceinline__ void vectors_any(uint32_t at, int live, int W, uint4 (&v)[kCount]) {
  constexpr int kV = 16 / sizeof(T), kPer = 4 / sizeof(T);
  const int lane = threadIdx.x % N;
  by_word<N>(at, [&](auto word) {
#pragma unroll
    for (int j = 0; j < kCount; ++j) {
      v[j] = make_uint4(0, 0, 0, 0);
      if (j < live) v[j] = load_any<T, decltype(word)::value>(at + (j * N + lane) * 16);
    }
  });
#pragma unroll
  for (int j = 0; j < kCount; ++j) {
    const int left = W - (j * N + lane) * kV;
    if (left < kV) {
      const auto cut = [&](uint32_t u, int i) {
        return left >= (i + 1) * kPer ? u : kPer == 2 && left == 2 * i + 1 ? u & 0xffffu : 0u;
      };
      v[j] = make_uint4(cut(v[j].x, 0), cut(v[j].y, 1), cut(v[j].z, 2), cut(v[j].w, 3));
    }
  }
}
// A row of shared memory, on 16 bytes, to `row`: whole 16-byte pieces, and the channels before and
// behind these, a thread each.
template <typename T, int N, int E>
__device__ __forceinline__ void store_any(uint32_t slot, T *row, int W) {
  constexpr int kV = 16 / sizeof(T);
  const int lane = threadIdx.x % N;
  const int before = (int)(reinterpret_cast<uintptr_t>(row) & 15) / (int)sizeof(T);
  const int head = min((kV - before) % kV, W), behind = W - (W - head) % kV;
  by_word<N>(slot - before * (int)sizeof(T), [&](auto word) {
#pragma unroll
    for (int j = 0; j <= E / kV; ++j) {
      const int c0 = (j * N + lane) * kV - before;       // first channel of the piece
      if (c0 >= 0 && c0 + kV <= W)
        *reinterpret_cast<uint4 *>(row + c0) =
            load_any<T, decltype(word)::value>(slot + c0 * (int)sizeof(T));
    }
  });
#pragma unroll
  for (int e0 = 0; e0 < 2 * kV; e0 += N) {
    const int e = e0 + lane, c = e < kV ? e : behind + e - kV;
    if (e < kV ? c < head : e < 2 * kV && c < W) {
      const uint32_t at = slot + c * (int)sizeof(T);
      if constexpr (sizeof(T) == 4) {
        uint32_t u;
        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(u) : "r"(at) : "memory");
        row[c] = __uint_as_float(u);
      } else {
        uint16_t u;
        asm volatile("ld.shared.u16 %0, [%1];" : "=h"(u) : "r"(at) : "memory");
        row[c] = __ushort_as_bfloat16(u);
      }
    }
  }
}

template <typename T, int N, int E, bool kAny>
__global__ void __launch_bounds__(kFwdThreads<N, E>, 1) kda_norm_fwd_ring_kernel(const NormArgs a) {
  using R = Row<T, N, E, true>;
  constexpr int kThreads = kFwdThreads<N, E>, kGroups = kThreads / N, kD = kFwdStages<T, N, E, kAny>;
  static_assert(kD >= 1, "a row ahead");
  constexpr uint32_t kStageBytes = kGroups * kSlot<T, N, E, kAny>;
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ float part[kGroups][2 * kPart<N>];
  const int lane = threadIdx.x % N, live = ((a.W + R::kV - 1) / R::kV - lane + N - 1) / N;
  const uint32_t slot = sm100::smem_u32(ring) + threadIdx.x / N * kSlot<T, N, E, kAny>;
  const uint32_t sm_w = sm100::smem_u32(ring) + kD * kStageBytes, sm_b = sm_w + N * E * 4;
  const int64_t step = (int64_t)gridDim.x * kGroups;
  int64_t row = (int64_t)blockIdx.x * kGroups + threadIdx.x / N;
  const T *x_at = static_cast<const T *>(a.x) + row * a.x_rs;
  const int64_t x_step = step * a.x_rs;
  const auto copy = [&](uint32_t to, const T *from) {
    if constexpr (kAny) copy_any<T, N, E>(to, from, a.W, a.x);
    else copy_row<T, N, E>(to, from, live);
  };
#pragma unroll
  for (int i = 0; i < kD; ++i) {
    if (row + i * step < a.n) copy(slot + i * kStageBytes, x_at + i * x_step);
    sm100::cp_async_commit();
  }
  keep_vector<T, N, E, kAny>(sm_w, a.weight, a.W, 1.f);
  keep_vector<T, N, E, kAny>(sm_b, a.bias, a.W, 0.f);
  __syncthreads();
  const uint32_t my_w = sm_w + lane * 16, my_b = sm_b + lane * 16;
  float *part_at = part[threadIdx.x / N];
  const float inv = 1.f / a.W;
  int stage = 0, turn = 0;
  for (; row < a.n; row += step, turn ^= 1) {
    copies_wait<kD - 1>();
    if constexpr (kAny) group_sync<N>();                 // others' pieces too
    const uint32_t at = slot + stage * kStageBytes, mine = at + lane * 16;
    uint4 v[R::kCount];
    if constexpr (kAny) {
      vectors_any<T, N>(at + (reinterpret_cast<uintptr_t>(x_at) & 15), live, a.W, v);
    } else {
#pragma unroll
      for (int j = 0; j < R::kCount; ++j) {
        v[j] = make_uint4(0, 0, 0, 0);
        if (j < live) v[j] = sm100::ld_shared_v4(mine + j * N * 16);
      }
    }
    R x;
#pragma unroll
    for (int j = 0; j < R::kCount; ++j) {
      x.raw[4 * j] = v[j].x;
      x.raw[4 * j + 1] = v[j].y;
      x.raw[4 * j + 2] = v[j].z;
      x.raw[4 * j + 3] = v[j].w;
    }
    float m = 0.f;
    if (a.center) {
      F2 t[2] = {F2(0.f, 0.f), F2(0.f, 0.f)};
#pragma unroll
      for (int i = 0; i < E / 2; ++i) t[i & 1] = t[i & 1] + x.two(i);
      float s[1] = {(t[0] + t[1]).sum()};
      row_sum<N, 1>(s, part_at);
      m = s[0] * inv;
    }
    const F2 m2(-m, -m);
    F2 t[2] = {F2(0.f, 0.f), F2(0.f, 0.f)};
#pragma unroll
    for (int j = 0; j < R::kCount; ++j)
      if (j < live) {
        if (kAny && (j * N + lane + 1) * R::kV > a.W) {
#pragma unroll
          for (int k = 0; k < R::kV / 2; ++k) {            // past the row x is 0
            const int c = (j * N + lane) * R::kV + 2 * k;
            const F2 d = x.two(j * R::kV / 2 + k) + F2(c < a.W ? -m : 0.f, c + 1 < a.W ? -m : 0.f);
            t[k & 1] = fma2(d, d, t[k & 1]);
          }
        } else {
#pragma unroll
          for (int k = 0; k < R::kV / 2; ++k) {
            const F2 d = x.two(j * R::kV / 2 + k) + m2;
            t[k & 1] = fma2(d, d, t[k & 1]);
          }
        }
      }
    float s[1] = {(t[0] + t[1]).sum()};
    row_sum<N, 1>(s, part_at + (a.center || turn ? kPart<N> : 0));
    const float r = rsqrtf(fmaf(s[0], inv, a.eps));
    if (lane == 0) {
      if (a.mean) a.mean[row] = m;
      if (a.rstd) a.rstd[row] = r;
    }
    const F2 r2(r, r);
    T *out = static_cast<T *>(a.out) + row * a.out_rs;
    if constexpr (kAny && N <= 32) group_sync<N>();      // all have read (longer rows: in their sums)
#pragma unroll
    for (int j = 0; j < R::kCount; ++j)
      if (j < live) {
        float2 y[R::kV / 2];
#pragma unroll
        for (int k = 0; k < R::kV / 2; k += 2) {
          const int q = j * R::kV / 4 + k / 2, i = 2 * q;
          const float4 w = sm100::ld_shared_f32x4(my_w + q * N * 16);
          const float4 b = sm100::ld_shared_f32x4(my_b + q * N * 16);
          y[k] = fma2((x.two(i) + m2) * r2, F2(w.x, w.y), F2(b.x, b.y)).get();
          y[k + 1] = fma2((x.two(i + 1) + m2) * r2, F2(w.z, w.w), F2(b.z, b.w)).get();
        }
        const uint4 packed = pack16<T>(y);
        if constexpr (kAny) put16(mine + j * N * 16, packed);
        else *reinterpret_cast<uint4 *>(out + (j * N + lane) * R::kV) = packed;
      }
    if constexpr (kAny) {
      group_sync<N>();
      store_any<T, N, E>(at, out, a.W);
      group_sync<N>();
    }
    if (row + kD * step < a.n) copy(at, x_at + kD * x_step);   // what has been used may go
    sm100::cp_async_commit();
    x_at += x_step;
    stage = stage + 1 == kD ? 0 : stage + 1;
  }
}

// Floats of a row of the scratch.
__host__ __device__ inline int32_t padded(int32_t W) { return (W + 3) / 4 * 4; }
// A block's sums, its groups' added in their order: rows 2 blockIdx (dw) and 2 blockIdx + 1 (db)
// of the scratch.  dw, db: a thread's, vectors of kV; sums: [2][kGroups][N E] of shared memory.
template <int N, int E, int kGroups, int kV>
__device__ __forceinline__ void leave_sums(const NormArgs &a, const F2 (&dw)[E / 2], const F2 (&db)[E / 2],
                                           float *sums) {
  float *to = a.partial + (int64_t)blockIdx.x * 2 * padded(a.W);
  constexpr int kNext = kGroups * N * E;                 // from dw to db
  float *at = sums + (int)threadIdx.x / N * (N * E) + threadIdx.x % N * kV;
#pragma unroll
  for (int i = 0; i < E; i += 4) {
    float *p = at + i / kV * N * kV + i % kV;
    const float2 w0 = dw[i / 2].get(), w1 = dw[i / 2 + 1].get();
    const float2 b0 = db[i / 2].get(), b1 = db[i / 2 + 1].get();
    *reinterpret_cast<float4 *>(p) = make_float4(w0.x, w0.y, w1.x, w1.y);
    *reinterpret_cast<float4 *>(p + kNext) = make_float4(b0.x, b0.y, b1.x, b1.y);
  }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * a.W; c += blockDim.x) {
    const float *from = sums + (c < a.W ? c : c - a.W + kNext);
    float all = 0.f;
#pragma unroll 16
    for (int p = 0; p < kGroups; ++p) all += from[p * N * E];
    to[c < a.W ? c : c - a.W + padded(a.W)] = all;
  }
}

template <typename T, int N, int E, bool kAny>
__global__ void __launch_bounds__(kBwdThreads, E * N <= kShort ? 2 : 1) kda_norm_bwd_ring_kernel(const NormArgs a) {
  using R = Row<T, N, E, true>;
  constexpr int kGroups = kBwdThreads / N, kD = kBwdStages<T, N, E, kAny>, kV = R::kV;
  static_assert(kD >= 1, "a row ahead");
  constexpr uint32_t kRowBytes = kGroups * kSlot<T, N, E, kAny>;
  static_assert(kD * 2 * kRowBytes + N * E * 4 >= kGroups * N * E * 8, "room for the groups' sums");
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ float part[kGroups][2][2 * kPart<N>];
  latent::pdl_launch_dependents();
  const int lane = threadIdx.x % N, live = ((a.W + kV - 1) / kV - lane + N - 1) / N;
  const uint32_t slot = sm100::smem_u32(ring) + threadIdx.x / N * kSlot<T, N, E, kAny>;
  const int64_t step = (int64_t)gridDim.x * kGroups;
  int64_t row = (int64_t)blockIdx.x * kGroups + threadIdx.x / N;
  const T *x_at = static_cast<const T *>(a.x) + row * a.x_rs;
  const T *g_at = static_cast<const T *>(a.d_out) + row * a.do_rs;
  const int64_t x_step = step * a.x_rs, g_step = step * a.do_rs;
  // The addresses stay at the row itself where they tell how it lies, and where there are few
  // registers; else they are the next copy's (16384 x 7168 bf16 113.5 -> 110.5 us).
  constexpr bool kHere = kAny || N * E <= kShort;
  const auto copy = [&](uint32_t to, int ahead) {
    if constexpr (kAny) {
      copy_any<T, N, E>(to, x_at + ahead * x_step, a.W, a.x);
      copy_any<T, N, E>(to + kRowBytes, g_at + ahead * g_step, a.W, a.d_out);
    } else {
      copy_row<T, N, E>(to, x_at + (kHere ? ahead : 0) * x_step, live);
      copy_row<T, N, E>(to + kRowBytes, g_at + (kHere ? ahead : 0) * g_step, live);
    }
  };
#pragma unroll
  for (int i = 0; i < kD; ++i) {
    if (row + i * step < a.n) copy(slot + 2 * i * kRowBytes, i);
    sm100::cp_async_commit();
    if constexpr (!kHere) {
      x_at += x_step;
      g_at += g_step;
    }
  }
  keep_vector<T, N, E, kAny>(sm100::smem_u32(ring) + kD * 2 * kRowBytes, a.weight, a.W, 1.f);
  __syncthreads();
  const uint32_t my_w = sm100::smem_u32(ring) + kD * 2 * kRowBytes + lane * 16;
  const float inv = 1.f / a.W;
  F2 dw[E / 2], db[E / 2];
#pragma unroll
  for (int i = 0; i < E / 2; ++i) dw[i] = db[i] = F2(0.f, 0.f);
  int stage = 0, turn = 0;
  float m = 0.f, r = 0.f;
  if (row < a.n) {
    if (a.center) m = a.mean[row];
    r = a.rstd[row];
  }
  for (; row < a.n; row += step, turn ^= 1) {
    float m_next = 0.f, r_next = 0.f;
    if (row + step < a.n) {
      if (a.center) m_next = a.mean[row + step];
      r_next = a.rstd[row + step];
    }
    copies_wait<kD - 1>();
    const uint32_t at = slot + 2 * stage * kRowBytes, mine = at + lane * 16;
    if constexpr (kAny) {                                // vectors to their places, x, then g
      group_sync<N>();                                   // others' pieces too
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        const uint32_t place = at + which * kRowBytes;
        const uint32_t from = place + (reinterpret_cast<uintptr_t>(which ? g_at : x_at) & 15);
        uint4 v[R::kCount];
        vectors_any<T, N>(from, live, a.W, v);
        group_sync<N>();
#pragma unroll
        for (int j = 0; j < R::kCount; ++j)
          if (j < live) put16(place + (j * N + lane) * 16, v[j]);
      }
    }
    // A vector at a time, and all again for the second half: registers hold dw and db.
    const F2 m2(-m, -m), r2(r, r);
    F2 s0(0.f, 0.f), s1(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < R::kCount; ++j)
      if (j < live) {
        const Piece<T> x(mine + j * N * 16), g(mine + kRowBytes + j * N * 16);
#pragma unroll
        for (int k = 0; k < kV / 2; k += 2) {
          const float4 w = sm100::ld_shared_f32x4(my_w + (j * kV / 4 + k / 2) * N * 16);
#pragma unroll
          for (int l = k; l < k + 2; ++l) {
            const int i = j * kV / 2 + l;
            const F2 z = (x.two(l) + m2) * r2, d = g.two(l);
            const F2 e = d * (l == k ? F2(w.x, w.y) : F2(w.z, w.w));
            dw[i] = fma2(d, z, dw[i]);
            db[i] = db[i] + d;
            s0 = s0 + e;
            s1 = fma2(e, z, s1);
          }
        }
      }
    float s[2] = {s0.sum(), s1.sum()};
    row_sum<N, 2>(s, part[threadIdx.x / N][turn]);
    const float c1 = a.center ? -s[0] * inv : 0.f, c2 = -s[1] * inv;
    const F2 c1_2(c1, c1), c2_2(c2, c2);
    T *d_x = static_cast<T *>(a.d_x) + row * a.dx_rs;
#pragma unroll
    for (int j = 0; j < R::kCount; ++j)
      if (j < live) {
        const Piece<T> x(mine + j * N * 16), g(mine + kRowBytes + j * N * 16);
        float2 y[kV / 2];
#pragma unroll
        for (int k = 0; k < kV / 2; k += 2) {
          const float4 w = sm100::ld_shared_f32x4(my_w + (j * kV / 4 + k / 2) * N * 16);
#pragma unroll
          for (int l = k; l < k + 2; ++l) {
            const F2 z = (x.two(l) + m2) * r2;
            const F2 e = fma2(g.two(l), l == k ? F2(w.x, w.y) : F2(w.z, w.w), c1_2);
            y[l] = (fma2(z, c2_2, e) * r2).get();
          }
        }
        const uint4 packed = pack16<T>(y);
        if constexpr (kAny) put16(mine + j * N * 16, packed);
        else *reinterpret_cast<uint4 *>(d_x + (j * N + lane) * kV) = packed;
      }
    if constexpr (kAny) {
      group_sync<N>();
      store_any<T, N, E>(at, d_x, a.W);
      group_sync<N>();
    }
    if (row + kD * step < a.n) copy(at, kD);             // what has been used may go
    sm100::cp_async_commit();
    x_at += x_step;
    g_at += g_step;
    stage = stage + 1 == kD ? 0 : stage + 1;
    m = m_next;
    r = r_next;
  }
  copies_wait<0>();
  __syncthreads();                                       // the ring is free
  if (!a.partial) return;
  leave_sums<N, E, kGroups, kV>(a, dw, db, reinterpret_cast<float *>(ring));
}

// Sums of the blocks' rows, in their order: 32 stretches of consecutive blocks, a warp each,
// then the stretches.  Block (x: 128 channels, y: dw, db).
constexpr int kJoinWarps = 32;
__global__ void __launch_bounds__(32 * kJoinWarps)
kda_norm_join_kernel(const float *__restrict__ partial, int32_t blocks, int32_t W, float *d_weight,
                     float *d_bias) {
  __shared__ float4 s[kJoinWarps][32];
  latent::pdl_wait();
  float *out = blockIdx.y ? d_bias : d_weight;
  if (!out) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = (blockIdx.x * 32 + lane) * 4;
  const int per = (blocks + kJoinWarps - 1) / kJoinWarps;
  const int b0 = warp * per, b1 = min(blocks, b0 + per);
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kBatch = 5;                // rows in flight
  for (int b = b0; b < b1; b += kBatch) {
    float4 x[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (b + i < b1 && c < W)
        x[i] = *reinterpret_cast<const float4 *>(
            partial + ((int64_t)(b + i) * 2 + blockIdx.y) * padded(W) + c);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      sum.x += x[i].x;
      sum.y += x[i].y;
      sum.z += x[i].z;
      sum.w += x[i].w;
    }
  }
  s[warp][lane] = sum;
  __syncthreads();
  if (threadIdx.x >= 128) return;
  const int o = blockIdx.x * 128 + threadIdx.x;
  if (o >= W) return;
  float all = 0.f;
#pragma unroll
  for (int i = 0; i < kJoinWarps; ++i) all += reinterpret_cast<const float *>(s[i])[threadIdx.x];
  out[o] = all;
}

int sms() { return latent::sm_count() > 0 ? latent::sm_count() : 1; }

// Blocks of the gradient at most: one an SM, of short rows four, whose sums are short too.
int64_t most_blocks(int32_t W) { return W <= kShort ? 4 * sms() : sms(); }
int bwd_blocks(int64_t n, int32_t W, int N) {
  const int64_t need = (n + kBwdThreads / N - 1) / (kBwdThreads / N), most = most_blocks(W);
  return (int)(need < most ? need : most);
}

// Rows enough that every group has some to walk over.
template <int N, int E>
bool many(int64_t n) { return n >= (int64_t)4 * (kFwdThreads<N, E> / N) * sms(); }
// The same for rows that start anywhere, against single channels: one row a group, but for the
// longest (608 x 7169 bf16 9.4 us and 11.2; 4864 x 999 8.8 and 9.2; 304 x 16383 13.3 and 10.2).
// Not where few of a group's threads have a vector of their own and its steps tell: 65 to 256
// channels (524288 x 100 bf16 105 us, by single channels 82), fp32 513 to 1024 (32768 x 999 76, 56).
template <int N, int E>
bool many_any(int64_t n, int32_t W) {
  constexpr int kGroups = kFwdThreads<N, E> / N;
  if (E == 8 && N >= 16) return false;
  if (N == 128 && W <= 1024) return false;
  return n >= (int64_t)(kGroups > 4 ? kGroups : 4) * sms();
}

template <typename T, int N, int E, bool kAny>
cudaError_t fwd_ring(const NormArgs &a, cudaStream_t stream) {
  constexpr int kThreads = kFwdThreads<N, E>, kD = kFwdStages<T, N, E, kAny>;
  constexpr int kBytes = kD * (kThreads / N) * kSlot<T, N, E, kAny> + 2 * N * E * 4;
  if (!latent::kernel_ready<kda_norm_fwd_ring_kernel<T, N, E, kAny>>(kBytes, 0)) return cudaErrorNotSupported;
  kda_norm_fwd_ring_kernel<T, N, E, kAny><<<sms(), kThreads, kBytes, stream>>>(a);
  return cudaGetLastError();
}
template <typename T, int N, int E, bool kVector>
cudaError_t fwd_direct(const NormArgs &a, cudaStream_t stream) {
  constexpr int kRows = kBlock<N> / N;
  const int64_t blocks = (a.n + kRows - 1) / kRows;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  kda_norm_fwd_kernel<T, N, E, kVector><<<(unsigned)blocks, kBlock<N>, 0, stream>>>(a);
  return cudaGetLastError();
}

template <typename T, int N, int E, bool kAny>
cudaError_t bwd(const NormArgs &a, cudaStream_t stream) {
  constexpr int kD = kBwdStages<T, N, E, kAny>;
  constexpr int kBytes = kD * 2 * (kBwdThreads / N) * kSlot<T, N, E, kAny> + N * E * 4;
  if (!latent::kernel_ready<kda_norm_bwd_ring_kernel<T, N, E, kAny>>(kBytes, 0))
    return cudaErrorNotSupported;
  const int blocks = bwd_blocks(a.n, a.W, N);
  kda_norm_bwd_ring_kernel<T, N, E, kAny><<<blocks, kBwdThreads, kBytes, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.partial) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.W + 127) / 128), 2);
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kda_norm_join_kernel, (const float *)a.partial, (int32_t)blocks, a.W,
                            a.d_weight, a.d_bias);
}

bool rows_of_16(const void *p, int64_t rs, int esz) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && rs * esz % 16 == 0;
}

// Threads of a row: four to 32 for a short one with eight channels each, else the fewest that hold
// it with 64 bytes of it each, of the longest fp32 rows 128.
template <typename T, class F>
cudaError_t classes(int32_t W, F go) {
  using std::integral_constant;
  constexpr integral_constant<int, 32> warp{};
  constexpr integral_constant<int, 512> half{};
  constexpr integral_constant<int, 8> least{};
  constexpr integral_constant<int, 64 / sizeof(T)> E{};
  static_assert(kShort == 32 * 8, "a short row is a warp's with eight channels each");
  if (W <= kShort / 8) return go(integral_constant<int, 4>{}, least);
  if (W <= kShort / 4) return go(integral_constant<int, 8>{}, least);
  if (W <= kShort / 2) return go(integral_constant<int, 16>{}, least);
  if (W <= kShort) return go(warp, least);
  if constexpr (E > 16)
    if (W <= 32 * 16) return go(warp, integral_constant<int, 16>{});
  if (W <= 32 * E) return go(warp, E);
  if (W <= 128 * E) return go(integral_constant<int, 128>{}, E);
  if (W <= 256 * E) return go(integral_constant<int, 256>{}, E);
  if (W <= 512 * E) return go(half, E);
  if constexpr (512 * E < kNormMax) return go(half, integral_constant<int, kNormMax / 512>{});
  return cudaErrorInvalidValue;
}
// The same for few rows that start anywhere: eight channels each, of the longest 16.
template <typename T, class F>
cudaError_t single_classes(int32_t W, F go) {
  using std::integral_constant;
  constexpr integral_constant<int, 1024> all{};
  constexpr integral_constant<int, 8> least{};
  if (W <= kShort / 2) return go(integral_constant<int, 16>{}, least);
  if (W <= kShort) return go(integral_constant<int, 32>{}, least);
  if (W <= 128 * least) return go(integral_constant<int, 128>{}, least);
  if (W <= 256 * least) return go(integral_constant<int, 256>{}, least);
  if (W <= 512 * least) return go(integral_constant<int, 512>{}, least);
  if (W <= 1024 * least) return go(all, least);
  return go(all, integral_constant<int, kNormMax / 1024>{});
}

// vector: rows start on 16 bytes; whole: and end there.  The gradient's rows go by the ring at any
// number (few rows that start anywhere, 16 x 7169 bf16 10.9 us: by single channels 9.3).
template <typename T>
cudaError_t run_fwd(const NormArgs &a, bool vector, bool whole, cudaStream_t stream) {
  bool few = false;
  const cudaError_t e = classes<T>(a.W, [&](auto n, auto e) {
    constexpr int N = decltype(n)::value, E = decltype(e)::value;
    if (whole && many<N, E>(a.n)) return fwd_ring<T, N, E, false>(a, stream);
    if (!whole && many_any<N, E>(a.n, a.W)) return fwd_ring<T, N, E, true>(a, stream);
    if (vector) return fwd_direct<T, N, E, true>(a, stream);
    few = true;
    return cudaSuccess;
  });
  if (!few) return e;
  return single_classes<T>(a.W, [&](auto n, auto e) {
    return fwd_direct<T, decltype(n)::value, decltype(e)::value, false>(a, stream);
  });
}
template <typename T>
cudaError_t run_bwd(const NormArgs &a, bool whole, cudaStream_t stream) {
  return classes<T>(a.W, [&](auto n, auto e) {
    constexpr int N = decltype(n)::value, E = decltype(e)::value;
    return whole ? bwd<T, N, E, false>(a, stream) : bwd<T, N, E, true>(a, stream);
  });
}

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs &a, cudaStream_t stream) {
  if (a.n == 0) return cudaSuccess;
  const int esz = a.bf16 ? 2 : 4;
  const bool vector = rows_of_16(a.x, a.x_rs, esz) && rows_of_16(a.out, a.out_rs, esz) &&
                      rows_of_16(a.weight, 0, 1) && rows_of_16(a.bias, 0, 1);
  const bool whole = vector && a.W * esz % 16 == 0;
  return a.bf16 ? run_fwd<__nv_bfloat16>(a, vector, whole, stream)
                : run_fwd<float>(a, vector, whole, stream);
}

size_t norm_bwd_scratch_bytes(int64_t n, int32_t W, bool bf16) {
  (void)bf16;
  const int64_t most = most_blocks(W);
  return (size_t)(n < most ? n : most) * 2 * padded(W) * sizeof(float);
}

cudaError_t launch_norm_bwd(const NormArgs &a, cudaStream_t stream) {
  if (a.n == 0) {
    for (float *p : {a.d_weight, a.d_bias})
      if (p) {
        const cudaError_t e = cudaMemsetAsync(p, 0, (size_t)a.W * 4, stream);
        if (e != cudaSuccess) return e;
      }
    return cudaSuccess;
  }
  const int esz = a.bf16 ? 2 : 4;
  const bool whole = a.W * esz % 16 == 0 && rows_of_16(a.x, a.x_rs, esz) &&
                     rows_of_16(a.d_out, a.do_rs, esz) && rows_of_16(a.d_x, a.dx_rs, esz) &&
                     rows_of_16(a.weight, 0, 1);
  return a.bf16 ? run_bwd<__nv_bfloat16>(a, whole, stream) : run_bwd<float>(a, whole, stream);
}

}  // namespace kda
