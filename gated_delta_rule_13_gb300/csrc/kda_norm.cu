// Norm over a row's channels, with or without its mean (kda_norm_fwd), and its gradient
// (kda_norm_bwd).
//
//   m = mean x (0 without), r = 1 / sqrt(mean (x - m)^2 + eps),  z = (x - m) r
//   y = z w + b
//   dx = r (w g - mean(w g) - z mean(w g z))   (without the mean: no second term)
//   dw = sum over rows of g z,  db = sum over rows of g
//
// Bound by HBM: two passes of bytes forward, three back.  A row is read once: by half a warp or
// up to 512 threads, into registers (few rows) or, many rows, some rows ahead into shared memory.
// The variance is the mean square of what the mean leaves, from the row on chip, so that a mean
// far from zero costs no digits.  Statistics and sums are fp32; values are taken in pairs, which
// halves the instructions (with one at a time the gradient of 16384 x 7168 was bound by them:
// 167 us).  The gradient's blocks walk over the rows with the sums of dw and db in registers and
// leave one pair of rows each in the workspace; a second kernel adds these in the blocks' order,
// so that results do not vary between calls.
//
// Measured (cold): 16384 x 7168 bf16 forward 75 us (6.3 TB/s), gradient 114 us (6.2); gradient of
// 16384 x 512 fp32 22.8 us (4.4), of which the two sums are 4.5; 64 x 7168 2.9 us; 1 M x 128 bf16
// 88 us (6.1).  Rows that do not lie on 16 bytes go one channel at a time: 8192 x 7169 bf16 152 and
// 268 us (1.5 and 1.3 TB/s).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "kda_latent_tc.cuh"
#include "kda_rows.h"

namespace kda {
namespace {

constexpr int kShort = 256;              // channels of a short row: a warp's or half a warp's

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

// One row a group of N threads, straight from memory: for few rows, and rows whose address or
// distance is no multiple of 16 bytes.
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
template <typename T, int N, int E>
constexpr int kFwdStages = stages(kFwdThreads<N, E> *E *(int)sizeof(T), 2 * N *E * 4);
template <typename T, int N, int E>
constexpr int kBwdStages = stages(2 * kBwdThreads * E * (int)sizeof(T), N * E * 4);

// An fp32 vector [W] into shared memory, laid out as threads read it: [E / 4][N] 16 bytes.
template <typename T, int N, int E>
__device__ __forceinline__ void keep_vector(uint32_t dst, const float *p, int W, float none) {
  if (threadIdx.x >= N) return;
  float w[E];
  Row<T, N, E, true>::load_vector(p, W, none, w);
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
__device__ __forceinline__ void store16(T *to, const float2 *y) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (sizeof(T) == 4) w[k] = __float_as_uint(k & 1 ? y[k / 2].y : y[k / 2].x);
    else w[k] = sm100::pack_bf16x2(y[k].x, y[k].y);
  }
  *reinterpret_cast<uint4 *>(to) = make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int kLeft>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}
// This thread's vectors of a row, `live` of them, which starts at `row` for its first.
template <typename T, int N, int E, int kThreads>
__device__ __forceinline__ void copy_row(uint32_t dst, const T *row, int live) {
  constexpr int kV = 16 / sizeof(T);
#pragma unroll
  for (int j = 0; j < E / kV; ++j)
    if (j < live) copy16(dst + j * kThreads * 16, row + j * N * kV);
}

template <typename T, int N, int E>
__global__ void __launch_bounds__(kFwdThreads<N, E>, 1) kda_norm_fwd_ring_kernel(const NormArgs a) {
  using R = Row<T, N, E, true>;
  constexpr int kThreads = kFwdThreads<N, E>, kGroups = kThreads / N, kD = kFwdStages<T, N, E>;
  static_assert(kD >= 1, "a row ahead");
  constexpr uint32_t kStageBytes = kThreads * E * sizeof(T);
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ float part[kGroups][2 * kPart<N>];
  const int lane = threadIdx.x % N, live = (a.W / R::kV - lane + N - 1) / N;
  const uint32_t mine = sm100::smem_u32(ring) + threadIdx.x * 16;
  const uint32_t sm_w = sm100::smem_u32(ring) + kD * kStageBytes, sm_b = sm_w + N * E * 4;
  const int64_t step = (int64_t)gridDim.x * kGroups;
  int64_t row = (int64_t)blockIdx.x * kGroups + threadIdx.x / N;
  const T *x_at = static_cast<const T *>(a.x) + row * a.x_rs + lane * R::kV;
  const int64_t x_step = step * a.x_rs;
#pragma unroll
  for (int i = 0; i < kD; ++i) {
    if (row + i * step < a.n)
      copy_row<T, N, E, kThreads>(mine + i * kStageBytes, x_at + i * x_step, live);
    sm100::cp_async_commit();
  }
  x_at += kD * x_step;
  keep_vector<T, N, E>(sm_w, a.weight, a.W, 1.f);
  keep_vector<T, N, E>(sm_b, a.bias, a.W, 0.f);
  __syncthreads();
  const uint32_t my_w = sm_w + lane * 16, my_b = sm_b + lane * 16;
  float *part_at = part[threadIdx.x / N];
  const float inv = 1.f / a.W;
  int stage = 0, turn = 0;
  for (; row < a.n; row += step, turn ^= 1) {
    copies_wait<kD - 1>();
    const uint32_t at = mine + stage * kStageBytes;
    R x;
#pragma unroll
    for (int j = 0; j < R::kCount; ++j) {
      uint4 v = make_uint4(0, 0, 0, 0);
      if (j < live) v = sm100::ld_shared_v4(at + j * kThreads * 16);
      x.raw[4 * j] = v.x;
      x.raw[4 * j + 1] = v.y;
      x.raw[4 * j + 2] = v.z;
      x.raw[4 * j + 3] = v.w;
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
      if (j < live)
#pragma unroll
        for (int k = 0; k < R::kV / 2; ++k) {
          const F2 d = x.two(j * R::kV / 2 + k) + m2;
          t[k & 1] = fma2(d, d, t[k & 1]);
        }
    float v[1] = {(t[0] + t[1]).sum()};
    row_sum<N, 1>(v, part_at + (a.center || turn ? kPart<N> : 0));
    const float r = rsqrtf(fmaf(v[0], inv, a.eps));
    if (lane == 0) {
      if (a.mean) a.mean[row] = m;
      if (a.rstd) a.rstd[row] = r;
    }
    const F2 r2(r, r);
    T *out = static_cast<T *>(a.out) + row * a.out_rs + lane * R::kV;
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
        store16(out + j * N * R::kV, y);
      }
    if (row + kD * step < a.n) copy_row<T, N, E, kThreads>(at, x_at, live);  // what has been used may go
    sm100::cp_async_commit();
    x_at += x_step;
    stage = stage + 1 == kD ? 0 : stage + 1;
  }
}

// First half of a row's gradient: the sums of w g and w g z, and this row's part of dw, db.
// four(q): weights of this thread's channels 4 q ... 4 q + 3.
template <int N, int E, class R, class F>
__device__ __forceinline__ void grad_sums(const NormArgs &a, const R &x, const R &g, float m, float r,
                                          F four, float (&dw)[E], float (&db)[E], float *part,
                                          float &c1, float &c2) {
  const float inv = 1.f / a.W;
  float s[2] = {0.f, 0.f};
#pragma unroll
  for (int q = 0; q < E / 4; ++q) {
    const float4 w4 = four(q);
    const float w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = 4 * q + k;
      // past the row g is 0, and z, with no infinity, is of no account
      const float z = R::channel(i) < a.W ? (x.get(i) - m) * r : 0.f, d = g.get(i), e = d * w[k];
      dw[i] = fmaf(d, z, dw[i]);
      db[i] += d;
      s[0] += e;
      s[1] = fmaf(e, z, s[1]);
    }
  }
  row_sum<N, 2>(s, part);
  c1 = a.center ? s[0] * inv : 0.f;
  c2 = s[1] * inv;
}
template <int N, int E, class R, class F, class T>
__device__ __forceinline__ void grad_finish(const NormArgs &a, const R &x, const R &g, float m, float r,
                                            float c1, float c2, F four, T *d_x) {
  float4 w4;
  R::store(d_x, a.W, [&](int i) {
    if (i % 2 == 0) w4 = four(i / 2);
    const float z0 = (x.get(2 * i) - m) * r, z1 = (x.get(2 * i + 1) - m) * r;
    return make_float2(r * (g.get(2 * i) * (i % 2 ? w4.z : w4.x) - c1 - z0 * c2),
                       r * (g.get(2 * i + 1) * (i % 2 ? w4.w : w4.y) - c1 - z1 * c2));
  });
}
// A block's sums, its groups' added in their order: rows 2 blockIdx (dw) and 2 blockIdx + 1 (db)
// of the scratch.  sums: [2][kGroups][W], where there are several; dw[i], db[i]: functions.
template <int N, int E, int kGroups, class R, class F, class G>
__device__ __forceinline__ void leave_sums(const NormArgs &a, F dw, G db, float *sums) {
  float *to = a.partial + (int64_t)blockIdx.x * 2 * a.W;
  float *at = kGroups > 1 ? sums + (int)threadIdx.x / N * a.W : to;
  const int next = kGroups > 1 ? kGroups * a.W : a.W;    // from dw to db
#pragma unroll
  for (int i = 0; i < E; ++i)
    if (R::channel(i) < a.W) {
      at[R::channel(i)] = dw(i);
      at[next + R::channel(i)] = db(i);
    }
  if (kGroups == 1) return;
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * a.W; c += blockDim.x) {
    const float *from = sums + (c < a.W ? c : c - a.W + next);
    float all = 0.f;
#pragma unroll 16
    for (int p = 0; p < kGroups; ++p) all += from[p * a.W];
    to[c] = all;
  }
}

// Rows whose address or distance is no multiple of 16 bytes, one channel at a time.
constexpr int kSingleThreads = 1024;
template <typename T, int N, int E>
__global__ void __launch_bounds__(kSingleThreads, 1) kda_norm_bwd_kernel(const NormArgs a) {
  using R = Row<T, N, E, false>;
  constexpr int kGroups = kSingleThreads / N;
  __shared__ float part[kGroups][2][2 * kPart<N>];
  extern __shared__ float sums[];                        // [2][kGroups][W], where there are several
  latent::pdl_launch_dependents();
  float dw[E], db[E];
#pragma unroll
  for (int i = 0; i < E; ++i) dw[i] = db[i] = 0.f;
  const auto four = [&](int q) {
    const auto one = [&](int i) {
      return a.weight && R::channel(i) < a.W ? __ldg(a.weight + R::channel(i)) : 1.f;
    };
    return make_float4(one(4 * q), one(4 * q + 1), one(4 * q + 2), one(4 * q + 3));
  };
  int turn = 0;
  for (int64_t row = (int64_t)blockIdx.x * kGroups + threadIdx.x / N; row < a.n;
       row += (int64_t)gridDim.x * kGroups, turn ^= 1) {
    R x, g;
    x.load(static_cast<const T *>(a.x) + row * a.x_rs, a.W);
    g.load(static_cast<const T *>(a.d_out) + row * a.do_rs, a.W);
    const float m = a.center ? a.mean[row] : 0.f, r = a.rstd[row];
    float c1, c2;
    grad_sums<N, E>(a, x, g, m, r, four, dw, db, part[threadIdx.x / N][turn], c1, c2);
    grad_finish<N, E>(a, x, g, m, r, c1, c2, four, static_cast<T *>(a.d_x) + row * a.dx_rs);
  }
  if (!a.partial) return;
  leave_sums<N, E, kGroups, R>(a, [&](int i) { return dw[i]; }, [&](int i) { return db[i]; }, sums);
}

template <typename T, int N, int E>
__global__ void __launch_bounds__(kBwdThreads, E * N <= kShort ? 2 : 1) kda_norm_bwd_ring_kernel(const NormArgs a) {
  using R = Row<T, N, E, true>;
  constexpr int kGroups = kBwdThreads / N, kD = kBwdStages<T, N, E>, kV = R::kV;
  static_assert(kD >= 1, "a row ahead");
  constexpr uint32_t kRowBytes = kBwdThreads * E * sizeof(T);
  extern __shared__ __align__(128) unsigned char ring[];
  __shared__ float part[kGroups][2][2 * kPart<N>];
  latent::pdl_launch_dependents();
  const int lane = threadIdx.x % N, live = (a.W / kV - lane + N - 1) / N;
  const uint32_t mine = sm100::smem_u32(ring) + threadIdx.x * 16;
  const int64_t step = (int64_t)gridDim.x * kGroups;
  int64_t row = (int64_t)blockIdx.x * kGroups + threadIdx.x / N;
  const T *x_at = static_cast<const T *>(a.x) + row * a.x_rs + lane * kV;
  const T *g_at = static_cast<const T *>(a.d_out) + row * a.do_rs + lane * kV;
#pragma unroll
  for (int i = 0; i < kD; ++i) {
    if (row + i * step < a.n) {
      const uint32_t to = mine + 2 * i * kRowBytes;
      copy_row<T, N, E, kBwdThreads>(to, x_at, live);
      copy_row<T, N, E, kBwdThreads>(to + kRowBytes, g_at, live);
    }
    sm100::cp_async_commit();
    x_at += step * a.x_rs;
    g_at += step * a.do_rs;
  }
  keep_vector<T, N, E>(sm100::smem_u32(ring) + kD * 2 * kRowBytes, a.weight, a.W, 1.f);
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
    // A vector at a time, and all again for the second half: registers hold dw and db.
    const uint32_t at = mine + 2 * stage * kRowBytes;
    const F2 m2(-m, -m), r2(r, r);
    F2 s0(0.f, 0.f), s1(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < R::kCount; ++j)
      if (j < live) {
        const Piece<T> x(at + j * kBwdThreads * 16), g(at + kRowBytes + j * kBwdThreads * 16);
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
    T *d_x = static_cast<T *>(a.d_x) + row * a.dx_rs + lane * kV;
#pragma unroll
    for (int j = 0; j < R::kCount; ++j)
      if (j < live) {
        const Piece<T> x(at + j * kBwdThreads * 16), g(at + kRowBytes + j * kBwdThreads * 16);
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
        store16(d_x + j * N * kV, y);
      }
    if (row + kD * step < a.n) {                         // what has been used may go
      copy_row<T, N, E, kBwdThreads>(at, x_at, live);
      copy_row<T, N, E, kBwdThreads>(at + kRowBytes, g_at, live);
    }
    sm100::cp_async_commit();
    x_at += step * a.x_rs;
    g_at += step * a.do_rs;
    stage = stage + 1 == kD ? 0 : stage + 1;
    m = m_next;
    r = r_next;
  }
  copies_wait<0>();
  __syncthreads();                                       // the ring is free
  if (!a.partial) return;
  const auto one = [](const F2 (&v)[E / 2], int i) { return i % 2 ? v[i / 2].get().y : v[i / 2].get().x; };
  leave_sums<N, E, kGroups, R>(a, [&](int i) { return one(dw, i); }, [&](int i) { return one(db, i); },
                               reinterpret_cast<float *>(ring));
}

// Sums of the blocks' rows, in their order: 32 stretches of consecutive blocks, a warp each,
// then the stretches.  Block (x: 32 V channels, y: dw, db).
constexpr int kJoinWarps = 32;
template <int V>
__global__ void __launch_bounds__(32 * kJoinWarps)
kda_norm_join_kernel(const float *__restrict__ partial, int32_t blocks, int32_t W, float *d_weight,
                     float *d_bias) {
  __shared__ float s[kJoinWarps][32 * V];
  latent::pdl_wait();
  float *out = blockIdx.y ? d_bias : d_weight;
  if (!out) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = (blockIdx.x * 32 + lane) * V;
  const int per = (blocks + kJoinWarps - 1) / kJoinWarps;
  const int b0 = warp * per, b1 = min(blocks, b0 + per);
  float sum[V];
#pragma unroll
  for (int k = 0; k < V; ++k) sum[k] = 0.f;
  constexpr int kBatch = 5;                // rows in flight
  for (int b = b0; b < b1; b += kBatch) {
    float x[kBatch][V];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const float *at = partial + ((int64_t)(b + i) * 2 + blockIdx.y) * W + c;
      const bool live = b + i < b1 && c < W;
      if constexpr (V == 4) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (live) v = *reinterpret_cast<const float4 *>(at);
        x[i][0] = v.x;
        x[i][1] = v.y;
        x[i][2] = v.z;
        x[i][3] = v.w;
      } else {
        x[i][0] = live ? *at : 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
#pragma unroll
      for (int k = 0; k < V; ++k) sum[k] += x[i][k];
  }
#pragma unroll
  for (int k = 0; k < V; ++k) s[warp][lane * V + k] = sum[k];
  __syncthreads();
  if (threadIdx.x >= 32 * V) return;
  const int o = blockIdx.x * 32 * V + threadIdx.x;
  if (o >= W) return;
  float all = 0.f;
#pragma unroll
  for (int i = 0; i < kJoinWarps; ++i) all += s[i][threadIdx.x];
  out[o] = all;
}

int sms() { return latent::sm_count() > 0 ? latent::sm_count() : 1; }

// Blocks of the gradient at most: one an SM, of short rows four, whose sums are short too.
int64_t most_blocks(int32_t W) { return W <= kShort ? 4 * sms() : sms(); }
template <int kThreads>
int bwd_blocks(int64_t n, int32_t W, int N) {
  const int64_t need = (n + kThreads / N - 1) / (kThreads / N), most = most_blocks(W);
  return (int)(need < most ? need : most);
}

template <typename T, int N, int E, bool kVector>
cudaError_t fwd(const NormArgs &a, cudaStream_t stream) {
  constexpr int kRows = kBlock<N> / N;
  if constexpr (kVector && kFwdStages<T, N, E> >= 1) {
    constexpr int kThreads = kFwdThreads<N, E>, kGroups = kThreads / N;
    constexpr int kBytes = kFwdStages<T, N, E> * kThreads * E * (int)sizeof(T) + 2 * N * E * 4;
    // Rows enough that every group has some to walk over.
    if (a.W % (16 / (int)sizeof(T)) == 0 && a.n >= (int64_t)4 * kGroups * sms() &&
        latent::kernel_ready<kda_norm_fwd_ring_kernel<T, N, E>>(kBytes, 0)) {
      kda_norm_fwd_ring_kernel<T, N, E><<<sms(), kThreads, kBytes, stream>>>(a);
      return cudaGetLastError();
    }
  }
  const int64_t blocks = (a.n + kRows - 1) / kRows;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  kda_norm_fwd_kernel<T, N, E, kVector><<<(unsigned)blocks, kBlock<N>, 0, stream>>>(a);
  return cudaGetLastError();
}

template <typename T, int N, int E, bool kVector>
cudaError_t bwd(const NormArgs &a, cudaStream_t stream) {
  int blocks;
  if constexpr (kVector) {
    constexpr int kBytes = kBwdStages<T, N, E> * 2 * kBwdThreads * E * (int)sizeof(T) + N * E * 4;
    if (!latent::kernel_ready<kda_norm_bwd_ring_kernel<T, N, E>>(kBytes, 0))
      return cudaErrorNotSupported;
    blocks = bwd_blocks<kBwdThreads>(a.n, a.W, N);
    kda_norm_bwd_ring_kernel<T, N, E><<<blocks, kBwdThreads, kBytes, stream>>>(a);
  } else {
    blocks = bwd_blocks<kSingleThreads>(a.n, a.W, N);
    const size_t smem = kSingleThreads / N > 1 ? (size_t)(kSingleThreads / N) * a.W * 8 : 0;
    if (smem > 0 && !latent::kernel_ready<kda_norm_bwd_kernel<T, N, E>>(2 * kSingleThreads * E * 4, 0))
      return cudaErrorNotSupported;
    kda_norm_bwd_kernel<T, N, E><<<blocks, kSingleThreads, smem, stream>>>(a);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.partial) return e;
  const int V = a.W % 4 == 0 ? 4 : 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.W + 32 * V - 1) / (32 * V)), 2);
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, V == 4 ? kda_norm_join_kernel<4> : kda_norm_join_kernel<1>,
                            (const float *)a.partial, (int32_t)blocks, a.W, a.d_weight, a.d_bias);
}

bool rows_of_16(const void *p, int64_t rs, int esz) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && rs * esz % 16 == 0;
}

// Threads of a row.  With vectors: half a warp or a warp for a short one, the fewest that hold it with 64 bytes
// of it each, of the longest fp32 rows 128.  Single channels: eight each, of the longest 16, which
// leaves registers for 1024 threads an SM.
template <typename T, bool kVector, bool kForward>
cudaError_t pick(const NormArgs &a, cudaStream_t stream) {
  const auto go = [&](auto n, auto e) {
    if constexpr (kForward) return fwd<T, decltype(n)::value, decltype(e)::value, kVector>(a, stream);
    else return bwd<T, decltype(n)::value, decltype(e)::value, kVector>(a, stream);
  };
  using std::integral_constant;
  constexpr integral_constant<int, 32> warp{};
  constexpr integral_constant<int, 128> four{};
  constexpr integral_constant<int, 256> eight{};
  constexpr integral_constant<int, 512> half{};
  constexpr integral_constant<int, 1024> all{};
  constexpr integral_constant<int, 8> least{};
  static_assert(kShort == 32 * 8, "a short row is a warp's with eight channels each");
  if (a.W <= kShort / 2) return go(integral_constant<int, 16>{}, least);
  if (a.W <= kShort) return go(warp, least);
  if constexpr (kVector) {
    constexpr integral_constant<int, 64 / sizeof(T)> E{};
    if constexpr (E > 16)
      if (a.W <= 32 * 16) return go(warp, integral_constant<int, 16>{});
    if (a.W <= 32 * E) return go(warp, E);
    if (a.W <= 128 * E) return go(four, E);
    if (a.W <= 256 * E) return go(eight, E);
    if (a.W <= 512 * E) return go(half, E);
    if constexpr (512 * E < kNormMax) return go(half, integral_constant<int, kNormMax / 512>{});
  } else {
    if (a.W <= 128 * least) return go(four, least);
    if (a.W <= 512 * least) return go(half, least);
    if (a.W <= 1024 * least) return go(all, least);
    return go(all, integral_constant<int, kNormMax / 1024>{});
  }
  return cudaErrorInvalidValue;
}

template <bool kForward>
cudaError_t launch(const NormArgs &a, bool vector, cudaStream_t stream) {
  vector = vector && rows_of_16(a.weight, 0, 1) && rows_of_16(a.bias, 0, 1);
  if (a.bf16)
    return vector ? pick<__nv_bfloat16, true, kForward>(a, stream)
                  : pick<__nv_bfloat16, false, kForward>(a, stream);
  return vector ? pick<float, true, kForward>(a, stream) : pick<float, false, kForward>(a, stream);
}

}  // namespace

cudaError_t launch_norm_fwd(const NormArgs &a, cudaStream_t stream) {
  if (a.n == 0) return cudaSuccess;
  const int esz = a.bf16 ? 2 : 4;
  return launch<true>(a, rows_of_16(a.x, a.x_rs, esz) && rows_of_16(a.out, a.out_rs, esz), stream);
}

size_t norm_bwd_scratch_bytes(int64_t n, int32_t W, bool bf16) {
  (void)bf16;
  const int64_t most = most_blocks(W);
  return (size_t)(n < most ? n : most) * 2 * W * sizeof(float);
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
  return launch<false>(a, a.W * esz % 16 == 0 && rows_of_16(a.x, a.x_rs, esz) && rows_of_16(a.d_out, a.do_rs, esz) &&
                              rows_of_16(a.d_x, a.dx_rs, esz), stream);
}

}  // namespace kda
