// Norm over a row's channels, with or without its mean (kda_norm_fwd), and its gradient
// (kda_norm_bwd).
//
//   m = mean x (0 without), r = 1 / sqrt(mean (x - m)^2 + eps),  z = (x - m) r
//   y = z w + b
//   dx = r (w g - mean(w g) - z mean(w g z))   (without the mean: no second term)
//   dw = sum over rows of g z,  db = sum over rows of g
//
// A row is read once and held in registers, as it was loaded, by a warp or by up to 1024
// threads; the variance is the mean square of what the mean leaves, from the same
// registers, so that a mean far from zero costs no digits.  Statistics and sums are fp32.
// The gradient's blocks walk over the rows with the sums of dw and db in registers and
// leave one pair of rows each in the workspace; a second kernel adds these in the blocks'
// order, so that results do not vary between calls.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "kda_latent_tc.cuh"
#include "kda_rows.h"

namespace kda {
namespace {

template <typename T>
constexpr int kEach = 64 / sizeof(T);    // channels of a thread

// What a thread holds of a row: 16-byte vectors tid, tid + N, ..., or single channels.  A
// vector that the row ends in is put together from single channels.
template <typename T, int N, bool kVector>
struct Row {
  static constexpr int kV = kVector ? 16 / (int)sizeof(T) : 1;
  static constexpr int kCount = kEach<T> / kV;
  uint32_t raw[16];
  static __device__ __forceinline__ int channel(int i) {  // of element i of this thread
    const int lane = N == 32 ? threadIdx.x & 31 : threadIdx.x % N;
    return (i / kV * N + lane) * kV + i % kV;
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
  __device__ __forceinline__ void load(const T *row, int W) {
#pragma unroll
    for (int i = 0; i < 16; ++i) raw[i] = 0;
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
  // f: element -> value
  template <class F>
  __device__ __forceinline__ void store(T *row, int W, F f) const {
#pragma unroll
    for (int j = 0; j < kCount; ++j) {
      const int c = channel(j * kV);
      if (c >= W) continue;
      T v[kV];
#pragma unroll
      for (int e = 0; e < kV; ++e) {
        const float y = f(j * kV + e, c + e);
        if constexpr (sizeof(T) == 4) v[e] = y;
        else v[e] = __float2bfloat16_rn(y);
      }
      if constexpr (kVector) {
        if (c + kV <= W) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (sizeof(T) == 4) w[k] = __float_as_uint(v[k]);
            else w[k] = (uint32_t)__bfloat16_as_ushort(v[2 * k]) |
                        (uint32_t)__bfloat16_as_ushort(v[2 * k + 1]) << 16;
          }
          *reinterpret_cast<uint4 *>(row + c) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
#pragma unroll
          for (int e = 0; e < kV; ++e)
            if (c + e < W) row[c + e] = v[e];
        }
      } else {
        row[c] = v[0];
      }
    }
  }
};

// Sums over the N threads of a row; `slot` alternates between calls, so that one barrier a
// call is enough.  Every thread of the block calls.
template <int N, int K>
__device__ __forceinline__ void row_sum(float (&x)[K], float (*part)[32 * K]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) x[k] += __shfl_xor_sync(0xffffffffu, x[k], o);
  if constexpr (N > 32) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int kWarps = N / 32;
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) (*part)[k * 32 + warp] = x[k];
    __syncthreads();
    const int first = warp / kWarps * kWarps;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float y = lane < kWarps ? (*part)[k * 32 + first + lane] : 0.f;
#pragma unroll
      for (int o = kWarps / 2; o > 0; o >>= 1) y += __shfl_xor_sync(0xffffffffu, y, o);
      x[k] = __shfl_sync(0xffffffffu, y, 0);
    }
  }
}

template <int N>
constexpr int kBlock = N < 256 ? 256 : N;

template <typename T, int N, bool kVector>
__global__ void __launch_bounds__(kBlock<N>) kda_norm_fwd_kernel(const NormArgs a) {
  __shared__ float part[2][32];
  constexpr int kRows = kBlock<N> / N;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / N;
  const bool live = row < a.n;
  Row<T, N, kVector> x;
  if (live) x.load(static_cast<const T *>(a.x) + row * a.x_rs, a.W);
  const float inv = 1.f / a.W;
  float m[1] = {0.f};
  if (a.center) {
    if (live)
#pragma unroll
      for (int i = 0; i < kEach<T>; ++i) m[0] += x.get(i);
    row_sum<N, 1>(m, &part[0]);
    m[0] *= inv;
  }
  float v[1] = {0.f};
  if (live)
#pragma unroll
    for (int i = 0; i < kEach<T>; ++i)
      if (x.channel(i) < a.W) {
        const float d = x.get(i) - m[0];
        v[0] = fmaf(d, d, v[0]);
      }
  row_sum<N, 1>(v, &part[1]);
  if (!live) return;
  const float r = rsqrtf(fmaf(v[0], inv, a.eps));
  if (threadIdx.x % N == 0) {
    if (a.mean) a.mean[row] = m[0];
    if (a.rstd) a.rstd[row] = r;
  }
  x.store(static_cast<T *>(a.out) + row * a.out_rs, a.W, [&](int i, int c) {
    c = min(c, a.W - 1);
    float y = (x.get(i) - m[0]) * r;
    if (a.weight) y *= a.weight[c];
    if (a.bias) y += a.bias[c];
    return y;
  });
}

constexpr int kJoinCols = 32;

template <typename T, int N, bool kVector>
__global__ void __launch_bounds__(kBlock<N>) kda_norm_bwd_kernel(const NormArgs a) {
  __shared__ float part[2][64];
  extern __shared__ float sums[];                        // [W], where a block has several rows
  constexpr int kRows = kBlock<N> / N, kE = kEach<T>;
  latent::pdl_launch_dependents();
  const float inv = 1.f / a.W;
  float dw[kE], db[kE];
#pragma unroll
  for (int i = 0; i < kE; ++i) dw[i] = db[i] = 0.f;
  int turn = 0;
  for (int64_t r0 = (int64_t)blockIdx.x * kRows; r0 < a.n; r0 += (int64_t)gridDim.x * kRows) {
    const int64_t row = r0 + threadIdx.x / N;
    const bool live = row < a.n;
    Row<T, N, kVector> x, g;
    float m = 0.f, r = 0.f;
    if (live) {
      x.load(static_cast<const T *>(a.x) + row * a.x_rs, a.W);
      g.load(static_cast<const T *>(a.d_out) + row * a.do_rs, a.W);
      if (a.center) m = a.mean[row];
      r = a.rstd[row];
    }
    float s[2] = {0.f, 0.f};                             // sums of w g and of w g z
    if (live)
#pragma unroll
      for (int i = 0; i < kE; ++i) {
        const int c = x.channel(i);
        if (c < a.W) {
          const float z = (x.get(i) - m) * r, d = g.get(i);
          dw[i] = fmaf(d, z, dw[i]);
          db[i] += d;
          const float e = a.weight ? d * a.weight[c] : d;
          s[0] += e;
          s[1] = fmaf(e, z, s[1]);
        }
      }
    row_sum<N, 2>(s, &part[turn]);
    turn ^= 1;
    if (!live) continue;
    const float c1 = a.center ? s[0] * inv : 0.f, c2 = s[1] * inv;
    x.store(static_cast<T *>(a.d_x) + row * a.dx_rs, a.W, [&](int i, int c) {
      c = min(c, a.W - 1);
      const float z = (x.get(i) - m) * r, e = a.weight ? g.get(i) * a.weight[c] : g.get(i);
      return r * (e - c1 - z * c2);
    });
  }
  if (!a.partial) return;
  // this block's sums: rows 2 blockIdx (dw) and 2 blockIdx + 1 (db) of the scratch
  for (int which = 0; which < 2; ++which) {
    float *to = a.partial + ((int64_t)blockIdx.x * 2 + which) * a.W;
    for (int p = 0; p < kRows; ++p) {
      if (threadIdx.x / N == p) {
#pragma unroll
        for (int i = 0; i < kE; ++i) {
          const int c = Row<T, N, kVector>::channel(i);
          if (c < a.W) {
            const float v = which ? db[i] : dw[i];
            if (kRows == 1) to[c] = v;
            else if (p == 0) sums[c] = v;
            else sums[c] += v;
          }
        }
      }
      if (kRows > 1) __syncthreads();
    }
    if (kRows > 1) {
      for (int c = threadIdx.x; c < a.W; c += kBlock<N>) to[c] = sums[c];
      __syncthreads();
    }
  }
}

// Sums of the blocks' rows, in their order: 32 groups of consecutive blocks, then the
// groups.  Block (x: 32 channels, y: dw, db).
__global__ void __launch_bounds__(1024)
kda_norm_join_kernel(const float *__restrict__ partial, int32_t blocks, int32_t W, float *d_weight,
                     float *d_bias) {
  __shared__ float s[32][kJoinCols + 1];
  latent::pdl_wait();
  float *out = blockIdx.y ? d_bias : d_weight;
  if (!out) return;
  const int lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
  const int c = blockIdx.x * kJoinCols + lane;
  const int per = (blocks + 31) / 32, b0 = grp * per, b1 = min(blocks, b0 + per);
  float sum = 0.f;
  if (c < W)
#pragma unroll 8
    for (int b = b0; b < b1; ++b) sum += partial[((int64_t)b * 2 + blockIdx.y) * W + c];
  s[grp][lane] = sum;
  __syncthreads();
  if (grp > 0 || c >= W) return;
  float all = 0.f;
#pragma unroll
  for (int i = 0; i < 32; ++i) all += s[i][lane];
  out[c] = all;
}

template <typename T, int N, bool kVector>
cudaError_t fwd(const NormArgs &a, cudaStream_t stream) {
  constexpr int kRows = kBlock<N> / N;
  const int64_t blocks = (a.n + kRows - 1) / kRows;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  kda_norm_fwd_kernel<T, N, kVector><<<(unsigned)blocks, kBlock<N>, 0, stream>>>(a);
  return cudaGetLastError();
}

// Blocks of the gradient: 1024 threads an SM, or as many as there are rows for.
int bwd_blocks(int64_t n, int threads_of_row) {
  const int block = threads_of_row < 256 ? 256 : threads_of_row, rows = block / threads_of_row;
  const int sms = latent::sm_count() > 0 ? latent::sm_count() : 1;
  const int64_t most = (int64_t)sms * (block < 512 ? 512 / block : 1), need = (n + rows - 1) / rows;
  return (int)(need < most ? need : most);
}

template <typename T, int N, bool kVector>
cudaError_t bwd(const NormArgs &a, cudaStream_t stream) {
  const int blocks = bwd_blocks(a.n, N);
  const size_t smem = kBlock<N> / N > 1 ? (size_t)a.W * 4 : 0;
  kda_norm_bwd_kernel<T, N, kVector><<<blocks, kBlock<N>, smem, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.partial) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.W + kJoinCols - 1) / kJoinCols), 2);
  cfg.blockDim = dim3(1024);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kda_norm_join_kernel, (const float *)a.partial, (int32_t)blocks,
                            a.W, a.d_weight, a.d_bias);
}

// Threads of a row: the fewest that hold it.
int threads_of(int32_t W, bool bf16) {
  const int each = bf16 ? kEach<__nv_bfloat16> : kEach<float>;
  for (const int n : {32, 128, 256, 512})
    if (W <= n * each) return n;
  return 1024;
}

bool rows_of_16(const void *p, int64_t rs, int esz) {
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && rs * esz % 16 == 0;
}

template <typename T, bool kVector, bool kForward>
cudaError_t pick(const NormArgs &a, cudaStream_t stream) {
  const auto go = [&](auto n) {
    constexpr int N = decltype(n)::value;
    if constexpr (kForward) return fwd<T, N, kVector>(a, stream);
    else return bwd<T, N, kVector>(a, stream);
  };
  switch (threads_of(a.W, std::is_same_v<T, __nv_bfloat16>)) {
    case 32: return go(std::integral_constant<int, 32>{});
    case 128: return go(std::integral_constant<int, 128>{});
    case 256: return go(std::integral_constant<int, 256>{});
    case 512: return go(std::integral_constant<int, 512>{});
    default:
      if constexpr (std::is_same_v<T, float>) return go(std::integral_constant<int, 1024>{});
      else return cudaErrorInvalidValue;                 // 512 threads hold 16384 channels
  }
}

template <bool kForward>
cudaError_t launch(const NormArgs &a, bool vector, cudaStream_t stream) {
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
  return n == 0 ? 0 : (size_t)bwd_blocks(n, threads_of(W, bf16)) * 2 * W * sizeof(float);
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
  return launch<false>(a, rows_of_16(a.x, a.x_rs, esz) && rows_of_16(a.d_out, a.do_rs, esz) &&
                              rows_of_16(a.d_x, a.dx_rs, esz), stream);
}

}  // namespace kda
