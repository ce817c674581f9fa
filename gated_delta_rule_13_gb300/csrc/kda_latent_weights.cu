// The attention weight that cached rows have been given (kda_latent_weights).
//
//   w_j <- decay w_j + sum over tokens t and heads h that see j of exp(scale q_th . c_j - lse_th)
//
// One thread block per 32 cached rows of a sequence, held in shared memory; a warp takes
// every eighth query row, a lane is a cached row.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kda_latent_tc.cuh"
#include "kda_rows.h"

namespace kda {
namespace {

constexpr int kRows = 32, kWarps = 8;

__global__ void __launch_bounds__(32 * kWarps) kda_latent_weights_kernel(const LatentWeightsArgs a) {
  extern __shared__ uint32_t tile[];       // [32][W / 2 + 1]
  __shared__ float part[kWarps][kRows];
  __shared__ int bad;
  const int b = blockIdx.y, W = kLatentC + a.dr, words = W / 2, R = a.T * a.H;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cap = a.max_pages * a.page_size;
  const int n = a.seq_lens[b];
  if (threadIdx.x == 0) bad = n < 0 || n > cap;
  __syncthreads();
  const int32_t *table = a.block_table + (int64_t)b * a.max_pages;
  if (!bad) {
    bool wrong = false;
    for (int i = threadIdx.x; i < (n + a.page_size - 1) / a.page_size; i += 32 * kWarps)
      wrong = wrong || table[i] < 0 || table[i] >= a.n_pages;
    if (wrong) bad = 2;
  }
  __syncthreads();
  if (bad) {
    if (threadIdx.x == 0 && blockIdx.x == 0)
      record_device_status(a.status, KDA_ERR_INVALID_ARG, bad, b, 0);
    return;
  }
  for (int64_t j0 = (int64_t)blockIdx.x * kRows; j0 < n; j0 += (int64_t)gridDim.x * kRows) {
    const int live = (int)min((int64_t)kRows, n - j0);
    __syncthreads();
    for (int i = threadIdx.x; i < live * words; i += 32 * kWarps) {
      const int r = i / words, c = i - r * words;
      const int pos = (int)j0 + r, pg = pos / a.page_size;
      const uint32_t *row = static_cast<const uint32_t *>(a.cache) +
                            ((int64_t)table[pg] * a.page_size + (pos - pg * a.page_size)) * words;
      tile[r * (words + 1) + c] = row[c];
    }
    __syncthreads();
    const int j = (int)j0 + lane, draft = j - (n - a.T);
    float sum = 0.f;
    for (int r = warp; r < R; r += kWarps) {
      const int t = r / a.H;
      const float lse = a.lse[(int64_t)b * R + r];
      bool seen = lane < live && !isinf(lse);
      if (draft >= 0)
        seen = seen && (a.tree_mask ? (a.tree_mask[(int64_t)b * a.T + t] >> draft & 1) != 0 : draft <= t);
      const uint32_t *q = static_cast<const uint32_t *>(a.q) + ((int64_t)b * R + r) * words;
      float s = 0.f;
      for (int c = 0; c < words; ++c) {
        const float2 x = sm100::unpack_bf16x2(q[c]);
        const float2 y = sm100::unpack_bf16x2(tile[(lane < live ? lane : 0) * (words + 1) + c]);
        s = fmaf(x.x, y.x, s);
        s = fmaf(x.y, y.y, s);
      }
      if (seen) sum += exp2f((s * a.scale - lse) * latent::kLog2e);
    }
    part[warp][lane] = sum;
    __syncthreads();
    if (warp == 0 && lane < live) {
      float all = 0.f;
      for (int k = 0; k < kWarps; ++k) all += part[k][lane];
      float *to = a.weights + (int64_t)b * cap + j;
      *to = a.decay == 0.f ? all : fmaf(*to, a.decay, all);
    }
  }
}

}  // namespace

size_t latent_weights_scratch_bytes(int32_t, int32_t, int32_t, int32_t) { return 0; }

cudaError_t launch_latent_weights(const LatentWeightsArgs &a, cudaStream_t stream) {
  const cudaError_t e = cudaMemsetAsync(a.status, 0, sizeof(DeviceStatus), stream);
  if (e != cudaSuccess || a.B == 0) return e;
  const size_t smem = (size_t)kRows * ((kLatentC + a.dr) / 2 + 1) * 4;
  int64_t tiles = ((int64_t)a.max_pages * a.page_size + kRows - 1) / kRows;
  if (tiles > 4096) tiles = 4096;
  kda_latent_weights_kernel<<<dim3((unsigned)tiles, (unsigned)a.B), 32 * kWarps, smem, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace kda
