// Host-side declarations of the operators around a cached latent row: rotation, norm,
// the attention weight it has been given, eviction.  Not part of the public ABI.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_latent.h"

namespace kda {

constexpr int kRopeMax = 512;     // rotary channels of a row at most
constexpr int kNormMax = 16384;   // channels of a normalised row at most

// Strides in elements.  k: one row a token, rotated as one more head (nullptr: none).
struct RopeArgs {
  const void *x;              // [n, H, dr]
  void *out;
  int64_t x_ts, x_hs, o_ts, o_hs;
  const void *k;              // [n, dr]
  void *k_out;
  int64_t k_ts, ko_ts;
  const int32_t *positions;   // [n]
  const double *inv_freq;     // [dr / 2]
  int64_t n;
  int32_t H, dr;
  bool interleaved, transpose, bf16;
  float scale;
};
cudaError_t launch_rope(const RopeArgs &a, cudaStream_t stream);

struct NormArgs {
  const void *x;              // [n, W], rows x_rs elements apart
  int64_t x_rs, n;
  const float *weight, *bias; // [W] or nullptr
  int32_t W;
  bool bf16, center;
  float eps;
  void *out;                  // forward
  int64_t out_rs;
  float *mean, *rstd;         // [n]; forward: or nullptr
  const void *d_out;          // backward
  int64_t do_rs;
  void *d_x;
  int64_t dx_rs;
  float *d_weight, *d_bias;   // [W] or nullptr
  float *partial;             // norm_bwd_scratch_bytes()
};
cudaError_t launch_norm_fwd(const NormArgs &a, cudaStream_t stream);
cudaError_t launch_norm_bwd(const NormArgs &a, cudaStream_t stream);
size_t norm_bwd_scratch_bytes(int64_t n, int32_t W, bool bf16);

struct LatentWeightsArgs {
  const void *q;              // [B, T, H, 512 + dr]
  const void *cache;          // [n_pages, page_size, 512 + dr]
  const int32_t *block_table; // [B, max_pages]
  const int32_t *seq_lens;    // [B]
  const int64_t *tree_mask;   // [B, T] or nullptr
  const float *lse;           // [B, T, H]
  int32_t B, T, H, dr, n_pages, page_size, max_pages;
  float scale, decay;
  float *weights;             // [B, max_pages * page_size]
  DeviceStatus *status;
  void *scratch;              // latent_weights_scratch_bytes()
  WaitTest test;
};
cudaError_t launch_latent_weights(const LatentWeightsArgs &a, cudaStream_t stream);
size_t latent_weights_scratch_bytes(int32_t B, int32_t T, int32_t H, int32_t dr);

struct CacheEvictArgs {
  void *cache;                // [L, n_pages, page_size, row_bytes]
  const int32_t *block_table; // [B, max_pages]
  const int32_t *seq_lens;    // [B]
  const float *weights;       // [L, B, max_pages * page_size]
  float *weights_out;         // the same, or weights itself
  int32_t L, n_pages, page_size, B, max_pages, budget, first, recent;
  int64_t row_bytes;
  int32_t *new_lens;          // [B]
  int32_t *origin;            // [L, B, budget]
  int32_t *moves;             // scratch: cache_evict_scratch_bytes()
  int32_t *status;
};
cudaError_t launch_cache_evict(const CacheEvictArgs &a, cudaStream_t stream);
size_t cache_evict_scratch_bytes(int32_t L, int32_t B, int32_t budget);

}  // namespace kda
