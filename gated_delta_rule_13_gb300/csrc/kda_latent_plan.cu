// Tile counts before every sequence, for calls with more sequences than a warp has
// lanes: with them a block finds its tile in a few probes instead of reading both
// cu_seqlens arrays (at 4096 sequences, 128 reads of 0.6 us one after another).
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/kda.h"
#include "kda_latent.h"

namespace kda {
namespace {

constexpr int kThreads = 1024;

// One block; sequence by sequence in rounds of 1024, the sum carried along.  Bound by
// latency: 5.3 us for 64 sequences, 9 for 4096.
__global__ void __launch_bounds__(kThreads)
kda_latent_plan_kernel(const Packed p, int32_t *mem, int64_t stride, DeviceStatus *status) {
  __shared__ int32_t warp_sum[kThreads / 32];
  __shared__ int32_t s_bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0)
    s_bad = cu_at(p.cu_q, 0, p.n_q) != 0 || cu_at(p.cu_k, 0, p.n_k) != 0 ||
            cu_at(p.cu_q, p.n_seqs, p.n_q) != p.n_q || cu_at(p.cu_k, p.n_seqs, p.n_k) != p.n_k;
  __syncthreads();
  bool bad = false;
  for (int s = tid; s < p.n_seqs; s += kThreads) {
    const int32_t qa = cu_at(p.cu_q, s, p.n_q), qb = cu_at(p.cu_q, s + 1, p.n_q);
    const int32_t ka = cu_at(p.cu_k, s, p.n_k), kb = cu_at(p.cu_k, s + 1, p.n_k);
    bad = bad || qb < qa || kb < ka || qa < 0 || ka < 0 || qb > p.n_q || kb > p.n_k;
  }
  if (bad) s_bad = 1;
  __syncthreads();
  const bool wrong = s_bad != 0;
  if (tid == 0) set_device_status(status, wrong ? KDA_ERR_INVALID_ARG : KDA_OK, wrong);
  for (int kind = 0; kind < kTileKinds; ++kind) {
    const int32_t rows = p.rows[kind];
    int32_t *before = mem + kind * stride;
    if (rows == 0) continue;
    if (wrong) {
      if (tid == 0) before[p.n_seqs] = -1;
      continue;
    }
    int32_t carry = 0;
    for (int32_t s0 = 0; s0 < p.n_seqs; s0 += kThreads) {
      const int32_t s = s0 + tid;
      int32_t tiles = 0;
      if (s < p.n_seqs) {
        const int32_t n = p.by_key[kind]
                              ? cu_at(p.cu_k, s + 1, p.n_k) - cu_at(p.cu_k, s, p.n_k)
                              : cu_at(p.cu_q, s + 1, p.n_q) - cu_at(p.cu_q, s, p.n_q);
        tiles = (n + rows - 1) / rows;
      }
      int32_t inc = tiles;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += y;
      }
      if (lane == 31) warp_sum[warp] = inc;
      __syncthreads();
      int32_t base = carry, all = 0;
      for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) base += warp_sum[w];
        all += warp_sum[w];
      }
      if (s < p.n_seqs) before[s] = base + inc - tiles;
      carry += all;
      __syncthreads();
    }
    if (tid == 0) before[p.n_seqs] = carry;
  }
}

int64_t plan_stride(int32_t n_seqs) { return ((int64_t)n_seqs + 1 + 63) / 64 * 64; }

}  // namespace

size_t latent_plan_bytes(int32_t n_seqs) {
  return n_seqs > kLaneSeqs ? (size_t)plan_stride(n_seqs) * kTileKinds * sizeof(int32_t) : 0;
}

cudaError_t launch_latent_plan(Packed &p, void *mem, DeviceStatus *status, cudaStream_t stream) {
  int32_t *at = static_cast<int32_t *>(mem);
  for (int kind = 0; kind < kTileKinds; ++kind) p.before[kind] = at + kind * plan_stride(p.n_seqs);
  if (p.n_seqs <= kLaneSeqs) return cudaSuccess;
  kda_latent_plan_kernel<<<1, kThreads, 0, stream>>>(p, at, plan_stride(p.n_seqs), status);
  return cudaGetLastError();
}

}  // namespace kda
