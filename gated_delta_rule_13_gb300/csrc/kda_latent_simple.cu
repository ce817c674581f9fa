// Latent attention, first form: one warp per row on the CUDA cores, fp32 throughout.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <stdint.h>

#include "../../include/kda.h"
#include "kda_latent.h"

namespace kda {
namespace {

constexpr int kRows = 8;  // rows (warps) per block
using bf16 = __nv_bfloat16;

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
__device__ __forceinline__ float4 ld4(const bf16 *p) {
  const uint2 r = *reinterpret_cast<const uint2 *>(p);
  return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u),
                     __uint_as_float(r.y << 16), __uint_as_float(r.y & 0xffff0000u));
}
__device__ __forceinline__ float2 ld2(const bf16 *p) {
  const uint32_t r = *reinterpret_cast<const uint32_t *>(p);
  return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
}
__device__ __forceinline__ float dot4(float4 a, float4 b) {
  return a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w;
}
__device__ __forceinline__ void st4(bf16 *p, float4 v) {
  p[0] = __float2bfloat16(v.x); p[1] = __float2bfloat16(v.y);
  p[2] = __float2bfloat16(v.z); p[3] = __float2bfloat16(v.w);
}
__device__ __forceinline__ void axpy(float4 &y, float a, float4 x) {
  y.x += a * x.x; y.y += a * x.y; y.z += a * x.z; y.w += a * x.w;
}

// A query row and its head: rows of the packed sequence, or false.
__device__ bool row_tile(const LatentArgs &a, bool by_key, SeqTile &t) {
  __shared__ SeqTile st;
  if (threadIdx.x < 32) {
    const SeqTile f =
        find_seq_tile(a.cu_q, a.cu_k, a.n_seqs, a.n_q, a.n_k, kRows, by_key, blockIdx.x);
    if (threadIdx.x == 0) st = f;
  }
  __syncthreads();
  t = st;
  if (t.bad && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
    record_device_status(a.status, KDA_ERR_INVALID_ARG, 0, 0, 0);
  return t.seq >= 0;
}

struct Row {
  float4 qn, g;
  float2 qr;
  float lse, delta;
};
__device__ Row load_row(const LatentArgs &a, int64_t r, int h, int lane) {
  Row x;
  const int W = kLatentD + a.dr;
  const int64_t rh = r * a.H + h;
  const bf16 *q = static_cast<const bf16 *>(a.q) + rh * W;
  x.qn = ld4(q + 4 * lane);
  x.qr = a.dr ? ld2(q + kLatentD + 2 * lane) : make_float2(0, 0);
  x.g = ld4(static_cast<const bf16 *>(a.d_out) + rh * kLatentD + 4 * lane);
  x.delta = warp_sum(dot4(x.g, ld4(static_cast<const bf16 *>(a.out) + rh * kLatentD + 4 * lane)));
  x.lse = a.lse[rh];
  return x;
}
// p and ds of one pair
__device__ void pair_grad(const LatentArgs &a, const Row &x, float4 kn, float2 kr, float4 v,
                          float &p, float &ds) {
  const float s = warp_sum(dot4(x.qn, kn) + x.qr.x * kr.x + x.qr.y * kr.y) * a.scale;
  const float dp = warp_sum(dot4(x.g, v));
  p = x.lse == -CUDART_INF_F ? 0.f : expf(s - x.lse);
  ds = p * (dp - x.delta) * a.scale;
}

__global__ void bwd_q_kernel(LatentArgs a) {
  SeqTile t;
  if (!row_tile(a, false, t)) return;
  const int lane = threadIdx.x & 31, i = t.tile * kRows + (threadIdx.x >> 5), h = blockIdx.y;
  if (i >= t.nq) return;
  const Row x = load_row(a, t.q0 + i, h, lane);
  const int n = a.causal ? min(t.nk, max(0, t.nk - t.nq + i + 1)) : t.nk;
  float4 dn = make_float4(0, 0, 0, 0);
  float2 dr = make_float2(0, 0);
  for (int j = 0; j < n; ++j) {
    const int64_t kj = t.k0 + j;
    const float4 kn = ld4(static_cast<const bf16 *>(a.k) + kj * a.k_ts + h * a.k_hs + 4 * lane);
    const float2 kr = a.dr ? ld2(static_cast<const bf16 *>(a.k_rope) + kj * a.dr + 2 * lane)
                           : make_float2(0, 0);
    float p, ds;
    pair_grad(a, x, kn, kr, ld4(static_cast<const bf16 *>(a.v) + kj * a.v_ts + h * a.v_hs + 4 * lane),
              p, ds);
    axpy(dn, ds, kn);
    dr.x += ds * kr.x; dr.y += ds * kr.y;
  }
  const int W = kLatentD + a.dr;
  bf16 *dq = static_cast<bf16 *>(a.dq) + ((int64_t)(t.q0 + i) * a.H + h) * W;
  st4(dq + 4 * lane, dn);
  if (a.dr) {
    dq[kLatentD + 2 * lane] = __float2bfloat16(dr.x);
    dq[kLatentD + 2 * lane + 1] = __float2bfloat16(dr.y);
  }
}

// One warp per key; the heads in turn, so that the shared rope gradient is one sum.
__global__ void bwd_kv_kernel(LatentArgs a) {
  SeqTile t;
  if (!row_tile(a, true, t)) return;
  const int lane = threadIdx.x & 31, j = t.tile * kRows + (threadIdx.x >> 5);
  if (j >= t.nk) return;
  const int64_t kj = t.k0 + j;
  const float2 kr = a.dr ? ld2(static_cast<const bf16 *>(a.k_rope) + kj * a.dr + 2 * lane)
                         : make_float2(0, 0);
  float2 dr = make_float2(0, 0);
  for (int h = 0; h < a.H; ++h) {
    const float4 kn = ld4(static_cast<const bf16 *>(a.k) + kj * a.k_ts + h * a.k_hs + 4 * lane);
    const float4 v = ld4(static_cast<const bf16 *>(a.v) + kj * a.v_ts + h * a.v_hs + 4 * lane);
    float4 dk = make_float4(0, 0, 0, 0), dv = dk;
    for (int i = a.causal ? max(0, j - (t.nk - t.nq)) : 0; i < t.nq; ++i) {
      const Row x = load_row(a, t.q0 + i, h, lane);
      float p, ds;
      pair_grad(a, x, kn, kr, v, p, ds);
      axpy(dv, p, x.g);
      axpy(dk, ds, x.qn);
      dr.x += ds * x.qr.x; dr.y += ds * x.qr.y;
    }
    st4(static_cast<bf16 *>(a.dk) + kj * a.dk_ts + h * a.dk_hs + 4 * lane, dk);
    st4(static_cast<bf16 *>(a.dv) + kj * a.dv_ts + h * a.dv_hs + 4 * lane, dv);
  }
  if (a.dr) {
    bf16 *p = static_cast<bf16 *>(a.d_k_rope) + kj * a.dr + 2 * lane;
    p[0] = __float2bfloat16(dr.x);
    p[1] = __float2bfloat16(dr.y);
  }
}

unsigned tiles(int64_t n, int32_t n_seqs) { return (unsigned)(n / kRows + n_seqs); }

}  // namespace

size_t latent_bwd_scratch_bytes(int64_t, int64_t, int32_t, int32_t) { return 0; }

cudaError_t launch_latent_bwd(const LatentArgs &a, cudaStream_t stream) {
  if (a.n_q > 0)
    bwd_q_kernel<<<dim3(tiles(a.n_q, a.n_seqs), a.H), 32 * kRows, 0, stream>>>(a);
  if (a.n_k > 0) bwd_kv_kernel<<<tiles(a.n_k, a.n_seqs), 32 * kRows, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace kda
