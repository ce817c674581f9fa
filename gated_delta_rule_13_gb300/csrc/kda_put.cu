// A host array to the device as launch parameters: the numbers are taken before the call
// returns, and a captured launch keeps its own copy.  (A copy from host memory reads it
// when the stream gets there, from pinned memory, and at every replay, from any.)
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "kda_internal.h"

namespace kda {
namespace {

template <int kCap>
struct Ints {
  int32_t v[kCap];
};
template <int kCap>
__global__ void kda_put_kernel(const __grid_constant__ Ints<kCap> p, int32_t *dst, int n) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) dst[i] = p.v[i];
}

template <int kCap>
cudaError_t put(int32_t *dst, const int32_t *src, int n, cudaStream_t stream) {
  Ints<kCap> p;
  memcpy(p.v, src, sizeof(int32_t) * n);
  kda_put_kernel<kCap><<<(n + 255) / 256, 256, 0, stream>>>(p, dst, n);
  return cudaGetLastError();
}

}  // namespace

cudaError_t put_ints(int32_t *dst, const int32_t *src, int64_t n, cudaStream_t stream) {
  // a launch carries at most 32,764 bytes of parameters; a short one costs less to send
  constexpr int kFew = 256, kMany = 8000;
  for (int64_t at = 0; at < n; at += kMany) {
    const int now = (int)(n - at < kMany ? n - at : kMany);
    const cudaError_t e = now <= kFew ? put<kFew>(dst + at, src + at, now, stream)
                                      : put<kMany>(dst + at, src + at, now, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace kda
