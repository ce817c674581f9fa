// Moves of a paged cache: rows appended or compacted through a block table, and
// whole pages copied (a fork's private page, a snapshot made a running state).
// Pure data movement: bytes in, the same bytes out, 16 at a time.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/kda.h"
#include "kda_latent.h"

namespace kda {
namespace {

__device__ __forceinline__ void flag_status(int32_t *status) {
  if (status) atomicCAS(status, 0, (int32_t)KDA_ERR_INVALID_ARG);
}

// Position `pos` of sequence b as a row of the pool, or -1 (no such page).
__device__ __forceinline__ int64_t row_of(const int32_t *__restrict__ table, int32_t b,
                                          int32_t max_pages, int32_t page_size, int32_t n_pages,
                                          int64_t pos) {
  if (pos < 0) return -1;
  const int64_t pg = pos / page_size;
  if (pg >= max_pages) return -1;
  const int32_t id = table[(int64_t)b * max_pages + pg];
  if (id < 0 || id >= n_pages) return -1;
  return (int64_t)id * page_size + (pos - pg * page_size);
}

constexpr int kWriteThreads = 128;
constexpr int kWriteBatch = 4;   // rows in flight per thread

// Block (x: 16-byte columns, y: sequence, z: layer).  The sequence's row moves
// (source row, destination row) are worked out once per block, in shared memory,
// then every thread carries its own column through them.
//
// Compaction moves row start + path[i] to row start + i inside the pool.  With a
// strictly increasing path, path[i] >= i, and a thread reads its column of rows
// i .. i + 3 before it writes them: a later read path[j] >= j > i + 3 never meets
// a row already written, and no other thread touches the column.  So no second
// buffer and no barrier between reads and writes is needed.  A path that is not
// increasing is refused for its sequence (status).
//
// Bound by latency (three dependent reads: start, block table, row), then by HBM: one
// row of 1,152 bytes for each of 64 sequences 4.3 us on the device, 7.8 with the call;
// the accepted rows of 16 drafts, 256 sequences, 24 layers at once, 12.3 us with the
// pool's rows in L2, 15.7 without.  With 1, 4, 8 and 16 rows in flight a thread: 12.4,
// 12.3, 12.8, 20.6 us (one row at a time: 5.8 us for the first).
template <bool kCompact>
__global__ void __launch_bounds__(kWriteThreads)
kda_cache_write_kernel(CacheWriteArgs a) {
  extern __shared__ int64_t moves[];   // [T][2] pool row from / to, -1: none
  __shared__ int bad;
  const int32_t b = blockIdx.y;
  const int64_t start = a.start[b];
  int32_t n = a.n_write ? a.n_write[b] : a.T;
  n = n < 0 ? 0 : n > a.T ? a.T : n;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kWriteThreads) {
    const int32_t p = a.path ? a.path[(int64_t)b * a.T + i] : i;
    const int64_t to = row_of(a.block_table, b, a.max_pages, a.page_size, a.n_pages, start + i);
    int64_t from = p;
    bool wrong = p < 0 || p >= a.T || to < 0;
    if (kCompact) {
      from = row_of(a.block_table, b, a.max_pages, a.page_size, a.n_pages, start + p);
      wrong = wrong || from < 0 || (i > 0 && a.path[(int64_t)b * a.T + i - 1] >= p);
    }
    if (wrong || start < 0) bad = 1;
    moves[2 * i] = from;
    moves[2 * i + 1] = to;
  }
  __syncthreads();
  if (bad) {  // nothing of this sequence is written
    if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.z == 0) flag_status(a.status);
    return;
  }
  const int64_t col = ((int64_t)blockIdx.x * kWriteThreads + threadIdx.x) * 16;
  if (col >= a.row_bytes) return;
  unsigned char *pool = static_cast<unsigned char *>(a.cache) +
                        (int64_t)blockIdx.z * a.n_pages * a.page_size * a.row_bytes + col;
  const unsigned char *src =
      kCompact ? pool
               : static_cast<const unsigned char *>(a.rows) + (int64_t)blockIdx.z * a.rows_ls +
                     (int64_t)b * a.rows_bs + col;
  const int64_t src_row = kCompact ? a.row_bytes : a.rows_ts;
  for (int i0 = 0; i0 < n; i0 += kWriteBatch) {
    uint4 x[kWriteBatch];
#pragma unroll
    for (int j = 0; j < kWriteBatch; ++j)
      if (i0 + j < n)
        x[j] = *reinterpret_cast<const uint4 *>(src + moves[2 * (i0 + j)] * src_row);
#pragma unroll
    for (int j = 0; j < kWriteBatch; ++j)
      if (i0 + j < n && (!kCompact || moves[2 * (i0 + j)] != moves[2 * (i0 + j) + 1]))
        *reinterpret_cast<uint4 *>(pool + moves[2 * (i0 + j) + 1] * a.row_bytes) = x[j];
  }
}

constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;   // 16-byte loads in flight per thread

// Block (x: piece of a page, y: layer, z: pair).  A pair out of range, or a page
// copied onto itself, moves nothing.  Each byte is read and written once, past the
// caches: 16 states of 3 layers, 604 MB both ways, 89.6 us, 6.7 TB/s, the rate of a
// plain copy; one page of 24 layers 5.9 us, the launch.
__global__ void __launch_bounds__(kCopyThreads)
kda_cache_copy_pages_kernel(unsigned char *pool, const int32_t *__restrict__ src,
                            const int32_t *__restrict__ dst, int32_t n_pages, int64_t page_bytes,
                            int32_t *status) {
  const int32_t s = src[blockIdx.z], d = dst[blockIdx.z];
  if (s < 0 || s >= n_pages || d < 0 || d >= n_pages) {
    if (threadIdx.x == 0 && blockIdx.x == 0 && blockIdx.y == 0) flag_status(status);
    return;
  }
  if (s == d) return;
  unsigned char *layer = pool + (int64_t)blockIdx.y * n_pages * page_bytes;
  const uint4 *from = reinterpret_cast<const uint4 *>(layer + (int64_t)s * page_bytes);
  uint4 *to = reinterpret_cast<uint4 *>(layer + (int64_t)d * page_bytes);
  const int64_t n = page_bytes / 16;
  const int64_t step = (int64_t)gridDim.x * kCopyThreads * kCopyUnroll;
  for (int64_t i0 = (int64_t)blockIdx.x * kCopyThreads * kCopyUnroll + threadIdx.x; i0 < n;
       i0 += step) {
    uint4 x[kCopyUnroll];
#pragma unroll
    for (int j = 0; j < kCopyUnroll; ++j)
      if (i0 + j * kCopyThreads < n) x[j] = __ldcs(from + i0 + j * kCopyThreads);
#pragma unroll
    for (int j = 0; j < kCopyUnroll; ++j)
      if (i0 + j * kCopyThreads < n) __stcs(to + i0 + j * kCopyThreads, x[j]);
  }
}

}  // namespace

cudaError_t launch_cache_write(const CacheWriteArgs &a, cudaStream_t stream) {
  if (a.B == 0 || a.L == 0) return cudaSuccess;
  const int64_t cols = a.row_bytes / 16;
  const int64_t gx = (cols + kWriteThreads - 1) / kWriteThreads;
  if (gx > 0x7fffffffLL) return cudaErrorInvalidValue;
  const size_t smem = (size_t)a.T * 16;
  // grid y and z reach 65535: longer batches go in pieces
  for (int32_t b0 = 0; b0 < a.B; b0 += 65535)
    for (int32_t l0 = 0; l0 < a.L; l0 += 65535) {
      CacheWriteArgs c = a;
      c.B = a.B - b0 < 65535 ? a.B - b0 : 65535;
      c.L = a.L - l0 < 65535 ? a.L - l0 : 65535;
      c.block_table = a.block_table + (int64_t)b0 * a.max_pages;
      c.start = a.start + b0;
      c.path = a.path ? a.path + (int64_t)b0 * a.T : nullptr;
      c.n_write = a.n_write ? a.n_write + b0 : nullptr;
      c.cache = static_cast<unsigned char *>(a.cache) +
                (int64_t)l0 * a.n_pages * a.page_size * a.row_bytes;
      if (a.rows)
        c.rows = static_cast<const unsigned char *>(a.rows) + l0 * a.rows_ls + b0 * a.rows_bs;
      const dim3 grid((unsigned)gx, (unsigned)c.B, (unsigned)c.L);
      if (a.rows)
        kda_cache_write_kernel<false><<<grid, kWriteThreads, smem, stream>>>(c);
      else
        kda_cache_write_kernel<true><<<grid, kWriteThreads, smem, stream>>>(c);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
  return cudaSuccess;
}

cudaError_t launch_cache_copy_pages(void *cache, const int32_t *src, const int32_t *dst, int32_t n,
                                    int32_t L, int32_t n_pages, int64_t page_bytes,
                                    int32_t *status, cudaStream_t stream) {
  if (n == 0 || L == 0) return cudaSuccess;
  const int64_t per_block = (int64_t)kCopyThreads * kCopyUnroll * 16;
  int64_t gx = (page_bytes + per_block - 1) / per_block;
  if (gx > 4096) gx = 4096;
  unsigned char *pool = static_cast<unsigned char *>(cache);
  for (int32_t n0 = 0; n0 < n; n0 += 65535)
    for (int32_t l0 = 0; l0 < L; l0 += 65535) {
      const dim3 grid((unsigned)gx, (unsigned)(L - l0 < 65535 ? L - l0 : 65535),
                      (unsigned)(n - n0 < 65535 ? n - n0 : 65535));
      kda_cache_copy_pages_kernel<<<grid, kCopyThreads, 0, stream>>>(
          pool + (int64_t)l0 * n_pages * page_bytes, src + n0, dst + n0, n_pages, page_bytes,
          status);
      const cudaError_t e = cudaGetLastError();
      if (e != cudaSuccess) return e;
    }
  return cudaSuccess;
}

}  // namespace kda
