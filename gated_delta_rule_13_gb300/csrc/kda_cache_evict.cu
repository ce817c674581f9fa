// Eviction of cached rows by the weight they have been given (kda_cache_evict).
//
// A sequence of n > budget rows keeps its first `first` rows, its last `recent` rows and,
// of those between, the budget - first - recent of the greatest weight (of equal ones the
// earlier).  Kept rows in front of `last` = budget - recent stay where they are; the places
// there that fall free (holes) take the kept rows from behind (movers), the i-th hole the
// i-th mover; the last rows move up together.  So nothing moves that need not: there are
// as many movers as holes, they come from [last, n - recent) and go to [first, last), and
// the cache's rows have no order but the last ones.
//
// Selection: one block a (layer, sequence).  A weight becomes an unsigned number of the
// same order; its bytes are fixed one after another, from the top, by counting the
// candidates that share the bytes before (a radix selection), which leaves the last kept
// value and how many of its equals are kept.  Each warp then walks its own stretch of the
// candidates in order with the counts of the stretches before it, so that ranks need no
// sorting.  The moves follow in a second kernel.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/kda.h"
#include "kda_latent_tc.cuh"
#include "kda_rows.h"

namespace kda {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;

// Scratch of a (layer, sequence): [0] moves, [1] rows that move up, [2], [3] unused, then
// `budget` destinations and `budget` sources.
constexpr int kHead = 4;
__host__ __device__ inline int64_t scratch_ints(int32_t budget) {
  return kHead + 2 * (int64_t)((budget + 3) / 4 * 4);
}

// In the order of the weights; one that is no number is below all others.
__device__ __forceinline__ uint32_t order_of(float w) {
  if (w != w) return 0;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return u >> 31 ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kThreads) kda_evict_select_kernel(const CacheEvictArgs a) {
  __shared__ int hist[256], counts[3][kWarps], pick[2], bad;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t lb = blockIdx.x;
  const int b = (int)(lb % a.B);
  const int cap = a.max_pages * a.page_size;
  const int n = a.seq_lens[b];
  const float *w = a.weights + lb * cap;
  float *to = a.weights_out + lb * cap;
  int32_t *origin = a.origin + lb * a.budget;
  int32_t *moves = a.moves + lb * scratch_ints(a.budget);
  int32_t *dst = moves + kHead, *src = dst + (a.budget + 3) / 4 * 4;
  const bool same = w == to;
  latent::pdl_launch_dependents();

  if (tid == 0) bad = n < 0 || n > cap;
  __syncthreads();
  if (!bad) {
    const int pages = (n + a.page_size - 1) / a.page_size;
    bool wrong = false;
    for (int i = tid; i < pages; i += kThreads) {
      const int32_t id = a.block_table[(int64_t)b * a.max_pages + i];
      wrong = wrong || id < 0 || id >= a.n_pages;
    }
    if (wrong) bad = 1;
  }
  __syncthreads();
  const bool refused = bad != 0;
  if (tid == 0) {
    moves[0] = moves[1] = 0;
    if (refused && a.status) atomicCAS(a.status, 0, (int32_t)KDA_ERR_INVALID_ARG);
    if (lb < a.B) a.new_lens[b] = refused ? n : min(n, a.budget);
  }
  if (refused || n <= a.budget) {          // all rows stay
    for (int i = tid; i < a.budget; i += kThreads) origin[i] = !refused && i < n ? i : -1;
    const int live = refused ? cap : n;
    if (!same)
      for (int i = tid; i < live; i += kThreads) to[i] = w[i];
    for (int i = live + tid; i < cap; i += kThreads) to[i] = 0.f;
    return;
  }

  // candidates [lo, hi), `keep` of them stay
  const int lo = a.first, hi = n - a.recent, last = a.budget - a.recent;
  const int keep = last - lo;
  uint32_t prefix = 0, known = 0;          // the last kept value's upper bytes
  int left = keep;                         // kept ones among those that share them
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += kThreads) hist[i] = 0;
    __syncthreads();
    for (int i = lo + tid; i < hi; i += kThreads) {
      const uint32_t u = order_of(w[i]);
      if ((u & known) == prefix) atomicAdd(&hist[u >> shift & 255], 1);
    }
    __syncthreads();
    if (warp == 0) {                       // the byte of the left-th from the top
      int mine[8], sum = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) sum += mine[k] = hist[255 - (8 * lane + k)];
      int upto = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      int above = upto - sum;
      if (above < left && upto >= left)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          if (above < left && above + mine[k] >= left) {
            pick[0] = 255 - (8 * lane + k);
            pick[1] = left - above;
          }
          above += mine[k];
        }
      if (left == 0 && lane == 0) {        // none is kept: above every value there is
        pick[0] = 255;
        pick[1] = 0;
      }
    }
    __syncthreads();
    prefix |= (uint32_t)pick[0] << shift;
    known |= 255u << shift;
    left = pick[1];
    __syncthreads();
  }
  // kept: above `prefix`, and the first `left` of its equals.  (With none to keep, prefix is
  // all ones, which no weight becomes, and left is 0.)
  const int stretch = ((hi - lo + kWarps - 1) / kWarps + 31) / 32 * 32;
  const int s0 = min(lo + warp * stretch, hi), s1 = min(s0 + stretch, hi);
  int equal = 0;
  for (int i = s0 + lane; i < s1; i += 32) equal += order_of(w[i]) == prefix;
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) counts[0][warp] = equal;
  __syncthreads();
  const auto before = [&](const int *c) {
    return __reduce_add_sync(0xffffffffu, lane < warp ? c[lane] : 0);
  };
  const int equal0 = before(counts[0]);
  // Two walks over the stretch: holes and movers are counted, then listed.
  int hole0 = 0, mover0 = 0;
  for (int pass = 0; pass < 2; ++pass) {
    int eq = equal0, holes = 0, movers = 0;
    for (int i0 = s0; i0 < s1; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t u = i < s1 ? order_of(w[i]) : 0;
      const unsigned same_value = __ballot_sync(0xffffffffu, i < s1 && u == prefix);
      const unsigned under = (1u << lane) - 1;
      const bool kept = i < s1 && (u > prefix || (u == prefix && eq + __popc(same_value & under) < left));
      eq += __popc(same_value);
      const bool hole = i < s1 && !kept && i < last, mover = kept && i >= last;
      const unsigned hs = __ballot_sync(0xffffffffu, hole), ms = __ballot_sync(0xffffffffu, mover);
      if (pass == 1) {
        if (hole) dst[hole0 + holes + __popc(hs & under)] = i;
        if (mover) src[mover0 + movers + __popc(ms & under)] = i;
        if (i < last && kept) origin[i] = i;
        if (i < last && kept && !same) to[i] = w[i];
      }
      holes += __popc(hs);
      movers += __popc(ms);
    }
    if (pass == 0) {
      if (lane == 0) {
        counts[1][warp] = holes;
        counts[2][warp] = movers;
      }
      __syncthreads();
      hole0 = before(counts[1]);
      mover0 = before(counts[2]);
    }
  }
  __syncthreads();
  int total = 0;
  for (int k = 0; k < kWarps; ++k) total += counts[1][k];
  if (tid == 0) {
    moves[0] = total;
    moves[1] = a.recent;
  }
  for (int i = tid; i < lo; i += kThreads) {
    origin[i] = i;
    if (!same) to[i] = w[i];
  }
  for (int i = tid; i < total; i += kThreads) {
    origin[dst[i]] = src[i];
    to[dst[i]] = w[src[i]];
  }
  __syncthreads();
  // The last rows move up by n - budget: chunks in order, a chunk read before it is written.
  for (int i0 = 0; i0 < a.recent; i0 += kThreads) {
    const int i = i0 + tid;
    float v = 0.f;
    if (i < a.recent) {
      v = w[hi + i];
      origin[last + i] = hi + i;
    }
    __syncthreads();
    if (i < a.recent) to[last + i] = v;
  }
  __syncthreads();
  for (int i = a.budget + tid; i < cap; i += kThreads) to[i] = 0.f;
}

constexpr int kMoveThreads = 256;
constexpr int kSlice = 8;                  // 16-byte columns of a block
constexpr int kMoveRows = kMoveThreads / kSlice;
constexpr int kMoveBatch = 8;              // rows in flight per thread

// Block (x: 128-byte column slice and piece of the moves, y: layer and sequence).  Movers'
// places and holes have no row in common, so they move in any order.  The last rows may
// take movers' old places, and one another's: they move after the movers (within the
// block, or in a launch of its own), chunks in order, a chunk read before it is written.
template <bool kMoves, bool kUp>
__global__ void __launch_bounds__(kMoveThreads)
kda_evict_move_kernel(const CacheEvictArgs a, const int32_t slices, const int32_t pieces,
                      const int64_t lb0) {
  const int64_t lb = lb0 + blockIdx.y;
  const int b = (int)(lb % a.B);
  const int64_t layer = lb / a.B;
  const int slice = blockIdx.x % slices, piece = blockIdx.x / slices;
  const int row = threadIdx.x / kSlice;
  const int64_t col = ((int64_t)slice * kSlice + threadIdx.x % kSlice) * 16;
  const bool live = col < a.row_bytes;
  unsigned char *pool = static_cast<unsigned char *>(a.cache) +
                        layer * a.n_pages * a.page_size * a.row_bytes + col;
  const int32_t *table = a.block_table + (int64_t)b * a.max_pages;
  const int32_t *moves = a.moves + lb * scratch_ints(a.budget);
  const int32_t *dst = moves + kHead, *src = dst + (a.budget + 3) / 4 * 4;
  const auto at = [&](int pos) {
    const int pg = pos / a.page_size;
    return reinterpret_cast<uint4 *>(
        pool + ((int64_t)table[pg] * a.page_size + (pos - pg * a.page_size)) * a.row_bytes);
  };
  latent::pdl_wait();
  if (kMoves && live) {
    const int n = moves[0];
    constexpr int kStep = kMoveRows * kMoveBatch;
    for (int i0 = piece * kStep; i0 < n; i0 += pieces * kStep) {
      uint4 x[kMoveBatch];
#pragma unroll
      for (int j = 0; j < kMoveBatch; ++j) {
        const int i = i0 + j * kMoveRows + row;
        if (i < n) x[j] = *at(src[i]);
      }
#pragma unroll
      for (int j = 0; j < kMoveBatch; ++j) {
        const int i = i0 + j * kMoveRows + row;
        if (i < n) *at(dst[i]) = x[j];
      }
    }
  }
  if (kUp) {
    const int n = moves[1];
    if (n == 0) return;
    if (kMoves) __syncthreads();           // the movers have been read
    const int hi = a.seq_lens[b] - n, last = a.budget - n;
    constexpr int kStep = kMoveRows * kMoveBatch;
    for (int i0 = 0; i0 < n; i0 += kStep) {
      uint4 x[kMoveBatch];
#pragma unroll
      for (int j = 0; j < kMoveBatch; ++j) {
        const int i = i0 + j * kMoveRows + row;
        if (live && i < n) x[j] = *at(hi + i);
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < kMoveBatch; ++j) {
        const int i = i0 + j * kMoveRows + row;
        if (live && i < n) *at(last + i) = x[j];
      }
    }
  }
}

template <bool kMoves, bool kUp>
cudaError_t launch_moves(const CacheEvictArgs &a, int32_t slices, int32_t pieces, bool overlap,
                         cudaStream_t stream) {
  const int64_t all = (int64_t)a.L * a.B;
  for (int64_t lb = 0; lb < all; lb += 65535) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(slices * pieces), (unsigned)(all - lb < 65535 ? all - lb : 65535));
    cfg.blockDim = dim3(kMoveThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = overlap && lb == 0 ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kda_evict_move_kernel<kMoves, kUp>, a, slices,
                                             pieces, lb);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t cache_evict_scratch_bytes(int32_t L, int32_t B, int32_t budget) {
  return (size_t)L * B * scratch_ints(budget) * sizeof(int32_t);
}

cudaError_t launch_cache_evict(const CacheEvictArgs &a, cudaStream_t stream) {
  const int64_t all = (int64_t)a.L * a.B;
  if (all == 0) return cudaSuccess;
  kda_evict_select_kernel<<<(unsigned)all, kThreads, 0, stream>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int64_t cols = a.row_bytes / 16;
  const int32_t slices = (int32_t)((cols + kSlice - 1) / kSlice);
  const int sms = latent::sm_count() > 0 ? latent::sm_count() : 1;
  const int64_t blocks = all * slices;
  // Blocks enough that each may have its columns of all rows: one launch.  Else the moves
  // are shared out, and the last rows follow by themselves.
  if (blocks >= sms / 2) return launch_moves<true, true>(a, slices, 1, true, stream);
  const int64_t most = (a.budget - a.first + kMoveRows * kMoveBatch - 1) / (kMoveRows * kMoveBatch);
  int64_t pieces = 2 * sms / blocks;
  if (pieces > most) pieces = most;
  if (pieces < 1) pieces = 1;
  e = launch_moves<true, false>(a, slices, (int32_t)pieces, true, stream);
  if (e != cudaSuccess) return e;
  return a.recent > 0 ? launch_moves<false, true>(a, slices, 1, false, stream) : cudaSuccess;
}

}  // namespace kda
