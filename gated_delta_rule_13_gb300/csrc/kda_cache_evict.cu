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
// Selection, one block a (layer, sequence): a weight becomes an unsigned number of the same
// order.  Counts by its upper 11 bits (four bins an octave) tell in which bin the last kept one
// is; counts by the bits below do so within the bin, 11 and 10 more (a radix selection), until
// all that share the bits are kept or few do, which are ranked against each other.  Equal weights
// go by their order.  Each warp then walks its own stretch of the candidates in order and, with
// the counts of the stretches before it, lists holes and movers in the workspace.
//
// Moves, in a second kernel that starts beside the first.  The last rows take places that movers
// leave, and where n - budget < recent also one another's.  Where they do not, a place and all
// that goes through it are one warp's: first the mover leaves, then the last row comes.  Where
// they do (and then there are few movers), a block has some columns of all rows and takes the
// movers first.  No block waits for another.
//
// Measured: prompts of 3000 .. 8192 rows cut to 2048, 8 sequences, 24 layers, 131 us, of which the
// selection is 19 (latency: a dozen dependent steps) and the moves 110 (638 MB both ways, 5.8
// TB/s, rows of 1,152 bytes at random places; 95 at a plain copy's rate).  Fewer bytes in flight
// than 144 a thread, or more threads with less, took 133 to 184 us in all.  One row of each of 16
// requests of 2049 (a table of 2112 places): 7.8 us in one launch, 7.9 in place, which takes two.
//
// A call writes every place of the weights, so that it costs by the table's capacity too, the zeros
// of a sequence being one block's: the same row with 16 K places 8.9 us in place (10.9 to another
// buffer), with 128 K 16 (18); of 24 layers of these requests, in place, 28, 32 and 66.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/kda.h"
#include "kda_latent_tc.cuh"
#include "kda_rows.h"

namespace kda {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
// Candidates in shared memory, by the table's capacity, which is what the host knows: of up to
// kKeep places room for all; of more so many that three blocks fit an SM, and a sequence with more
// candidates than these reads its weights again in every walk, also where SMs have one block each
// (60000 rows to 8000 80 to 90 us, one load in flight 163; 20000 rows in place 30).
constexpr int kKeep = 49152, kKeepLong = 16384;
constexpr int kBins = 2048;
constexpr int kFew = 256;                  // ranked directly
constexpr int kShort = 4096, kLeast = 4;   // one launch: places of the table at most, blocks at least
static_assert(kBins % kThreads == 0 && kBins <= 4 * kThreads, "a thread has four bins at most");

// Scratch of a (layer, sequence): what to move, then as many numbers as the budget each of
// destinations and sources of movers (the moves), then where the row at each of the last
// `recent` places goes, -1: nowhere.
struct Moves {
  int32_t movers, near, recent, n;         // near: movers from places that the last rows take
};
constexpr int kHead = 4;
static_assert(sizeof(Moves) == kHead * sizeof(int32_t), "head of the scratch");
__host__ __device__ inline int64_t list_ints(int32_t budget) { return ((int64_t)budget + 3) / 4 * 4; }
__host__ __device__ inline int64_t scratch_ints(int32_t budget) { return kHead + 3 * list_ints(budget); }

// In the order of the weights; one that is no number is below all others.
__device__ __forceinline__ uint32_t order_of(float w) {
  if (w != w) return 0;
  const uint32_t u = __float_as_uint(w == 0.f ? 0.f : w);
  return u >> 31 ? ~u : u | 0x80000000u;
}

constexpr int kMoveThreads = 256;
constexpr int kLeastPieces = 8;            // blocks of a sequence's moves
constexpr int kSlots = 9, kColSlots = 5;   // 16-byte pieces in flight per thread: rows, columns

// The moves of a (layer, sequence), shared out over `pieces` blocks of kN threads.
template <int kN>
__device__ __forceinline__ void move_rows(const CacheEvictArgs &a, const int64_t lb, const Moves m,
                                          const int32_t *via, const int piece, const int pieces) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int32_t *table = a.block_table + (int64_t)(lb % a.B) * a.max_pages;
  const int32_t *dst = a.moves + lb * scratch_ints(a.budget) + kHead, *src = dst + list_ints(a.budget);
  unsigned char *pool = static_cast<unsigned char *>(a.cache) +
                        lb / a.B * a.n_pages * a.page_size * a.row_bytes;
  const int vecs = (int)(a.row_bytes / 16);
  const auto pool_row = [&](int pos) {
    const int pg = pos / a.page_size;
    return table[pg] * a.page_size + (pos - pg * a.page_size);
  };
  const auto piece_at = [&](int row, int col) {
    return reinterpret_cast<uint4 *>(pool + row * a.row_bytes + (int64_t)col * 16);
  };
  if (m.movers == 0 && m.recent == 0) return;
  const int hi = m.n - m.recent, last = a.budget - m.recent;

  if (m.n - a.budget >= m.recent) {
    // ---- whole rows, some at a time for each warp: the places of the last rows, then the
    // movers from behind these
    const int wide = min(vecs, 32 * kSlots);             // pieces of a row at a time
    const int group = min(32, 32 * kSlots / wide);       // rows at a time
    int place[kSlots];                                   // row of the group, piece
#pragma unroll
    for (int j = 0; j < kSlots; ++j) {
      const int v = lane + 32 * j, r = v / wide;
      place[j] = r < group ? r << 16 | (v - r * wide) : -1;
    }
    // rows s to rows d, each by the lane that has that row of the group; -1: none
    const auto copy = [&](int s, int d) {
      for (int c0 = 0; c0 < vecs; c0 += wide) {
        uint4 x[kSlots];
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
          const int row = __shfl_sync(0xffffffffu, s, place[j] < 0 ? 0 : place[j] >> 16);
          const int col = c0 + (place[j] & 0xffff);
          if (place[j] >= 0 && row >= 0 && col < vecs) x[j] = *piece_at(row, col);
        }
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
          const int row = __shfl_sync(0xffffffffu, d, place[j] < 0 ? 0 : place[j] >> 16);
          const int col = c0 + (place[j] & 0xffff);
          if (place[j] >= 0 && row >= 0 && col < vecs) *piece_at(row, col) = x[j];
        }
      }
    };
    const int far = m.movers - m.near, all = m.recent + far;
    for (int i0 = (piece * (kN / 32) + warp) * group; i0 < all; i0 += pieces * (kN / 32) * group) {
      const int i = i0 + lane;
      int s = -1, d = -1, out = -1;
      if (lane < group && i < all) {
        if (i < m.recent) {
          s = pool_row(hi + i);
          d = pool_row(last + i);
          out = via[i] >= 0 ? pool_row(via[i]) : -1;
        } else {
          s = pool_row(src[m.near + i - m.recent]);
          d = pool_row(dst[m.near + i - m.recent]);
        }
      }
      if (__any_sync(0xffffffffu, out >= 0)) copy(out >= 0 ? d : -1, out);   // the same lanes, in order
      copy(s, d);
    }
    return;
  }

  // ---- some columns of all rows, chunks in order, a chunk read before it is written
  // (of few rows of many sequences two pieces, each of half the columns: 384 times 65 rows 33 us,
  // with eight 44; 1500 rows 338 and 326.  Where between these the two meet has not been measured.)
  const int use = kN == kMoveThreads && pieces == kLeastPieces && m.movers + m.recent < 1024 ? 2 : pieces;
  if (piece >= use) return;
  const int per = (vecs + use - 1) / use, c0 = piece * per, c1 = min(c0 + per, vecs);
  for (int cc = c0; cc < c1; cc += kN) {
    const int width = min(c1 - cc, kN), lanes = kN / width;
    const int col = cc + tid % width, r = tid / width;
    for (int kind = 0; kind < 2; ++kind) {               // movers, then the last rows
      const int rows = kind ? m.recent : m.movers;
      for (int i0 = 0; i0 < rows; i0 += lanes * kColSlots) {
        uint4 x[kColSlots];
#pragma unroll
        for (int j = 0; j < kColSlots; ++j) {
          const int i = i0 + j * lanes + r;
          if (r < lanes && i < rows) x[j] = *piece_at(pool_row(kind ? hi + i : src[i]), col);
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kColSlots; ++j) {
          const int i = i0 + j * lanes + r;
          if (r < lanes && i < rows) *piece_at(pool_row(kind ? last + i : dst[i]), col) = x[j];
        }
      }
    }
  }
}

// Where sequences are few, their table is short and the weights go to another buffer, one launch:
// each of `pieces` blocks of a (layer, sequence) selects by itself (they write the same to the
// lists, and in place would write what the others read), and takes its share of the moves.
template <bool kMove>
__global__ void __launch_bounds__(kThreads, kMove ? 1 : 3)
kda_evict_select_kernel(const CacheEvictArgs a, const int32_t room, const int32_t pieces) {
  extern __shared__ uint32_t keys[];       // [room] candidates, as numbers
  __shared__ int hist[kBins], counts[2][kWarps], pick[3], bad, gathered;
  __shared__ uint2 few[kFew];              // value, position
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t lb = kMove ? blockIdx.x / pieces : blockIdx.x;
  const int piece = kMove ? (int)(blockIdx.x - lb * pieces) : 0;
  const int b = (int)(lb % a.B);
  const int cap = a.max_pages * a.page_size;
  const int n = a.seq_lens[b];
  const float *w = a.weights + lb * cap;
  float *to = a.weights_out + lb * cap;
  int32_t *origin = a.origin + lb * a.budget;
  int32_t *scratch = a.moves + lb * scratch_ints(a.budget);
  int32_t *dst = scratch + kHead, *src = dst + list_ints(a.budget);
  // (a block that moves has it to itself: it is not the same at all times)
  int32_t *via = kMove ? reinterpret_cast<int32_t *>(keys + room) : src + list_ints(a.budget);
  const int32_t *table = a.block_table + (int64_t)b * a.max_pages;
  const bool same = w == to;
  // candidates [lo, hi), a stretch a warp; `keep` of them stay
  const int lo = a.first, hi = (n < 0 || n > cap ? 0 : n) - a.recent, last = a.budget - a.recent;
  const int stretch = ((max(hi - lo, 0) + kWarps - 1) / kWarps + 31) / 32 * 32;
  const int s0 = min(lo + warp * stretch, hi), s1 = min(s0 + stretch, hi);
  if constexpr (!kMove) latent::pdl_launch_dependents();

  if (tid == 0) bad = n < 0 || n > cap;
  __syncthreads();
  const bool here = hi - lo <= room;
  if (!bad) {
    const int pages = (n + a.page_size - 1) / a.page_size;
    const int32_t id0 = tid < pages ? table[tid] : 0;
    if (here && n > a.budget)              // each its own ones
#pragma unroll 4
      for (int i = s0 + lane; i < s1; i += 32) keys[i - lo] = order_of(w[i]);
    bool wrong = id0 < 0 || id0 >= a.n_pages;
    for (int i = tid + kThreads; i < pages; i += kThreads)
      wrong = wrong || table[i] < 0 || table[i] >= a.n_pages;
    if (wrong) bad = 1;
  }
  __syncthreads();
  const bool refused = bad != 0;
  if (tid == 0) {
    if (refused && a.status) atomicCAS(a.status, 0, (int32_t)KDA_ERR_INVALID_ARG);
    if (lb < a.B) a.new_lens[b] = refused ? n : min(n, a.budget);
  }
  if (refused || n <= a.budget) {          // all rows stay
    if (piece > 0) return;
    if (!kMove && tid == 0) *reinterpret_cast<Moves *>(scratch) = Moves{0, 0, 0, 0};
    for (int i = tid; i < a.budget; i += kThreads) origin[i] = !refused && i < n ? i : -1;
    const int live = refused ? cap : n;
    if (!same)
      for (int i = tid; i < live; i += kThreads) to[i] = w[i];
    for (int i = live + tid; i < cap; i += kThreads) to[i] = 0.f;
    return;
  }

  const float recent0 = tid < a.recent ? w[hi + tid] : 0.f;   // needed at the end

  // f(position, value), the warp together, in order; positions >= s1 are none
  const auto each = [&](auto f) {
    if (here) {
#pragma unroll 2
      for (int i0 = s0; i0 < s1; i0 += 32) f(i0 + lane, i0 + lane < s1 ? keys[i0 + lane - lo] : 0);
    } else {
      constexpr int kAhead = 8;              // in flight
#pragma unroll 1
      for (int i0 = s0; i0 < s1; i0 += 32 * kAhead) {
        float v[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) v[k] = i0 + 32 * k + lane < s1 ? w[i0 + 32 * k + lane] : 0.f;
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
          if (i0 + 32 * k < s1)
            f(i0 + 32 * k + lane, i0 + 32 * k + lane < s1 ? order_of(v[k]) : 0);
      }
    }
  };
  // Of counts in hist[0 .. bins), the bin of the `left`-th from the top: pick = bin, what is
  // left of it there, its count.
  const auto find = [&](int bins, int left) {
    constexpr int kPer = kBins / kThreads;
    int c[kPer], sum = 0;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int at = bins - 1 - (kPer * tid + k);
      sum += c[k] = at >= 0 ? hist[at] : 0;
    }
    int upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) counts[0][warp] = upto;
    __syncthreads();
    upto += __reduce_add_sync(0xffffffffu, lane < warp ? counts[0][lane] : 0);
    int above = upto - sum;
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      if (above < left && above + c[k] >= left) {
        pick[0] = bins - 1 - (kPer * tid + k);
        pick[1] = left - above;
        pick[2] = c[k];
      }
      above += c[k];
    }
    __syncthreads();
  };
  // Kept: what is above `value`, and of its equals those up to `place`.
  uint32_t value = last > lo ? 0 : ~0u, known = 0;
  int place = last > lo ? 0x7fffffff : -1, left = last - lo;
  for (int shift = 21; last > lo && shift >= 0; shift = shift == 21 ? 10 : shift - 10) {
    const uint32_t mask = shift > 0 ? 2047 : 1023;
    for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
    if (tid == 0) gathered = 0;
    __syncthreads();
    each([&](int i, uint32_t u) {
      if (i < s1 && (u & known) == value) atomicAdd(&hist[u >> shift & mask], 1);
    });
    __syncthreads();
    find((int)mask + 1, left);
    value |= (uint32_t)pick[0] << shift;
    known |= mask << shift;
    left = pick[1];
    const int inside = pick[2];
    if (left == inside) break;               // all that share the bits are kept
    if (inside <= kFew) {
      each([&](int i, uint32_t u) {
        if (i < s1 && (u & known) == value) few[atomicAdd(&gathered, 1)] = make_uint2(u, (uint32_t)i);
      });
      __syncthreads();
      for (int k0 = 0; k0 < inside; k0 += kThreads / 4) {   // four threads each
        const int k = k0 + tid / 4;
        const uint2 me = few[min(k, inside - 1)];
        int rank = 0;
#pragma unroll 4
        for (int l = tid % 4; l < inside; l += 4) {
          const uint2 x = few[l];
          rank += x.x > me.x || (x.x == me.x && x.y < me.y);
        }
        rank += __shfl_xor_sync(0xffffffffu, rank, 1);
        rank += __shfl_xor_sync(0xffffffffu, rank, 2);
        if (k < inside && rank == left - 1) {
          pick[0] = (int)me.x;
          pick[1] = (int)me.y;
        }
      }
      __syncthreads();
      value = (uint32_t)pick[0];
      place = pick[1];
      break;
    }
    if (shift == 0) {                        // more equals: the place of the left-th
      int equal = 0;
      each([&](int i, uint32_t u) { equal += __popc(__ballot_sync(0xffffffffu, i < s1 && u == value)); });
      if (lane == 0) counts[0][warp] = equal;
      __syncthreads();
      int seen = __reduce_add_sync(0xffffffffu, lane < warp ? counts[0][lane] : 0);
      each([&](int i, uint32_t u) {
        const unsigned alike = __ballot_sync(0xffffffffu, i < s1 && u == value);
        if (alike >> lane & 1 && seen + __popc(alike & ((1u << lane) - 1)) == left - 1) pick[0] = i;
        seen += __popc(alike);
      });
      __syncthreads();
      place = pick[0];
    }
  }
  __syncthreads();                         // counts are free

  // ---- holes and movers, counted and listed
  const auto kept = [&](int i, uint32_t u) {
    return i < s1 && (u > value || (u == value && i <= place));
  };
  int holes = 0, movers = 0;
  each([&](int i, uint32_t u) {
    const bool yes = kept(i, u);
    holes += i < s1 && !yes && i < last;
    movers += yes && i >= last;
  });
  holes = __reduce_add_sync(0xffffffffu, holes);
  movers = __reduce_add_sync(0xffffffffu, movers);
  if (lane == 0) {
    counts[0][warp] = holes;
    counts[1][warp] = movers;
  }
  for (int i = tid; i < a.recent; i += kThreads) via[i] = -1;
  __syncthreads();
  int hole = __reduce_add_sync(0xffffffffu, lane < warp ? counts[0][lane] : 0);
  int mover = __reduce_add_sync(0xffffffffu, lane < warp ? counts[1][lane] : 0);
  const int total = __reduce_add_sync(0xffffffffu, lane < kWarps ? counts[0][lane] : 0);
  const unsigned under = (1u << lane) - 1;
  each([&](int i, uint32_t u) {
    const bool yes = kept(i, u), h = i < s1 && !yes && i < last, m = yes && i >= last;
    const unsigned hs = __ballot_sync(0xffffffffu, h), ms = __ballot_sync(0xffffffffu, m);
    if (h) dst[hole + __popc(hs & under)] = i;
    if (m) src[mover + __popc(ms & under)] = i;
    hole += __popc(hs);
    mover += __popc(ms);
  });
  constexpr int kBatch = 4;                // in flight per thread
  for (int i0 = tid; i0 < last && piece == 0; i0 += kBatch * kThreads) {   // what stays in place
    float v[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) v[k] = w[min(i0 + k * kThreads, last - 1)];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * kThreads;
      const uint32_t u = order_of(v[k]);
      if (i < last && (i < lo || u > value || (u == value && i <= place))) {
        origin[i] = i;
        if (!same) to[i] = v[k];
      }
    }
  }
  __syncthreads();                         // the lists; and no weight is looked at again

  // ---- weights of movers and of the last rows (chunks in order, read before written)
  int near = 0;
  for (int i0 = tid; i0 < total; i0 += kBatch * kThreads) {
    int from[kBatch], at[kBatch];
    float v[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = min(i0 + k * kThreads, total - 1);
      from[k] = src[i];
      at[k] = dst[i];
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) v[k] = w[from[k]];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (i0 + k * kThreads < total) {
        if (piece == 0) {
          origin[at[k]] = from[k];
          to[at[k]] = v[k];
        }
        if (from[k] < a.budget) {
          via[from[k] - last] = at[k];
          ++near;
        }
      }
  }
  near = __reduce_add_sync(0xffffffffu, near);
  if (lane == 0) counts[0][warp] = near;
  __syncthreads();
  near = __reduce_add_sync(0xffffffffu, lane < kWarps ? counts[0][lane] : 0);
  const Moves moves{total, near, a.recent, n};
  if (!kMove && tid == 0) *reinterpret_cast<Moves *>(scratch) = moves;
  if (piece == 0) {
    for (int i0 = 0; i0 < a.recent; i0 += kThreads) {
      const int i = i0 + tid;
      float v = recent0;
      if (i < a.recent) {
        if (i0 > 0) v = w[hi + i];
        origin[last + i] = hi + i;
      }
      __syncthreads();
      if (i < a.recent) to[last + i] = v;
    }
    __syncthreads();
    for (int i = a.budget + tid; i < cap; i += kThreads) to[i] = 0.f;
  }
  if constexpr (kMove) {
    __syncthreads();                       // the lists, of which this block has written all
    move_rows<kThreads>(a, lb, moves, via, piece, pieces);
  }
}

// Block (x: one of `pieces`, y: layer and sequence).
__global__ void __launch_bounds__(kMoveThreads, 2)
kda_evict_move_kernel(const CacheEvictArgs a, const int32_t pieces, const int64_t lb0) {
  const int64_t lb = lb0 + blockIdx.y;
  const int32_t *scratch = a.moves + lb * scratch_ints(a.budget);
  latent::pdl_wait();
  move_rows<kMoveThreads>(a, lb, *reinterpret_cast<const Moves *>(scratch),
                          scratch + kHead + 2 * list_ints(a.budget), blockIdx.x, pieces);
}


}  // namespace

size_t cache_evict_scratch_bytes(int32_t L, int32_t B, int32_t budget) {
  return (size_t)L * B * scratch_ints(budget) * sizeof(int32_t);
}

cudaError_t launch_cache_evict(const CacheEvictArgs &a, cudaStream_t stream) {
  const int64_t all = (int64_t)a.L * a.B;
  if (all == 0) return cudaSuccess;
  const int64_t cap = (int64_t)a.max_pages * a.page_size;
  const int64_t sms = latent::sm_count() > 0 ? latent::sm_count() : 1;
  const int32_t room = (int32_t)(cap <= kKeep ? cap : kKeepLong);
  const int64_t want = 2 * sms / all;      // blocks of a (layer, sequence)
  const int64_t one = sms / all;           // where one of them is on an SM
  if (cap <= kShort && one >= kLeast && a.weights != a.weights_out) {
    const int32_t pieces = (int32_t)(one < 32 ? one : 32);
    const int64_t via = a.recent < cap ? a.recent : cap;
    if (!latent::kernel_ready<kda_evict_select_kernel<true>>(2 * kShort * 4, 0))
      return cudaErrorNotSupported;
    kda_evict_select_kernel<true>
        <<<(unsigned)(all * pieces), kThreads, (size_t)(room + via) * 4, stream>>>(a, room, pieces);
    return cudaGetLastError();
  }
  if (!latent::kernel_ready<kda_evict_select_kernel<false>>(kKeep * 4, 0)) return cudaErrorNotSupported;
  kda_evict_select_kernel<false><<<(unsigned)all, kThreads, (size_t)room * 4, stream>>>(a, room, 1);
  cudaError_t e = cudaGetLastError();
  const int32_t pieces = (int32_t)(want < kLeastPieces ? kLeastPieces : want > 64 ? 64 : want);
  for (int64_t lb = 0; lb < all && e == cudaSuccess; lb += 65535) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)pieces, (unsigned)(all - lb < 65535 ? all - lb : 65535));
    cfg.blockDim = dim3(kMoveThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = lb == 0 ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, kda_evict_move_kernel, a, pieces, lb);
  }
  return e;
}

}  // namespace kda
