// Internal declarations of the latent-attention operators and of the paged-cache
// moves (kda_latent_*, kda_cache_*).  Not part of the public ABI (include/kda.h).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "kda_internal.h"

namespace kda {

constexpr int kLatentD = 128;    // head dimension of the expanded form (keys without rope, values)
constexpr int kLatentC = 512;    // latent channels of a cached row
constexpr int kLatentRope = 64;  // rotary channels (or none)
constexpr int kTreeMax = 64;     // drafts a tree mask can describe

// The bound on any wait in these kernels and, for a test, a block (none: -1) whose loader
// withholds tile `tile` of its first item, so that the waits for that tile run out.
struct WaitTest {
  uint64_t wait_ns;
  int32_t block, tile;
};
// What kda_latent_test_timeout armed for this workspace, or the usual bounds.
WaitTest take_wait_test(const void *workspace);
constexpr uint64_t kWaitNs = 2000000000ull;

// Expanded form: packed sequences, keys and values per head.
struct LatentArgs {
  const void *q;       // [n_q, H, 128 + dr]
  const void *k, *v;   // [n_k, H, 128] with the strides below (elements)
  const void *k_rope;  // [n_k, dr] or nullptr
  int64_t k_ts, k_hs, v_ts, v_hs;
  const int32_t *cu_q, *cu_k;  // device, [n_seqs + 1]; nullptr: one sequence of n_q / n_k
  int32_t n_seqs;
  int64_t n_q, n_k;
  int32_t H, dr;
  float scale;
  bool causal;
  void *out;           // [n_q, H, 128]
  float *lse;          // [n_q, H]
  DeviceStatus *status;
  // gradients
  const void *d_out;
  void *dq, *dk, *dv, *d_k_rope;
  int64_t dk_ts, dk_hs, dv_ts, dv_hs;
  void *scratch;       // latent_fwd_scratch_bytes() or latent_bwd_scratch_bytes()
  WaitTest test;
};
cudaError_t launch_latent_fwd(const LatentArgs &a, cudaStream_t stream);
cudaError_t launch_latent_bwd(const LatentArgs &a, cudaStream_t stream);
size_t latent_fwd_scratch_bytes(int32_t n_seqs, int64_t n_q, int64_t n_k, int32_t H);
size_t latent_bwd_scratch_bytes(int32_t n_seqs, int64_t n_q, int64_t n_k, int32_t H, int32_t dr);

// Absorbed form over a paged cache.
struct LatentDecodeArgs {
  const void *q;              // [B, T, H, 512 + dr]
  const void *cache;          // [n_pages, page_size, 512 + dr]
  const int32_t *block_table; // [B, max_pages]
  const int32_t *seq_lens;    // [B]
  const int64_t *tree_mask;   // [B, T] or nullptr
  int32_t B, T, H, dr, n_pages, page_size, max_pages;
  float scale;
  void *out;                  // [B, T, H, 512]
  float *lse;                 // [B, T, H] or nullptr
  DeviceStatus *status;
  void *scratch;              // latent_decode_scratch_bytes()
  WaitTest test;
};
cudaError_t launch_latent_decode(const LatentDecodeArgs &a, cudaStream_t stream);
size_t latent_decode_scratch_bytes(int32_t B, int32_t T, int32_t H, int32_t dr);

// Paged-cache moves; sizes and strides in bytes, multiples of 16.
struct CacheWriteArgs {
  void *cache;                // [L, n_pages, page_size, row_bytes]
  const void *rows;           // [L, B, T] rows with the strides below, or nullptr (compaction)
  int64_t rows_ls, rows_bs, rows_ts;
  const int32_t *block_table, *start, *path, *n_write;
  int32_t L, page_size, B, T, max_pages;
  int32_t n_pages;
  int64_t row_bytes;
  int32_t *status;
};
cudaError_t launch_cache_write(const CacheWriteArgs &a, cudaStream_t stream);
cudaError_t launch_cache_copy_pages(void *cache, const int32_t *src, const int32_t *dst, int32_t n,
                                    int32_t L, int32_t n_pages, int64_t page_bytes,
                                    int32_t *status, cudaStream_t stream);

#ifdef __CUDACC__
__device__ __forceinline__ void record_device_status(DeviceStatus *st, int32_t code, int32_t detail,
                                                     int32_t chain, int32_t chunk) {
  if (atomicCAS(&st->code, 0, code) == 0) {
    st->detail = detail;
    st->chain = chain;
    st->chunk = chunk;
  }
}

// Status of a call that has one writer of its validity: cleared, or the error.
__device__ __forceinline__ void set_device_status(DeviceStatus *st, int32_t code, int32_t detail) {
  *st = DeviceStatus{code, detail, 0, 0, 0, 0};
}

// A tile of consecutive rows of one sequence.
struct SeqTile {
  int32_t seq, tile, n_tiles;      // n_tiles of the sequence; seq < 0: no such tile
  int32_t q0, nq, k0, nk;          // the sequence's queries and keys
  int32_t bad;                     // cu_q or cu_k is not a prefix sum of n_q / n_k
};

// Entry s of a prefix sum; without one, a single sequence of n rows.
__device__ __forceinline__ int32_t cu_at(const int32_t *__restrict__ cu, int32_t s, int64_t n) {
  return cu ? cu[s] : s == 0 ? 0 : (int32_t)n;
}

// The packed sequences of a call, as its kernels need them to find their work.  Each
// kind of tile they are cut into (kTileRows) has, for more than kLaneSeqs sequences,
// the number of tiles before every sequence in memory.
enum TileKind { kTileA = 0, kTileB = 1, kTileC = 2, kTileKinds = 3 };
constexpr int kLaneSeqs = 32;
struct Packed {
  const int32_t *cu_q, *cu_k;
  int32_t n_seqs, H, sms;
  int64_t n_q, n_k;
  int32_t rows[kTileKinds];        // rows of a tile; 0: no such kind
  bool by_key[kTileKinds];         // of keys (else of queries)
  const int32_t *before[kTileKinds];  // [n_seqs + 1], -1 in the last entry: malformed arrays
};

// The calling warp's view of the sequences: up to 32 of them are in its lanes, loaded
// once; more are looked up.
struct LaneSeqs {
  int32_t q0, nq, k0, nk;
  bool bad, many;
  __device__ explicit LaneSeqs(const Packed &p)
      : q0(0), nq(0), k0(0), nk(0), bad(false), many(p.n_seqs > kLaneSeqs) {
    if (many) return;
    const int lane = threadIdx.x & 31;
    int32_t qb = 0, kb = 0;
    if (lane < p.n_seqs) {
      q0 = cu_at(p.cu_q, lane, p.n_q);
      qb = cu_at(p.cu_q, lane + 1, p.n_q);
      k0 = cu_at(p.cu_k, lane, p.n_k);
      kb = cu_at(p.cu_k, lane + 1, p.n_k);
    }
    nq = qb - q0;
    nk = kb - k0;
    bad = __any_sync(0xffffffffu,
                     q0 < 0 || k0 < 0 || nq < 0 || nk < 0 || qb > p.n_q || kb > p.n_k ||
                         (lane == 0 && (q0 != 0 || k0 != 0)) ||
                         (lane == p.n_seqs - 1 && (qb != p.n_q || kb != p.n_k)));
  }
};

// All tiles of a kind, or -1 for malformed arrays; by one warp.
__device__ inline int32_t count_tiles(const Packed &p, const LaneSeqs &l, TileKind kind) {
  if (l.many) return p.before[kind][p.n_seqs];
  if (l.bad) return -1;
  return __reduce_add_sync(
      0xffffffffu, ((p.by_key[kind] ? l.nk : l.nq) + p.rows[kind] - 1) / p.rows[kind]);
}

// Tile `index` of all sequences, by one warp: every sequence's tile 0, then every
// sequence's tile 1, and so on (more than 32 sequences: in sequence order, where a
// sequence is a small part of the whole anyway).  Callers count tiles from the end
// of a sequence that has the most work.
__device__ inline SeqTile ordered_tile(const Packed &p, const LaneSeqs &l, TileKind kind,
                                       int32_t index) {
  const int lane = threadIdx.x & 31;
  SeqTile r;
  r.bad = 0;
  if (l.many) {
    // the last sequence with at most `index` tiles before it, 32 probes a step
    const int32_t *before = p.before[kind];
    int32_t lo = 0, hi = p.n_seqs;
    while (hi - lo > 1) {
      const int32_t step = (hi - lo + 31) / 32, at = lo + lane * step;
      const unsigned le =
          __ballot_sync(0xffffffffu, at < hi && before[at < hi ? at : lo] <= index);
      lo += (31 - __clz(le)) * step;     // lane 0 always holds
      hi = lo + step < hi ? lo + step : hi;
    }
    r.seq = lo;
    r.tile = index - before[lo];
    r.n_tiles = before[lo + 1] - before[lo];
    r.q0 = cu_at(p.cu_q, lo, p.n_q);
    r.nq = cu_at(p.cu_q, lo + 1, p.n_q) - r.q0;
    r.k0 = cu_at(p.cu_k, lo, p.n_k);
    r.nk = cu_at(p.cu_k, lo + 1, p.n_k) - r.k0;
    return r;
  }
  const int32_t tiles = ((p.by_key[kind] ? l.nk : l.nq) + p.rows[kind] - 1) / p.rows[kind];
  // the largest tile number with at most `index` tiles before it
  int lo = 0, s = 0;
  if (p.n_seqs == 1) {
    lo = index;
  } else {
    int hi = __reduce_max_sync(0xffffffffu, tiles);
    while (lo + 1 < hi) {
      const int mid = (lo + hi) / 2;
      if (__reduce_add_sync(0xffffffffu, min(tiles, mid)) <= index) lo = mid;
      else hi = mid;
    }
    const int rank = index - __reduce_add_sync(0xffffffffu, min(tiles, lo));
    const unsigned have = __ballot_sync(0xffffffffu, tiles > lo);
    // the sequence that `rank` others with such a tile come before
    const bool it = tiles > lo && __popc(have & ((1u << lane) - 1)) == rank;
    s = __ffs(__ballot_sync(0xffffffffu, it)) - 1;
  }
  r.seq = s;
  r.tile = lo;
  const int from = max(s, 0);
  r.n_tiles = __shfl_sync(0xffffffffu, tiles, from);
  r.q0 = __shfl_sync(0xffffffffu, l.q0, from);
  r.nq = __shfl_sync(0xffffffffu, l.nq, from);
  r.k0 = __shfl_sync(0xffffffffu, l.k0, from);
  r.nk = __shfl_sync(0xffffffffu, l.nk, from);
  return r;
}

// Tile and head of work item `index` of `tiles` * H (a grid's blocks: below 2^31).
// Items run in groups of as many heads as fill the SMs once, inside a group tile by tile.
__device__ inline SeqTile place_item(const Packed &p, const LaneSeqs &l, TileKind kind,
                                     uint32_t tiles, uint32_t index, int *head) {
  const uint32_t fill = (uint32_t)p.sms / tiles, group = fill > 1 ? fill : 1;
  const uint32_t g = index / (tiles * group), left = (uint32_t)p.H - g * group;
  const uint32_t heads = group < left ? group : left, in = index - g * tiles * group;
  *head = (int)(g * group + in % heads);
  return ordered_tile(p, l, kind, (int32_t)(in / heads));
}
#endif

#ifdef __CUDACC__
// Fills the `before` arrays (and the status) of a call with more than kLaneSeqs
// sequences: one kernel before the others.  `mem`: plan_bytes().
cudaError_t launch_latent_plan(Packed &p, void *mem, DeviceStatus *status, cudaStream_t stream);
#endif
size_t latent_plan_bytes(int32_t n_seqs);

}  // namespace kda
