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
};
cudaError_t launch_latent_fwd(const LatentArgs &a, cudaStream_t stream);
cudaError_t launch_latent_bwd(const LatentArgs &a, cudaStream_t stream);
size_t latent_fwd_scratch_bytes(int64_t n_q, int64_t n_k, int32_t H);
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

// A tile of `rows` packed rows of one sequence: which sequence and which rows.
struct SeqTile {
  int32_t seq, tile, n_tiles;      // n_tiles of the sequence; seq < 0: no such tile
  int32_t q0, nq, k0, nk;          // the sequence's queries and keys
  int32_t bad;                     // cu_q or cu_k is not a prefix sum of n_q / n_k
};

// Entry s of a prefix sum; without one, a single sequence of n rows.
__device__ __forceinline__ int32_t cu_at(const int32_t *__restrict__ cu, int32_t s, int64_t n) {
  return cu ? cu[s] : s == 0 ? 0 : (int32_t)n;
}

// Tile `index` of the packed sequences, cut into tiles of `rows` queries
// (by_key: keys), by one whole warp.  Every entry of both arrays is read, so a
// malformed array is seen by every caller, whatever its tile.
__device__ inline SeqTile find_seq_tile(const int32_t *__restrict__ cu_q,
                                        const int32_t *__restrict__ cu_k, int32_t n_seqs,
                                        int64_t n_q, int64_t n_k, int32_t rows, bool by_key,
                                        int64_t index) {
  const int lane = threadIdx.x & 31;
  SeqTile r;
  r.seq = -1; r.tile = 0; r.n_tiles = 0; r.q0 = r.nq = r.k0 = r.nk = 0;
  bool bad = cu_at(cu_q, 0, n_q) != 0 || cu_at(cu_k, 0, n_k) != 0 ||
             cu_at(cu_q, n_seqs, n_q) != n_q || cu_at(cu_k, n_seqs, n_k) != n_k;
  int64_t base = 0;
  for (int32_t s0 = 0; s0 < n_seqs; s0 += 32) {
    const int32_t s = s0 + lane;
    int32_t qa = 0, qb = 0, ka = 0, kb = 0;
    if (s < n_seqs) {
      qa = cu_at(cu_q, s, n_q); qb = cu_at(cu_q, s + 1, n_q);
      ka = cu_at(cu_k, s, n_k); kb = cu_at(cu_k, s + 1, n_k);
    }
    bad = bad || qb < qa || kb < ka || qa < 0 || ka < 0 || qb > n_q || kb > n_k;
    bad = __any_sync(0xffffffffu, bad);
    if (bad) break;
    const int32_t len = by_key ? kb - ka : qb - qa;
    const int32_t t = (int32_t)(((int64_t)len + rows - 1) / rows);
    int32_t inc = t;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int32_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const int64_t lo = base + inc - t;
    const unsigned hit = __ballot_sync(0xffffffffu, index >= lo && index < lo + t);
    if (hit) {
      const int w = __ffs(hit) - 1;
      r.seq = s0 + w;
      r.tile = (int32_t)__shfl_sync(0xffffffffu, (int)(index - lo), w);
      r.n_tiles = __shfl_sync(0xffffffffu, t, w);
      r.q0 = __shfl_sync(0xffffffffu, qa, w);
      r.nq = __shfl_sync(0xffffffffu, qb - qa, w);
      r.k0 = __shfl_sync(0xffffffffu, ka, w);
      r.nk = __shfl_sync(0xffffffffu, kb - ka, w);
    }
    base += __shfl_sync(0xffffffffu, inc, 31);
  }
  r.bad = __any_sync(0xffffffffu, bad) ? 1 : 0;
  if (r.bad) r.seq = -1;
  return r;
}
// The packed sequences of a call, as its kernels need them to find their work.
struct Packed {
  const int32_t *cu_q, *cu_k;
  int32_t n_seqs, H, sms;
  int64_t n_q, n_k;
};

// Up to 32 sequences, one a lane, loaded once; `bad`: the arrays are malformed.
struct LaneSeqs {
  int32_t q0, nq, k0, nk;
  bool bad, many;  // many: more than 32, looked up in memory instead
  __device__ explicit LaneSeqs(const Packed &p) : q0(0), nq(0), k0(0), nk(0), many(p.n_seqs > 32) {
    const int lane = threadIdx.x & 31;
    int32_t qb = 0, kb = 0;
    if (!many && lane < p.n_seqs) {
      q0 = cu_at(p.cu_q, lane, p.n_q);
      qb = cu_at(p.cu_q, lane + 1, p.n_q);
      k0 = cu_at(p.cu_k, lane, p.n_k);
      kb = cu_at(p.cu_k, lane + 1, p.n_k);
    }
    nq = qb - q0;
    nk = kb - k0;
    bool wrong = q0 < 0 || k0 < 0 || nq < 0 || nk < 0 || qb > p.n_q || kb > p.n_k;
    wrong = wrong || (!many && ((lane == 0 && (q0 != 0 || k0 != 0)) ||
                                (lane == p.n_seqs - 1 && (qb != p.n_q || kb != p.n_k))));
    bad = __any_sync(0xffffffffu, wrong);
  }
};

// All tiles (of `rows` queries, by_key: keys), or -1 for malformed arrays; by one warp.
__device__ inline int64_t count_tiles(const Packed &p, const LaneSeqs &l, int32_t rows,
                                      bool by_key) {
  if (!l.many) {
    if (l.bad) return -1;
    return __reduce_add_sync(0xffffffffu, ((by_key ? l.nk : l.nq) + rows - 1) / rows);
  }
  const int lane = threadIdx.x & 31;
  bool bad = cu_at(p.cu_q, 0, p.n_q) != 0 || cu_at(p.cu_k, 0, p.n_k) != 0 ||
             cu_at(p.cu_q, p.n_seqs, p.n_q) != p.n_q || cu_at(p.cu_k, p.n_seqs, p.n_k) != p.n_k;
  int mine = 0;
  for (int s = lane; s < p.n_seqs; s += 32) {
    const int qa = cu_at(p.cu_q, s, p.n_q), qb = cu_at(p.cu_q, s + 1, p.n_q);
    const int ka = cu_at(p.cu_k, s, p.n_k), kb = cu_at(p.cu_k, s + 1, p.n_k);
    bad = bad || qb < qa || kb < ka || qa < 0 || ka < 0 || qb > p.n_q || kb > p.n_k;
    if (!bad) mine += ((by_key ? kb - ka : qb - qa) + rows - 1) / rows;
  }
  if (__any_sync(0xffffffffu, bad)) return -1;
  return __reduce_add_sync(0xffffffffu, mine);
}

// Tile `index` of all sequences, by one warp: every sequence's tile 0, then every
// sequence's tile 1, and so on (up to 32 sequences; more of them in sequence order,
// where a sequence is a small part of the whole anyway).  Callers count tiles from
// the end of a sequence that has the most work.
__device__ inline SeqTile ordered_tile(const Packed &p, const LaneSeqs &l, int32_t rows,
                                       bool by_key, int64_t index) {
  if (l.many)
    return find_seq_tile(p.cu_q, p.cu_k, p.n_seqs, p.n_q, p.n_k, rows, by_key, index);
  const int tiles = ((by_key ? l.nk : l.nq) + rows - 1) / rows;
  // the largest tile number with at most `index` tiles before it
  int lo = 0, s = 0;
  if (p.n_seqs == 1) {
    lo = (int)index;
  } else {
    int hi = __reduce_max_sync(0xffffffffu, tiles);
    while (lo + 1 < hi) {
      const int mid = (lo + hi) / 2;
      if (__reduce_add_sync(0xffffffffu, min(tiles, mid)) <= index) lo = mid;
      else hi = mid;
    }
    const int rank = (int)(index - __reduce_add_sync(0xffffffffu, min(tiles, lo)));
    const unsigned have = __ballot_sync(0xffffffffu, tiles > lo);
    s = __popc(have) > rank ? (int)__fns(have, 0, rank + 1) : -1;
  }
  SeqTile r;
  r.bad = 0;
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

// Tile and head of work item `index` of `tiles` * H.  Items run in groups of as many
// heads as fill the SMs once, inside a group tile by tile.
__device__ inline SeqTile place_item(const Packed &p, const LaneSeqs &l, int32_t rows, bool by_key,
                                     int64_t tiles, int64_t index, int *head) {
  const int64_t fill = p.sms / tiles, group = fill > 1 ? fill : 1;
  const int64_t g = index / (tiles * group), left = p.H - g * group;
  const int64_t heads = group < left ? group : left, in = index - g * tiles * group;
  *head = (int)(g * group + in % heads);
  return ordered_tile(p, l, rows, by_key, in / heads);
}
#endif

}  // namespace kda
