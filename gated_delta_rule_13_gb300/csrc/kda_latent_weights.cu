// The attention weight that cached rows have been given (kda_latent_weights), tcgen05 /
// TMEM / TMA, sm_103a.
//
//   w_j <- decay w_j + sum over tokens t and heads h that see j of exp(scale q_th . c_j - lse_th)
//
// Scores once more, but transposed: S [keys x query rows] = C Q^T, so that a thread of the
// epilogue has a key, and its sum over the R = T * H query rows is a sum along its own row
// of the accumulator, in registers, in a fixed order, whatever R is.  With lse from the decode
// pass every term is final, and there is no maximum to follow.  No key is touched by two CTAs,
// but where there are few tiles of many query rows: then a tile is cut into ranges of its rows,
// and who comes last to 32 keys adds the ranges' sums, in their order, so that nothing depends
// on the order of CTAs.  Into how many ranges goes by the tiles of the whole call, so that the
// last bits of a sequence depend on what else the call holds.
//
// A cached row is 2 W = 1,024 or 1,152 bytes against 2 R W operations: at R = 96 the card's
// 289 operations a byte leave it bound by HBM, from R = 145 on by the matrix work.  So there
// are two forms, by what stays in shared memory while the other operand streams past it, in
// blocks of 64 channels:
//   R <= 128  the queries of a sequence stay (at most 147 KB), 128-key tiles stream: every
//             cached row is read once, 64 to 190 KB of copies in flight an SM.
//   R > 128   a 256-key tile stays, half in each CTA of a pair, and the query rows stream
//             from L2, 256 at a time, half to each CTA; cta_group::2 products (256 keys x
//             256 rows) read both halves.  One CTA by itself would have to stream 64 bytes
//             of queries a cycle from L2 to keep its tensor cores busy; a pair 32 a CTA.
// Steps (one accumulator each) are double-buffered in TMEM: the products of one run beside
// the exponentials of the other.  What stays and what streams have a loader each, so that the
// next tile's keys are under way as soon as a block of the last one's is done with.
//
// Measured (96 heads): one token of 128 sequences of up to 16384 rows, dr = 64, 1.23 GB, 188 to
// 209 us cold on several boxes (5.9 to 6.5 TB/s); trees of 16 drafts, 32 sequences, 310 to 331 us
// (1.6 to 1.7 PFLOP/s, tensor cores 84 % busy, the clock held down by power); one token over
// 3001 rows, dr = 0, 8.1 us (replayed): start, 230 KB an SM, one tile's way.  One tree of 16
// drafts over 8000 rows 25 us (tiles whole: 35), of 24 over 300 16 us (46), 70 tokens of 128
// heads over 1000 rows 21 us (131).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <string.h>

#include "kda_latent_tc.cuh"
#include "kda_rows.h"

namespace kda {
namespace {

using namespace latent;

constexpr int kThreads = 384;            // 2 x 4 epilogue warps, two loaders, MMA, lse
constexpr int kLoadWarp = 8, kMmaWarp = 9, kLseWarp = 10, kKeepWarp = 11;
constexpr uint32_t kBlock = 16384;       // 128 rows x 64 channels
constexpr uint32_t kSmem = 232448;
constexpr int kMaxBlocks = 9, kMostTiles = 0x7fff0000;
// A pair's tile in several parts, of a range of the query rows each, where there are few tiles.
constexpr int kMostUnits = 4;            // parts in all, for each pair of the grid
constexpr int kTileCounts = 8;           // of a tile: parts that have come, for each 32 keys
constexpr int kUnitKeys = 256;

template <bool kPair>
constexpr int kKeysLog = kPair ? 8 : 7;  // keys of a tile
template <bool kPair>
constexpr int kCols = kPair ? 256 : 128; // query rows of a step at most

template <bool kPair>
constexpr int kMaxSlots = kPair ? 5 : 12;
template <bool kPair>
struct Shared {
  // Of a pair, the barriers that the products wait for are rank 0's.
  uint64_t full[kMaxSlots<kPair>], empty[kMaxSlots<kPair>], kept_full[kMaxBlocks], kept_free[kMaxBlocks];
  uint64_t s_full[2], s_free[2], lse_full[2], lse_free[2], part_ready[4], part_free[4], fin;
  uint32_t tmem;
  int abort;
  int seq0, tile0, total;                // the CTA's first sequence and tile; all tiles
  int parts;                             // of a tile
  DeviceStatus error;
  // Of a pair: the parts of tiles it takes, one ahead (sequence, -1: no more; tile; length; the
  // part's number among all).
  uint64_t unit_full[2], unit_free[2];
  int4 unit[2];
  uint32_t load_ring, load_kept;         // blocks the loader asked for
  alignas(16) float lse[2][kCols<kPair>];            // times log2(e); +inf where a row gives nothing
  union {
    float part[128];                     // the second warpgroup's sums
    int64_t warp_sum[kThreads / 32];     // at the start
  };
};
constexpr uint32_t kSharedBytes = 3 * 1024;
static_assert(sizeof(Shared<false>) <= kSharedBytes, "fits beside the tiles");
static_assert(sizeof(Shared<true>) <= kSharedBytes, "fits beside the tiles");

struct Params {
  const int32_t *table, *lens;
  const int64_t *mask;
  const float *lse;
  int32_t B, T, H, R, n_pages, page_size, max_pages, box_rows;
  int32_t blocks;       // of 64 channels
  int32_t cols;         // query rows of a step, a multiple of 16
  int32_t row_steps;    // steps for all of them (1 where they stay)
  int32_t slots;        // of the ring
  int32_t groups;       // CTAs, or pairs of them
  uint32_t kept_bytes;  // a kept block's place
  float scale2, decay;  // scale * log2(e), see launch_latent_weights
  float lse_hi, lse_lo; // what lse is multiplied by, in two parts
  float *weights;
  DeviceStatus *status;
  int32_t *taken;       // parts that pairs have taken beyond their first
  int32_t *come;        // [tile][kTileCounts]
  float *part;          // [part][kUnitKeys]
  WaitTest test;
};

// Length of sequence b, 0 when it is out of range.
__device__ __forceinline__ int seq_len(const Params &p, int b) {
  const int n = p.lens[b];
  return n < 0 || n > (int64_t)p.max_pages * p.page_size ? 0 : n;
}
template <bool kPair>
__device__ __forceinline__ int key_tiles(int n) {
  return (n >> kKeysLog<kPair>)+((n & ((1 << kKeysLog<kPair>)-1)) != 0);
}

// First tile of group c of G when the list has `total`: the first total % G take one more.
__device__ __forceinline__ int group_begin(int c, int G, int total) {
  const int each = total / G, more = total - each * G;
  return c * each + min(c, more);
}

// The steps of one CTA, which has consecutive tiles; every role walks over them by itself.
struct OneSteps {
  const Params &p;
  int next_b, next_t, left;       // next sequence, its next tile, tiles left
  int b = 0, n = 0, ta = 0, tb = 0, t = 0;   // current: sequence, its length, tiles [ta, tb), tile
  static constexpr int rs = 0;
  __device__ OneSteps(const Params &p_, int b_, int t_, int left_)
      : p(p_), next_b(b_), next_t(t_), left(left_) {}
  template <bool kLane>
  __device__ bool next() {
    if (t + 1 < tb) {
      ++t;
      return true;
    }
    if (left <= 0) return false;
    for (; next_b < p.B; ++next_b, next_t = 0) {
      n = seq_len(p, next_b);
      const int k = key_tiles<false>(n);
      if (next_t >= k) continue;
      b = next_b;
      t = ta = next_t;
      tb = k - ta <= left ? k : ta + left;
      left -= tb - ta;
      next_t = tb;                // at the end of the sequence the loop passes on
      return true;
    }
    return false;
  }
  // of what stays in shared memory; of a tile of keys
  __device__ bool first() const { return t == ta; }
  __device__ bool last() const { return t + 1 == tb; }
  __device__ bool tile_begins() const { return true; }
  __device__ bool tile_ends() const { return true; }
  __device__ int number() const { return t - ta; }
};
// Into how many parts to cut tiles: in rounds of all pairs, the steps of one and what it takes to
// start and to end (about two more).  By a warp.
__device__ __forceinline__ int best_parts(int tiles, int steps, int groups) {
  const int most = min(steps, kMostUnits * groups / max(tiles, 1));
  uint32_t least = ~0u;                      // cost, parts
  for (int s = 1 + (int)(threadIdx.x & 31); s <= most; s += 32) {
    const int cost = (tiles * s + groups - 1) / groups * ((steps + s - 1) / s + 2);
    least = min(least, (uint32_t)cost << 12 | (uint32_t)s);
  }
  least = __reduce_min_sync(0xffffffffu, least);
  return most < 2 ? 1 : (int)(least & 4095);
}
// The steps of a pair.  Pairs are not equally fast (by 20 % in the same work), so that each takes
// a tile, or a part of one, when it needs it: rank 0 counts them up and tells both CTAs, one ahead.
struct PairSteps {
  const Params &p;
  Shared<true> &m;
  const WaitCtx &cx;
  const uint32_t rank;
  uint32_t taken = 0;
  int b = 0, n = 0, t = 0, rs = 0;           // current: sequence, its length, tile, row step
  int r0 = 0, r1 = 0, unit = 0;              // row steps of the part, its number
  __device__ PairSteps(const Params &p_, Shared<true> &m_, const WaitCtx &cx_, uint32_t rank_)
      : p(p_), m(m_), cx(cx_), rank(rank_) {}
  template <bool kLane>                      // by one lane, or by a converged warp
  __device__ bool next() {
    if (taken > 0 && rs + 1 < r1) {
      ++rs;
      return true;
    }
    const uint32_t s = taken & 1, par = (taken >> 1) & 1;
    if (!(kLane ? wait_or_abort<2>(cx, &m.unit_full[s], par, 50, (int)taken)
                : warp_wait<2>(cx, &m.unit_full[s], par, 50, (int)taken)))
      return false;
    const int4 u = m.unit[s];
    // (the vote has consumed what was read: the place may be written again)
    const bool more = kLane ? u.x >= 0 : __all_sync(0xffffffffu, u.x >= 0) != 0;
    if (kLane || (threadIdx.x & 31) == 0) {
      if (rank == 0) mbar_arrive(&m.unit_free[s]);
      else remote_arrive_relaxed(map_rank(smem_u32(&m.unit_free[s]), 0));
    }
    ++taken;
    b = u.x;
    t = u.y;
    n = u.z;
    unit = u.w;
    const int parts = m.parts, part = unit % parts;
    rs = r0 = part * p.row_steps / parts;
    r1 = (part + 1) * p.row_steps / parts;
    return more;
  }
  __device__ bool first() const { return rs == r0; }
  __device__ bool last() const { return rs + 1 == r1; }
  __device__ bool tile_begins() const { return first(); }
  __device__ bool tile_ends() const { return last(); }
  __device__ int number() const { return (int)taken - 1; }
};
constexpr int kUnitReaders = 12 + 11;        // loaders, lse, sums of both CTAs, products

// Sequence, tile and length of the x-th tile of all, x not falling from call to call; by a warp.
struct Finder {
  const Params &p;
  int base = -32, before = 0;                // 32 sequences from `base` on, tiles before them
  int n = 0, upto = 0;                       // of this lane's: length, tiles with those before it
  int all = 0;                               // tiles of the 32
  __device__ explicit Finder(const Params &p_) : p(p_) {}
  __device__ int4 find(int x) {
    const int lane = threadIdx.x & 31;
    while (x >= before + all) {
      before += all;
      base += 32;
      n = base + lane < p.B ? seq_len(p, base + lane) : 0;
      upto = key_tiles<true>(n);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
      }
      all = __shfl_sync(0xffffffffu, upto, 31);
      if (base >= p.B) return make_int4(-1, 0, 0, 0);
    }
    const int at = __ffs(__ballot_sync(0xffffffffu, x - before < upto)) - 1;
    const int k = __shfl_sync(0xffffffffu, upto, at), len = __shfl_sync(0xffffffffu, n, at);
    return make_int4(base + at, x - before - (k - key_tiles<true>(len)), len, 0);
  }
};

// What differs between one CTA and a pair: the products and who hears of their end.
template <bool kPair>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  if constexpr (!kPair) {
    umma_ss(d, a, b, idesc, add);
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
  }
}
template <bool kPair>
__device__ __forceinline__ void commit(uint64_t *bar) {
  if constexpr (!kPair) {
    umma_commit(bar);
  } else {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
  }
}
template <bool kPair>
__device__ __forceinline__ void tmem_get(uint32_t *dst) {
  if constexpr (!kPair) {
    tmem_alloc(dst, 256);
    tmem_relinquish();
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     smem_u32(dst))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <bool kPair>
__device__ __forceinline__ void tmem_give(uint32_t addr) {
  if constexpr (!kPair) tmem_dealloc(addr, 256);
  else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(addr) : "memory");
}
// Copies counted by barrier `bar` (an address of the cluster's shared memory).
template <bool kPair>
__device__ __forceinline__ void copy_2d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int32_t c0,
                                        int32_t c1) {
  if constexpr (!kPair)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}
template <bool kPair>
__device__ __forceinline__ void copy_3d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int32_t c0,
                                        int32_t c1, int32_t c2) {
  if constexpr (!kPair)
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
        : "memory");
}

// The call's status and counts are cleared by a kernel of its own, beside which the next one starts.
__global__ void kda_latent_weights_begin_kernel(DeviceStatus *status, int32_t *counts, int32_t n) {
  pdl_launch_dependents();
  if (threadIdx.x == 0) set_device_status(status, KDA_OK, 0);
  for (int i = threadIdx.x; i < n; i += blockDim.x) counts[i] = 0;
}

template <bool kPair>
__device__ __forceinline__ void weights_body(const CUtensorMap &map_q, const CUtensorMap &map_c,
                                             const Params &p) {
  using Sh = Shared<kPair>;
  constexpr int kN = kCols<kPair>;
  extern __shared__ __align__(1024) unsigned char tiles[];
  const uint32_t base = smem_u32(tiles);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = kPair ? cluster_rank() : 0;
  const int group = kPair ? blockIdx.x >> 1 : blockIdx.x;
  const int NB = p.blocks, NS = p.slots;
  const uint32_t sm_kept = base, sm_ring = base + NB * p.kept_bytes;
  Sh &m = *reinterpret_cast<Sh *>(tiles + (kSmem - kSharedBytes));

  if (tid == 0) {
    for (int i = 0; i < kMaxSlots<kPair>; ++i) {
      mbar_init(&m.full[i], 1);
      mbar_init(&m.empty[i], 1);
    }
    for (int i = 0; i < kMaxBlocks; ++i) {
      mbar_init(&m.kept_full[i], 1);
      mbar_init(&m.kept_free[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&m.s_full[i], 1);
      mbar_init(&m.s_free[i], kPair ? 16 : 8);
      mbar_init(&m.lse_full[i], 1);
      mbar_init(&m.lse_free[i], 8);
    }
    for (int w = 0; w < 4; ++w) {
      mbar_init(&m.part_ready[w], 1);
      mbar_init(&m.part_free[w], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&m.unit_full[i], 1);
      mbar_init(&m.unit_free[i], kUnitReaders);
    }
    mbar_init(&m.fin, 1);
    m.abort = 0;
    m.seq0 = p.B;
    m.tile0 = 0;
    m.error = DeviceStatus{0, 0, 0, 0, 0, 0};
    fence_mbarrier_init();
  }
  if (warp == kLoadWarp && lane == 0) {
    prefetch_tensormap(&map_q);
    prefetch_tensormap(&map_c);
  }
  if (warp == kMmaWarp) tmem_get<kPair>(&m.tmem);
  {  // the group's share of the tile list
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = tid * per, b1 = min(p.B, b0 + per);
    int64_t mine = 0;                    // sequences may share pages: no pool bounds the sum
    bool bad = false;
    for (int b = b0; b < b1; ++b) {
      const int n = p.lens[b];
      if (n < 0 || n > (int64_t)p.max_pages * p.page_size) bad = true;
      else mine += key_tiles<kPair>(n);
    }
    int64_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) m.warp_sum[warp] = inc;
    __syncthreads();
    if (bad) record_device_status(&m.error, KDA_ERR_INVALID_ARG, 1, b0, 0);
    int64_t before = inc - mine, all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += m.warp_sum[w];
      all += m.warp_sum[w];
    }
    // tiles are counted in 32 bits from here on, by pairs a little past the last; a list that is
    // longer is refused
    const int total = all > kMostTiles ? 0 : (int)all;
    if (all > kMostTiles && tid == 0)
      record_device_status(&m.error, KDA_ERR_INVALID_ARG, 3, 0, 0);
    const int begin = group_begin(group, p.groups, total);
    if (!kPair && total > 0 && begin >= before && begin < before + mine) {
      int at = (int)before;
      for (int b = b0; b < b1; ++b) {
        const int k = key_tiles<kPair>(seq_len(p, b));
        if (begin < at + k) {
          m.seq0 = b;
          m.tile0 = begin - at;
          break;
        }
        at += k;
      }
    }
    if (warp == 0) {
      const int parts = kPair ? best_parts(total, p.row_steps, p.groups) : 1;
      if (lane == 0) {
        m.total = total;
        m.parts = parts;
      }
    }
  }
  tc_fence_before();
  if constexpr (kPair) cluster_sync_all();  // barriers of both CTAs are ready
  else __syncthreads();
  tc_fence_after();
  const uint32_t tm = m.tmem;
  const WaitCtx cx{&m.abort, &m.error, (int)blockIdx.x, p.test.wait_ns};
  auto st = [&] {
    if constexpr (kPair) {
      return PairSteps(p, m, cx, rank);
    } else {
      const int begin = group_begin(group, p.groups, m.total);
      return OneSteps(p, m.seq0, m.tile0, group_begin(group + 1, p.groups, m.total) - begin);
    }
  }();

  if (warp == kLoadWarp || warp == kKeepWarp) {
    // ---- loaders, of what streams and of what stays: each is as far ahead as its places are
    // free.  A lane has a piece of the tile's keys (the rows of one page), lane 0 the queries.
    const bool streams = warp == kLoadWarp, keys = streams != kPair;
    const int pieces = 128 / p.box_rows;
    const uint32_t piece_bytes = p.box_rows * 128;
    const auto lead = [&](uint64_t *bar) { return kPair ? map_rank(smem_u32(bar), 0) : smem_u32(bar); };
    uint32_t count = 0, round = 0;           // blocks asked for, parity of the places' rounds
    int s = 0, row = -1;                     // place; this lane's pool row
    uint32_t bytes = p.cols * 128;           // of a block, in both CTAs
    bool ok = true;
    while (ok && st.template next<false>()) {
      if (!streams && !st.first()) continue;
      if (keys) {
        const int at0 = st.t << kKeysLog<kPair>, at = at0 + (int)rank * 128 + lane * p.box_rows;
        row = -1;
        if (lane < pieces && at < st.n) {
          const int page = at / p.page_size;
          const int32_t id = p.table[(int64_t)st.b * p.max_pages + page];
          if (id < 0 || id >= p.n_pages) {
            record_device_status(&m.error, KDA_ERR_INVALID_ARG, 2, st.b, at);
            row = p.n_pages * p.page_size;   // past the pool: reads zeros
          } else {
            row = id * p.page_size + at - page * p.page_size;
          }
        }
        const int live = min(st.n - at0, 1 << kKeysLog<kPair>);
        bytes = (live + p.box_rows - 1) / p.box_rows * piece_bytes;
      }
      if (p.test.block == (int)blockIdx.x && p.test.tile == st.number()) break;  // a test
      const int places = streams ? NS : NB;
      uint64_t *full = streams ? m.full : m.kept_full, *empty = streams ? m.empty : m.kept_free;
      const uint32_t base_at = streams ? sm_ring : sm_kept, place_bytes = streams ? kBlock : p.kept_bytes;
      for (int c = 0; c < NB; ++c) {
        if (count >= (uint32_t)places) ok = warp_wait<2>(cx, &empty[s], round ^ 1, streams ? 11 : 10, st.t);
        if (!ok) break;
        if (lane == 0 && rank == 0) mbar_arrive_expect_tx(&full[s], bytes);
        __syncwarp();
        const uint32_t dst = base_at + s * place_bytes;
        if (keys) {
          if (row >= 0) copy_2d<kPair>(dst + lane * piece_bytes, &map_c, lead(&full[s]), c * 64, row);
        } else if (lane == 0) {
          copy_3d<kPair>(dst, &map_q, lead(&full[s]), c * 64, st.rs * kN + (int)rank * 128, st.b);
        }
        ++count;
        if (++s == places) {
          s = 0;
          round ^= 1;
        }
      }
    }
    if (lane == 0) (streams ? m.load_ring : m.load_kept) = count;
  } else if (warp == kMmaWarp) {
    // ---- products: one lane of rank 0
    if (rank == 0 && elect_one()) {
      const uint32_t idesc = idesc_bf16(kPair ? 256 : 128, p.cols, false, false);
      const Desc d_kept(sm_kept, 16), d_ring(sm_ring, 16);
      uint32_t round = 0, step = 0, outer = 0;
      int s = 0;
      bool ok = true;
      while (ok && st.template next<true>()) {
        const uint32_t buf = step & 1;
        if (step > 1) ok = wait_or_abort(cx, &m.s_free[buf], ((step >> 1) - 1) & 1, 20, st.t);
        if (!ok) break;
        tc_fence_after();
        for (int c = 0; c < NB; ++c) {
          if (st.first()) ok = wait_or_abort(cx, &m.kept_full[c], outer & 1, 21, st.t);
          ok = ok && wait_or_abort(cx, &m.full[s], round, 22, st.t);
          if (!ok) break;
          tc_fence_after();
          const uint32_t k_at = kPair ? c * kBlock : s * kBlock;
          const uint32_t q_at = kPair ? s * kBlock : c * p.kept_bytes;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint64_t a = kPair ? d_kept.at(k_at + k * 32) : d_ring.at(k_at + k * 32);
            const uint64_t q = kPair ? d_ring.at(q_at + k * 32) : d_kept.at(q_at + k * 32);
            mma<kPair>(tm + buf * kN, a, q, idesc, c > 0 || k > 0);
          }
          commit<kPair>(&m.empty[s]);
          if (st.last()) commit<kPair>(&m.kept_free[c]);
          if (++s == NS) {
            s = 0;
            round ^= 1;
          }
        }
        if (!ok) break;
        commit<kPair>(&m.s_full[buf]);
        outer += st.last();
        ++step;
      }
    }
  } else if (warp == kLseWarp) {
    // ---- lse of a step's rows (where the queries stay: of a sequence's), and a pair's tiles
    uint32_t item = 0, told = 0;
    bool ok = true, ended = false;
    Finder finder(p);
    // Tile number `told` of this pair to both CTAs: the first is its own, the others as they come.
    const auto tell = [&] {
      const uint32_t s = told & 1;
      if (rank == 0) {
        int x = group;
        if (told > 0) {
          if (lane == 0) x = p.groups + atomicAdd(p.taken, 1);
          x = __shfl_sync(0xffffffffu, x, 0);
        }
        const int parts = m.parts;
        int4 u = make_int4(-1, 0, 0, 0);
        if (x / parts < m.total) {
          u = finder.find(x / parts);
          u.w = x;
        }
        if (told > 1) ok = warp_wait<2>(cx, &m.unit_free[s], ((told >> 1) - 1) & 1, 31, (int)told);
        if (ok && lane == 0) {
          st_async_v4(map_rank(smem_u32(&m.unit[s]), 1), (uint32_t)u.x, (uint32_t)u.y, (uint32_t)u.z,
                      (uint32_t)u.w, map_rank(smem_u32(&m.unit_full[s]), 1));
          m.unit[s] = u;
          mbar_arrive(&m.unit_full[s]);
        }
        ended = u.x < 0;
      } else if (lane == 0) {
        mbar_arrive_expect_tx(&m.unit_full[s], 16);
      }
      ++told;
    };
    if constexpr (kPair) {
      tell();
      pdl_wait();                            // the count, from the second on, has been cleared
    }
    while (ok && st.template next<false>()) {
      if constexpr (kPair) {
        if (st.first() && !ended) tell();
        if (!ok) break;
      } else {
        if (!st.first()) continue;
      }
      const uint32_t i = item & 1;
      if (item > 1) ok = warp_wait<2>(cx, &m.lse_free[i], ((item >> 1) - 1) & 1, 30, st.t);
      if (!ok) break;
      const float *src = p.lse + (int64_t)st.b * p.R;
      for (int c = lane; c < p.cols; c += 32) {
        const int r = st.rs * kN + c;
        const float v = r < p.R ? src[r] : CUDART_INF_F;
        m.lse[i][c] = isinf(v) ? CUDART_INF_F : fmaf(v, p.lse_hi, v * p.lse_lo);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&m.lse_full[i]);
      ++item;
    }
  } else if (warp < 8) {
    // ---- sums: thread = key; the warpgroups take 16 of the step's rows in turn
    const int wg = warp >> 2, w4 = warp & 3, key = w4 * 32 + lane;
    const uint32_t ts = tm + ((uint32_t)w4 << 21);
    const int chunks = p.cols / 16;
    const uint32_t credit0 = kPair ? map_rank(smem_u32(&m.s_free[0]), 0) : 0;
    uint32_t step = 0, item = 0, tile = 0;
    float sum = 0.f, old = 0.f;
    bool ok = true;
    while (ok && st.template next<false>()) {
      const uint32_t buf = step & 1, par = (step >> 1) & 1;
      const int j = (st.t << kKeysLog<kPair>)+(int)rank * 128 + key;
      float *to = p.weights + (int64_t)st.b * p.max_pages * p.page_size + j;
      if (st.tile_begins()) {
        sum = 0.f;
        if (wg == 0 && p.decay != 0.f && j < st.n && (!kPair || m.parts == 1)) old = *to;
      }
      if (kPair || st.first()) {
        ok = warp_wait<2>(cx, &m.lse_full[item & 1], (item >> 1) & 1, 40, st.t);
        if (!ok) break;
      }
      const float *lse = m.lse[item & 1];
      ok = warp_wait<2>(cx, &m.s_full[buf], par, 41, st.t);
      if (!ok) break;
      tc_fence_after();
      // drafts: which of the step's rows see this key
      const int draft = j - (st.n - p.T);
      const bool masked = (p.T > 1 || p.mask) && ((st.t + 1) << kKeysLog<kPair>) > st.n - p.T;
      constexpr int kBatch = 4;              // chunks of 16 in registers
#pragma unroll 1
      for (int c0 = wg; c0 < chunks; c0 += 2 * kBatch) {
        uint32_t x[kBatch][16];
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          if (c0 + 2 * i < chunks) tmem_ld16(ts + buf * kN + 16 * (c0 + 2 * i), x[i]);
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          if (c0 + 2 * i < chunks) tmem_ld_wait(x[i]);
        if (c0 + 2 * kBatch >= chunks) {     // the accumulator has been read
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            if constexpr (kPair) remote_arrive_relaxed(credit0 + 8 * buf);
            else mbar_arrive(&m.s_free[buf]);
          }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int c = 16 * (c0 + 2 * i);
          if (c >= p.cols) continue;
          if (masked) {
            // a bit a row, a token's rows at a time
            int tok = (st.rs * kN + c) / p.H, left = (tok + 1) * p.H - (st.rs * kN + c);
            uint32_t seen = 0;
#pragma unroll 1
            for (int k = 0; k < 16 && tok < p.T; k += left, left = p.H, ++tok) {
              const bool see = draft < 0 || (p.mask ? (p.mask[(int64_t)st.b * p.T + tok] >>
                                                       (draft & 63) & 1) != 0
                                                    : draft <= tok);
              if (see) seen |= (left < 16 ? (1u << left) - 1 : 0xffffu) << k;
            }
#pragma unroll
            for (int k = 0; k < 16; ++k)
              if (!(seen >> k & 1)) x[i][k] = __float_as_uint(-CUDART_INF_F);
          }
          const float4 *l4 = reinterpret_cast<const float4 *>(lse + c);
          float part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float4 l = l4[k];
            part[0] += ex2(fmaf(__uint_as_float(x[i][4 * k]), p.scale2, -l.x));
            part[1] += ex2(fmaf(__uint_as_float(x[i][4 * k + 1]), p.scale2, -l.y));
            part[2] += ex2(fmaf(__uint_as_float(x[i][4 * k + 2]), p.scale2, -l.z));
            part[3] += ex2(fmaf(__uint_as_float(x[i][4 * k + 3]), p.scale2, -l.w));
          }
          sum += (part[0] + part[1]) + (part[2] + part[3]);
        }
      }
      if (wg >= chunks) {                    // nothing for this warpgroup: it has read it all
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.s_free[buf]);
      }
      if (kPair || st.last()) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.lse_free[item & 1]);
        ++item;
      }
      ++step;
      if (!st.tile_ends()) continue;
      const uint32_t turn = tile & 1;
      if (wg == 1) {
        if (tile > 0) ok = warp_wait<2>(cx, &m.part_free[w4], turn ^ 1, 42, st.t);
        if (!ok) break;
        m.part[key] = sum;
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.part_ready[w4]);
      } else {
        ok = warp_wait<2>(cx, &m.part_ready[w4], turn, 43, st.t);
        if (!ok) break;
        float all = sum + m.part[key];
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.part_free[w4]);
        if constexpr (kPair)
          if (m.parts > 1) {                 // whose part of 32 keys comes last adds all, in order
            const int parts = m.parts, x = st.unit / parts;
            float *mine = p.part + (int64_t)x * parts * kUnitKeys + rank * 128 + key;
            mine[(st.unit - x * parts) * kUnitKeys] = all;
            __threadfence();
            pdl_wait();                      // counts have been cleared
            __syncwarp();
            int come = 0;
            if (lane == 0) come = atomicAdd(&p.come[x * kTileCounts + rank * 4 + w4], 1);
            come = __shfl_sync(0xffffffffu, come, 0);
            if (come + 1 < parts) {
              ++tile;
              continue;
            }
            __threadfence();
            all = 0.f;
            for (int k = 0; k < parts; ++k) all += __ldcg(mine + k * kUnitKeys);
            if (p.decay != 0.f && j < st.n) old = *to;
          }
        if (j < st.n) *to = p.decay == 0.f ? all : fmaf(old, p.decay, all);
      }
      ++tile;
    }
  }

  __syncwarp();
  __syncthreads();
  if (m.abort) {
    // Nothing in flight outlives the block: the last copies, whose barriers tell rank 0 so,
    // and the products; then time for the copies of a pair's other CTA.
    if (tid == 32 * kLoadWarp && rank == 0) {
      const uint32_t ring = m.load_ring, kept = m.load_kept;
      for (uint32_t k = ring > (uint32_t)NS ? ring - NS : 0; k < ring; ++k)
        mbar_wait(&m.full[k % NS], (k / NS) & 1, 1000000);
      for (uint32_t k = kept > (uint32_t)NB ? kept - NB : 0; k < kept; ++k)
        mbar_wait(&m.kept_full[k % NB], (k / NB) & 1, 1000000);
    }
    if (warp == kMmaWarp && rank == 0 && elect_one()) {  // of the lane that issued them
      commit<kPair>(&m.fin);
      mbar_wait(&m.fin, 0, kWaitNs);
    }
    const uint64_t t0 = global_timer_ns();
    while (kPair && global_timer_ns() - t0 < 200000) {}
    __syncthreads();
  }
  tc_fence_before();
  if constexpr (kPair) cluster_sync_all();  // what one CTA signals in the other has arrived
  else __syncthreads();
  tc_fence_after();
  if (tid == 0) {
    pdl_wait();                // the status has been cleared
    if (m.error.code != 0)
      record_device_status(p.status, m.error.code, m.error.detail, m.error.chain, m.error.chunk);
  }
  if (warp == kMmaWarp) tmem_give<kPair>(tm);
  if constexpr (kPair) cluster_sync_all();
}

__global__ void __launch_bounds__(kThreads, 1)
kda_latent_weights_kernel(const __grid_constant__ CUtensorMap map_q,
                          const __grid_constant__ CUtensorMap map_c, const Params p) {
  weights_body<false>(map_q, map_c, p);
}
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
kda_latent_weights_pair_kernel(const __grid_constant__ CUtensorMap map_q,
                               const __grid_constant__ CUtensorMap map_c, const Params p) {
  weights_body<true>(map_q, map_c, p);
}

// Pairs of CTAs the device runs at once (0 without a device).
int resident_pairs() {
  static std::atomic<int> cache[kMaxDevices];
  return per_device(cache, [](int) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = 2;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    if (!kernel_ready<kda_latent_weights_pair_kernel>(kSmem, 0) ||
        cudaOccupancyMaxActiveClusters(&n, kda_latent_weights_pair_kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    return n;
  });
}

}  // namespace

// The count of parts taken, and for pairs those of parts that have come, and the parts.
static int counts_of(bool pair) {
  return pair ? 4 + kMostUnits / 2 * resident_pairs() * kTileCounts : 1;
}
size_t latent_weights_scratch_bytes(int32_t, int32_t T, int32_t H, int32_t) {
  const bool pair = (int64_t)T * H > 128;
  return ((size_t)counts_of(pair) + (pair ? kMostUnits * resident_pairs() * kUnitKeys : 0)) * 4;
}

cudaError_t launch_latent_weights(const LatentWeightsArgs &a, cudaStream_t stream) {
  if (a.B == 0) return cudaMemsetAsync(a.status, 0, sizeof(DeviceStatus), stream);
  const int W = kLatentC + a.dr, R = a.T * a.H;
  const bool pair = R > 128;
  if (!latent::encode_tiled() || (pair ? resident_pairs() : sm_count()) < 1 ||
      !kernel_ready<kda_latent_weights_kernel>(kSmem, 0))
    return cudaErrorNotSupported;
  Params p;
  p.table = a.block_table; p.lens = a.seq_lens; p.mask = a.tree_mask; p.lse = a.lse;
  p.B = a.B; p.T = a.T; p.H = a.H; p.R = R; p.n_pages = a.n_pages; p.page_size = a.page_size;
  p.max_pages = a.max_pages;
  p.box_rows = 128;                      // rows of a copied box: as many as lie in one page
  while (a.page_size % p.box_rows) p.box_rows >>= 1;
  p.blocks = W / 64;
  p.cols = pair ? 256 : (R + 15) / 16 * 16;
  p.row_steps = pair ? (R + 255) / 256 : 1;
  p.kept_bytes = pair ? kBlock : (uint32_t)p.cols * 128;  // whole 1,024s
  const uint32_t space = kSmem - kSharedBytes - p.blocks * p.kept_bytes;
  p.slots = (int)(space / kBlock);
  const int most = pair ? kMaxSlots<true> : kMaxSlots<false>;
  if (p.slots > most) p.slots = most;
  p.groups = pair ? resident_pairs() : sm_count();
  // Scores are made up for what is cut off of them, and lse is taken times what the rounded scale
  // stands for, so that the rounding cancels in the exponent: with an lse of 64 bits a short
  // sequence's weights went from 1.5e-6 to 3e-7.
  const double more = latent::cut_off(W, 1);
  p.scale2 = (float)(a.scale * 1.4426950408889634 * more);
  const double lse_by = p.scale2 > 1e-30f && p.scale2 < 1e30f ? p.scale2 / (a.scale * more) : 1.4426950408889634;
  p.lse_hi = (float)lse_by;
  p.lse_lo = (float)(lse_by - p.lse_hi);
  p.decay = a.decay; p.weights = a.weights; p.status = a.status;
  const int counts = counts_of(pair);
  p.taken = static_cast<int32_t *>(a.scratch);
  p.come = p.taken + 4;
  p.part = reinterpret_cast<float *>(p.taken + counts);
  p.test = a.test;
  CUtensorMap mq, mc;
  const cuuint64_t qd[3] = {(cuuint64_t)W, (cuuint64_t)R, (cuuint64_t)a.B};
  const cuuint64_t qs[2] = {(cuuint64_t)W * 2, (cuuint64_t)W * 2 * R};
  const cuuint32_t qb[3] = {64, (cuuint32_t)(pair ? 128 : p.cols), 1};
  const cuuint64_t cd[2] = {(cuuint64_t)W, (cuuint64_t)a.n_pages * a.page_size};
  const cuuint64_t cs[1] = {(cuuint64_t)W * 2};
  const cuuint32_t cb[2] = {64, (cuuint32_t)p.box_rows};
  if (!latent::make_bf16_map(&mq, a.q, 3, qd, qs, qb) ||
      !latent::make_bf16_map(&mc, a.cache, 2, cd, cs, cb))
    return cudaErrorInvalidValue;
  kda_latent_weights_begin_kernel<<<1, pair ? 512 : 32, 0, stream>>>(a.status, p.taken, counts);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(pair ? 2 * p.groups : p.groups));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return pair ? cudaLaunchKernelEx(&cfg, kda_latent_weights_pair_kernel, mq, mc, p)
              : cudaLaunchKernelEx(&cfg, kda_latent_weights_kernel, mq, mc, p);
}

}  // namespace kda
