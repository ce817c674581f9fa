// Latent attention in its absorbed form over a paged cache (kda_latent_decode),
// tcgen05 / TMEM / TMA, clusters of two CTAs, sm_103a.
//
// For one sequence, with R = T * H query rows of W = 512 + dr channels and cached
// rows c_j: s_rj = scale q_r . c_j, o_r = sum_j softmax(s_r)_j c_j[0:512].  The
// cached row is key and value at once: 2 W bytes of HBM and 2 R (W + 512)
// operations, at R = 96 181 operations a byte against the card's 289, so that
// decoding one token is bound by HBM when the matrix work runs near its rate, and
// a tree of drafts (R = 1536) by the matrix work.
//
// O [128 rows x 512] in fp32 would fill TMEM, and a 64-key tile beside all of Q
// would fill shared memory, so that one SM can neither hold the problem nor stream
// it.  Two SMs can: the CTAs of a pair share rows and keys and split the channels,
// rank 0 taking 0 .. 255 and the rotary ones, rank 1 256 .. 511.  Each loads its
// half of every cached row once, computes a partial S = Q C^T over its channels,
// sends it to the other through distributed shared memory (24 KB a tile at 96
// rows) and adds what it gets; both then do the same softmax, and each multiplies
// P with its own half of the values, which is the very tile it used as keys.  The
// sum of the two parts is the same in both CTAs, bit for bit.
//
// The way of a tile, S -> exchange -> softmax -> P -> O, takes about three times as
// long as the tensor cores need for it, so the ways of several tiles overlap: two
// warpgroups take the tiles in turn, each a tile all the way, and S of the next tile
// is issued as soon as S of this one is in registers.  TMEM (512 columns): Q 128
// (first operand of S; its rotary block is in shared memory), P 2 x 32 (first operand
// of O), O 256, S 64.  The rotary blocks of the tiles have a ring of their own,
// because they are done with S.  A thread owns a row of every other tile; exponents
// are taken against a reference per row, handed from tile to tile, that moves only
// when a score exceeds it by more than 8 (log2), and only then O is rescaled.  P is
// rounded to bf16 (half a step, 2^-8 of the value) as an operand of the tensor cores;
// the exchanged scores, sums, references and O are fp32.
//
// The 64-key tiles of all sequences form one list, cut evenly over the pairs
// whatever the lengths.  A pair's first and last sequence may be shared with its
// neighbours: it leaves (reference, sum, O) in the workspace and a second small
// kernel joins the parts in the list's order.  Every tile of 128 query rows has
// pairs / row tiles pairs, rounded down: with 76 pairs 12 row tiles use 72 of them, 20
// use 60, 39 use 39, and 77 take a second round for one.
//
// Measured (96 heads, dr = 64; whole calls, cold inputs): one token of 128 sequences of
// up to 16384 rows, 1.2 GB, 297 us, 4.1 TB/s (DRAM 55 % busy, tensor cores 42 %); trees
// of 16 drafts, 32 sequences, 1,114 us, 0.91 PFLOP/s (DRAM 5 %, tensor cores 37 %); one
// token over 3001 rows, dr = 0, 20.5 us (replayed), all of it start, one tile's way and
// the join.  A pair takes about 2,750 cycles a tile at 96 rows and 2,850 at 128, though
// it then exchanges 32 KB and not 24 in each direction (1,490 and 1,100 cycles at the 22
// bytes a cycle that distributed shared memory gave by itself).  The products take
// 1,200, the copies at 96 rows 1,740 (by themselves, in the same ring, 7.3 TB/s).  So
// none of them is the bound alone; what is left is a tile's way, of which two at most
// overlap.  How its steps share the time has not been measured.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <string.h>

#include "kda_latent_tc.cuh"

namespace kda {
namespace {

using namespace latent;

constexpr int kTile = 64;                // keys per tile
constexpr int kRows = 128;               // query rows of a pair
constexpr int kHalf = kLatentC / 2;      // channels of a CTA's values
constexpr int kThreads = 384;            // 2 x 4 softmax warps, loader, MMA, cleaner, spare
constexpr int kLoadWarp = 8, kMmaWarp = 11, kCleanWarp = 10, kSpareWarp = 9;
constexpr uint32_t kBlock = 8192;        // 64 keys x 64 channels
constexpr uint32_t kStage = 4 * kBlock;  // a CTA's half of a tile without the rotary block
constexpr uint32_t kQBlock = 16384;      // 128 rows x 64 channels
constexpr uint32_t kSmem = 232448;
constexpr float kSlack = 8.f;            // log2 units a score may exceed its reference by
constexpr int kMaxStages = 6;
constexpr uint32_t TM_Q = 0, TM_P = 128, TM_O = 192, TM_S = 448;

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages], clean_req[kMaxStages], clean[kMaxStages];
  uint64_t rope_free[kMaxStages], s_full[2], recv_full[2], send_ok[2], p_ready[2];
  uint64_t q_full, q_ready, q_empty[2], s_free, pv_done[2], o_free, fin;
  uint64_t ref_ready[4][2], l_ready[4], l_taken[4];  // by warp of a warpgroup
  uint32_t tmem;
  int abort;
  int seq0, tile0, total;                // the pair's first sequence and tile, all tiles
  int64_t warp_sum[kThreads / 32];
  uint32_t load_pos;                     // tiles loaded, segments begun (loader)
  int load_seg;
  DeviceStatus error;                    // the CTA's first error
  float ref[2][kRows];                   // reference after a tile, by its parity
  float2 part[kRows];                    // the last but one tile's warpgroup: its sum, and of what
};
constexpr uint32_t kSharedBytes = 3 * 1024;
static_assert(sizeof(Shared) <= kSharedBytes, "fits beside the tiles");

struct Params {
  const int32_t *table, *lens;
  const int64_t *mask;
  const __nv_bfloat16 *q;
  int32_t B, T, H, W, R, n_pages, page_size, max_pages, box_rows;
  int32_t row_tiles;    // row tiles of 128
  int32_t G;            // pairs per row tile
  int32_t warps;        // 32-row groups in use
  int32_t stages[2];    // of either rank
  int32_t rope_slots;   // of rank 0
  float scale2;         // scale * log2(e), see launch_latent_decode
  float ln_hi, ln_lo;   // a logarithm by that scale to the natural one, in two parts
  __nv_bfloat16 *out;
  float *lse;
  DeviceStatus *status;
  DeviceStatus *errors; // [CTAs]
  int4 *joins;          // [G] of the border before a pair: sequence, parts (0: none), slot
  float *part_o;        // [row tiles][G][2][512 / 4][128 rows][4]
  float *part_ml;       // [row tiles][G][2][2][128]
  WaitTest test;
};

__device__ __forceinline__ float natural(const Params &p, float x) {
  return fmaf(x, p.ln_hi, x * p.ln_lo);
}

// Length of sequence b, 0 when it is out of range.
__device__ __forceinline__ int seq_len(const Params &p, int b) {
  const int n = p.lens[b];
  return n < 0 || n > (int64_t)p.max_pages * p.page_size ? 0 : n;
}
static_assert(kTile == 64, "tiles are counted with shifts");
// (n reaches 2^31 - 1: nothing may be added to it.)
__device__ __forceinline__ int key_tiles(int n) { return (n >> 6) + ((n & 63) != 0); }

// First tile of pair c of G when the list has `total` tiles: the first total % G
// pairs take one more than the others.
__device__ __forceinline__ int pair_begin(int c, int G, int total) {
  const int each = total / G, more = total - each * G;
  return c * each + min(c, more);
}
// The pair of tile x.
__device__ __forceinline__ int pair_of(int x, int G, int total) {
  const int each = total / G, more = total - each * G, wide = more * (each + 1);
  return x < wide ? x / (each + 1) : more + (x - wide) / max(each, 1);
}

// Walks the pair's tiles sequence by sequence; every role does so by itself.
struct Walk {
  const Params &p;
  int b, t, left;       // next sequence, its next tile, tiles left
  int n, ta, tb;        // current segment: length of the sequence, tiles [ta, tb)
  __device__ Walk(const Params &p_, int b_, int t_, int left_) : p(p_), b(b_), t(t_), left(left_) {}
  __device__ bool next(int *seq) {
    if (left <= 0) return false;
    while (b < p.B) {
      n = seq_len(p, b);
      const int k = key_tiles(n);
      if (t < k) {
        ta = t;
        tb = k - t <= left ? k : t + left;
        left -= tb - ta;
        *seq = b;
        if (tb == k) { ++b; t = 0; } else { t = tb; }
        return true;
      }
      ++b;
      t = 0;
    }
    return false;
  }
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
kda_latent_decode_kernel(const __grid_constant__ CUtensorMap map_q,
                         const __grid_constant__ CUtensorMap map_c, const Params p) {
  constexpr uint32_t ID_S = idesc_bf16(128, kTile, false, false);
  constexpr uint32_t ID_PV = idesc_bf16(128, kHalf, false, true);

  extern __shared__ __align__(1024) unsigned char tiles[];
  const uint32_t base = smem_u32(tiles);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank(), peer = rank ^ 1u;
  const int pair = blockIdx.x >> 1, rt = pair % p.row_tiles, slice = pair / p.row_tiles;
  const bool rope = rank == 0 && p.W > kLatentC;
  const int nb = rope ? 5 : 4;                          // blocks of a tile
  const int NS = p.stages[rank], NR = p.rope_slots;
  const int rows = p.warps * 32;                        // rows in use
  // shared memory: two tiles that the other CTA sends (at one offset in both), the
  // rotary block of Q, tiles, their rotary blocks, the rest
  const uint32_t sm_recv = base, recv_bytes = rows * kTile * 4, sm_q = sm_recv + 2 * recv_bytes;
  const uint32_t sm_ring = sm_q + (rope ? kQBlock : 0), sm_rope = sm_ring + NS * kStage;
  Shared &m = *reinterpret_cast<Shared *>(tiles + (kSmem - kSharedBytes));

  if (tid == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&m.full[i], 1);
      mbar_init(&m.empty[i], 1);
      mbar_init(&m.clean_req[i], 1);
      mbar_init(&m.clean[i], 1);
      mbar_init(&m.rope_free[i], 1);
    }
    mbar_init(&m.q_full, 1);
    mbar_init(&m.q_ready, p.warps);
    mbar_init(&m.q_empty[0], 1);
    mbar_init(&m.q_empty[1], 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&m.s_full[i], 1);
      mbar_init(&m.p_ready[i], p.warps);
      mbar_init(&m.recv_full[i], 1);
      mbar_init(&m.send_ok[i], p.warps);
    }
    mbar_init(&m.s_free, p.warps);
    mbar_init(&m.pv_done[0], 1);
    mbar_init(&m.pv_done[1], 1);
    mbar_init(&m.o_free, p.warps);
    for (int i = 0; i < 4; ++i) {
      mbar_init(&m.ref_ready[i][0], 1);
      mbar_init(&m.ref_ready[i][1], 1);
      mbar_init(&m.l_ready[i], 1);
      mbar_init(&m.l_taken[i], 1);
    }
    mbar_init(&m.fin, 1);
    m.abort = 0;
    m.seq0 = p.B;
    m.tile0 = 0;
    m.load_pos = 0;
    m.load_seg = 0;
    m.error = DeviceStatus{0, 0, 0, 0, 0, 0};
    fence_mbarrier_init();
  }
  if (warp == kLoadWarp && lane == 0) {
    prefetch_tensormap(&map_q);
    prefetch_tensormap(&map_c);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&m.tmem, 512);
    tmem_relinquish();
  }
  {  // the pair's share of the tile list
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = tid * per, b1 = min(p.B, b0 + per);
    int64_t mine = 0;                    // sequences may share pages: no pool bounds the sum
    bool bad = false;
    for (int b = b0; b < b1; ++b) {
      const int n = p.lens[b];
      if (n < 0 || n > (int64_t)p.max_pages * p.page_size) bad = true;
      else mine += key_tiles(n);
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
    // tiles are counted in 32 bits from here on; a list that is longer is refused
    const int total = all > 0x7fffffff ? 0 : (int)all;
    if (all > 0x7fffffff && tid == 0)
      record_device_status(&m.error, KDA_ERR_INVALID_ARG, 3, 0, 0);
    const int begin = pair_begin(slice, p.G, total);
    if (total > 0 && begin >= before && begin < before + mine) {
      int at = (int)before;
      for (int b = b0; b < b1; ++b) {
        const int k = key_tiles(seq_len(p, b));
        if (begin < at + k) {
          m.seq0 = b;
          m.tile0 = begin - at;
          break;
        }
        at += k;
      }
    }
    if (tid == 0) m.total = total;
  }
  tc_fence_before();
  cluster_sync_all();  // barriers of both CTAs are ready, and their shared memory mapped
  tc_fence_after();
  pdl_launch_dependents();
  const uint32_t tm = m.tmem;
  if (rt == 0 && rank == 0 && tid == 0) {  // for the kernel that joins the parts
    // The first border inside a sequence joins its parts, from the pair before it to the
    // pair of its last tile.  A pair's first segment is in slot 0, its last in slot 1.
    const int at = pair_begin(slice, p.G, m.total), start = at - m.tile0;
    const int before = slice > 0 ? pair_begin(slice - 1, p.G, m.total) : 0;
    int parts = 0;
    if (slice > 0 && m.tile0 > 0 && before <= start)
      parts = pair_of(start + key_tiles(seq_len(p, m.seq0)) - 1, p.G, m.total) - slice + 2;
    p.joins[slice] = make_int4(m.seq0, parts, 2 * (slice - 1) + (before < start ? 1 : 0), 0);
  }
  const int begin = pair_begin(slice, p.G, m.total);
  const int mine = pair_begin(slice + 1, p.G, m.total) - begin;
  const WaitCtx cx{&m.abort, &m.error, (int)blockIdx.x, p.test.wait_ns};
  Walk walk(p, m.seq0, m.tile0, mine);
  int b;

  if (warp == kLoadWarp) {
    // ---- loader: every lane has one box of a tile, block lane % nb of piece lane / nb
    uint32_t pos = 0;                    // tiles loaded
    int s = 0, sr = 0, seg = 0;          // stage and rotary slot of the next tile
    bool ok = true;
    const int piece = lane / nb, blk = lane - piece * nb, pieces = kTile / p.box_rows;
    const int col = rank ? kHalf + 64 * blk : blk < 4 ? 64 * blk : kLatentC;
    const uint32_t off = (blk < 4 ? blk * kBlock : 0) + piece * p.box_rows * 128;
    while (ok && walk.next(&b)) {
      const int n = walk.n;
      // pool row of this lane's box of tile t, -1: nothing to load
      auto box_row = [&](int t) {
        if (piece >= pieces || t >= walk.tb) return -1;
        const int at = t * kTile + piece * p.box_rows;
        if (at >= n) return -1;
        const int page = at / p.page_size;
        const int32_t id = p.table[(int64_t)b * p.max_pages + page];
        if (id < 0 || id >= p.n_pages) {
          record_device_status(&m.error, KDA_ERR_INVALID_ARG, 2, b, at);
          return p.n_pages * p.page_size;  // past the pool: reads zeros
        }
        return id * p.page_size + at - page * p.page_size;
      };
      int row = box_row(walk.ta);
      if (rope) {
        if (seg > 0)
          ok = warp_wait(cx, &m.q_empty[(seg - 1) & 1], ((seg - 1) >> 1) & 1, 10, seg);
        if (!ok) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(&m.q_full, kQBlock);
          tma_load_3d_u(sm_q, &map_q, &m.q_full, kLatentC, rt * kRows, b);
        }
      }
      ++seg;
      for (int t = walk.ta; t < walk.tb; ++t) {
        if ((int)pos == p.test.tile && p.test.block == (int)blockIdx.x) {
          ok = false;                    // a test: the waits for this tile run out
          break;
        }
        const int row_next = box_row(t + 1);
        if (pos >= NS) ok = warp_wait(cx, &m.empty[s], (pos / NS - 1) & 1, 11, t);
        if (ok && rope && pos >= NR) ok = warp_wait(cx, &m.rope_free[sr], (pos / NR - 1) & 1, 12, t);
        if (!ok) break;
        const int have = __popc(__ballot_sync(0xffffffffu, row >= 0));
        if (lane == 0) mbar_arrive_expect_tx(&m.full[s], have * p.box_rows * 128);
        __syncwarp();
        if (row >= 0)
          tma_load_2d((blk < 4 ? sm_ring + s * kStage : sm_rope + sr * kBlock) + off, &map_c,
                      &m.full[s], col, row);
        __syncwarp();
        if (lane == 0 && n - t * kTile < kTile) mbar_arrive(&m.clean_req[s]);
        row = row_next;
        ++pos;
        s = s + 1 == NS ? 0 : s + 1;
        sr = sr + 1 == NR ? 0 : sr + 1;
      }
    }
    if (lane == 0) {
      m.load_pos = pos;
      m.load_seg = seg;
    }
  } else if (warp == kMmaWarp && elect_one()) {
    // ---- MMA issue: whichever of the next O and the next S has its operands, O first
    // (stages wait for it).  S waits until the S before it has been read, and is at
    // most three tiles ahead of O.
    const Desc q_s(sm_q, 16), c_s(sm_ring, 16), r_s(sm_rope, 16), c_v(sm_ring, kBlock);
    uint32_t pos = 0, done = 0, cleaned = 0;  // S and O issued; parity bit per stage
    uint32_t first = 0, ragged = 0;      // of the tiles in between, bit 0 the oldest
    int s = 0, sr = 0, sv = 0, seg = -1, seg_o = -1, t = 0;
    bool more = walk.next(&b);           // a tile is left for S
    t = walk.ta;
    uint64_t idle = 0;                   // since when nothing could be issued
    while (more || done < pos) {
      if (done < pos && mbar_test_wait(&m.p_ready[done & 1], (done >> 1) & 1) &&
                 (!(ragged & 1) || mbar_test_wait(&m.clean[sv], cleaned >> sv & 1)) &&
                 (!(first & 1) || seg_o < 0 || mbar_test_wait(&m.o_free, seg_o & 1))) {
        idle = 0;
        tc_fence_after();
        if (first & 1) ++seg_o;
        if (ragged & 1) cleaned ^= 1u << sv;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_ts(tm + TM_O, tm + TM_P + 32 * (done & 1) + 8 * k, c_v.at(sv * kStage + k * 2048), ID_PV,
                  k > 0 || !(first & 1));
        umma_commit(&m.empty[sv]);
        umma_commit(&m.pv_done[done & 1]);
        ++done;
        first >>= 1;
        ragged >>= 1;
        sv = sv + 1 == NS ? 0 : sv + 1;
      } else if (more && pos - done < 3 && mbar_test_wait(&m.full[s], (pos / NS) & 1) &&
          (pos < 1 || mbar_test_wait(&m.s_free, (pos - 1) & 1)) &&
          (t > walk.ta || (mbar_test_wait(&m.q_ready, (seg + 1) & 1) &&
                           (!rope || mbar_test_wait(&m.q_full, (seg + 1) & 1))))) {
        idle = 0;
        tc_fence_after();
        if (t == walk.ta) ++seg;
        const uint32_t at = s * kStage, ts = tm + TM_S;
#pragma unroll
        for (int k = 0; k < 16; ++k)
          umma_ts(ts, tm + TM_Q + 8 * k, c_s.at(at + (k >> 2) * kBlock + (k & 3) * 32), ID_S, k > 0);
        if (rope) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_ss(ts, q_s.at(k * 32), r_s.at(sr * kBlock + k * 32), ID_S, 1);
          umma_commit(&m.rope_free[sr]);
          sr = sr + 1 == NR ? 0 : sr + 1;
        }
        umma_commit(&m.s_full[pos & 1]);
        if (t + 1 == walk.tb) umma_commit(&m.q_empty[seg & 1]);
        const uint32_t bit = pos - done;
        first |= (t == walk.ta ? 1u : 0u) << bit;
        ragged |= (walk.n - t * kTile < kTile ? 1u : 0u) << bit;
        ++pos;
        s = s + 1 == NS ? 0 : s + 1;
        if (++t == walk.tb) {
          more = walk.next(&b);
          t = walk.ta;
        }
      } else {
        if (*cx.abort) break;
        const uint64_t now = global_timer_ns();
        if (idle == 0) idle = now;
        if (now - idle > cx.wait_ns) {
          record_device_status(cx.status, KDA_ERR_TIMEOUT, 20, cx.chain, (int)pos);
          *cx.abort = 1;
          break;
        }
      }
    }
  } else if (warp == kCleanWarp) {
    // ---- cleaner: rows past a sequence's end may hold anything; as values they are
    // zeroed in shared memory (0 * NaN would reach the sum).  The loader asks once
    // the copies of the tile are under way, and nothing overtakes a request of the
    // same stage, because its product waits for the answer.
    uint32_t asked = 0;                  // parity bit per stage
    uint32_t pos = 0;
    bool ok = true;
    while (ok && walk.next(&b)) {
      pos += walk.tb - walk.ta;
      const int live = walk.n - (walk.tb - 1) * kTile;
      if (live >= kTile) continue;
      const int s = (pos - 1) % NS;
      ok = warp_wait<kLongWaits>(cx, &m.clean_req[s], asked >> s & 1, 30, walk.tb) &&
           warp_wait(cx, &m.full[s], ((pos - 1) / NS) & 1, 31, walk.tb);
      if (!ok) break;
      asked ^= 1u << s;
      const uint32_t dst = sm_ring + s * kStage + live * 128;
      for (int i = lane; i < (kTile - live) * 8; i += 32)
#pragma unroll
        for (int c = 0; c < 4; ++c) st_shared_v4(dst + c * kBlock + i * 16, 0, 0, 0, 0);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&m.clean[s]);
    }
  } else if (warp < 8 && (warp & 3) < p.warps) {
    // ---- softmax and output: thread = row; warpgroup = parity of the tiles
    const int wg = warp >> 2, w4 = warp & 3;
    const int r = w4 * 32 + lane, row = rt * kRows + r, tok = row / p.H;
    const uint32_t lanes = (uint32_t)w4 << 21;
    const uint32_t ts = tm + lanes + TM_S;
    const uint32_t src = sm_recv + wg * recv_bytes + r * 16;
    const uint32_t dst = map_rank(src, peer), bar = map_rank(smem_u32(&m.recv_full[wg]), peer);
    const uint32_t credit = map_rank(smem_u32(&m.send_ok[wg]), peer);
    uint32_t pos = 0;
    int seg = 0, joined = 0;             // segments; those of two tiles and more
    bool ok = true;
    for (; ok && walk.next(&b); ++seg) {
      const int n = walk.n, t_draft = n - p.T;          // position of the first draft
      const bool several = walk.tb - walk.ta > 1;
      if ((pos & 1) == (uint32_t)wg) {
        // Q of the segment into TMEM, once the segment before has used its own.  A
        // warpgroup has a tile in at least one of two consecutive segments, so with
        // a barrier for each parity it is never two phases behind.
        if (seg > 0)
          ok = warp_wait(cx, &m.q_empty[(seg - 1) & 1], ((seg - 1) >> 1) & 1, 40, seg);
        if (!ok) break;
        tc_fence_after();
        const __nv_bfloat16 *q = p.q + ((int64_t)b * p.R + row) * p.W + rank * kHalf;
#pragma unroll
        for (int c = 0; c < 4; c += 2) {                // 16 loads in flight
          uint32_t x[2][32];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (row < p.R) v = *reinterpret_cast<const uint4 *>(q + 64 * c + 8 * j);
            uint32_t *y = &x[j >> 3][4 * (j & 7)];
            y[0] = v.x; y[1] = v.y; y[2] = v.z; y[3] = v.w;
          }
          tmem_st32(tm + lanes + TM_Q + 32 * c, x[0]);
          tmem_st32(tm + lanes + TM_Q + 32 * c + 32, x[1]);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.q_ready);
      }
      // the drafts this row sees, by index
      uint64_t seen = 0;
      if (p.mask && tok < p.T) seen = (uint64_t)p.mask[(int64_t)b * p.T + tok];
      if (p.T < 64) seen &= (1ull << p.T) - 1;
      float ref = kNoRef, l = 0.f;                      // l is relative to ref
      for (int t = walk.ta; t < walk.tb; ++t, ++pos) {
        if ((pos & 1) != (uint32_t)wg) continue;
        const uint32_t par = (pos >> 1) & 1;
        if (w4 == 0 && lane == 0) mbar_arrive_expect_tx(&m.recv_full[wg], recv_bytes);
        ok = warp_wait(cx, &m.s_full[wg], par, 41, t);
        if (!ok) break;
        tc_fence_after();
        uint32_t x[2][32];
        tmem_ld32(ts, x[0]);
        tmem_ld32(ts + 32, x[1]);
        tmem_ld_wait(x[0]);
        tmem_ld_wait(x[1]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.s_free);
        // this CTA's part to the other one, which has read the tile that the buffer had
        if (pos > 1) ok = warp_wait(cx, &m.send_ok[wg], par ^ 1, 42, t);
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            st_async_v4(dst + (8 * c + j) * rows * 16, x[c][4 * j], x[c][4 * j + 1],
                        x[c][4 * j + 2], x[c][4 * j + 3], bar);
        ok = warp_wait(cx, &m.recv_full[wg], par, 43, t);
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 y = ld_shared_f32x4(src + (8 * c + j) * rows * 16);
            x[c][4 * j] = __float_as_uint(__uint_as_float(x[c][4 * j]) + y.x);
            x[c][4 * j + 1] = __float_as_uint(__uint_as_float(x[c][4 * j + 1]) + y.y);
            x[c][4 * j + 2] = __float_as_uint(__uint_as_float(x[c][4 * j + 2]) + y.z);
            x[c][4 * j + 3] = __float_as_uint(__uint_as_float(x[c][4 * j + 3]) + y.w);
          }
        if (t_draft - t * kTile < kTile) {              // the drafts' own tiles and the end
          const int live = min(kTile, n - t * kTile), d0 = t_draft - t * kTile;
          // bit j: this row sees key j of the tile
          uint64_t see = live >= 64 ? ~0ull : (1ull << live) - 1;
          const auto below = [](int k) { return k <= 0 ? 0ull : k >= 64 ? ~0ull : (1ull << k) - 1; };
          if (p.mask)
            see &= below(d0) | (d0 >= 0 ? (d0 < 64 ? seen << d0 : 0ull)
                                        : (d0 > -64 ? seen >> -d0 : 0ull));
          else
            see &= below(d0 + tok + 1);
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (!(see >> (32 * c + j) & 1)) x[c][j] = __float_as_uint(-CUDART_INF_F);
        }
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          mx[c] = __uint_as_float(x[c >> 1][16 * (c & 1)]);
#pragma unroll
          for (int j = 1; j < 16; ++j)
            mx[c] = fmaxf(mx[c], __uint_as_float(x[c >> 1][16 * (c & 1) + j]));
        }
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale2;
        // The reference after the tile before, from the other warpgroup's same warp
        // (across segments only the turn: it has read what is overwritten below).
        if (pos > 0) ok = warp_wait(cx, &m.ref_ready[w4][wg ^ 1], ((pos - 1) >> 1) & 1, 44, t);
        if (!ok) break;
        const float before = t > walk.ta ? m.ref[wg ^ 1][r] : kNoRef;
        const bool move = __any_sync(0xffffffffu, top > before + kSlack);
        // The vote has consumed every value read from what the other CTA sent: it may
        // send into the buffer again.
        if (lane == 0) remote_arrive_relaxed(credit);
        const float now = move ? fmaxf(before, top) : before;
        m.ref[wg][r] = now;
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.ref_ready[w4][wg]);
        l *= ex2(ref - now);
        ref = now;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t pk[32];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float u = ex2(fmaf(__uint_as_float(x[c][j]), p.scale2, -ref));
            const float v = ex2(fmaf(__uint_as_float(x[c][j + 1]), p.scale2, -ref));
            sum[(j >> 1) & 3] += u + v;
            pk[16 * c + j / 2] = pack_bf16x2(u, v);
          }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
        // this P's buffer is free once the product of two tiles before is done
        if (pos > 1) ok = warp_wait(cx, &m.pv_done[wg], par ^ 1, 45, t);
        if (!ok) break;
        tc_fence_after();
        if (move && t > walk.ta) {  // and O once that of the tile before is
          ok = warp_wait(cx, &m.pv_done[wg ^ 1], ((pos - 1) >> 1) & 1, 48, t);
          if (!ok) break;
          tc_fence_after();
          const float f = ex2(before - now);
#pragma unroll 1
          for (int c = 0; c < kHalf / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tm + lanes + TM_O + 32 * c, o);
            tmem_ld_wait(o);
#pragma unroll
            for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            tmem_st32(tm + lanes + TM_O + 32 * c, o);
          }
        }
        tmem_st32(tm + lanes + TM_P + 32 * wg, pk);
        tmem_st_wait();
        tc_fence_before();
        if (t + 1 == walk.tb && several) {
          ok = warp_wait(cx, &m.l_ready[w4], joined & 1, 46, seg);
          if (!ok) break;
          const float2 other = m.part[r];
          l += other.x * ex2(other.y - ref);
          __syncwarp();
          if (lane == 0) mbar_arrive(&m.l_taken[w4]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.p_ready[wg]);
        if (t + 2 == walk.tb) {  // the other warpgroup ends the segment: hand it the sum
          if (joined > 0) ok = warp_wait(cx, &m.l_taken[w4], (joined - 1) & 1, 49, t);
          if (!ok) break;
          m.part[r] = make_float2(l, ref);
          __syncwarp();
          if (lane == 0) mbar_arrive(&m.l_ready[w4]);
        }
      }
      if (!ok) break;
      joined += several;
      if (((pos - 1) & 1) != (uint32_t)wg) continue;    // the other warpgroup's last tile
      // ---- the segment's output
      ok = warp_wait(cx, &m.pv_done[wg], ((pos - 1) >> 1) & 1, 47, seg);
      if (!ok) break;
      tc_fence_after();
      const bool whole = walk.ta == 0 && walk.tb == key_tiles(n);
      // slot of a part: a pair's first segment 0, its last 1
      const int64_t slot = ((int64_t)rt * p.G + slice) * 2 + (seg == 0 ? 0 : 1);
      const int64_t out_row = (int64_t)b * p.R + row;
      if (rank == 0) {
        if (whole) {
          if (p.lse && row < p.R)
            p.lse[out_row] = l == 0.f ? -CUDART_INF_F : natural(p, ref + log2f(l));
        } else {
          p.part_ml[slot * 2 * kRows + r] = ref;
          p.part_ml[slot * 2 * kRows + kRows + r] = l;
        }
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
      for (int c = 0; c < kHalf / 32; ++c) {
        uint32_t o[32];
        tmem_ld32(tm + lanes + TM_O + 32 * c, o);
        tmem_ld_wait(o);
        if (whole) {
          uint4 *to = reinterpret_cast<uint4 *>(p.out + out_row * kLatentC + rank * kHalf + 32 * c);
          if (row < p.R)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t w[4];
#pragma unroll
              for (int k = 0; k < 4; ++k)
                w[k] = pack_bf16x2(__uint_as_float(o[8 * j + 2 * k]) * inv,
                                   __uint_as_float(o[8 * j + 2 * k + 1]) * inv);
              to[j] = make_uint4(w[0], w[1], w[2], w[3]);
            }
        } else {
          // four channels of the 32 rows beside one another
          uint4 *to = reinterpret_cast<uint4 *>(p.part_o) +
                      (slot * (kLatentC / 4) + (rank * kHalf + 32 * c) / 4) * kRows + r;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            to[j * kRows] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&m.o_free);
    }
  }

  if (warp == kSpareWarp) {
    // ---- rows of empty sequences see nothing
    for (int e = slice; e < p.B; e += p.G)
      if (key_tiles(seq_len(p, e)) == 0)
        for (int i = lane; i < kRows * kHalf / 8; i += 32) {
          const int row = rt * kRows + i / (kHalf / 8), c = i % (kHalf / 8);
          if (row >= p.R) break;
          const int64_t at = (int64_t)e * p.R + row;
          *reinterpret_cast<uint4 *>(p.out + at * kLatentC + rank * kHalf + 8 * c) =
              make_uint4(0, 0, 0, 0);
          if (p.lse && rank == 0 && c == 0) p.lse[at] = -CUDART_INF_F;
        }
  }

  __syncwarp();
  __syncthreads();
  if (m.abort) {
    // nothing in flight outlives the CTA: the last copy into every stage, the last
    // Q, the products; then time for what is on its way between the CTAs
    if (tid == 32 * kLoadWarp) {
      const uint32_t pos = m.load_pos;
      for (uint32_t k = pos > (uint32_t)NS ? pos - NS : 0; k < pos; ++k)
        mbar_wait(&m.full[k % NS], (k / NS) & 1, kWaitNs);
      if (rope && m.load_seg > 0) mbar_wait(&m.q_full, (m.load_seg - 1) & 1, kWaitNs);
    }
    if (warp == kMmaWarp && elect_one()) {  // of the lane that issued the products
      umma_commit(&m.fin);
      mbar_wait(&m.fin, 0, kWaitNs);
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < 20000) {}
    }
    __syncthreads();
  }
  if (tid == 0) p.errors[blockIdx.x] = m.error;
  if (warp == kMmaWarp) {
    __syncwarp();
    tmem_dealloc(tm, 512);
  }
  cluster_sync_all();  // the other CTA is done with this one's shared memory
}

// Joins the parts of sequences that several pairs shared, in the list's order.
// Block (x: 32 rows and some channels, y: the y-th border that joins a sequence; the
// last y: the call's status, which is the first error of any CTA, or none).  A lane is
// a row.  With few sequences there are many parts to each: a block has 16 channels, its
// warps take the parts in turn, and their sums are added in warp order.  With many
// there are few: a block has 128 channels, 16 a warp, and every warp takes all parts.
// Whole calls, first form against second, 96 rows: 1 x 3000 keys 20.5 / 48.4 us, 8 x
// 4000 30.6 / 35.0, 12 x 4000 (six parts and a half each) 37.0 / 37.7, 19 x 4000 49.2 /
// 45.2, 64 x 2000 85.9 / 61.5.  Both wait for memory: a border, its parts, their sum.
constexpr int kJoinWarps = 8, kJoinCh = 16;
template <bool kMany>
__global__ void __launch_bounds__(32 * kJoinWarps)
kda_latent_join_kernel(const Params p) {
  constexpr int kStep = kMany ? kJoinWarps : 1;         // warps that share the parts
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  if (blockIdx.y + 1 == gridDim.y) {
    if (blockIdx.x > 0 || warp > 0) return;
    int at = 0x7fffffff;
    const int ctas = p.G * p.row_tiles * 2;
#pragma unroll 8
    for (int i = lane; i < ctas; i += 32)
      if (p.errors[i].code != 0) at = min(at, i);
    at = __reduce_min_sync(0xffffffffu, at);
    if (lane == 0) {
      DeviceStatus st{0, 0, 0, 0, 0, 0};
      if (at < ctas) st = p.errors[at];
      *p.status = st;
    }
    return;
  }
  int4 join = make_int4(0, 0, 0, 0);
  int skip = blockIdx.y;                 // joining borders still to be passed over
#pragma unroll 3
  for (int i = lane; i - lane < p.G; i += 32) {
    const int4 v = i < p.G ? p.joins[i] : make_int4(0, 0, 0, 0);
    const unsigned have = __ballot_sync(0xffffffffu, v.y > 0);
    const int src =
        __ffs(__ballot_sync(0xffffffffu,
                            v.y > 0 && __popc(have & ((1u << lane) - 1)) == skip)) - 1;
    if (src >= 0) {
      join.x = __shfl_sync(0xffffffffu, v.x, src);
      join.y = __shfl_sync(0xffffffffu, v.y, src);
      join.z = __shfl_sync(0xffffffffu, v.z, src);
    }
    skip -= __popc(have);                // below 0 once found, and never 0 again
  }
  const int parts = join.y;
  if (parts == 0) return;
  const int groups = (p.R + 31) / 32;
  const int group = blockIdx.x % groups;
  const int ch = (blockIdx.x / groups * (kMany ? 1 : kJoinWarps) + (kMany ? 0 : warp)) * kJoinCh;
  const int rt = group / 4, r = (group & 3) * 32 + lane, row = group * 32 + lane;
  const int64_t slot0 = (int64_t)rt * p.G * 2 + join.z;
  float ref = kNoRef, l = 0.f, o[kJoinCh];
#pragma unroll
  for (int c = 0; c < kJoinCh; ++c) o[c] = 0.f;
#pragma unroll 4
  for (int i = kMany ? warp : 0; i < parts; i += kStep) {
    const int64_t slot = i == 0 ? slot0 : (slot0 & ~(int64_t)1) + 2 * i;
    const float4 *x = reinterpret_cast<const float4 *>(p.part_o) +
                      (slot * (kLatentC / 4) + ch / 4) * kRows + r;
    float4 v[kJoinCh / 4];
#pragma unroll
    for (int c = 0; c < kJoinCh / 4; ++c) v[c] = x[c * kRows];
    const float m = p.part_ml[slot * 2 * kRows + r], s = p.part_ml[slot * 2 * kRows + kRows + r];
    const float now = m > ref || m != m ? m : ref;
    const float a = ex2(ref - now), b = ex2(m - now);
    ref = now;
    l = l * a + s * b;
#pragma unroll
    for (int c = 0; c < kJoinCh / 4; ++c) {
      o[4 * c] = o[4 * c] * a + v[c].x * b;
      o[4 * c + 1] = o[4 * c + 1] * a + v[c].y * b;
      o[4 * c + 2] = o[4 * c + 2] * a + v[c].z * b;
      o[4 * c + 3] = o[4 * c + 3] * a + v[c].w * b;
    }
  }
  const int64_t out_row = (int64_t)join.x * p.R + row;
  if (!kMany) {
    if (row >= p.R) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint32_t w[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) w[c] = pack_bf16x2(o[2 * c] * inv, o[2 * c + 1] * inv);
    uint4 *to = reinterpret_cast<uint4 *>(p.out + out_row * kLatentC + ch);
    to[0] = make_uint4(w[0], w[1], w[2], w[3]);
    to[1] = make_uint4(w[4], w[5], w[6], w[7]);
    if (p.lse && ch == 0)
      p.lse[out_row] = l == 0.f ? -CUDART_INF_F : natural(p, ref + log2f(l));
    return;
  }
  __shared__ float s_o[kJoinWarps][kJoinCh][32], s_ref[kJoinWarps][32], s_l[kJoinWarps][32];
  s_ref[warp][lane] = ref;
  s_l[warp][lane] = l;
#pragma unroll
  for (int c = 0; c < kJoinCh; ++c) s_o[warp][c][lane] = o[c];
  __syncthreads();
  // warp w: channels 2 w and 2 w + 1 of all rows
  ref = s_ref[0][lane];
#pragma unroll
  for (int w = 1; w < kJoinWarps; ++w) {
    const float y = s_ref[w][lane];
    ref = y > ref || y != y ? y : ref;
  }
  l = 0.f;
  float u = 0.f, v = 0.f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    const float f = ex2(s_ref[w][lane] - ref);
    l += f * s_l[w][lane];
    u += f * s_o[w][2 * warp][lane];
    v += f * s_o[w][2 * warp + 1][lane];
  }
  if (row >= p.R) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *reinterpret_cast<uint32_t *>(p.out + out_row * kLatentC + ch + 2 * warp) =
      pack_bf16x2(u * inv, v * inv);
  if (p.lse && ch == 0 && warp == 0)
    p.lse[out_row] = l == 0.f ? -CUDART_INF_F : natural(p, ref + log2f(l));
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
    if (!kernel_ready<kda_latent_decode_kernel>(kSmem, 0) ||
        cudaOccupancyMaxActiveClusters(&n, kda_latent_decode_kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
    }
    return n;
  });
}

struct Plan {
  int row_tiles, G;
  size_t joins, errors, ml, o;          // bytes of the workspace's pieces
};
Plan make_plan(int T, int H) {
  Plan pl;
  pl.row_tiles = (T * H + kRows - 1) / kRows;
  const int pairs = resident_pairs();
  pl.G = pairs / pl.row_tiles;
  if (pl.G < 1) pl.G = 1;
  auto round = [](size_t x) { return (x + 255) / 256 * 256; };
  // partial results: none when one pair has all keys of its rows
  const size_t parts = pl.G > 1 ? (size_t)pl.row_tiles * pl.G * 2 : 0;
  pl.joins = round((size_t)pl.G * sizeof(int4));
  pl.errors = round((size_t)pl.row_tiles * pl.G * 2 * sizeof(DeviceStatus));
  pl.ml = parts * 2 * kRows * sizeof(float);
  pl.o = parts * kRows * kLatentC * sizeof(float);
  return pl;
}

}  // namespace

size_t latent_decode_scratch_bytes(int32_t B, int32_t T, int32_t H, int32_t dr) {
  (void)B;
  (void)dr;
  const Plan pl = make_plan(T, H);
  return pl.joins + pl.errors + pl.ml + pl.o;
}

cudaError_t launch_latent_decode(const LatentDecodeArgs &a, cudaStream_t stream) {
  if (a.B == 0) return cudaMemsetAsync(a.status, 0, sizeof(DeviceStatus), stream);
  if (!latent::encode_tiled() || resident_pairs() < 1) return cudaErrorNotSupported;
  const Plan pl = make_plan(a.T, a.H);
  const int W = kLatentC + a.dr, R = a.T * a.H;
  // Rows of a copied box: as many as lie in one page and one tile.
  int box = kTile;
  while (a.page_size % box) box >>= 1;
  CUtensorMap mq, mc;
  const cuuint64_t qd[3] = {(cuuint64_t)W, (cuuint64_t)R, (cuuint64_t)a.B};
  const cuuint64_t qs[2] = {(cuuint64_t)W * 2, (cuuint64_t)W * 2 * R};
  const cuuint32_t qb[3] = {64, kRows, 1};
  const cuuint64_t cd[2] = {(cuuint64_t)W, (cuuint64_t)a.n_pages * a.page_size};
  const cuuint64_t cs[1] = {(cuuint64_t)W * 2};
  const cuuint32_t cb[2] = {64, (cuuint32_t)box};
  if (!latent::make_bf16_map(&mq, a.q, 3, qd, qs, qb) ||
      !latent::make_bf16_map(&mc, a.cache, 2, cd, cs, cb))
    return cudaErrorInvalidValue;
  Params p;
  p.table = a.block_table; p.lens = a.seq_lens; p.mask = a.tree_mask;
  p.q = static_cast<const __nv_bfloat16 *>(a.q);
  p.B = a.B; p.T = a.T; p.H = a.H; p.W = W; p.R = R; p.n_pages = a.n_pages;
  p.page_size = a.page_size; p.max_pages = a.max_pages; p.box_rows = box;
  p.row_tiles = pl.row_tiles; p.G = pl.G;
  p.warps = ((R < kRows ? R : kRows) + 31) / 32;
  const uint32_t space = kSmem - kSharedBytes - 2 * p.warps * 32 * kTile * 4;
  // rank 0: two rotary slots at least, more where a stage does not fit
  const uint32_t space0 = space - (a.dr ? kQBlock : 0);
  p.stages[0] = (int)((space0 - (a.dr ? 2 * kBlock : 0)) / kStage);
  p.stages[1] = (int)(space / kStage);
  for (int &n : p.stages)
    if (n > kMaxStages) n = kMaxStages;
  p.rope_slots = a.dr ? (int)((space0 - p.stages[0] * kStage) / kBlock) : 1;
  if (p.rope_slots > kMaxStages) p.rope_slots = kMaxStages;
  // Scores are made up for what the tensor cores cut off of their two parts: lse was 5e-6 too small
  // at scores of 24, and the probabilities that kda_latent_weights takes from it, whose scores are
  // one sum, by as much too large.  The scale's rounding is taken back from lse.
  const double more = latent::cut_off(W, 2);
  p.scale2 = (float)(a.scale * 1.4426950408889634 * more);
  const double ln = p.scale2 > 1e-30f && p.scale2 < 1e30f ? a.scale * more / p.scale2 : 0.6931471805599453;
  p.ln_hi = (float)ln;
  p.ln_lo = (float)(ln - p.ln_hi);
  p.out = static_cast<__nv_bfloat16 *>(a.out); p.lse = a.lse; p.status = a.status;
  unsigned char *ws = static_cast<unsigned char *>(a.scratch);
  p.joins = reinterpret_cast<int4 *>(ws);
  p.errors = reinterpret_cast<DeviceStatus *>(ws + pl.joins);
  p.part_ml = reinterpret_cast<float *>(ws + pl.joins + pl.errors);
  p.part_o = reinterpret_cast<float *>(ws + pl.joins + pl.errors + pl.ml);
  p.test = a.test;
  kda_latent_decode_kernel<<<2 * pl.G * pl.row_tiles, kThreads, kSmem, stream>>>(mq, mc, p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const bool many = pl.G > 7 * (int64_t)a.B;           // parts of a sequence
  const int borders = pl.G - 1 < a.B ? pl.G - 1 : a.B;  // a sequence is joined at one
  cfg.gridDim = dim3((unsigned)((R + 31) / 32 * (kLatentC / kJoinCh / (many ? 1 : kJoinWarps))),
                     (unsigned)(borders + 1));
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(
      &cfg, many ? kda_latent_join_kernel<true> : kda_latent_join_kernel<false>, p);
}

}  // namespace kda
