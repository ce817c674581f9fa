// Gradient of latent attention in its expanded form (kda_latent_bwd), tcgen05 /
// TMEM / TMA, sm_103a.
//
//   p_ij = exp(s_ij - lse_i),  ds_ij = p_ij (do_i . v_j - delta_i),
//   delta_i = do_i . o_i
//   dv_j = sum_i p_ij do_i,  dk_j = scale sum_i ds_ij q_i,  dq_i = scale sum_j ds_ij k_j
//
// Two passes in one launch, each output element owned by one CTA (no atomics, so the
// result does not depend on the order of execution; the price is that s and dp are
// computed twice, 1,152 multiply-adds a pair at dr = 64 instead of 832).  A CTA keeps
// 128 rows X1, X2 and streams tiles of rows Y1, Y2 past them:
//   S  = X1 Y1^T,  dP = X2 Y2^T              (fp32, TMEM)
//   P  = exp2(S scale log2e - lse log2e),  dS = P (dP - delta)
//   A1 += dS Y1,   A2 += P Y2                (fp32, TMEM, over all tiles)
// keys pass:    X = (keys, values), Y = (queries, d_out), 64 rows: A1 = dk, A2 = dv
// queries pass: X = (queries, d_out), Y = (keys, values), 128 rows: A1 = dq
// P and dS are rounded to bf16 (half a step, 2^-8 of the value): they are operands of
// the tensor cores, in TMEM over the columns they were computed from.
//
// A block works through items, taking over blocks of the grid that have not started;
// the next item's rows and first tiles arrive beside this one's last products and its
// output, which leaves from registers because the buffers are the next item's by then
// (none of this holds across the change of pass, where the pipeline runs empty: with
// under four items a block that costs more than it gains).
// 4 x 4096 tokens, 16 heads: 920 us with a block for each item, 855 so; 32 x 512: 350 and
// 288; five sequences of 1,847 tokens together, at under four items a block, 59 and 64.
//
// Measured (16 heads, dr = 64): 4 x 4096 tokens 855 us (L2 warm, replayed), of it
// statistics 27, both passes 813, rotary sums 14: 1.05 PFLOP/s of the formulas, 1.4 of
// what the two passes compute, whose products alone are 2,624 tensor-core cycles for
// 64 x 128 pairs (S and dP of the keys pass have 64 columns, which the tensor cores take
// at two thirds of their rate).  The whole call on cold inputs: 917 us, 0.97 PFLOP/s.
// 4 x 2048 tokens, the passes: 250 us with the tensor cores busy 54 % of the time and
// DRAM 22 %; dr = 0: 215 us, 49 % and 21 %.  Bound by the products and by the way
// S -> P -> dP -> dS between them.
//
// The rotary key is shared by the heads: every head leaves its fp32 gradient in
// the workspace and a last kernel adds them in head order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <string.h>

#include "kda_latent_tc.cuh"

namespace kda {
namespace {

using namespace latent;

constexpr int kX = 128, kY = 64;
constexpr int kThreads = 384;            // 8 elementwise warps; loader, MMA, cleaner, items
constexpr int kLoadWarp = 8, kMmaWarp = 9, kCleanWarp = 10, kItemWarp = 11;
constexpr int kMaxStages = 4;
constexpr uint32_t kXBlock = 16384, kYBlock = 8192;  // 128 or 64 rows x 64 channels

// Barriers of the keys pass and of the queries pass.  Their phases run on over the
// items of a pass and start again with the next one (counted from a constant, they
// leave what the MMA warp computes in uniform registers).
struct KeysBars {
  uint64_t full[kMaxStages], empty[kMaxStages], s_full[2], clean_req[2], clean[2];
  uint64_t x_full, x_free, dp_full, acc_full;  // of one arrival, down to here
  uint64_t p_ready[2], ds_ready;               // of eight
  uint32_t loaded, loaded_x;             // tiles, blocks of X
};
struct QueriesBars {
  uint64_t k_full[4], k_empty[4], v_full[2], v_empty[2], clean_req[2], clean[2];
  uint64_t x_full, x_free, g_full, s_full, dp_full, acc_full;  // of one arrival, down to here
  uint64_t x2_ready, s_free, ds_ready;                         // of eight
  uint32_t loaded_k, loaded_v, loaded_x, loaded_g;
};
// What a block works on, and the one after it (seq < 0: nothing, the block ends).
struct Item {
  SeqTile tile;
  int head, keys;                        // keys: of the keys pass
};
struct Shared {
  KeysBars keys;
  QueriesBars queries;
  uint64_t item_full[2], item_free[2], want, taken, fin;
  alignas(16) uint32_t answer[4];
  uint32_t tmem;
  int abort, pass, next;                 // next: number of the item after the pass
  Item item[2];
};
enum { kNoPass, kKeysPass, kQueriesPass };
constexpr int kItemUsers = 11;           // loader, MMA, cleaner, eight elementwise warps
// Tiles before an item's last, the next is asked for: finding it takes about 2 us.
// (4 x 4096 tokens: 871 us; 874 with 2, 878 with 1.)
constexpr int kAhead = 4;
// What a role has behind it in a pass: streamed tiles, items that streamed any, and
// those of them whose last tile was cleaned.
struct Behind {
  uint32_t tiles, items, cleans;
};

template <class Bars>
__device__ __forceinline__ void init_bars(Bars &b, uint64_t *of_eight, bool again) {
  uint64_t *const all = reinterpret_cast<uint64_t *>(&b);
  for (uint64_t *x = all; x < of_eight + 3; ++x) {
    if (again) mbar_inval(x);
    mbar_init(x, x < of_eight ? 1 : 8);
  }
}
__device__ __forceinline__ void init_keys(KeysBars &b, bool again) {
  init_bars(b, b.p_ready, again);
  b.loaded = b.loaded_x = 0;
}
__device__ __forceinline__ void init_queries(QueriesBars &b, bool again) {
  init_bars(b, &b.x2_ready, again);
  b.loaded_k = b.loaded_v = b.loaded_x = b.loaded_g = 0;
}

template <int DR>
constexpr uint32_t x_bytes() { return ((kLatentD + DR) / 64 + 2) * kXBlock; }
template <int DR>
constexpr uint32_t stage_bytes() { return ((kLatentD + DR) / 64 + 2) * kYBlock; }
template <int DR>
constexpr int stages() { return DR ? 3 : 4; }
constexpr uint32_t kSmem = 232448 - 1024;  // dynamic; Shared is static
static_assert(sizeof(Shared) <= 1024, "shared memory");
// of the keys pass: X, the streamed tiles, their statistics
template <int DR>
constexpr uint32_t keys_bytes() { return x_bytes<DR>() + stages<DR>() * stage_bytes<DR>(); }
template <int DR>
constexpr uint32_t stat_bytes() { return stages<DR>() * kY * 4; }
static_assert(keys_bytes<64>() + 2 * stat_bytes<64>() <= kSmem &&
              keys_bytes<0>() + 2 * stat_bytes<0>() <= kSmem, "shared memory");

struct Params : Packed {
  int64_t stat_rows;
  float scale, scale2;
  int causal;
  __nv_bfloat16 *dq, *dk, *dv;
  int64_t dk_ts, dk_hs, dv_ts, dv_hs;
  const float *lse2, *delta;             // [H][stat_rows]
  float *rope;                           // [H][n_k][64]
  DeviceStatus *status;
  WaitTest test;
};

// A test lets the waits for tile i of the block's item k run out.
__device__ __forceinline__ bool withheld(const Params &p, int k, int i) {
  return k == 0 && i == p.test.tile && p.test.block == (int)blockIdx.x;
}

// Row statistics are kept per head in tiles of 64 that no two sequences share:
// the first tile of sequence s is floor(q0 / 64) + s.
__host__ __device__ inline int64_t stat_tile(int64_t q0, int64_t s) { return q0 / kY + s; }

struct Maps {
  CUtensorMap q128, q64, g128, g64, k128, v128, r128;
};

// The 64 columns at `col` of a warp's 32 accumulator rows, times `mul`, as bf16 rows of
// dst (row stride `stride` elements); rows >= n_rows are not written.  Straight from
// registers: the buffers are the next item's by now.
__device__ __forceinline__ void store_cols(uint32_t col, float mul, bool zero, __nv_bfloat16 *dst,
                                           int64_t stride, int n_rows, int lane) {
  uint32_t o[2][32];
  if (zero) {
#pragma unroll
    for (int j = 0; j < 32; ++j) o[0][j] = o[1][j] = 0;
  } else {
    tmem_ld32(col, o[0]);
    tmem_ld32(col + 32, o[1]);
    tmem_ld_wait(o[0]);
    tmem_ld_wait(o[1]);
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint4 v[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = pack_bf16x2(__uint_as_float(o[c][8 * q + 2 * j]) * mul,
                           __uint_as_float(o[c][8 * q + 2 * j + 1]) * mul);
      v[q] = make_uint4(w[0], w[1], w[2], w[3]);
    }
    store_rows(v, dst + 32 * c, stride * 2, n_rows, lane);
  }
}

// Zeroes rows [from, n) of the `blocks` 64-channel blocks of a streamed tile: they are
// another sequence's and may hold anything, and as operands of the sums 0 * NaN would
// reach the result.
__device__ __forceinline__ void clean_rows(uint32_t tile, int blocks, uint32_t block_bytes,
                                           int from, int n, int lane) {
  for (int b = 0; b < blocks; ++b)
    for (int j = lane; j < (n - from) * 8; j += 32)
      st_shared_v4(tile + b * block_bytes + from * 128 + j * 16, 0, 0, 0, 0);
  fence_proxy_async_smem();
  __syncwarp();
}

// The keys pass: X = 128 keys and their values.  A1 (192 columns) and A2 (128) leave 192
// columns of TMEM: two S buffers and one dP, so the tensor cores run S two tiles ahead
// and dP one ahead of the elementwise work.  Tiles of 64 queries: with the 80 KB of X,
// 96 of them fit shared memory only once, and S and dP would need 288 columns.
// Of an item: its rows from x0, n streamed tiles from `first` on, `live` rows of the last.
struct Span {
  int x0, first, n, live;
};
// Longest first: the first keys are seen by the most queries.
__device__ __forceinline__ Span keys_span(const SeqTile &st, int causal) {
  Span s;
  s.x0 = st.tile * kX;
  s.first = causal ? max(0, s.x0 - (st.nk - st.nq)) / kY : 0;  // query i sees keys <= i + nk - nq
  s.n = max(0, (st.nq + kY - 1) / kY - s.first);
  s.live = min(kY, st.nq - (s.first + s.n - 1) * kY);
  return s;
}

template <int DR>
__device__ __forceinline__ void keys_pass(const Maps &maps, const Params &p, Shared &sh, int k,
                                          uint32_t base, uint32_t tm, const WaitCtx &cx) {
  constexpr int KB = (kLatentD + DR) / 64, ST = stages<DR>();
  constexpr uint32_t kStage = x_bytes<DR>(), SB = stage_bytes<DR>();
  constexpr uint32_t kLse = keys_bytes<DR>(), kDelta = kLse + stat_bytes<DR>();
  constexpr int N1 = kLatentD + DR;
  constexpr uint32_t TM_A1 = 0, TM_A2 = 192, TM_S = 320, TM_DP = 448;
  constexpr uint32_t ID_S = idesc_bf16(128, kY, false, false);
  constexpr uint32_t ID_A1 = idesc_bf16(128, N1, false, true);
  constexpr uint32_t ID_A2 = idesc_bf16(128, kLatentD, false, true);
  KeysBars &m = sh.keys;
  Behind did = {0, 0, 0};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the item numbered k, which the pass goes on with if it is one of its own
  auto mine = [&](int k) { return sh.item[k & 1].tile.seq >= 0 && sh.item[k & 1].keys; };

  if (warp == kLoadWarp && lane == 0) {
    // ---- loader
    bool ok = true;
    for (; ok; ++k) {
      ok = wait_or_abort(cx, &sh.item_full[k & 1], (k >> 1) & 1, 13, k);
      if (!ok || !mine(k)) break;
      const SeqTile st = sh.item[k & 1].tile;
      const int head = sh.item[k & 1].head;
      const Span sp = keys_span(st, p.causal);
      const int xr = st.k0 + sp.x0;
      if (sp.n == 0) {
        mbar_arrive(&sh.want);
        mbar_arrive(&sh.item_free[k & 1]);
        continue;
      }
      if (did.items > 0) ok = wait_or_abort(cx, &m.x_free, (did.items - 1) & 1, 14, k);
      if (!ok) break;
      mbar_arrive_expect_tx(&m.x_full, (KB + 2) * kXBlock);
      for (int kb = 0; kb < KB; ++kb) {
        const uint32_t dst = base + kb * kXBlock;
        if (kb < 2) tma_load_3d_u(dst, &maps.k128, &m.x_full, 64 * kb, head, xr);
        else tma_load_2d(dst, &maps.r128, &m.x_full, 0, xr);
      }
      for (int c = 0; c < 2; ++c)
        tma_load_3d_u(base + (KB + c) * kXBlock, &maps.v128, &m.x_full, 64 * c, head, xr);
      ++did.items;
      for (int i = 0; i < sp.n; ++i) {
        if (withheld(p, k, i)) ok = false;
        if (!ok) break;
        if (i == max(0, sp.n - kAhead)) mbar_arrive(&sh.want);
        const uint32_t g = did.tiles, s = g % ST;
        if (g >= ST) ok = wait_or_abort(cx, &m.empty[s], (g / ST - 1) & 1, 10, i);
        if (!ok) break;
        const int yr = st.q0 + (sp.first + i) * kY;
        const uint32_t dst = base + kStage + s * SB;
        mbar_arrive_expect_tx(&m.full[s], SB + 2 * kY * 4);
        for (int kb = 0; kb < KB; ++kb)
          tma_load_3d_u(dst + kb * kYBlock, &maps.q64, &m.full[s], 64 * kb, head, yr);
        for (int c = 0; c < 2; ++c)
          tma_load_3d_u(dst + (KB + c) * kYBlock, &maps.g64, &m.full[s], 64 * c, head, yr);
        const int64_t at = head * p.stat_rows + (stat_tile(st.q0, st.seq) + sp.first + i) * kY;
        bulk_load(base + kLse + s * kY * 4, p.lse2 + at, kY * 4, &m.full[s]);
        bulk_load(base + kDelta + s * kY * 4, p.delta + at, kY * 4, &m.full[s]);
        ++did.tiles;
      }
      if (ok && sp.live < kY) mbar_arrive(&m.clean_req[did.cleans++ & 1]);
      mbar_arrive(&sh.item_free[k & 1]);
    }
    m.loaded = did.tiles;
    m.loaded_x = did.items;
    // no arrival is on its way when the barriers start again
    for (uint32_t g = did.tiles > ST ? did.tiles - ST : 0; ok && g < did.tiles; ++g)
      ok = wait_or_abort(cx, &m.empty[g % ST], (g / ST) & 1, 17, k);
    if (ok && did.items > 0) wait_or_abort(cx, &m.x_free, (did.items - 1) & 1, 18, k);
  } else if (warp == kMmaWarp && elect_one()) {
    // ---- MMA issue
    const Desc x_s(base, 16), y_s(base + kStage, 16), y_a(base + kStage, kYBlock);
    bool ok = true;
    for (; ok; ++k) {
      ok = wait_or_abort(cx, &sh.item_full[k & 1], (k >> 1) & 1, 25, k);
      if (!ok || !mine(k)) break;
      const Span sp = keys_span(sh.item[k & 1].tile, p.causal);
      mbar_arrive(&sh.item_free[k & 1]);
      const int n = sp.n;
      if (n == 0) continue;
      const uint32_t T = did.tiles;
      ok = wait_or_abort(cx, &m.x_full, did.items & 1, 20, k);
      auto issue_s = [&](int i, int s) {   // s: stage of tile i
        const uint32_t g = T + i;
        ok = ok && wait_or_abort(cx, &m.full[s], (g / ST) & 1, 21, i);
        if (!ok) return;
#pragma unroll
        for (int k = 0; k < 4 * KB; ++k)
          umma_ss(tm + TM_S + 64 * (g & 1), x_s.at((k >> 2) * kXBlock + (k & 3) * 32),
                  y_s.at(s * SB + (k >> 2) * kYBlock + (k & 3) * 32), ID_S, k > 0);
        umma_commit(&m.s_full[g & 1]);
      };
      auto issue_dp = [&](int i, int s) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          umma_ss(tm + TM_DP, x_s.at((KB + (k >> 2)) * kXBlock + (k & 3) * 32),
                  y_s.at(s * SB + (KB + (k >> 2)) * kYBlock + (k & 3) * 32), ID_S, k > 0);
        umma_commit(&m.dp_full);
        if (i + 1 == n) umma_commit(&m.x_free);
      };
      int s0 = T % ST;                     // stage of tile i
      const int s_1 = s0 + 1 == ST ? 0 : s0 + 1;
      issue_s(0, s0);
      if (ok) issue_dp(0, s0);
      if (n > 1) issue_s(1, s_1);
      for (int i = 0; ok && i < n; ++i) {
        const int s1 = s0 + 1 == ST ? 0 : s0 + 1, s2 = s1 + 1 == ST ? 0 : s1 + 1;
        const uint32_t g = T + i;
        // P Y2 while the elementwise warps are still at dS, which needs dP.  (P of the
        // next tile may be ready before this wait: a barrier for each parity.)
        ok = wait_or_abort(cx, &m.p_ready[g & 1], (g >> 1) & 1, 24, i);
        if (ok && i + 1 == n && sp.live < kY)
          ok = wait_or_abort(cx, &m.clean[did.cleans & 1], (did.cleans >> 1) & 1, 23, i);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sb = tm + TM_S + 64 * (g & 1);
#pragma unroll
        for (int k = 0; k < 4; ++k)  // bf16 columns: rows 0 .. 31 at +0, 32 .. 63 at +32
          umma_ts(tm + TM_A2, sb + (k >> 1) * 32 + (k & 1) * 8,
                  y_a.at(s0 * SB + KB * kYBlock + k * 2048), ID_A2, i + k > 0);
        ok = wait_or_abort(cx, &m.ds_ready, g & 1, 22, i);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_ts(tm + TM_A1, tm + TM_DP + (k >> 1) * 32 + (k & 1) * 8, y_a.at(s0 * SB + k * 2048),
                  ID_A1, i + k > 0);
        umma_commit(&m.empty[s0]);
        if (i + 1 < n) issue_dp(i + 1, s1);
        if (i + 2 < n) issue_s(i + 2, s2);
        s0 = s1;
      }
      if (ok) umma_commit(&m.acc_full);
      did.tiles += n;
      ++did.items;
      did.cleans += sp.live < kY;
    }
  } else if (warp == kCleanWarp) {
    // ---- cleaner: the loader asks once the copy of an item's last tile is under way;
    // the products that read it wait.  The loader may ask for the next item's too
    // before this one's is used, but no further: two barriers each.
    bool ok = true;
    for (; ok; ++k) {
      ok = warp_wait_idle(cx, &sh.item_full[k & 1], (k >> 1) & 1, 32, k);
      if (!ok || !mine(k)) break;
      const Span sp = keys_span(sh.item[k & 1].tile, p.causal);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.item_free[k & 1]);
      did.tiles += sp.n;
      if (sp.n == 0 || sp.live == kY) continue;
      const uint32_t g = did.tiles - 1;
      ok = warp_wait_idle(cx, &m.clean_req[did.cleans & 1], (did.cleans >> 1) & 1, 30, k);
      ok = ok && warp_wait(cx, &m.full[g % ST], (g / ST) & 1, 31, k);
      if (!ok) break;
      clean_rows(base + kStage + g % ST * SB, KB + 2, kYBlock, sp.live, kY, lane);
      if (lane == 0) mbar_arrive(&m.clean[did.cleans & 1]);
      ++did.cleans;
    }
  } else if (warp < 8) {
    // ---- elementwise: thread = row of X, warpgroup = half of a tile's columns
    const int wg = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21, col = 32 * wg;
    bool ok = true;
    for (; ok; ++k) {
      ok = warp_wait(cx, &sh.item_full[k & 1], (k >> 1) & 1, 43, k);
      if (!ok || !mine(k)) break;
      const Item &item = sh.item[k & 1];
      const Span sp = keys_span(item.tile, p.causal);
      const int xr = sp.x0 + row, ny = item.tile.nq;
      // queries [lo, ny) see this row's key
      const int lo = p.causal ? max(0, xr - (item.tile.nk - ny)) : 0;
      for (int i = 0; ok && i < sp.n; ++i) {
        const uint32_t g = did.tiles + i;
        ok = warp_wait(cx, &m.s_full[g & 1], (g >> 1) & 1, 40, i);
        if (!ok) break;
        tc_fence_after();
        uint32_t r[32];
        const uint32_t ts = tm + lanes + TM_S + 64 * (g & 1) + col, td = tm + lanes + TM_DP + col;
        tmem_ld32(ts, r);
        tmem_ld_wait(r);
        const int y0 = (sp.first + i) * kY + (int)col;
        const bool edge = __any_sync(0xffffffffu, y0 < lo || y0 + 32 > ny);
        float pr[32];
        const uint32_t sl = base + kLse + (g % ST * kY + col) * 4;
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 l = ld_shared_f32x4(sl + 4 * j);
          pr[j] = ex2(fmaf(__uint_as_float(r[j]), p.scale2, -l.x));
          pr[j + 1] = ex2(fmaf(__uint_as_float(r[j + 1]), p.scale2, -l.y));
          pr[j + 2] = ex2(fmaf(__uint_as_float(r[j + 2]), p.scale2, -l.z));
          pr[j + 3] = ex2(fmaf(__uint_as_float(r[j + 3]), p.scale2, -l.w));
        }
        if (edge) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (y0 + j < lo || y0 + j >= ny) pr[j] = 0.f;
        }
        uint32_t pk[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) pk[j] = pack_bf16x2(pr[2 * j], pr[2 * j + 1]);
        tmem_st16(ts, pk);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.p_ready[g & 1]);
        ok = warp_wait(cx, &m.dp_full, g & 1, 41, i);
        if (!ok) break;
        tc_fence_after();
        tmem_ld32(td, r);
        tmem_ld_wait(r);
        const uint32_t sd = base + kDelta + (g % ST * kY + col) * 4;
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 d = ld_shared_f32x4(sd + 4 * j);
          r[j] = __float_as_uint(pr[j] * (__uint_as_float(r[j]) - d.x));
          r[j + 1] = __float_as_uint(pr[j + 1] * (__uint_as_float(r[j + 1]) - d.y));
          r[j + 2] = __float_as_uint(pr[j + 2] * (__uint_as_float(r[j + 2]) - d.z));
          r[j + 3] = __float_as_uint(pr[j + 3] * (__uint_as_float(r[j + 3]) - d.w));
        }
        if (edge) {  // dP of a pair outside may be anything
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (y0 + j < lo || y0 + j >= ny) r[j] = 0;
        }
#pragma unroll
        for (int j = 0; j < 16; ++j)
          pk[j] = pack_bf16x2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
        tmem_st16(td, pk);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.ds_ready);
      }
      if (ok && sp.n > 0) ok = warp_wait(cx, &m.acc_full, did.items & 1, 42, k);
      if (!ok) break;
      if (sp.n > 0) tc_fence_after();
      did.tiles += sp.n;
      did.items += sp.n > 0;
      // ---- output: a warpgroup half of each result's columns
      const bool zero = sp.n == 0;
      const uint32_t acc = tm + lanes;
      const int from = sp.x0 + (warp & 3) * 32, rows = item.tile.nk - from;  // of this warp
      const int64_t kr = item.tile.k0 + from;
      store_cols(acc + TM_A2 + 64 * wg, 1.f, zero, p.dv + kr * p.dv_ts + item.head * p.dv_hs + 64 * wg,
                 p.dv_ts, rows, lane);
      store_cols(acc + TM_A1 + 64 * wg, p.scale, zero,
                 p.dk + kr * p.dk_ts + item.head * p.dk_hs + 64 * wg, p.dk_ts, rows, lane);
      if (DR) {  // fp32
        uint32_t o[32];
        if (zero) {
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = 0;
        } else {
          tmem_ld32(acc + TM_A1 + kLatentD + 32 * wg, o);
          tmem_ld_wait(o);
        }
        float *dst = p.rope + ((int64_t)item.head * p.n_k + kr) * kLatentRope + 32 * wg;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint4 v[4];
#pragma unroll
          for (int q = 0; q < 4; ++q)
            v[q] = make_uint4(o[16 * c + 4 * q], o[16 * c + 4 * q + 1], o[16 * c + 4 * q + 2],
                              o[16 * c + 4 * q + 3]);
          store_rows(v, dst + 16 * c, kLatentRope * 4, rows, lane);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.item_free[k & 1]);
    }
    if (threadIdx.x == 0) sh.next = k;
  }
}

// The queries pass: X = 128 queries and their d_out, streamed tiles of 128 keys.  S and
// dP have one buffer each (128 columns): S of the next tile is issued as soon as S of
// this one is in registers, dP of the next tile after the product that read dS.  d_out
// moves to TMEM (64 columns, the first operand of dP), which gives its 32 KB to the
// streamed tiles: keys in three (dr = 0: four) buffers, because they are held from S
// to the product with dS, values in one (two), because they are done with dP.
// Longest first: the last queries of a sequence see the most keys.
__device__ __forceinline__ Span queries_span(const SeqTile &st, int causal) {
  Span s;
  s.x0 = (st.n_tiles - 1 - st.tile) * kX;
  const int end = causal ? min(st.nk, min(s.x0 + kX, st.nq) + st.nk - st.nq) : st.nk;
  s.first = 0;
  s.n = end > 0 ? (end + 127) / 128 : 0;
  s.live = min(128, st.nk - (s.n - 1) * 128);
  return s;
}

template <int DR>
__device__ __forceinline__ void queries_pass(const Maps &maps, const Params &p, Shared &sh, int k,
                                             uint32_t base, uint32_t tm, const WaitCtx &cx) {
  constexpr int KB = (kLatentD + DR) / 64, KT = DR ? 3 : 4, VT = DR ? 1 : 2;
  constexpr uint32_t kRingK = KB * kXBlock, kRingV = kRingK + KT * KB * kXBlock;
  static_assert(kRingV + VT * 2 * kXBlock <= kSmem, "shared memory");
  constexpr int N1 = kLatentD + DR;
  constexpr uint32_t TM_A1 = 0, TM_X2 = 192, TM_S = 256, TM_DP = 384;
  constexpr uint32_t ID_S = idesc_bf16(128, 128, false, false);
  constexpr uint32_t ID_A1 = idesc_bf16(128, N1, false, true);
  QueriesBars &m = sh.queries;
  Behind did = {0, 0, 0};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto mine = [&](int k) { return sh.item[k & 1].tile.seq >= 0 && !sh.item[k & 1].keys; };
  // d_out of the item whose first tile is `tile` comes in where the keys of its third go
  auto x2_place = [&](uint32_t tile) { return base + kRingK + (tile + 2) % KT * KB * kXBlock; };

  if (warp == kLoadWarp && lane == 0) {
    // ---- loader
    bool ok = true;
    uint32_t loaded_v = 0, loaded_g = 0;
    for (; ok; ++k) {
      ok = wait_or_abort(cx, &sh.item_full[k & 1], (k >> 1) & 1, 13, k);
      if (!ok || !mine(k)) break;
      const SeqTile st = sh.item[k & 1].tile;
      const int head = sh.item[k & 1].head;
      const Span sp = queries_span(st, p.causal);
      const int xr = st.q0 + sp.x0;
      if (sp.n == 0) {
        mbar_arrive(&sh.want);
        mbar_arrive(&sh.item_free[k & 1]);
        continue;
      }
      if (did.items > 0) ok = wait_or_abort(cx, &m.x_free, (did.items - 1) & 1, 14, k);
      if (!ok) break;
      mbar_arrive_expect_tx(&m.x_full, KB * kXBlock);
      for (int kb = 0; kb < KB; ++kb)
        tma_load_3d_u(base + kb * kXBlock, &maps.q128, &m.x_full, 64 * kb, head, xr);
      const uint32_t x2 = did.items++ & 1;       // phase of this item's d_out
      for (int i = 0; i < sp.n; ++i) {
        if (withheld(p, k, i)) ok = false;
        if (!ok) break;
        if (i == max(0, sp.n - kAhead)) mbar_arrive(&sh.want);
        const int yr = st.k0 + i * 128;
        const uint32_t g = did.tiles, sk = g % KT, sv = g % VT;
        if (g >= KT) ok = wait_or_abort(cx, &m.k_empty[sk], (g / KT - 1) & 1, 10, i);
        if (ok && i == 2) ok = wait_or_abort(cx, &m.x2_ready, x2, 11, i);
        if (!ok) break;
        mbar_arrive_expect_tx(&m.k_full[sk], KB * kXBlock);
        const uint32_t dk = base + kRingK + sk * KB * kXBlock;
        for (int kb = 0; kb < KB; ++kb) {
          if (kb < 2) tma_load_3d_u(dk + kb * kXBlock, &maps.k128, &m.k_full[sk], 64 * kb, head, yr);
          else tma_load_2d(dk + kb * kXBlock, &maps.r128, &m.k_full[sk], 0, yr);
        }
        ++did.tiles;
        if (i == 0) {
          const uint32_t t = g + 2;              // the tile before in d_out's place is used
          if (t >= KT) ok = wait_or_abort(cx, &m.k_empty[t % KT], (t / KT - 1) & 1, 15, k);
          if (!ok) break;
          mbar_arrive_expect_tx(&m.g_full, 2 * kXBlock);
          for (int c = 0; c < 2; ++c)
            tma_load_3d_u(x2_place(g) + c * kXBlock, &maps.g128, &m.g_full, 64 * c, head, xr);
          ++loaded_g;
        }
        if (g >= VT) ok = wait_or_abort(cx, &m.v_empty[sv], (g / VT - 1) & 1, 12, i);
        if (!ok) break;
        mbar_arrive_expect_tx(&m.v_full[sv], 2 * kXBlock);
        const uint32_t dv = base + kRingV + sv * 2 * kXBlock;
        for (int c = 0; c < 2; ++c)
          tma_load_3d_u(dv + c * kXBlock, &maps.v128, &m.v_full[sv], 64 * c, head, yr);
        ++loaded_v;
      }
      if (ok && sp.live < 128) mbar_arrive(&m.clean_req[did.cleans++ & 1]);
      // the next item's second or third tile would go where d_out is
      if (ok && sp.n <= 2) ok = wait_or_abort(cx, &m.x2_ready, x2, 16, k);
      mbar_arrive(&sh.item_free[k & 1]);
    }
    m.loaded_k = did.tiles;
    m.loaded_v = loaded_v;
    m.loaded_x = did.items;
    m.loaded_g = loaded_g;
    // no arrival is on its way when the barriers start again
    for (uint32_t g = did.tiles > KT ? did.tiles - KT : 0; ok && g < did.tiles; ++g)
      ok = wait_or_abort(cx, &m.k_empty[g % KT], (g / KT) & 1, 17, k);
    for (uint32_t g = did.tiles > VT ? did.tiles - VT : 0; ok && g < did.tiles; ++g)
      ok = wait_or_abort(cx, &m.v_empty[g % VT], (g / VT) & 1, 19, k);
    if (ok && did.items > 0) wait_or_abort(cx, &m.x_free, (did.items - 1) & 1, 18, k);
  } else if (warp == kMmaWarp && elect_one()) {
    // ---- MMA issue
    const Desc x_s(base, 16), k_s(base + kRingK, 16), v_s(base + kRingV, 16),
        k_a(base + kRingK, kXBlock);
    bool ok = true;
    for (; ok; ++k) {
      ok = wait_or_abort(cx, &sh.item_full[k & 1], (k >> 1) & 1, 27, k);
      if (!ok || !mine(k)) break;
      const Span sp = queries_span(sh.item[k & 1].tile, p.causal);
      mbar_arrive(&sh.item_free[k & 1]);
      const int n = sp.n;
      if (n == 0) continue;
      const uint32_t T = did.tiles;
      auto issue_s = [&](int i) {
        const uint32_t g = T + i, sk = g % KT;
        ok = ok && wait_or_abort(cx, &m.k_full[sk], (g / KT) & 1, 21, i);
        if (ok && g > 0) ok = wait_or_abort(cx, &m.s_free, (g - 1) & 1, 22, i);
        if (!ok) return;
        tc_fence_after();
        const uint32_t off = sk * KB * kXBlock;
#pragma unroll
        for (int k = 0; k < 4 * KB; ++k)
          umma_ss(tm + TM_S, x_s.at((k >> 2) * kXBlock + (k & 3) * 32),
                  k_s.at(off + (k >> 2) * kXBlock + (k & 3) * 32), ID_S, k > 0);
        umma_commit(&m.s_full);
        if (i + 1 == n) umma_commit(&m.x_free);
      };
      auto issue_dp = [&](int i) {
        const uint32_t g = T + i, sv = g % VT;
        ok = ok && wait_or_abort(cx, &m.v_full[sv], (g / VT) & 1, 23, i);
        if (!ok) return;
        const uint32_t off = sv * 2 * kXBlock;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          umma_ts(tm + TM_DP, tm + TM_X2 + 8 * k, v_s.at(off + (k >> 2) * kXBlock + (k & 3) * 32),
                  ID_S, k > 0);
        umma_commit(&m.dp_full);
        umma_commit(&m.v_empty[sv]);
      };
      ok = wait_or_abort(cx, &m.x_full, did.items & 1, 20, k);
      issue_s(0);
      ok = ok && wait_or_abort(cx, &m.x2_ready, did.items & 1, 26, k);
      if (!ok) break;
      tc_fence_after();
      issue_dp(0);
      if (n > 1) issue_s(1);
      for (int i = 0; ok && i < n; ++i) {
        const uint32_t g = T + i;
        ok = wait_or_abort(cx, &m.ds_ready, g & 1, 24, i);
        if (ok && i + 1 == n && sp.live < 128)
          ok = wait_or_abort(cx, &m.clean[did.cleans & 1], (did.cleans >> 1) & 1, 25, i);
        if (!ok) break;
        tc_fence_after();
        // dS is over dP, keys 0 .. 63 at column 0, 64 .. 127 at column 64
        const uint32_t off = g % KT * KB * kXBlock;
#pragma unroll
        for (int k = 0; k < 8; ++k)
          umma_ts(tm + TM_A1, tm + TM_DP + (k >> 2) * 64 + (k & 3) * 8, k_a.at(off + k * 2048),
                  ID_A1, i + k > 0);
        umma_commit(&m.k_empty[g % KT]);
        if (i + 1 < n) issue_dp(i + 1);
        if (ok && i + 2 < n) issue_s(i + 2);
      }
      if (ok) umma_commit(&m.acc_full);
      did.tiles += n;
      ++did.items;
      did.cleans += sp.live < 128;
    }
  } else if (warp == kCleanWarp) {
    // ---- cleaner: keys of the last tile past the sequence's end, as in the other pass
    bool ok = true;
    for (; ok; ++k) {
      ok = warp_wait_idle(cx, &sh.item_full[k & 1], (k >> 1) & 1, 32, k);
      if (!ok || !mine(k)) break;
      const Span sp = queries_span(sh.item[k & 1].tile, p.causal);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.item_free[k & 1]);
      did.tiles += sp.n;
      if (sp.n == 0 || sp.live == 128) continue;
      const uint32_t g = did.tiles - 1;
      ok = warp_wait_idle(cx, &m.clean_req[did.cleans & 1], (did.cleans >> 1) & 1, 30, k);
      ok = ok && warp_wait(cx, &m.k_full[g % KT], (g / KT) & 1, 31, k);
      if (!ok) break;
      clean_rows(base + kRingK + g % KT * KB * kXBlock, KB, kXBlock, sp.live, 128, lane);
      if (lane == 0) mbar_arrive(&m.clean[did.cleans & 1]);
      ++did.cleans;
    }
  } else if (warp < 8) {
    // ---- elementwise: thread = query, warpgroup = half of a tile's keys
    const int wg = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    bool ok = true;
    for (; ok; ++k) {
      ok = warp_wait(cx, &sh.item_full[k & 1], (k >> 1) & 1, 44, k);
      if (!ok || !mine(k)) break;
      const Item &item = sh.item[k & 1];
      const Span sp = queries_span(item.tile, p.causal);
      const int xr = sp.x0 + row, n = sp.n;
      float lse2 = 0.f, delta = 0.f;
      if (xr < item.tile.nq) {
        const int64_t at =
            item.head * p.stat_rows + stat_tile(item.tile.q0, item.tile.seq) * kY + xr;
        lse2 = p.lse2[at];
        delta = p.delta[at];
      }
      const int nk = item.tile.nk;       // keys below hi are seen by this row
      const int hi = p.causal ? min(nk, xr + nk - item.tile.nq + 1) : nk;
      if (n > 0) {  // this row's 64 channels of d_out (a warpgroup's half) into TMEM
        ok = warp_wait(cx, &m.g_full, did.items & 1, 43, k);
        if (!ok) break;
        uint32_t x[32];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const uint4 v = ld_shared_v4(x2_place(did.tiles) + wg * kXBlock + sw128_offset(row, 16 * q));
          x[4 * q] = v.x; x[4 * q + 1] = v.y; x[4 * q + 2] = v.z; x[4 * q + 3] = v.w;
        }
        tmem_st32(tm + lanes + TM_X2 + 32 * wg, x);
        tmem_st_wait();
        tc_fence_before();
        fence_proxy_async_smem();        // its place is loaded again
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.x2_ready);
      }
      for (int i = 0; ok && i < n; ++i) {
        const uint32_t g = did.tiles + i;
        ok = warp_wait(cx, &m.s_full, g & 1, 40, i);
        if (!ok) break;
        tc_fence_after();
        uint32_t x[2][32];
        const uint32_t ts = tm + lanes + TM_S + 64 * wg, td = tm + lanes + TM_DP + 64 * wg;
        tmem_ld32(ts, x[0]);
        tmem_ld32(ts + 32, x[1]);
        tmem_ld_wait(x[0]);
        tmem_ld_wait(x[1]);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.s_free);
        const int seen = hi - (i * 128 + 64 * wg);       // columns below it are allowed
        const bool edge = __any_sync(0xffffffffu, seen < 64);
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int j = 0; j < 32; ++j)
            x[c][j] = __float_as_uint(ex2(fmaf(__uint_as_float(x[c][j]), p.scale2, -lse2)));
        if (edge) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (32 * c + j >= seen) x[c][j] = 0;
        }
        ok = warp_wait(cx, &m.dp_full, g & 1, 41, i);
        if (!ok) break;
        tc_fence_after();
        uint32_t pk[2][16];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t d[32];
          tmem_ld32(td + 32 * c, d);
          tmem_ld_wait(d);
#pragma unroll
          for (int j = 0; j < 32; ++j)
            d[j] = __float_as_uint(__uint_as_float(x[c][j]) * (__uint_as_float(d[j]) - delta));
          if (edge) {  // dP of a pair outside may be anything
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (32 * c + j >= seen) d[j] = 0;
          }
#pragma unroll
          for (int j = 0; j < 16; ++j)
            pk[c][j] = pack_bf16x2(__uint_as_float(d[2 * j]), __uint_as_float(d[2 * j + 1]));
        }
        // over dP, all of whose columns here are in registers
        tmem_st16(td, pk[0]);
        tmem_st16(td + 16, pk[1]);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.ds_ready);
      }
      if (ok && n > 0) ok = warp_wait(cx, &m.acc_full, did.items & 1, 42, k);
      if (!ok) break;
      if (n > 0) tc_fence_after();
      did.tiles += n;
      did.items += n > 0;
      const int from = sp.x0 + (warp & 3) * 32;
      const int64_t to = ((item.tile.q0 + from) * (int64_t)p.H + item.head) * N1;
      for (int c = wg; c < KB; c += 2)
        store_cols(tm + lanes + TM_A1 + 64 * c, p.scale, n == 0, p.dq + to + 64 * c,
                   (int64_t)p.H * N1, item.tile.nq - from, lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.item_free[k & 1]);
    }
    if (threadIdx.x == 0) sh.next = k;
  }
}

// What block `block` of the grid works on: the keys pass's items, then the queries
// pass's; both longest first (the first keys are seen by the most queries, the last
// queries see the most keys).
struct Finder {                          // of one warp
  const Params &p;
  const LaneSeqs seqs;
  const int nk, nq;                      // tiles of keys and of queries
  __device__ explicit Finder(const Params &params)
      : p(params), seqs(params), nk(count_tiles(params, seqs, kTileB)),
        nq(count_tiles(params, seqs, kTileA)) {}
  __device__ Item find(int64_t block) const {
    Item it;
    it.tile.seq = -1;
    it.head = it.keys = 0;
    const int64_t first_q = (int64_t)nk * p.H;
    if (nk < 0) {
      if (p.n_q == 0 && block == 0 && (threadIdx.x & 31) == 0)  // no kernel before this one
        set_device_status(p.status, KDA_ERR_INVALID_ARG, 1);
    } else if (block < first_q) {
      it.tile = place_item(p, seqs, kTileB, nk, (uint32_t)block, &it.head);
      it.keys = 1;
    } else if (block < first_q + (int64_t)nq * p.H) {
      it.tile = place_item(p, seqs, kTileA, nq, (uint32_t)(block - first_q), &it.head);
    }
    return it;
  }
};

// A block works through items until no block of the grid is left that has not started:
// the next item's rows and first tiles are loaded while this one's last products and
// its output are under way.
template <int DR>
__global__ void __launch_bounds__(kThreads, 1)
kda_latent_bwd_kernel(const __grid_constant__ Maps maps, const Params p) {
  extern __shared__ __align__(1024) unsigned char tiles[];
  __shared__ Shared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (warp == kMmaWarp) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
  }
  if (tid == 0) {
    init_keys(sh.keys, false);
    init_queries(sh.queries, false);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.item_full[i], 1);
      mbar_init(&sh.item_free[i], kItemUsers);
    }
    mbar_init(&sh.want, 1);
    mbar_init(&sh.taken, 1);
    mbar_init(&sh.fin, 1);
    sh.abort = 0;
    fence_mbarrier_init();
  }
  if (warp == kLoadWarp && lane == 0) {
    prefetch_tensormap(&maps.k128);
    prefetch_tensormap(&maps.v128);
    prefetch_tensormap(&maps.q64);
    prefetch_tensormap(&maps.g64);
    prefetch_tensormap(&maps.q128);
    prefetch_tensormap(&maps.g128);
    if (DR) prefetch_tensormap(&maps.r128);
  }
  const auto start = [] {
    pdl_wait();                          // the row statistics
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  };
  const WaitCtx cx{&sh.abort, p.status, (int)blockIdx.x, p.test.wait_ns};

  if (warp == kItemWarp) {
    // ---- items: publishes this block's, and takes over the next one when the loader
    // is about to be through with it
    const Finder finder(p);
    Item it = finder.find(blockIdx.x);
    bool more = true;
    start();
    int asked = 0, k = 0;
    for (bool ok = true; ok;) {
      if (!more || it.tile.seq >= 0) {
        if (k >= 2) ok = warp_wait(cx, &sh.item_free[k & 1], ((k >> 1) - 1) & 1, 50, k);
        if (!ok) break;
        if (lane == 0) {
          sh.item[k & 1] = it;
          mbar_arrive(&sh.item_full[k & 1]);
        }
        if (!more) break;
        ok = warp_wait_idle(cx, &sh.want, k & 1, 51, k);
        ++k;
        if (!ok) break;
      }
      if (lane == 0) {
        mbar_arrive_expect_tx(&sh.taken, 16);
        take_block(smem_u32(sh.answer), &sh.taken);
      }
      __syncwarp();
      // the answer is waited for whatever else fails: it is written to this block
      ok = __all_sync(0xffffffffu, mbar_wait(&sh.taken, asked & 1, kWaitNs));
      ++asked;
      if (!ok) {
        if (lane == 0) record_device_status(p.status, KDA_ERR_TIMEOUT, 52, (int)blockIdx.x, k);
        *(volatile int *)&sh.abort = 1;
        break;
      }
      const int64_t block = taken_block(smem_u32(sh.answer));
      fence_proxy_async_smem();
      __syncwarp();
      more = block >= 0;
      if (more) it = finder.find(block);
      else it.tile.seq = -1;
    }
  } else {
    start();
    const uint32_t base = smem_u32(tiles), tm = sh.tmem;
    for (int k = 0;;) {
      // one warp says for all what comes next, so that all meet at the same barriers
      if (warp == 0) {
        const bool ok = warp_wait(cx, &sh.item_full[k & 1], (k >> 1) & 1, 45, k);
        if (lane == 0)
          sh.pass = !ok || *cx.abort || sh.item[k & 1].tile.seq < 0 ? kNoPass
                    : sh.item[k & 1].keys                           ? kKeysPass
                                                                    : kQueriesPass;
      }
      __syncwarp();
      named_sync(1, kThreads - 32);
      const int pass = sh.pass;
      if (pass == kNoPass) break;
      if (pass == kKeysPass) keys_pass<DR>(maps, p, sh, k, base, tm, cx);
      else queries_pass<DR>(maps, p, sh, k, base, tm, cx);
      __syncwarp();
      named_sync(1, kThreads - 32);      // the passes lay out shared memory differently
      k = sh.next;
      if (tid == 0 && !*cx.abort) {
        if (pass == kKeysPass) init_keys(sh.keys, true);
        else init_queries(sh.queries, true);
        fence_mbarrier_init();
      }
    }
  }

  __syncwarp();
  __syncthreads();
  if (sh.abort) {  // nothing in flight outlives the CTA
    if (tid == 32 * kLoadWarp) {
      constexpr uint32_t ST = stages<DR>(), KT = DR ? 3 : 4, VT = DR ? 1 : 2;
      const KeysBars &a = sh.keys;
      const QueriesBars &b = sh.queries;
      auto drain = [](const uint64_t *bars, uint32_t loaded, uint32_t ring) {
        for (uint32_t g = loaded > ring ? loaded - ring : 0; g < loaded; ++g)
          mbar_wait(const_cast<uint64_t *>(&bars[g % ring]), (g / ring) & 1, kWaitNs);
      };
      drain(a.full, a.loaded, ST);
      drain(&a.x_full, a.loaded_x, 1);
      drain(b.k_full, b.loaded_k, KT);
      drain(b.v_full, b.loaded_v, VT);
      drain(&b.x_full, b.loaded_x, 1);
      drain(&b.g_full, b.loaded_g, 1);
    }
    if (warp == kMmaWarp && elect_one()) {
      umma_commit(&sh.fin);
      mbar_wait(&sh.fin, 0, kWaitNs);
    }
    __syncthreads();
  }
  if (warp == kMmaWarp) {
    __syncwarp();
    tmem_dealloc(sh.tmem, 512);
  }
}

// lse * log2(e) and delta = d_out . out of 64 rows of a head, in the padded layout.
// A row without any key has lse = -inf: +inf stands for it, so that exp2 gives 0.
// One pass over both tensors: 134 MB in 27 us (4 x 4096 tokens, 16 heads), 5 TB/s.
constexpr int kStatThreads = 256;
__global__ void __launch_bounds__(kStatThreads)
kda_latent_stat_kernel(const __nv_bfloat16 *__restrict__ out,
                       const __nv_bfloat16 *__restrict__ d_out, const float *__restrict__ lse,
                       float *__restrict__ lse2, float *__restrict__ delta, const Params p) {
  __shared__ SeqTile st;
  const int tid = threadIdx.x, head = blockIdx.y;
  pdl_launch_dependents();
  if (tid < 32) {
    const LaneSeqs seqs(p);
    const int32_t tiles = count_tiles(p, seqs, kTileC);
    SeqTile f;
    f.seq = -1;
    if ((int32_t)blockIdx.x < tiles) f = ordered_tile(p, seqs, kTileC, (int32_t)blockIdx.x);
    f.bad = tiles < 0;
    if (tid == 0) st = f;
  }
  __syncthreads();
  if (blockIdx.x == 0 && head == 0 && tid == 0)  // the call's first kernel
    set_device_status(p.status, st.bad ? KDA_ERR_INVALID_ARG : KDA_OK, st.bad);
  if (st.seq < 0) return;
  const int64_t at = head * p.stat_rows + (stat_tile(st.q0, st.seq) + st.tile) * kY;
#pragma unroll
  for (int k = 0; k < kY * 16 / kStatThreads; ++k) {  // 16 lanes a row, 8 channels each
    const int r = (k * kStatThreads + tid) >> 4, c = tid & 15, row = st.tile * kY + r;
    float sum = 0.f, l = -CUDART_INF_F;
    if (row < st.nq) {
      if (c == 0) l = lse[((int64_t)st.q0 + row) * p.H + head];
      const int64_t e = (((int64_t)st.q0 + row) * p.H + head) * kLatentD + 8 * c;
      const uint4 a = *reinterpret_cast<const uint4 *>(out + e);
      const uint4 b = *reinterpret_cast<const uint4 *>(d_out + e);
      const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 u = unpack_bf16x2(x[j]), v = unpack_bf16x2(y[j]);
        sum = fmaf(u.x, v.x, sum);
        sum = fmaf(u.y, v.y, sum);
      }
    }
#pragma unroll
    for (int o = 8; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (c == 0) {
      lse2[at + r] = l == -CUDART_INF_F ? CUDART_INF_F : l * kLog2e;
      delta[at + r] = sum;
    }
  }
}

// d_k_rope = scale * sum over the heads, in head order.  67 MB in 14 us (as above), 4.8
// TB/s, part of it from L2.
__global__ void kda_latent_rope_kernel(const float *__restrict__ rope, int64_t n, int32_t H,
                                       float scale, const DeviceStatus *status,
                                       __nv_bfloat16 *__restrict__ out) {
  const int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) * 4;
  if (i >= n || status->code == KDA_ERR_INVALID_ARG) return;
  float4 a = make_float4(0, 0, 0, 0);
#pragma unroll 8
  for (int h = 0; h < H; ++h) {
    const float4 x = *reinterpret_cast<const float4 *>(rope + h * n + i);
    a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
  }
  *reinterpret_cast<uint2 *>(out + i) =
      make_uint2(pack_bf16x2(a.x * scale, a.y * scale), pack_bf16x2(a.z * scale, a.w * scale));
}

int64_t stat_rows(int64_t n_q, int32_t n_seqs) { return (n_q / kY + n_seqs) * kY; }

template <int DR>
cudaError_t launch(const LatentArgs &a, cudaStream_t stream) {
  Maps mp;
  memset(&mp, 0, sizeof(mp));
  const cuuint64_t W = kLatentD + DR, H = a.H;
  const cuuint64_t nq = a.n_q > 0 ? a.n_q : 1, nk = a.n_k > 0 ? a.n_k : 1;
  // without queries or keys nothing is loaded; the maps only need a valid base
  const void *any = a.n_q > 0 ? a.q : a.k;
  const void *q = a.n_q > 0 ? a.q : any, *g = a.n_q > 0 ? a.d_out : any;
  const void *k = a.n_k > 0 ? a.k : any, *v = a.n_k > 0 ? a.v : any;
  const void *r = a.n_k > 0 ? a.k_rope : any;
  const cuuint64_t qd[3] = {W, H, nq}, qs[2] = {W * 2, H * W * 2};
  const cuuint64_t gd[3] = {kLatentD, H, nq}, gs[2] = {kLatentD * 2, H * kLatentD * 2};
  const cuuint64_t kd[3] = {kLatentD, H, nk};
  const cuuint64_t ks[2] = {(cuuint64_t)a.k_hs * 2, (cuuint64_t)a.k_ts * 2};
  const cuuint64_t vs[2] = {(cuuint64_t)a.v_hs * 2, (cuuint64_t)a.v_ts * 2};
  const cuuint64_t rd[2] = {64, nk}, rs[1] = {128};
  const cuuint32_t b128[3] = {64, 1, 128}, b64[3] = {64, 1, 64};
  const cuuint32_t r128[2] = {64, 128};
  if (!make_bf16_map(&mp.q128, q, 3, qd, qs, b128) || !make_bf16_map(&mp.q64, q, 3, qd, qs, b64) ||
      !make_bf16_map(&mp.g128, g, 3, gd, gs, b128) || !make_bf16_map(&mp.g64, g, 3, gd, gs, b64) ||
      !make_bf16_map(&mp.k128, k, 3, kd, ks, b128) ||
      !make_bf16_map(&mp.v128, v, 3, kd, vs, b128) ||
      (DR && !make_bf16_map(&mp.r128, r, 2, rd, rs, r128)))
    return cudaErrorInvalidValue;
  Params p;
  p.cu_q = a.cu_q; p.cu_k = a.cu_k; p.n_seqs = a.n_seqs; p.H = a.H; p.n_q = a.n_q; p.n_k = a.n_k;
  p.sms = sm_count();
  p.rows[kTileA] = kX; p.by_key[kTileA] = false;
  p.rows[kTileB] = kX; p.by_key[kTileB] = true;
  p.rows[kTileC] = kY; p.by_key[kTileC] = false;
  cudaError_t e = launch_latent_plan(p, a.scratch, a.status, stream);
  if (e != cudaSuccess) return e;
  p.stat_rows = stat_rows(a.n_q, a.n_seqs);
  p.scale = a.scale; p.scale2 = a.scale * kLog2e; p.causal = a.causal;
  p.dq = static_cast<__nv_bfloat16 *>(a.dq); p.dk = static_cast<__nv_bfloat16 *>(a.dk);
  p.dv = static_cast<__nv_bfloat16 *>(a.dv);
  p.dk_ts = a.dk_ts; p.dk_hs = a.dk_hs; p.dv_ts = a.dv_ts; p.dv_hs = a.dv_hs;
  float *lse2 = reinterpret_cast<float *>(static_cast<unsigned char *>(a.scratch) +
                                          latent_plan_bytes(a.n_seqs));
  float *delta = lse2 + p.stat_rows * a.H;
  p.lse2 = lse2; p.delta = delta; p.rope = delta + p.stat_rows * a.H;
  p.status = a.status;
  p.test = a.test;
  // as many items as there can be (one sequence: exactly that many)
  auto most = [&](int64_t n) {
    return n == 0 ? 0 : a.n_seqs == 1 ? (n + kX - 1) / kX : n / kX + a.n_seqs;
  };
  const int64_t blocks = (most(a.n_k) + most(a.n_q)) * a.H;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  auto kernel = kda_latent_bwd_kernel<DR>;
  if (!kernel_ready<kda_latent_bwd_kernel<DR>>(kSmem, 0)) return cudaErrorNotSupported;
  if (a.n_q > 0) {
    const dim3 grid((unsigned)(a.n_q / kY + a.n_seqs), (unsigned)a.H);
    kda_latent_stat_kernel<<<grid, kStatThreads, 0, stream>>>(
        static_cast<const __nv_bfloat16 *>(a.out), static_cast<const __nv_bfloat16 *>(a.d_out),
        a.lse, lse2, delta, p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  // starts while the statistics' kernel ends, and waits for it before it reads them.
  // (The kernel after this one starts in the usual way: launched early it makes this one
  // slower: all three, replayed from a graph, take 67 us and not 64 on 1,847 tokens in
  // five sequences, 16 heads.)
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = a.n_q > 0 ? 1 : 0;
  e = cudaLaunchKernelEx(&cfg, kernel, mp, p);
  if (e != cudaSuccess || !DR || a.n_k == 0) return e;
  const int64_t elems = a.n_k * kLatentRope;
  kda_latent_rope_kernel<<<(unsigned)((elems / 4 + 255) / 256), 256, 0, stream>>>(
      p.rope, elems, a.H, a.scale, a.status, static_cast<__nv_bfloat16 *>(a.d_k_rope));
  return cudaGetLastError();
}

}  // namespace

size_t latent_bwd_scratch_bytes(int32_t n_seqs, int64_t n_q, int64_t n_k, int32_t H, int32_t dr) {
  return latent_plan_bytes(n_seqs) + (size_t)H * sizeof(float) * (2 * (size_t)stat_rows(n_q, n_seqs) + (size_t)n_k * dr);
}

cudaError_t launch_latent_bwd(const LatentArgs &a, cudaStream_t stream) {
  if (a.n_q == 0 && a.n_k == 0) return cudaSuccess;
  if (!latent::encode_tiled()) return cudaErrorNotSupported;
  return a.dr ? launch<64>(a, stream) : launch<0>(a, stream);
}

}  // namespace kda
