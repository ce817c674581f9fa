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
constexpr int kThreads = 384;            // 8 elementwise warps; loader, MMA, cleaner, spare
constexpr int kLoadWarp = 8, kMmaWarp = 9, kCleanWarp = 10;
constexpr int kMaxStages = 4;
constexpr uint32_t kXBlock = 16384, kYBlock = 8192;  // 128 or 64 rows x 64 channels

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages], s_full[2];
  uint64_t x_full, dp_full, p_ready[2], ds_ready, clean_req, clean, acc_full, fin;
  int abort, loaded;
  alignas(16) float lse2[kMaxStages][kY];
  float delta[kMaxStages][kY];
};

template <int DR>
constexpr uint32_t x_bytes() { return ((kLatentD + DR) / 64 + 2) * kXBlock; }
template <int DR>
constexpr uint32_t stage_bytes() { return ((kLatentD + DR) / 64 + 2) * kYBlock; }
template <int DR>
constexpr int stages() { return DR ? 3 : 4; }
constexpr uint32_t kSmem = 232448 - 1024, kSharedBytes = 2048;  // dynamic; the item is static
struct QShared {                         // of the queries pass
  uint64_t k_full[4], k_empty[4], v_full[2], v_empty[2];
  uint64_t x_full, x2_ready, s_full, s_free, dp_full, ds_ready, clean_req, clean, acc_full, fin;
  int abort, loaded_k, loaded_v;
};
static_assert(sizeof(QShared) <= kSharedBytes, "shared memory");
template <int DR>
constexpr uint32_t keys_bytes() { return x_bytes<DR>() + stages<DR>() * stage_bytes<DR>(); }
static_assert(keys_bytes<64>() + sizeof(Shared) <= kSmem &&
              keys_bytes<0>() + sizeof(Shared) <= kSmem, "shared memory");

struct Params : Packed {
  int64_t stat_rows;
  float scale, scale2;
  int causal;
  __nv_bfloat16 *dq, *dk, *dv;
  int64_t dk_ts, dk_hs, dv_ts, dv_hs;
  const float *lse2, *delta;             // [H][stat_rows]
  float *rope;                           // [H][n_k][64]
  DeviceStatus *status;
};

// Row statistics are kept per head in tiles of 64 that no two sequences share:
// the first tile of sequence s is floor(q0 / 64) + s.
__host__ __device__ inline int64_t stat_tile(int64_t q0, int64_t s) { return q0 / kY + s; }

struct Maps {
  CUtensorMap q128, q64, g128, g64, k128, v128, r128;
};

// The 64 columns at `col` of this warpgroup's 128 accumulator rows, times `mul`, as
// bf16 rows of dst (row stride `stride` elements); rows >= n_rows are not written.
// `buf`: 4 KB of shared memory of this warp.
__device__ __forceinline__ void store_cols(uint32_t col, float mul, bool zero,
                                           __nv_bfloat16 *dst, int64_t stride, int n_rows,
                                           uint32_t buf, int warp4, int lane) {
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    uint32_t o[32];
    if (zero) {
#pragma unroll
      for (int j = 0; j < 32; ++j) o[j] = 0;
    } else {
      tmem_ld32(col + 32 * c, o);
      tmem_ld_wait(o);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[j] = pack_bf16x2(__uint_as_float(o[8 * q + 2 * j]) * mul,
                           __uint_as_float(o[8 * q + 2 * j + 1]) * mul);
      st_shared_v4(buf + lane * 128 + (((4 * c + q) ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
    }
  }
  __syncwarp();
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int rr = 4 * k + (lane >> 3), piece = lane & 7, row = warp4 * 32 + rr;
    const uint4 v = ld_shared_v4(buf + rr * 128 + ((piece ^ (rr & 7)) << 4));
    if (row < n_rows) *reinterpret_cast<uint4 *>(dst + row * stride + 8 * piece) = v;
  }
  __syncwarp();
}

// The keys pass: X = 128 keys and their values.  A1 (192 columns) and A2 (128) leave 192
// columns of TMEM: two S buffers and one dP, so the tensor cores run S two tiles ahead
// and dP one ahead of the elementwise work.  Tiles of 64 queries: with the 80 KB of X,
// 96 of them fit shared memory only once, and S and dP would need 288 columns.
template <int DR>
__device__ __forceinline__ void keys_pass(const Maps &maps, const Params &p, const SeqTile &st, int head,
                                          uint32_t base, uint32_t tm, Shared &m) {
  constexpr int KB = (kLatentD + DR) / 64, ST = stages<DR>();
  constexpr uint32_t kStage = x_bytes<DR>();
  constexpr int N1 = kLatentD + DR;
  constexpr uint32_t TM_A1 = 0, TM_A2 = 192, TM_S = 320, TM_DP = 448;
  constexpr uint32_t ID_S = idesc_bf16(128, kY, false, false);
  constexpr uint32_t ID_A1 = idesc_bf16(128, N1, false, true);
  constexpr uint32_t ID_A2 = idesc_bf16(128, kLatentD, false, true);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&m.full[i], 1);
      mbar_init(&m.empty[i], 1);
    }
    mbar_init(&m.s_full[0], 1);
    mbar_init(&m.s_full[1], 1);
    mbar_init(&m.x_full, 1);
    mbar_init(&m.dp_full, 1);
    mbar_init(&m.p_ready[0], 8);
    mbar_init(&m.p_ready[1], 8);
    mbar_init(&m.ds_ready, 8);
    mbar_init(&m.clean_req, 1);
    mbar_init(&m.clean, 1);
    mbar_init(&m.acc_full, 1);
    mbar_init(&m.fin, 1);
    m.abort = 0;
    m.loaded = 0;
    fence_mbarrier_init();
  }
  if (warp == kLoadWarp && lane == 0) {
    prefetch_tensormap(&maps.k128);
    prefetch_tensormap(&maps.v128);
    prefetch_tensormap(&maps.q64);
    prefetch_tensormap(&maps.g64);
    if (DR) prefetch_tensormap(&maps.r128);
  }
  __syncthreads();

  // The CTA's keys [x0, x0 + 128) of the sequence, longest first: the first keys are
  // seen by the most queries.  It streams tiles [y_first, y_first + n) of 64 queries.
  const int x0 = st.tile * kX;
  const int ny = st.nq;
  const int shift = st.nk - st.nq;       // query i sees keys <= i + shift
  const int y_first = p.causal ? max(0, x0 - shift) / kY : 0;
  int n = (ny + kY - 1) / kY - y_first;
  if (st.seq < 0 || n < 0) n = 0;
  const int live = min(kY, ny - (y_first + n - 1) * kY);  // rows of the last tile
  const WaitCtx cx{&m.abort, p.status, (int)blockIdx.x};

  if (warp == kLoadWarp && lane == 0 && n > 0) {
    // ---- loader
    const int xr = st.k0 + x0;
    mbar_arrive_expect_tx(&m.x_full, (KB + 2) * kXBlock);
    for (int kb = 0; kb < KB; ++kb) {
      const uint32_t dst = base + kb * kXBlock;
      if (kb < 2) tma_load_3d_u(dst, &maps.k128, &m.x_full, 64 * kb, head, xr);
      else tma_load_2d(dst, &maps.r128, &m.x_full, 0, xr);
    }
    for (int c = 0; c < 2; ++c)
      tma_load_3d_u(base + (KB + c) * kXBlock, &maps.v128, &m.x_full, 64 * c,
                    head, xr);
    bool ok = true;
    int i = 0;
    for (; i < n; ++i) {
      const int s = i % ST;
      if (i >= ST) ok = wait_or_abort(cx, &m.empty[s], (i / ST - 1) & 1, 10, i);
      if (!ok) break;
      const int yr = st.q0 + (y_first + i) * kY;
      const uint32_t dst = base + kStage + s * stage_bytes<DR>();
      mbar_arrive_expect_tx(&m.full[s], stage_bytes<DR>() + 2 * kY * 4);
      for (int kb = 0; kb < KB; ++kb)
        tma_load_3d_u(dst + kb * kYBlock, &maps.q64, &m.full[s], 64 * kb, head, yr);
      for (int c = 0; c < 2; ++c)
        tma_load_3d_u(dst + (KB + c) * kYBlock, &maps.g64, &m.full[s], 64 * c,
                      head, yr);
      const int64_t at = head * p.stat_rows + (stat_tile(st.q0, st.seq) + y_first + i) * kY;
      bulk_load(smem_u32(m.lse2[s]), p.lse2 + at, kY * 4, &m.full[s]);
      bulk_load(smem_u32(m.delta[s]), p.delta + at, kY * 4, &m.full[s]);
    }
    if (ok) mbar_arrive(&m.clean_req);
    m.loaded = i;
  } else if (warp == kMmaWarp && n > 0 && elect_one()) {
    // ---- MMA issue
    const Desc x_s(base, 16), y_s(base + kStage, 16), y_a(base + kStage, kYBlock);
    constexpr uint32_t SB = stage_bytes<DR>();
    bool ok = wait_or_abort(cx, &m.x_full, 0, 20, 0);
    auto issue_s = [&](int i, int s) {   // s: stage of tile i
      ok = ok && wait_or_abort(cx, &m.full[s], (i / ST) & 1, 21, i);
      if (!ok) return;
#pragma unroll
      for (int k = 0; k < 4 * KB; ++k)
        umma_ss(tm + TM_S + 64 * (i & 1), x_s.at((k >> 2) * kXBlock + (k & 3) * 32),
                y_s.at(s * SB + (k >> 2) * kYBlock + (k & 3) * 32), ID_S, k > 0);
      umma_commit(&m.s_full[i & 1]);
    };
    auto issue_dp = [&](int s) {
#pragma unroll
      for (int k = 0; k < 8; ++k)
        umma_ss(tm + TM_DP, x_s.at((KB + (k >> 2)) * kXBlock + (k & 3) * 32),
                y_s.at(s * SB + (KB + (k >> 2)) * kYBlock + (k & 3) * 32), ID_S, k > 0);
      umma_commit(&m.dp_full);
    };
    issue_s(0, 0);
    if (ok) issue_dp(0);
    if (n > 1) issue_s(1, 1);
    int s0 = 0;                          // stage of tile i
    for (int i = 0; ok && i < n; ++i) {
      const int s1 = s0 + 1 == ST ? 0 : s0 + 1, s2 = s1 + 1 == ST ? 0 : s1 + 1;
      // P Y2 while the elementwise warps are still at dS, which needs dP.  (P of the
      // tile after the next may be ready before this wait: a barrier for each parity.)
      ok = wait_or_abort(cx, &m.p_ready[i & 1], (i >> 1) & 1, 24, i);
      if (ok && i + 1 == n && live < kY) ok = wait_or_abort(cx, &m.clean, 0, 23, i);
      if (!ok) break;
      tc_fence_after();
      const uint32_t sb = tm + TM_S + 64 * (i & 1);
#pragma unroll
      for (int k = 0; k < 4; ++k)  // bf16 columns: rows 0 .. 31 at +0, 32 .. 63 at +32
        umma_ts(tm + TM_A2, sb + (k >> 1) * 32 + (k & 1) * 8,
                y_a.at(s0 * SB + KB * kYBlock + k * 2048), ID_A2, i + k > 0);
      ok = wait_or_abort(cx, &m.ds_ready, i & 1, 22, i);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < 4; ++k)
        umma_ts(tm + TM_A1, tm + TM_DP + (k >> 1) * 32 + (k & 1) * 8, y_a.at(s0 * SB + k * 2048),
                ID_A1, i + k > 0);
      umma_commit(&m.empty[s0]);
      if (i + 1 < n) issue_dp(s1);
      if (i + 2 < n) issue_s(i + 2, s2);
      s0 = s1;
    }
    if (ok) umma_commit(&m.acc_full);
  } else if (warp == kCleanWarp && n > 0 && live < kY) {
    // ---- cleaner: rows of the last tile past the sequence's end are another
    // sequence's and may hold anything; as operands of the sums they are zeroed
    // (0 * NaN would reach the result).  The loader asks once their copy is under
    // way; the products that read them wait for it.
    bool ok = warp_wait(cx, &m.clean_req, 0, 30, n);
    ok = ok && warp_wait(cx, &m.full[(n - 1) % ST], ((n - 1) / ST) & 1, 31, n);
    if (ok) {
      const uint32_t y = base + kStage + (uint32_t)((n - 1) % ST) * stage_bytes<DR>();
      for (int b = 0; b < KB + 2; ++b)
        for (int j = lane; j < (kY - live) * 8; j += 32)
          st_shared_v4(y + b * kYBlock + live * 128 + j * 16, 0, 0, 0, 0);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&m.clean);
    }
  } else if (warp < 8) {
    // ---- elementwise: thread = row of X, warpgroup = half of a tile's columns
    const int wg = warp >> 2, xr = x0 + (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t col = 32 * wg;
    // queries [lo, ny) see this row's key
    const int lo = p.causal ? max(0, xr - shift) : 0;
    bool ok = true;
    for (int i = 0; ok && i < n; ++i) {
      ok = warp_wait(cx, &m.s_full[i & 1], (i >> 1) & 1, 40, i);
      if (!ok) break;
      tc_fence_after();
      uint32_t r[32];
      const uint32_t ts = tm + lanes + TM_S + 64 * (i & 1) + col, td = tm + lanes + TM_DP + col;
      tmem_ld32(ts, r);
      tmem_ld_wait(r);
      const int y0 = (y_first + i) * kY + (int)col;
      const bool edge = __any_sync(0xffffffffu, y0 < lo || y0 + 32 > ny);
      float pr[32];
      const uint32_t sl = smem_u32(&m.lse2[i % ST][col]);
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
      if (lane == 0) mbar_arrive(&m.p_ready[i & 1]);
      ok = warp_wait(cx, &m.dp_full, i & 1, 41, i);
      if (!ok) break;
      tc_fence_after();
      tmem_ld32(td, r);
      tmem_ld_wait(r);
      const uint32_t sd = smem_u32(&m.delta[i % ST][col]);
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
    if (ok && n > 0) {
      ok = warp_wait(cx, &m.acc_full, 0, 42, n);
      tc_fence_after();
    }
    // ---- output, 64 columns at a time, through the rows of X (all products are done)
    if (ok && st.seq >= 0) {
      const bool zero = n == 0;
      const uint32_t buf = base + warp * 8192, acc = tm + lanes;
      const int rows = st.nk - x0, w4 = warp & 3;
      const int64_t kr = st.k0 + x0;
      store_cols(acc + TM_A2 + 64 * wg, 1.f, zero, p.dv + kr * p.dv_ts + head * p.dv_hs + 64 * wg,
                 p.dv_ts, rows, buf, w4, lane);
      store_cols(acc + TM_A1 + 64 * wg, p.scale, zero,
                 p.dk + kr * p.dk_ts + head * p.dk_hs + 64 * wg, p.dk_ts, rows, buf, w4, lane);
      if (DR) {  // fp32, 32 columns a warpgroup
        uint32_t o[32];
        if (zero) {
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = 0;
        } else {
          tmem_ld32(acc + TM_A1 + kLatentD + 32 * wg, o);
          tmem_ld_wait(o);
        }
#pragma unroll
        for (int q = 0; q < 8; ++q)
          st_shared_v4(buf + lane * 128 + ((q ^ (lane & 7)) << 4), o[4 * q], o[4 * q + 1],
                       o[4 * q + 2], o[4 * q + 3]);
        __syncwarp();
        float *dst = p.rope + ((int64_t)head * p.n_k + kr + w4 * 32) * kLatentRope + 32 * wg;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int rr = 4 * k + (lane >> 3), piece = lane & 7;
          const uint4 v = ld_shared_v4(buf + rr * 128 + ((piece ^ (rr & 7)) << 4));
          if (w4 * 32 + rr < rows)
            *reinterpret_cast<uint4 *>(dst + rr * kLatentRope + 4 * piece) = v;
        }
      }
    }
  }

  __syncwarp();
  __syncthreads();
  if (m.abort) {  // nothing in flight outlives the CTA
    if (tid == 32 * kLoadWarp && n > 0) {
      for (int k = max(0, m.loaded - ST); k < m.loaded; ++k)
        mbar_wait(&m.full[k % ST], (k / ST) & 1, kWaitNs);
      mbar_wait(&m.x_full, 0, kWaitNs);
    }
    if (tid == 32 * kMmaWarp) {
      umma_commit(&m.fin);
      mbar_wait(&m.fin, 0, kWaitNs);
    }
    __syncthreads();
  }
}

// The queries pass: X = 128 queries and their d_out, streamed tiles of 128 keys.  S and
// dP have one buffer each (128 columns): S of the next tile is issued as soon as S of
// this one is in registers, dP of the next tile after the product that read dS.  d_out
// moves to TMEM (64 columns, the first operand of dP), which gives its 32 KB to the
// streamed tiles: keys in three (dr = 0: four) buffers, because they are held from S
// to the product with dS, values in one (two), because they are done with dP.
template <int DR>
__device__ __forceinline__ void queries_pass(const Maps &maps, const Params &p, const SeqTile &st, int head,
                                             uint32_t base, uint32_t tm, QShared &m) {
  constexpr int KB = (kLatentD + DR) / 64, KT = DR ? 3 : 4, VT = DR ? 1 : 2;
  constexpr uint32_t kRingK = KB * kXBlock, kRingV = kRingK + KT * KB * kXBlock;
  constexpr uint32_t kX2 = kRingK + 2 * KB * kXBlock;    // d_out, where the keys of tile 2 go
  static_assert(kRingV + VT * 2 * kXBlock + kSharedBytes <= kSmem, "shared memory");
  constexpr int N1 = kLatentD + DR;
  constexpr uint32_t TM_A1 = 0, TM_X2 = 192, TM_S = 256, TM_DP = 384;
  constexpr uint32_t ID_S = idesc_bf16(128, 128, false, false);
  constexpr uint32_t ID_A1 = idesc_bf16(128, N1, false, true);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(&m.k_full[i], 1);
      mbar_init(&m.k_empty[i], 1);
      mbar_init(&m.v_full[i & 1], 1);
      mbar_init(&m.v_empty[i & 1], 1);
    }
    mbar_init(&m.x2_ready, 8);
    mbar_init(&m.x_full, 1);
    mbar_init(&m.s_full, 1);
    mbar_init(&m.s_free, 8);
    mbar_init(&m.dp_full, 1);
    mbar_init(&m.ds_ready, 8);
    mbar_init(&m.clean_req, 1);
    mbar_init(&m.clean, 1);
    mbar_init(&m.acc_full, 1);
    mbar_init(&m.fin, 1);
    m.abort = 0;
    m.loaded_k = m.loaded_v = 0;
    fence_mbarrier_init();
  }
  if (warp == kLoadWarp && lane == 0) {
    prefetch_tensormap(&maps.q128);
    prefetch_tensormap(&maps.g128);
    prefetch_tensormap(&maps.k128);
    prefetch_tensormap(&maps.v128);
    if (DR) prefetch_tensormap(&maps.r128);
  }
  __syncthreads();

  // longest first: the last queries of a sequence see the most keys
  const int x0 = (st.n_tiles - 1 - st.tile) * kX;
  const int shift = st.nk - st.nq;       // query i sees keys <= i + shift
  const int y_end = p.causal ? min(st.nk, min(x0 + kX, st.nq) + shift) : st.nk;
  const int n = st.seq >= 0 && y_end > 0 ? (y_end + 127) / 128 : 0;
  const int live = min(128, st.nk - (n - 1) * 128);      // keys of the last tile
  const WaitCtx cx{&m.abort, p.status, (int)blockIdx.x};

  if (warp == kLoadWarp && lane == 0 && n > 0) {
    // ---- loader
    const int xr = st.q0 + x0;
    mbar_arrive_expect_tx(&m.x_full, (KB + 2) * kXBlock);
    for (int c = 0; c < 2; ++c)
      tma_load_3d_u(base + kX2 + c * kXBlock, &maps.g128, &m.x_full, 64 * c, head, xr);
    for (int kb = 0; kb < KB; ++kb)
      tma_load_3d_u(base + kb * kXBlock, &maps.q128, &m.x_full, 64 * kb, head, xr);
    bool ok = true;
    int i = 0, iv = 0;
    for (; i < n; ++i) {
      const int yr = st.k0 + i * 128, sk = i % KT, sv = i % VT;
      if (i >= KT) ok = wait_or_abort(cx, &m.k_empty[sk], (i / KT - 1) & 1, 10, i);
      if (ok && i == 2) ok = wait_or_abort(cx, &m.x2_ready, 0, 11, i);
      if (!ok) break;
      mbar_arrive_expect_tx(&m.k_full[sk], KB * kXBlock);
      const uint32_t dk = base + kRingK + sk * KB * kXBlock;
      for (int kb = 0; kb < KB; ++kb) {
        if (kb < 2) tma_load_3d_u(dk + kb * kXBlock, &maps.k128, &m.k_full[sk], 64 * kb, head, yr);
        else tma_load_2d(dk + kb * kXBlock, &maps.r128, &m.k_full[sk], 0, yr);
      }
      if (i >= VT) ok = wait_or_abort(cx, &m.v_empty[sv], (i / VT - 1) & 1, 12, i);
      if (!ok) { ++i; break; }
      mbar_arrive_expect_tx(&m.v_full[sv], 2 * kXBlock);
      const uint32_t dv = base + kRingV + sv * 2 * kXBlock;
      for (int c = 0; c < 2; ++c)
        tma_load_3d_u(dv + c * kXBlock, &maps.v128, &m.v_full[sv], 64 * c, head, yr);
      iv = i + 1;
    }
    if (ok) mbar_arrive(&m.clean_req);
    m.loaded_k = i;
    m.loaded_v = iv;
  } else if (warp == kMmaWarp && n > 0 && elect_one()) {
    // ---- MMA issue
    const Desc x_s(base, 16), k_s(base + kRingK, 16), v_s(base + kRingV, 16),
        k_a(base + kRingK, kXBlock);
    bool ok = wait_or_abort(cx, &m.x_full, 0, 20, 0);
    auto issue_s = [&](int i) {
      const int sk = i % KT;
      ok = ok && wait_or_abort(cx, &m.k_full[sk], (i / KT) & 1, 21, i);
      if (ok && i > 0) ok = wait_or_abort(cx, &m.s_free, (i - 1) & 1, 22, i);
      if (!ok) return;
      tc_fence_after();
      const uint32_t off = sk * KB * kXBlock;
#pragma unroll
      for (int k = 0; k < 4 * KB; ++k)
        umma_ss(tm + TM_S, x_s.at((k >> 2) * kXBlock + (k & 3) * 32),
                k_s.at(off + (k >> 2) * kXBlock + (k & 3) * 32), ID_S, k > 0);
      umma_commit(&m.s_full);
    };
    auto issue_dp = [&](int i) {
      const int sv = i % VT;
      ok = ok && wait_or_abort(cx, &m.v_full[sv], (i / VT) & 1, 23, i);
      if (!ok) return;
      const uint32_t off = sv * 2 * kXBlock;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        umma_ts(tm + TM_DP, tm + TM_X2 + 8 * k, v_s.at(off + (k >> 2) * kXBlock + (k & 3) * 32),
                ID_S, k > 0);
      umma_commit(&m.dp_full);
      umma_commit(&m.v_empty[sv]);
    };
    issue_s(0);
    ok = ok && wait_or_abort(cx, &m.x2_ready, 0, 26, 0);
    tc_fence_after();
    issue_dp(0);
    if (n > 1) issue_s(1);
    for (int i = 0; ok && i < n; ++i) {
      ok = wait_or_abort(cx, &m.ds_ready, i & 1, 24, i);
      if (ok && i + 1 == n && live < 128) ok = wait_or_abort(cx, &m.clean, 0, 25, i);
      if (!ok) break;
      tc_fence_after();
      // dS is over dP, keys 0 .. 63 at column 0, 64 .. 127 at column 64
      const uint32_t off = (i % KT) * KB * kXBlock;
#pragma unroll
      for (int k = 0; k < 8; ++k)
        umma_ts(tm + TM_A1, tm + TM_DP + (k >> 2) * 64 + (k & 3) * 8, k_a.at(off + k * 2048), ID_A1,
                i + k > 0);
      umma_commit(&m.k_empty[i % KT]);
      if (i + 1 < n) issue_dp(i + 1);
      if (ok && i + 2 < n) issue_s(i + 2);
    }
    if (ok) umma_commit(&m.acc_full);
  } else if (warp == kCleanWarp && n > 0 && live < 128) {
    // ---- cleaner: keys of the last tile past the sequence's end, as in the other pass
    const int sk = (n - 1) % KT;
    bool ok = warp_wait(cx, &m.clean_req, 0, 30, n);
    ok = ok && warp_wait(cx, &m.k_full[sk], ((n - 1) / KT) & 1, 31, n);
    if (ok) {
      const uint32_t y = base + kRingK + sk * KB * kXBlock + live * 128;
      for (int kb = 0; kb < KB; ++kb)
        for (int j = lane; j < (128 - live) * 8; j += 32)
          st_shared_v4(y + kb * kXBlock + j * 16, 0, 0, 0, 0);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&m.clean);
    }
  } else if (warp < 8) {
    // ---- elementwise: thread = query, warpgroup = half of a tile's keys
    const int wg = warp >> 2, xr = x0 + (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    float lse2 = 0.f, delta = 0.f;
    if (st.seq >= 0 && xr < st.nq) {
      const int64_t at = head * p.stat_rows + stat_tile(st.q0, st.seq) * kY + xr;
      lse2 = p.lse2[at];
      delta = p.delta[at];
    }
    const int hi = p.causal ? min(st.nk, xr + shift + 1) : st.nk;  // keys this row sees
    bool ok = n == 0 || warp_wait(cx, &m.x_full, 0, 43, 0);
    if (ok && n > 0) {  // this row's 64 channels of d_out (a warpgroup's half) into TMEM
      uint32_t x[32];
      const int r = (warp & 3) * 32 + lane;
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const uint4 v = ld_shared_v4(base + kX2 + wg * kXBlock + sw128_offset(r, 16 * q));
        x[4 * q] = v.x; x[4 * q + 1] = v.y; x[4 * q + 2] = v.z; x[4 * q + 3] = v.w;
      }
      tmem_st32(tm + lanes + TM_X2 + 32 * wg, x);
      tmem_st_wait();
      tc_fence_before();
      fence_proxy_async_smem();          // its place is loaded again
      __syncwarp();
      if (lane == 0) mbar_arrive(&m.x2_ready);
    }
    for (int i = 0; ok && i < n; ++i) {
      ok = warp_wait(cx, &m.s_full, i & 1, 40, i);
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
      const int seen = hi - (i * 128 + 64 * wg);         // columns below it are allowed
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
      ok = warp_wait(cx, &m.dp_full, i & 1, 41, i);
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
    if (ok && n > 0) {
      ok = warp_wait(cx, &m.acc_full, 0, 42, n);
      tc_fence_after();
    }
    if (ok && st.seq >= 0) {
      const int64_t qr = st.q0 + x0;
      for (int c = wg; c < KB; c += 2)
        store_cols(tm + lanes + TM_A1 + 64 * c, p.scale, n == 0,
                   p.dq + (qr * p.H + head) * N1 + 64 * c, (int64_t)p.H * N1, st.nq - x0,
                   base + warp * 8192, warp & 3, lane);
    }
  }

  __syncwarp();
  __syncthreads();
  if (m.abort) {  // nothing in flight outlives the CTA
    if (tid == 32 * kLoadWarp && n > 0) {
      for (int k = max(0, m.loaded_k - KT); k < m.loaded_k; ++k)
        mbar_wait(&m.k_full[k % KT], (k / KT) & 1, kWaitNs);
      for (int k = max(0, m.loaded_v - VT); k < m.loaded_v; ++k)
        mbar_wait(&m.v_full[k % VT], (k / VT) & 1, kWaitNs);
      mbar_wait(&m.x_full, 0, kWaitNs);
    }
    if (tid == 32 * kMmaWarp) {
      umma_commit(&m.fin);
      mbar_wait(&m.fin, 0, kWaitNs);
    }
    __syncthreads();
  }
}

// The keys pass's items, then the queries pass's; both longest first (the first keys
// are seen by the most queries, the last queries see the most keys).
template <int DR>
__global__ void __launch_bounds__(kThreads, 1)
kda_latent_bwd_kernel(const __grid_constant__ Maps maps, const Params p) {
  extern __shared__ __align__(1024) unsigned char tiles[];
  __shared__ SeqTile s_tile;
  __shared__ int s_head, s_keys;
  __shared__ uint32_t s_tmem;
  const int warp = threadIdx.x >> 5;
  if (warp == kMmaWarp) {
    tmem_alloc(&s_tmem, 512);
    tmem_relinquish();
  }
  if (warp == 0) {
    SeqTile f;
    f.seq = -1;
    int head = 0;
    const LaneSeqs seqs(p);
    const int64_t nk = count_tiles(p, seqs, kTileB), nq = count_tiles(p, seqs, kTileA);
    const int64_t b = blockIdx.x, first_q = nk * p.H;
    const bool keys = nk >= 0 && b < first_q;
    if (nk < 0) {
      if (p.n_q == 0 && b == 0 && threadIdx.x == 0)      // no kernel before this one
        set_device_status(p.status, KDA_ERR_INVALID_ARG, 1);
    } else if (keys) {
      f = place_item(p, seqs, kTileB, nk, b, &head);
    } else if (b < first_q + nq * p.H) {
      f = place_item(p, seqs, kTileA, nq, b - first_q, &head);
    }
    if (threadIdx.x == 0) {
      s_tile = f;
      s_head = head;
      s_keys = keys;
    }
  }
  pdl_launch_dependents();
  pdl_wait();                            // the row statistics
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const SeqTile st = s_tile;
  const uint32_t base = smem_u32(tiles), tm = s_tmem;
  if (st.seq >= 0) {
    if (s_keys)
      keys_pass<DR>(maps, p, st, s_head, base, tm,
                    *reinterpret_cast<Shared *>(tiles + keys_bytes<DR>()));
    else
      queries_pass<DR>(maps, p, st, s_head, base, tm,
                       *reinterpret_cast<QShared *>(tiles + kSmem - kSharedBytes));
  }
  if (warp == kMmaWarp) {                // all warps have passed the pass's last barrier
    __syncwarp();
    tmem_dealloc(tm, 512);
  }
}

// lse * log2(e) and delta = d_out . out of 64 rows of a head, in the padded layout.
// A row without any key has lse = -inf: +inf stands for it, so that exp2 gives 0.
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
    float sum = 0.f;
    if (row < st.nq) {
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
      float l = CUDART_INF_F;
      if (row < st.nq) {
        l = lse[((int64_t)st.q0 + row) * p.H + head];
        l = l == -CUDART_INF_F ? CUDART_INF_F : l * kLog2e;
      }
      lse2[at + r] = l;
      delta[at + r] = sum;
    }
  }
}

// d_k_rope = scale * sum over the heads, in head order.
__global__ void kda_latent_rope_kernel(const float *__restrict__ rope, int64_t n, int32_t H,
                                       float scale, const DeviceStatus *status,
                                       __nv_bfloat16 *__restrict__ out) {
  pdl_wait();
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
  // as many items as there can be (one sequence: exactly that many)
  auto most = [&](int64_t n) { return n == 0 ? 0 : a.n_seqs == 1 ? (n + kX - 1) / kX : n / kX + a.n_seqs; };
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
  // each kernel starts while the one before ends, and waits for it where it reads its
  // results
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
  cfg.gridDim = dim3((unsigned)((elems / 4 + 255) / 256));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kda_latent_rope_kernel, (const float *)p.rope, elems, a.H, a.scale,
                            (const DeviceStatus *)a.status,
                            static_cast<__nv_bfloat16 *>(a.d_k_rope));
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
