// Latent attention in its absorbed form over a paged cache (kda_latent_decode),
// tcgen05 / TMEM / TMA, sm_103a.
//
// For one sequence, with R = T * H query rows of W = 512 + dr channels and cached
// rows c_j: s_rj = scale q_r . c_j, o_r = sum_j softmax(s_r)_j c_j[0:512].  The
// cached row is key and value at once, so a row costs 2 W bytes of HBM and
// 2 R (W + 512) operations: at R = 96 it is just below the ridge of the card
// (181 against 289 operations a byte), and the matrix work has to run near its
// rate for the memory to be the bound.
//
// Everything is computed transposed: S^T [128 keys x N rows] = C Q^T and
// O^T [512 x N rows] = C^T P^T.  The keys fill M = 128 whatever the number of
// rows, so that N follows the rows in steps (16, 32, 64, 96) instead of padding
// them to 128, and O^T (4 x N TMEM columns) leaves room for S^T at N = 96, where
// O [128 x 512] would fill TMEM alone.  The softmax runs over lanes (keys):
// - exponents are taken against a reference per row that only moves when some
//   score exceeds it by more than 8 (a factor 256), so nearly every tile needs a
//   vote and no column maximum; O^T is rescaled only then;
// - row sums stay per thread (one key, N / 2 rows) until the end of a segment.
//
// One CTA per SM; the key tiles of all sequences form one list, cut evenly over
// the CTAs whatever the lengths.  A CTA's first and last sequence may be shared
// with its neighbours: it leaves (reference, sum, O^T) in the workspace, and a
// second small kernel joins the parts in the list's order.
//
// Shared memory: Q (N x W), P (N x 128), and a ring of 16 KB slots.  A 128-key
// tile (147 KB at W = 576) does not fit beside Q, so the ring streams it twice:
// 64-channel blocks as keys, then 64-key x 128-channel blocks as values, the
// second time from L2.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <string.h>

#include "kda_latent_tc.cuh"

namespace kda {
namespace {

using namespace latent;

constexpr int kTile = 128;               // keys per tile
constexpr int kThreads = 384;            // 8 softmax warps, loader, MMA, cleaner, spare
constexpr int kLoadWarp = 8, kMmaWarp = 9, kCleanWarp = 10;
constexpr uint32_t kSlotBytes = 16384;
constexpr uint32_t kSmemMax = 232448;
constexpr float kSlack = 8.f;            // log2 units a score may exceed its reference by
constexpr int kMaxSlots = 12;               // fewer than a tile's 8 key and 2 x 4 value slots

struct Shared {                          // after the tiles
  uint64_t full[kMaxSlots], empty[kMaxSlots], clean[kMaxSlots];
  uint64_t q_full, q_empty, s_full, s_free, p_ready, pv_done, clean_req, fin;
  uint32_t tmem;
  int abort;
  int seq0, tile0, total;                // the CTA's first sequence and tile, all tiles
  int warp_sum[kThreads / 32];
  uint32_t load_pos;                     // ring slots filled, segments begun (loader)
  int load_seg;
  alignas(16) float ref[96];
  float fac[96], sum[96];
  float wmax[8][48];
  int32_t tok[96];                       // draft index of a column's row
  uint64_t seen[96];                     // its tree mask
};

template <int N>
constexpr int slots() {
  const int free = (int)kSmemMax - 1024 - (int)sizeof(Shared) - N * 128 * 9 - N * 256;
  const int n = free / (int)kSlotBytes;
  return n > kMaxSlots ? kMaxSlots : n;
}
template <int N>
constexpr uint32_t smem_bytes() {
  return 1024 + N * 128 * 9 + N * 256 + slots<N>() * kSlotBytes + sizeof(Shared);
}
constexpr uint32_t tmem_cols(int n) { return 5 * n <= 128 ? 128u : 5 * n <= 256 ? 256u : 512u; }

struct Params {
  const int32_t *table, *lens;
  const int64_t *mask;
  int32_t B, T, H, W, n_pages, page_size, max_pages, k_rows, v_rows;
  int32_t n_tiles;      // row tiles
  int32_t G;            // CTAs per row tile
  float scale2;         // scale * log2(e)
  __nv_bfloat16 *out;
  float *lse;
  DeviceStatus *status;
  int32_t *before;      // [B + 1] tiles before each sequence
  float *part_o;        // [row tiles][G][2][N][512]
  float *part_ml;       // [row tiles][G][2][2][96]
};

// Length of sequence b, 0 when it is out of range.
__device__ __forceinline__ int seq_len(const Params &p, int b) {
  const int n = p.lens[b];
  return n < 0 || n > (int64_t)p.max_pages * p.page_size ? 0 : n;
}
__device__ __forceinline__ int key_tiles(int n) { return (n + kTile - 1) / kTile; }

// First tile of CTA c of G when the list has `total` tiles: the first total % G
// CTAs take one more than the others.
__device__ __forceinline__ int cta_begin(int c, int G, int total) {
  const int each = total / G, more = total - each * G;
  return c * each + min(c, more);
}
// The CTA of tile x.
__device__ __forceinline__ int cta_of(int x, int G, int total) {
  const int each = total / G, more = total - each * G, wide = more * (each + 1);
  return x < wide ? x / (each + 1) : more + (x - wide) / max(each, 1);
}

// Walks the CTA's tiles sequence by sequence; every role does so by itself.
struct Walk {
  const Params &p;
  int b, t, left;       // next sequence, its next tile, tiles left for this CTA
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

// Sum over the 128 keys of C values a thread, for a warp's 32 keys: after it, lane
// L holds the warp's sum of value (L * C / 32) (C = 8, 16, 32) ...
template <int C>
__device__ __forceinline__ float warp_transpose_sum(float (&v)[C], int lane) {
  int width = C;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    if (width > 1) {
      width >>= 1;
      const bool up = lane & o;
#pragma unroll
      for (int i = 0; i < C / 2; ++i)
        if (i < width) {
          const float give = up ? v[i] : v[i + width];
          const float keep = up ? v[i + width] : v[i];
          v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
        }
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    }
  }
  return v[0];
}

template <int N>
__device__ __forceinline__ void ld_cols(uint32_t addr, uint32_t (&r)[N / 2]) {
  // N / 2 = 8, 16, 32 or 48 columns
  if constexpr (N / 2 == 8) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                   "=r"(r[6]), "=r"(r[7])
                 : "r"(addr));
  } else if constexpr (N / 2 == 16) {
    tmem_ld16(addr, r);
  } else if constexpr (N / 2 == 32) {
    tmem_ld32(addr, r);
  } else {
    tmem_ld32(addr, *reinterpret_cast<uint32_t(*)[32]>(&r[0]));
    tmem_ld16(addr + 32, *reinterpret_cast<uint32_t(*)[16]>(&r[32]));
  }
}
template <int N>
__device__ __forceinline__ void ld_cols_wait(uint32_t (&r)[N / 2]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N / 2; ++i) asm volatile("" : "+r"(r[i]));
}
template <int N>
__device__ __forceinline__ void st_cols(uint32_t addr, const uint32_t (&r)[N / 2]) {
  if constexpr (N / 2 == 8) {
    tmem_st8(addr, r);
  } else if constexpr (N / 2 == 16) {
    tmem_st16(addr, r);
  } else if constexpr (N / 2 == 32) {
    tmem_st32(addr, r);
  } else {
    tmem_st32(addr, *reinterpret_cast<const uint32_t(*)[32]>(&r[0]));
    tmem_st16(addr + 32, *reinterpret_cast<const uint32_t(*)[16]>(&r[32]));
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads, 1)
kda_latent_decode_kernel(const __grid_constant__ CUtensorMap map_q,
                         const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ CUtensorMap map_v, const Params p) {
  constexpr int S = slots<N>();
  constexpr int HN = N / 2;              // columns of a softmax warpgroup
  constexpr uint32_t kQ = 0, kP = N * 128 * 9, kRing = kP + N * 256;
  constexpr uint32_t TM_O = 0, TM_S = 4 * N;
  constexpr uint32_t ID_S = idesc_bf16(128, N, false, false);
  constexpr uint32_t ID_PV = idesc_bf16(128, N, true, false);

  extern __shared__ unsigned char raw[];
  const uint32_t base = round_up_1k(smem_u32(raw));
  Shared &m = *reinterpret_cast<Shared *>(raw + (base - smem_u32(raw)) + kRing + S * kSlotBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rt = blockIdx.x % p.n_tiles, cta = blockIdx.x / p.n_tiles;
  const int KB = p.W / 64;               // 64-channel blocks of a row

  // ---- the CTA's share of the tile list
  if (tid == 0) {
    for (int i = 0; i < S; ++i) {
      mbar_init(&m.full[i], 1);
      mbar_init(&m.empty[i], 1);
      mbar_init(&m.clean[i], 1);
    }
    mbar_init(&m.q_full, 1);
    mbar_init(&m.q_empty, 1);
    mbar_init(&m.s_full, 1);
    mbar_init(&m.s_free, 8);
    mbar_init(&m.p_ready, 8);
    mbar_init(&m.pv_done, 1);
    mbar_init(&m.clean_req, 1);
    mbar_init(&m.fin, 1);
    m.abort = 0;
    m.seq0 = p.B;
    m.tile0 = 0;
    fence_mbarrier_init();
  }
  if (warp == kLoadWarp && lane == 0) {
    prefetch_tensormap(&map_q);
    prefetch_tensormap(&map_k);
    prefetch_tensormap(&map_v);
  }
  {
    const int per = (p.B + kThreads - 1) / kThreads;
    const int b0 = tid * per, b1 = min(p.B, b0 + per);
    int mine = 0;
    for (int b = b0; b < b1; ++b) {
      const int n = p.lens[b];
      if (n < 0 || n > (int64_t)p.max_pages * p.page_size) {
        if (blockIdx.x == 0) record_device_status(p.status, KDA_ERR_INVALID_ARG, 1, b, n);
      } else {
        mine += key_tiles(n);
      }
    }
    int inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) m.warp_sum[warp] = inc;
    __syncthreads();
    int before = inc - mine, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += m.warp_sum[w];
      total += m.warp_sum[w];
    }
    if (blockIdx.x == 0) {
      int at = before;
      for (int b = b0; b < b1; ++b) {
        p.before[b] = at;
        at += key_tiles(seq_len(p, b));
      }
      if (tid == 0) p.before[p.B] = total;
    }
    const int begin = cta_begin(cta, p.G, total);
    if (begin >= before && begin < before + mine) {
      int at = before;
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
  if (warp == kMmaWarp) {
    tmem_alloc(&m.tmem, tmem_cols(N));
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_launch_dependents();
  const uint32_t tm = m.tmem;
  const int begin = cta_begin(cta, p.G, m.total);
  const int mine = cta_begin(cta + 1, p.G, m.total) - begin;
  const WaitCtx cx{&m.abort, p.status, (int)blockIdx.x};
  Walk walk(p, m.seq0, m.tile0, mine);
  int b;

  // A wait by a whole warp: its lanes leave together.
  auto wait_warp = [&](uint64_t *bar, uint32_t parity, int where, int step) {
    return __all_sync(0xffffffffu, wait_or_abort(cx, bar, parity, where, step)) != 0;
  };

  if (warp == kLoadWarp) {
    // ---- loader: per segment Q, then keys of tile i and values of tile i - 1
    uint32_t pos = 0;                    // ring slots filled so far
    int seg = 0;
    bool ok = true;
    const int pk = kTile / p.k_rows, pv = 64 / p.v_rows;  // pieces of a slot (pk = pv * (1 or 2))
    while (ok && walk.next(&b)) {
      const int n = walk.n;
      if (seg > 0) ok = wait_warp(&m.q_empty, (seg - 1) & 1, 10, seg);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&m.q_full, N * 128 * KB);
        for (int kb = 0; kb < KB; ++kb)
          tma_load_3d_u(base + kQ + kb * N * 128, &map_q, &m.q_full, 64 * kb, rt * N, b);
      }
      ++seg;
      // Pool row of this lane's piece of 16, 32, 64 or 128 keys of tile t (value
      // pieces have the same size but for pages of 128 keys and more).
      auto piece_row = [&](int t, int rows, int count) {
        const int at = t * kTile + lane * rows;
        if (lane >= count || at >= n) return -1;
        const int32_t id = p.table[(int64_t)b * p.max_pages + at / p.page_size];
        if (id < 0 || id >= p.n_pages) {
          record_device_status(p.status, KDA_ERR_INVALID_ARG, 2, b, at);
          return (int)((int64_t)p.n_pages * p.page_size);  // past the pool: reads zeros
        }
        return id * p.page_size + at % p.page_size;
      };
      int row = piece_row(walk.ta, p.k_rows, pk), row_before = 0;
      for (int t = walk.ta; ok && t <= walk.tb; ++t) {
        int row_next = -1;
        if (t + 1 < walk.tb) row_next = piece_row(t + 1, p.k_rows, pk);
        if (t < walk.tb) {  // keys: 64-channel blocks of 128 rows
          const int have = __popc(__ballot_sync(0xffffffffu, row >= 0));
          for (int kb = 0; kb < KB; ++kb, ++pos) {
            const uint32_t s = pos % S;
            if (pos >= S && !wait_warp(&m.empty[s], (pos / S - 1) & 1, 11, t)) { ok = false; break; }
            if (lane == 0) mbar_arrive_expect_tx(&m.full[s], have * p.k_rows * 128);
            __syncwarp();
            if (row >= 0)
              tma_load_2d(base + kRing + s * kSlotBytes + lane * p.k_rows * 128, &map_k,
                          &m.full[s], 64 * kb, row);
          }
        }
        if (ok && t > walk.ta) {  // values of tile t - 1: 64 keys x 128 channels
          const int live = n - (t - 1) * kTile;
          for (int hf = 0; ok && hf < (live > 64 ? 2 : 1); ++hf) {
            // this lane's piece of the half: from the key pieces' rows
            const int src = (hf * 64 + lane * p.v_rows) / p.k_rows;
            int vrow = __shfl_sync(0xffffffffu, row_before, src & 31);
            if (vrow >= 0) vrow += (hf * 64 + lane * p.v_rows) % p.k_rows;
            if (lane >= pv || hf * 64 + lane * p.v_rows >= live) vrow = -1;
            const int have = __popc(__ballot_sync(0xffffffffu, vrow >= 0));
            for (int mt = 0; mt < 4; ++mt, ++pos) {
              const uint32_t s = pos % S;
              if (pos >= S && !wait_warp(&m.empty[s], (pos / S - 1) & 1, 12, t)) { ok = false; break; }
              if (lane == 0) mbar_arrive_expect_tx(&m.full[s], have * p.v_rows * 256);
              __syncwarp();
              if (vrow >= 0) {
                const uint32_t dst = base + kRing + s * kSlotBytes + lane * p.v_rows * 128;
                tma_load_2d(dst, &map_v, &m.full[s], 128 * mt, vrow);
                tma_load_2d(dst + 8192, &map_v, &m.full[s], 128 * mt + 64, vrow);
              }
            }
            __syncwarp();
            if (ok && lane == 0 && live < 64 * (hf + 1)) mbar_arrive(&m.clean_req);
          }
        }
        row_before = row;
        row = row_next;
      }
    }
    if (lane == 0) {
      m.load_pos = pos;
      m.load_seg = seg;
    }
  } else if (warp == kMmaWarp) {
    // ---- MMA issue: S of tile i, then PV of tile i - 1
    if (lane == 0) {
      uint32_t pos = 0, it = 0, cleaned = 0;  // cleaned: parity bit per slot
      int seg = 0;
      bool ok = true;
      while (ok && walk.next(&b)) {
        const int n = walk.n;
        ok = wait_or_abort(cx, &m.q_full, seg & 1, 20, seg);
        for (int t = walk.ta; ok && t <= walk.tb; ++t) {
          if (t < walk.tb) {
            if (it > 0) ok = wait_or_abort(cx, &m.s_free, (it - 1) & 1, 21, t);
            tc_fence_after();
            for (int kb = 0; ok && kb < KB; ++kb, ++pos) {
              const uint32_t s = pos % S;
              ok = wait_or_abort(cx, &m.full[s], (pos / S) & 1, 22, t);
              if (!ok) break;
              const uint32_t a = base + kRing + s * kSlotBytes, q = base + kQ + kb * N * 128;
#pragma unroll
              for (int ks = 0; ks < 4; ++ks)
                umma_ss(tm + TM_S, sdesc_sw128(a + ks * 32, 16, 1024),
                        sdesc_sw128(q + ks * 32, 16, 1024), ID_S, kb + ks > 0);
              umma_commit(&m.empty[s]);
            }
            if (!ok) break;
            umma_commit(&m.s_full);
            if (t + 1 == walk.tb) umma_commit(&m.q_empty);
            ++it;
          }
          if (t > walk.ta) {
            // PV of tile t - 1, the (it - 2)th or, at the end of the segment, the last
            const uint32_t j = t < walk.tb ? it - 2 : it - 1;
            const int live = n - (t - 1) * kTile;
            ok = wait_or_abort(cx, &m.p_ready, j & 1, 23, t);
            if (!ok) break;
            tc_fence_after();
            const bool last_tile = live < kTile;
            for (int hf = 0; ok && hf < (live > 64 ? 2 : 1); ++hf) {
              const bool ragged = last_tile && live < 64 * (hf + 1);
              for (int mt = 0; mt < 4; ++mt, ++pos) {
                const uint32_t s = pos % S;
                ok = wait_or_abort(cx, &m.full[s], (pos / S) & 1, 24, t);
                if (ok && ragged) {
                  ok = wait_or_abort(cx, &m.clean[s], cleaned >> s & 1, 25, t);
                  cleaned ^= 1u << s;
                }
                if (!ok) break;
                const uint32_t v = base + kRing + s * kSlotBytes;
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                  umma_ss(tm + TM_O + mt * N, sdesc_sw128(v + ks * 2048, 8192, 1024),
                          sdesc_sw128(base + kP + hf * N * 128 + ks * 32, 16, 1024), ID_PV,
                          (t - 1 > walk.ta) || hf + ks > 0);
                umma_commit(&m.empty[s]);
              }
            }
            if (!ok) break;
            umma_commit(&m.pv_done);
          }
        }
        ++seg;
      }
    }
  } else if (warp == kCleanWarp) {
    // ---- cleaner: rows past a sequence's end may hold anything; as values they
    // are zeroed in shared memory (0 * NaN would reach the sum).  The loader asks
    // once the slots' copies are under way, so that the wait below is for the phase
    // next to complete; it cannot be two requests ahead, because between two of
    // them lie more slots than the ring has.
    uint32_t pos = 0, req = 0;
    bool ok = true;
    while (ok && walk.next(&b)) {
      const int live = walk.n - (walk.tb - 1) * kTile;  // keys of the segment's last tile
      const int cnt = walk.tb - walk.ta;
      const int halves = live > 64 ? 2 : 1;
      if (live < kTile && (live & 63) != 0) {
        const uint32_t first = pos + (uint32_t)cnt * KB + (uint32_t)(cnt - 1) * 8 +
                               (uint32_t)(halves - 1) * 4;
        const int from = live - 64 * (halves - 1);      // first dead row of the half
        ok = wait_warp(&m.clean_req, req++ & 1, 31, walk.tb);
        for (int mt = 0; ok && mt < 4; ++mt) {
          const uint32_t k = first + mt, s = k % S;
          ok = wait_warp(&m.full[s], (k / S) & 1, 30, walk.tb);
          if (!ok) break;
          const uint32_t dst = base + kRing + s * kSlotBytes;
          for (int i = lane; i < (64 - from) * 8; i += 32) {
            st_shared_v4(dst + (from * 8 + i) * 16, 0, 0, 0, 0);
            st_shared_v4(dst + 8192 + (from * 8 + i) * 16, 0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&m.clean[s]);
        }
      }
      pos += (uint32_t)cnt * KB + (uint32_t)(cnt - 1) * 8 + (uint32_t)halves * 4;
    }
  } else if (warp < 8) {
    // ---- softmax and output: thread = key of the tile, warpgroup = half of the rows
    const int wg = warp >> 2, key = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // lane base in a TMEM address
    const int c0 = wg * HN, wt = tid & 127;             // first column; thread of the warpgroup
    const uint32_t barid = 1 + wg;
    const uint32_t p_dst = base + kP + (key >> 6) * N * 128;
    const uint32_t p_col = (key & 63) * 2;
    uint32_t it = 0;
    bool failed = false, dead = false;
    int seg = 0;
    while (!dead && walk.next(&b)) {
      const int n = walk.n, t_draft = n - p.T;          // position of the first draft
      if (wt < HN) {
        const int r = rt * N + c0 + wt, tok = r / p.H;
        m.ref[c0 + wt] = kNoRef;
        m.tok[c0 + wt] = tok;
        m.seen[c0 + wt] = p.mask && tok < p.T ? (uint64_t)p.mask[(int64_t)b * p.T + tok] : 0;
      }
      named_sync(barid, 128);
      float l[HN];
#pragma unroll
      for (int i = 0; i < HN; ++i) l[i] = 0.f;
      for (int t = walk.ta; t < walk.tb; ++t, ++it) {
        failed |= !wait_or_abort(cx, &m.s_full, it & 1, 40, t);
        tc_fence_after();
        uint32_t r[HN];
        ld_cols<N>(tm + lanes + TM_S + c0, r);
        ld_cols_wait<N>(r);
        tc_fence_before();
        if (lane == 0) mbar_arrive(&m.s_free);
        const int pos = t * kTile + key;
        float x[HN];
#pragma unroll
        for (int i = 0; i < HN; ++i) x[i] = __uint_as_float(r[i]) * p.scale2;
        if (t * kTile + kTile > t_draft) {              // the drafts' own tiles (and the end)
          const int d = pos - t_draft;
#pragma unroll
          for (int i = 0; i < HN; ++i) {
            bool see = pos < n;
            if (d >= 0 && see)
              see = p.mask ? (m.seen[c0 + i] >> d & 1) != 0 : d <= m.tok[c0 + i];
            x[i] = see ? x[i] : -CUDART_INF_F;
          }
        }
        bool over = failed;
#pragma unroll
        for (int i = 0; i < HN; i += 4) {
          const float4 f = ld_shared_f32x4(smem_u32(&m.ref[c0 + i]));
          over |= x[i] - f.x > kSlack || x[i + 1] - f.y > kSlack || x[i + 2] - f.z > kSlack ||
                  x[i + 3] - f.w > kSlack;
        }
        if (bar_any(barid, 128, over)) {
          if (bar_any(barid, 128, failed)) { dead = true; break; }
          // move the references to the maxima met so far
#pragma unroll
          for (int i = 0; i < HN; ++i) {
            const int w = __reduce_max_sync(0xffffffffu, ordered(x[i]));
            if (lane == 0) m.wmax[warp][i] = unordered(w);
          }
          named_sync(barid, 128);
          if (wt < HN) {
            float mx = m.ref[c0 + wt];
            const float old = mx;
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const float y = m.wmax[wg * 4 + w][wt];
              mx = y > mx || y != y ? y : mx;
            }
            m.ref[c0 + wt] = mx;
            m.fac[c0 + wt] = ex2(old - mx);
          }
          named_sync(barid, 128);
#pragma unroll
          for (int i = 0; i < HN; ++i) l[i] *= m.fac[c0 + i];
          if (t > walk.ta) {  // O^T has the tiles before: their products are done first
            failed |= !wait_or_abort(cx, &m.pv_done, (it - 1) & 1, 41, t);
            tc_fence_after();
#pragma unroll 1
            for (int mt = 0; mt < 4; ++mt) {
              uint32_t o[HN];
              ld_cols<N>(tm + lanes + TM_O + mt * N + c0, o);
              ld_cols_wait<N>(o);
#pragma unroll
              for (int i = 0; i < HN; ++i)
                o[i] = __float_as_uint(__uint_as_float(o[i]) * m.fac[c0 + i]);
              st_cols<N>(tm + lanes + TM_O + mt * N + c0, o);
            }
            tmem_st_wait();
          }
        }
#pragma unroll
        for (int i = 0; i < HN; i += 4) {
          const float4 f = ld_shared_f32x4(smem_u32(&m.ref[c0 + i]));
          x[i] = ex2(x[i] - f.x);
          x[i + 1] = ex2(x[i + 1] - f.y);
          x[i + 2] = ex2(x[i + 2] - f.z);
          x[i + 3] = ex2(x[i + 3] - f.w);
        }
#pragma unroll
        for (int i = 0; i < HN; ++i) l[i] += x[i];
        // P is free once the product of the tile before has read it
        if (it > 0) failed |= !wait_or_abort(cx, &m.pv_done, (it - 1) & 1, 42, t);
#pragma unroll
        for (int i = 0; i < HN; ++i) {
          const __nv_bfloat16 h = __float2bfloat16(x[i]);
          st_shared_b16(p_dst + sw128_offset(c0 + i, p_col), __bfloat16_as_ushort(h));
        }
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.p_ready);
      }
      if (dead) break;
      // ---- the segment's sums and output
      failed |= !wait_or_abort(cx, &m.pv_done, (it - 1) & 1, 43, seg);
      tc_fence_after();
      // row sums: over the warp's keys, then over the four warps
      if constexpr (HN == 48) {
        float l2[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) l2[i] = l[32 + i];
        const float a = warp_transpose_sum<32>(*reinterpret_cast<float(*)[32]>(&l[0]), lane);
        const float c = warp_transpose_sum<16>(l2, lane);
        m.wmax[warp][lane] = a;
        if ((lane & 1) == 0) m.wmax[warp][32 + (lane >> 1)] = c;
      } else {
        const float a = warp_transpose_sum<HN>(l, lane);
        if (lane % (32 / HN) == 0) m.wmax[warp][lane / (32 / HN)] = a;
      }
      if (bar_any(barid, 128, failed)) { dead = true; break; }
      const bool whole = walk.ta == 0 && walk.tb == key_tiles(n);
      const int first = seg == 0 ? 0 : 1;               // slot of a partial segment
      const int64_t slot = ((int64_t)rt * p.G + cta) * 2 + first;
      if (wt < HN) {
        const float s = m.wmax[wg * 4][wt] + m.wmax[wg * 4 + 1][wt] + m.wmax[wg * 4 + 2][wt] +
                        m.wmax[wg * 4 + 3][wt];
        const int rr = rt * N + c0 + wt;
        if (whole) {
          m.sum[c0 + wt] = s == 0.f ? 0.f : 1.f / s;
          if (p.lse && rr < p.T * p.H)
            p.lse[(int64_t)b * p.T * p.H + rr] =
                s == 0.f ? -CUDART_INF_F : (m.ref[c0 + wt] + __log2f(s)) * kLn2;
        } else {
          p.part_ml[slot * 192 + c0 + wt] = m.ref[c0 + wt];
          p.part_ml[slot * 192 + 96 + c0 + wt] = s;
        }
      }
      named_sync(barid, 128);
#pragma unroll 1
      for (int mt = 0; mt < 4; ++mt) {
        uint32_t o[HN];
        ld_cols<N>(tm + lanes + TM_O + mt * N + c0, o);
        ld_cols_wait<N>(o);
        const int ch = mt * 128 + key;
        if (whole) {
          // pairs of lanes exchange rows, so that each stores two channels of one row
          __nv_bfloat16 *dst = p.out + ((int64_t)b * p.T * p.H + rt * N + c0) * kLatentC;
#pragma unroll
          for (int i = 0; i < HN; i += 2) {
            const float a = __uint_as_float(o[i]) * m.sum[c0 + i];
            const float c = __uint_as_float(o[i + 1]) * m.sum[c0 + i + 1];
            const float got = __shfl_xor_sync(0xffffffffu, lane & 1 ? a : c, 1);
            const uint32_t w = lane & 1 ? pack_bf16x2(got, c) : pack_bf16x2(a, got);
            const int row = i + (lane & 1);
            if (rt * N + c0 + row < p.T * p.H)
              *reinterpret_cast<uint32_t *>(dst + (int64_t)row * kLatentC + (ch & ~1)) = w;
          }
        } else {
          float *dst = p.part_o + (slot * N + c0) * kLatentC + ch;
#pragma unroll
          for (int i = 0; i < HN; ++i) dst[(int64_t)i * kLatentC] = __uint_as_float(o[i]);
        }
      }
      tc_fence_before();
      ++seg;
    }
  }

  __syncwarp();
  __syncthreads();
  if (m.abort) {
    // nothing in flight outlives the CTA: the last copy into every slot, the last
    // Q, then the products
    if (tid == 32 * kLoadWarp) {
      const uint32_t pos = m.load_pos;
      for (uint32_t k = pos > S ? pos - S : 0; k < pos; ++k)
        mbar_wait(&m.full[k % S], (k / S) & 1, kWaitNs);
      if (m.load_seg > 0) mbar_wait(&m.q_full, (m.load_seg - 1) & 1, kWaitNs);
    }
    if (tid == 32 * kMmaWarp) {
      umma_commit(&m.fin);
      mbar_wait(&m.fin, 0, kWaitNs);
    }
    __syncthreads();
  }
  if (warp == kMmaWarp) {
    __syncwarp();
    tmem_dealloc(tm, tmem_cols(N));
  }
}

// Joins the parts of sequences that several CTAs shared, in the list's order, and
// writes the rows of empty sequences.  A warp per row and 128 channels; the parts
// are read kJoinBatch at a time, all loads of a batch in flight.
constexpr int kJoinRows = 2, kJoinBatch = 8;
template <int N>
__global__ void __launch_bounds__(128 * kJoinRows)
kda_latent_join_kernel(const Params p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.y, r = blockIdx.x * kJoinRows + (warp >> 2);
  const int ch = (warp & 3) * 128 + 4 * lane;
  const bool lead = threadIdx.x % 128 == 0;
  pdl_wait();
  if (r >= p.T * p.H) return;
  const int before = p.before[b], k = p.before[b + 1] - before, all = p.before[p.B];
  const int64_t row = (int64_t)b * p.T * p.H + r;
  uint2 *out = reinterpret_cast<uint2 *>(p.out + row * kLatentC + ch);
  if (k <= 0) {
    *out = make_uint2(0, 0);
    if (p.lse && lead) p.lse[row] = -CUDART_INF_F;
    return;
  }
  const int first = cta_of(before, p.G, all), last = cta_of(before + k - 1, p.G, all);
  if (first == last) return;             // one CTA had it all and wrote the output
  const int rt = r / N, col = r % N;
  // a CTA's first segment is in slot 0, its last in slot 1
  const int64_t slot0 = ((int64_t)rt * p.G + first) * 2;
  const int late = cta_begin(first, p.G, all) < before ? 1 : 0;
  const int parts = last - first + 1;
  auto slot_of = [&](int i) { return slot0 + 2 * i + (i == 0 ? late : 0); };
  float ref = kNoRef;
  for (int i = lane; i < parts; i += 32) {
    const float y = p.part_ml[slot_of(i) * 192 + col];
    ref = y > ref || y != y ? y : ref;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float y = __shfl_xor_sync(0xffffffffu, ref, o);
    ref = y > ref || y != y ? y : ref;
  }
  float sum = 0.f;
  float4 acc = make_float4(0, 0, 0, 0);
  for (int i0 = 0; i0 < parts; i0 += kJoinBatch) {
    float4 x[kJoinBatch];
    float f[kJoinBatch], l[kJoinBatch];
#pragma unroll
    for (int j = 0; j < kJoinBatch; ++j)
      if (i0 + j < parts) {
        const int64_t slot = slot_of(i0 + j);
        x[j] = *reinterpret_cast<const float4 *>(p.part_o + (slot * N + col) * kLatentC + ch);
        f[j] = p.part_ml[slot * 192 + col];
        l[j] = p.part_ml[slot * 192 + 96 + col];
      }
#pragma unroll
    for (int j = 0; j < kJoinBatch; ++j)
      if (i0 + j < parts) {
        const float w = ex2(f[j] - ref);
        sum += w * l[j];
        acc.x += w * x[j].x; acc.y += w * x[j].y; acc.z += w * x[j].z; acc.w += w * x[j].w;
      }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  *out = make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
  if (p.lse && lead) p.lse[row] = sum == 0.f ? -CUDART_INF_F : (ref + __log2f(sum)) * kLn2;
}

// Rows of a CTA: the fewest tiles of at most 96 rows, each as narrow as they allow.
int rows_per_tile(int rows) {
  const int tiles = (rows + 95) / 96, per = (rows + tiles - 1) / tiles;
  return per <= 16 ? 16 : per <= 32 ? 32 : per <= 64 ? 64 : 96;
}

struct Plan {
  int N, n_tiles, G;
};
Plan make_plan(int T, int H) {
  Plan pl;
  pl.N = rows_per_tile(T * H);
  pl.n_tiles = (T * H + pl.N - 1) / pl.N;
  const int sms = sm_count();
  pl.G = sms / pl.n_tiles;
  if (pl.G < 1) pl.G = 1;
  return pl;
}

// Partial results: none when one CTA has all keys of its rows.
size_t parts_of(const Plan &pl) { return pl.G > 1 ? (size_t)pl.n_tiles * pl.G * 2 : 0; }
size_t before_bytes(int32_t B) { return (((size_t)B + 1) * sizeof(int32_t) + 255) / 256 * 256; }

template <int N>
cudaError_t launch(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                   const Params &p, cudaStream_t stream) {
  auto kernel = kda_latent_decode_kernel<N>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       smem_bytes<N>());
  if (e != cudaSuccess) return e;
  kernel<<<p.G * p.n_tiles, kThreads, smem_bytes<N>(), stream>>>(mq, mk, mv, p);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const unsigned gx = (unsigned)((p.T * p.H + kJoinRows - 1) / kJoinRows);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(gx, (unsigned)p.B);
  cfg.blockDim = dim3(128 * kJoinRows);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kda_latent_join_kernel<N>, p);
}

}  // namespace

size_t latent_decode_scratch_bytes(int32_t B, int32_t T, int32_t H, int32_t dr) {
  (void)dr;
  const Plan pl = make_plan(T, H);
  return before_bytes(B) + parts_of(pl) * (192 + (size_t)pl.N * kLatentC) * sizeof(float);
}

cudaError_t launch_latent_decode(const LatentDecodeArgs &a, cudaStream_t stream) {
  if (a.B == 0) return cudaSuccess;
  if (!latent::encode_tiled()) return cudaErrorNotSupported;
  const Plan pl = make_plan(a.T, a.H);
  const int W = kLatentC + a.dr, rows = a.T * a.H;
  // Rows of a copied box: as many as lie in one page and one slot.
  int k_rows = 128;
  while (a.page_size % k_rows) k_rows >>= 1;
  const int v_rows = k_rows < 64 ? k_rows : 64;
  CUtensorMap mq, mk, mv;
  const cuuint64_t pool_rows = (cuuint64_t)a.n_pages * a.page_size;
  const cuuint64_t qd[3] = {(cuuint64_t)W, (cuuint64_t)rows, (cuuint64_t)a.B};
  const cuuint64_t qs[2] = {(cuuint64_t)W * 2, (cuuint64_t)W * 2 * rows};
  const cuuint32_t qb[3] = {64, (cuuint32_t)pl.N, 1};
  const cuuint64_t cd[2] = {(cuuint64_t)W, pool_rows}, cs[1] = {(cuuint64_t)W * 2};
  const cuuint32_t kb[2] = {64, (cuuint32_t)k_rows}, vb[2] = {64, (cuuint32_t)v_rows};
  if (!latent::make_bf16_map(&mq, a.q, 3, qd, qs, qb) ||
      !latent::make_bf16_map(&mk, a.cache, 2, cd, cs, kb) ||
      !latent::make_bf16_map(&mv, a.cache, 2, cd, cs, vb))
    return cudaErrorInvalidValue;
  Params p;
  p.table = a.block_table; p.lens = a.seq_lens; p.mask = a.tree_mask;
  p.B = a.B; p.T = a.T; p.H = a.H; p.W = W; p.n_pages = a.n_pages; p.page_size = a.page_size;
  p.max_pages = a.max_pages; p.k_rows = k_rows; p.v_rows = v_rows;
  p.n_tiles = pl.n_tiles; p.G = pl.G; p.scale2 = a.scale * kLog2e;
  p.out = static_cast<__nv_bfloat16 *>(a.out); p.lse = a.lse; p.status = a.status;
  p.before = static_cast<int32_t *>(a.scratch);
  p.part_ml = reinterpret_cast<float *>(static_cast<unsigned char *>(a.scratch) + before_bytes(a.B));
  p.part_o = p.part_ml + parts_of(pl) * 192;
  switch (pl.N) {
    case 16: return launch<16>(mq, mk, mv, p, stream);
    case 32: return launch<32>(mq, mk, mv, p, stream);
    case 64: return launch<64>(mq, mk, mv, p, stream);
    default: return launch<96>(mq, mk, mv, p, stream);
  }
}

}  // namespace kda
