// Latent attention in its expanded form (kda_latent_fwd), tcgen05 / TMEM / TMA,
// sm_103a.
//
// Per (sequence, head): o_i = sum_j softmax_j(scale [q_i] . [k_j; k_rope_j]) v_j
// over the allowed keys.  A 256 x 128 tile of (query, key) pairs costs
// 2 * 256 * 128 * (128 + dr + 128) operations, 2,560 cycles of an SM's tensor
// cores at dr = 64, and reads 80 KB of keys and values: the matrix rate is the
// bound, then the exponentials (32,768 a tile).
//
// One CTA takes 256 consecutive queries of a head, as two tiles of 128.  While one
// tile's softmax runs on four warps, the tensor cores work for the other tile:
//   S_t = Q_t K^T     (shared-memory operands, 128 x 128 fp32 in TMEM)
//   P_t               bf16, written by the softmax over S_t's own columns
//   O_t += P_t V      (P_t from TMEM)
// so TMEM holds exactly S_0, S_1, O_0, O_1.  A thread owns a query row.  The softmax is
// the one-pass form of Milakov and Gimelshein ("Online normalizer calculation for
// softmax", 2018), with a reference that need not be the maximum: it only moves when a
// score exceeds it by more than 8 (log2).  O_t is then rescaled in TMEM, which after
// the first tiles hardly ever happens.  P is rounded to bf16 (half a step, 2^-8 of the
// value) because it is an operand of the tensor cores; its sum, the reference and O
// are fp32.
//
// Work items are (256 queries, head).  They run in groups of as many heads as fill the
// SMs once, inside a group longest first: a group's keys are read by its tiles at
// about the same time, and the last items to start are short ones.  What does not fill
// the SMs a whole time at the end has its keys shared out over the idle ones; these
// items leave (reference, sum, O) in the workspace and a second small kernel joins
// them (2048 queries over 32768 keys, 96 heads: 768 items on 152 SMs are five rounds
// and eight items, which as a sixth round cost a fifth of the time).
//
// Keys and values stream through a ring of 16 KB slots: 64-channel blocks of 128
// keys, 64-key x 128-channel blocks of values.
//
// A block that is through with its item takes over a block of the grid that has not
// started (the hardware's work stealing, so the order of the items is kept and no
// counter has to be reset): the next queries and keys are loaded, and the next scores
// computed, beside the last products and the output.  4 x 4096 tokens, 16 heads: 247
// us with a block for each item, 237 so.
//
// Measured (2,070 MHz, L2 warm, replayed): 4 x 4096 tokens, 16 heads, dr = 64: 237 us,
// 1.45 PFLOP/s, tensor cores busy 63 % of the time, DRAM 15 %.  2048 queries over 32768
// keys, 96 heads, dr = 0: 1,950 us, 1.64 PFLOP/s.  Whole calls on cold inputs, as a
// layer finds them: 254 and 2,077 us, 1.35 and 1.54 PFLOP/s.  What bounds it are the
// products with their waits: without the softmax (time only, warm) it takes 217 and
// 1,650 us, without the copies of keys and values 227 and 1,876.  A step of 256 x 128
// pairs at dr = 64 moves about 345 KB through shared memory (operands of the products
// and copies), 2,690 cycles at 128 bytes a cycle beside 2,560 of matrix work.
// Handing P over in quarters (253 us), exponentials before the maximum is known (247)
// and an issuing warp for each query tile (243; 2,150 for the second) were slower.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math_constants.h>
#include <string.h>

#include "kda_latent_tc.cuh"

namespace kda {
namespace {

using namespace latent;

constexpr int kRows = 256, kKeys = 128;
constexpr int kThreads = 384;            // two softmax warpgroups; loader, MMA, cleaner, items
constexpr int kLoadWarp = 8, kMmaWarp = 9, kCleanWarp = 10, kItemWarp = 11;
constexpr uint32_t kSlotBytes = 16384;
constexpr uint32_t kSmemMax = 232448;
constexpr float kSlack = 8.f;            // log2 units a score may exceed its reference by
// 168 registers a thread at launch: 256 x 208 + 128 x 88 = 384 x 168
constexpr uint32_t kLaunchRegs = 168, kSoftmaxRegs = 208, kIssueRegs = 88;
constexpr int kMaxSlots = 10;

// A unit of the ring is a key tile (KB slots) or a value tile (2 slots); units are
// loaded, used and released in the order K0 V0 K1 V1 .., so the barriers of eight
// consecutive units are enough (at most five are resident).
constexpr uint32_t kUnits = 8;
constexpr int kItemUsers = 11;           // loader, MMA, cleaner, eight softmax warps

// What a block works on: a tile of a sequence, a head, and part `part` of `parts` of
// its keys; seq < 0: nothing.
struct Item {
  SeqTile tile;
  int head, part, parts, slot;           // slot: of its partial results
  int i0, n_iter, nt[2];                 // key tiles [i0, i0 + n_iter); of each query tile
  int row0, last_live;                   // first query; keys of the last tile
};

struct Shared {
  uint64_t full[kUnits], empty[kUnits];
  uint64_t q_full[2], q_free[2], s_full[2], p_ready[2][2], o_full[2], clean_req[2], clean[2];
  uint64_t item_full[2], item_free[2], want, taken, fin;
  alignas(16) uint32_t answer[4];
  uint32_t tmem;
  uint32_t loaded, loaded_q[2];                // units loaded, tiles of queries loaded
  int abort;
  Item item[2];
};

template <int DR>
constexpr uint32_t q_bytes() { return kRows * (kLatentD + DR) * 2; }
template <int DR>
constexpr int slots() {
  const int n = (int)((kSmemMax - 1024 - sizeof(Shared) - q_bytes<DR>()) / kSlotBytes);
  return n > kMaxSlots ? kMaxSlots : n;
}
template <int DR>
constexpr uint32_t smem_bytes() {
  return 1024 + q_bytes<DR>() + slots<DR>() * kSlotBytes + sizeof(Shared);
}

// Key tiles before an item's last, the next item is asked for: finding it takes about
// 2 us.  (4 x 4096 tokens: 240 us; 242 with 2, 244 with 1.)
constexpr int kAhead = 4;
constexpr int kMinPart = 4;              // key tiles of a part, at least

struct Params : Packed {
  int32_t split;                         // whether keys may be shared out
  float scale2;
  int causal;
  __nv_bfloat16 *out;
  float *lse;
  DeviceStatus *status;
  float *part_o;                         // [slot][2][128 / 4 channels][128 rows][4]
  float *part_ml;                        // [slot][2][2][128]
  WaitTest test;
};

// Key tiles of query tile t (of 128) of a work item.
__device__ __forceinline__ int key_tiles(const SeqTile &st, int row0, int t, int causal) {
  const int first = row0 + 128 * t;
  if (st.seq < 0 || first >= st.nq) return 0;
  int n = st.nk;
  if (causal) n = min(n, min(first + 128, st.nq) + st.nk - st.nq);
  return n <= 0 ? 0 : (n + kKeys - 1) / kKeys;
}
// First query of a work item: the last queries of a sequence, which see the most
// keys, come first.
__device__ __forceinline__ int first_row(const SeqTile &st) {
  return (st.n_tiles - 1 - st.tile) * kRows;
}

// Items of whole rounds run undivided, one a block; item `whole` + j of the `rest` in
// `ways` parts each (fewer when its keys are few).
struct Rounds {
  int64_t whole;
  int rest, ways;
  __device__ Rounds(const Params &p, int64_t items) {
    whole = p.split ? items / p.sms * p.sms : items;
    rest = (int)(items - whole);
    ways = rest > 0 ? p.sms / rest : 1;
  }
};
__device__ __forceinline__ int parts_of(const SeqTile &st, int ways, int causal) {
  const int row0 = first_row(st);
  const int n = max(key_tiles(st, row0, 0, causal), key_tiles(st, row0, 1, causal));
  return max(1, min(ways, n / kMinPart));
}

__device__ inline Item find_item(const Params &p, int64_t block) {
  Item it;
  it.tile.seq = -1; it.tile.bad = 0; it.tile.n_tiles = it.tile.tile = 0;
  it.tile.q0 = it.tile.nq = it.tile.k0 = it.tile.nk = 0;
  it.head = it.part = it.slot = 0;
  it.parts = 1;
  const LaneSeqs seqs(p);
  const int64_t tiles = count_tiles(p, seqs, kTileA);
  if (tiles < 0) it.tile.bad = 1;
  if (tiles <= 0) return it;
  const Rounds r(p, tiles * p.H);
  if (block < r.whole) {
    it.tile = place_item(p, seqs, kTileA, (uint32_t)tiles, (uint32_t)block, &it.head);
  } else if (block - r.whole < (int64_t)r.rest * r.ways) {
    it.slot = (int)(block - r.whole);
    it.tile = place_item(p, seqs, kTileA, (uint32_t)tiles, (uint32_t)(r.whole + it.slot / r.ways),
                         &it.head);
    it.part = it.slot % r.ways;
    it.parts = parts_of(it.tile, r.ways, p.causal);
    if (it.part >= it.parts) it.tile.seq = -1;
  }
  it.row0 = first_row(it.tile);
  // Key tiles [i0, i0 + n_iter) of this part, and those of the two query tiles among
  // them (the second never has fewer, unless it has no queries).
  const int all0 = key_tiles(it.tile, it.row0, 0, p.causal);
  const int all1 = key_tiles(it.tile, it.row0, 1, p.causal);
  const int n_all = max(all0, all1);
  it.i0 = (int)((int64_t)n_all * it.part / it.parts);
  const int i1 = (int)((int64_t)n_all * (it.part + 1) / it.parts);
  it.nt[0] = max(0, min(all0, i1) - it.i0);
  it.nt[1] = max(0, min(all1, i1) - it.i0);
  it.n_iter = i1 - it.i0;
  it.last_live = min(kKeys, it.tile.nk - (i1 - 1) * kKeys);
  return it;
}

// kTest: the form for a test of the waits.  (Read from a parameter, the bound on the waits
// costs the ordinary form 2 %: 1,850 and 1,896 us for 2048 queries over 32768 keys.)
template <int DR, bool kTest>
__global__ void __launch_bounds__(kThreads, 1)
kda_latent_fwd_kernel(const __grid_constant__ CUtensorMap map_q,
                      const __grid_constant__ CUtensorMap map_k,
                      const __grid_constant__ CUtensorMap map_r,
                      const __grid_constant__ CUtensorMap map_v, const Params p) {
  constexpr int S = slots<DR>();
  constexpr int KB = (kLatentD + DR) / 64;   // 64-channel blocks of a key
  constexpr int PER = KB + 2;                // slots of a key tile
  constexpr uint32_t kRing = q_bytes<DR>();
  constexpr uint32_t kQTile = 128 * 128;     // bytes of a 128-row block
  constexpr uint32_t ID_S = idesc_bf16(128, 128, false, false);
  constexpr uint32_t ID_PV = idesc_bf16(128, 128, false, true);

  extern __shared__ unsigned char raw[];
  const uint32_t base = round_up_1k(smem_u32(raw));
  unsigned char *const tiles = raw + (base - smem_u32(raw));
  Shared &m = *reinterpret_cast<Shared *>(tiles + kRing + S * kSlotBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (uint32_t i = 0; i < kUnits; ++i) {
      mbar_init(&m.full[i], 1);
      mbar_init(&m.empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&m.q_full[t], 1);
      mbar_init(&m.q_free[t], 1);
      mbar_init(&m.s_full[t], 1);
      mbar_init(&m.p_ready[t][0], 4);
      mbar_init(&m.p_ready[t][1], 4);
      mbar_init(&m.o_full[t], 1);
      mbar_init(&m.clean_req[t], 1);
      mbar_init(&m.clean[t], 1);
      mbar_init(&m.item_full[t], 1);
      mbar_init(&m.item_free[t], kItemUsers);
    }
    mbar_init(&m.want, 1);
    mbar_init(&m.taken, 1);
    mbar_init(&m.fin, 1);
    m.abort = 0;
    m.loaded = m.loaded_q[0] = m.loaded_q[1] = 0;
    fence_mbarrier_init();
  }
  if (warp == kLoadWarp && lane == 0) {
    prefetch_tensormap(&map_q);
    prefetch_tensormap(&map_k);
    prefetch_tensormap(&map_v);
    if (DR) prefetch_tensormap(&map_r);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&m.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = m.tmem;
  const WaitCtx cx{&m.abort, p.status, (int)blockIdx.x, kTest ? p.test.wait_ns : kWaitNs};
  pdl_launch_dependents();

  if (warp >= 8) {
    setmaxnreg_dec<kIssueRegs>();
    if (warp == kItemWarp) {
      // ---- items: finds what a block of the grid works on, and takes over the next
      // block when the loader is about to be through with this one
      int64_t block = blockIdx.x;
      int asked = 0, k = 0;
      for (bool ok = true; ok;) {
        Item it;
        it.tile.seq = -1;
        if (block >= 0) {
          it = find_item(p, block);
          // every block sees a malformed array; block 0 says so, or clears the status
          // (a wait that gives up does so seconds later)
          if (block == 0 && lane == 0)
            set_device_status(p.status, it.tile.bad ? KDA_ERR_INVALID_ARG : KDA_OK, it.tile.bad);
        }
        if (block < 0 || it.tile.seq >= 0) {
          if (k >= 2) ok = warp_wait_idle(cx, &m.item_free[k & 1], ((k >> 1) - 1) & 1, 50, k);
          if (!ok) break;
          if (lane == 0) {
            m.item[k & 1] = it;
            mbar_arrive(&m.item_full[k & 1]);
          }
          if (block < 0) break;
          ok = warp_wait_idle(cx, &m.want, k & 1, 51, k);
          ++k;
          if (!ok) break;
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(&m.taken, 16);
          take_block(smem_u32(m.answer), &m.taken);
        }
        __syncwarp();
        // the answer is waited for whatever else fails: it is written to this block
        ok = __all_sync(0xffffffffu, mbar_wait(&m.taken, asked & 1, kWaitNs));
        ++asked;
        if (!ok) {
          if (lane == 0) record_device_status(p.status, KDA_ERR_TIMEOUT, 52, (int)blockIdx.x, k);
          *(volatile int *)&m.abort = 1;
          break;
        }
        block = taken_block(smem_u32(m.answer));
        fence_proxy_async_smem();
        __syncwarp();
      }
    } else if (warp == kLoadWarp && lane == 0) {
      // ---- loader
      // Slots [at, at + PER) hold key tile i and its values; before a unit is loaded,
      // the last unit that had one of its slots has been released.
      bool ok = true;
      uint32_t at = 0;
      uint32_t u = 0, cleans = 0;
      uint32_t q_loads[2] = {0, 0};
      auto before = [&](int count) {  // slots `at` .. `at + count` of unit u
        // unit of slot position end - S, where positions run on without wrapping
        const int end = (int)(u >> 1) * PER + (int)(u & 1) * KB + count - 1 - S;
        if (end < 0) return;
        const int v = end / PER * 2 + (end % PER >= KB ? 1 : 0);
        ok = wait_or_abort(cx, &m.empty[v % kUnits], (v / kUnits) & 1, 10, u);
      };
      auto next = [&]() {
        const uint32_t dst = base + kRing + at * kSlotBytes;
        at = at + 1 == S ? 0 : at + 1;
        return dst;
      };
      for (int k = 0; ok; ++k) {
        ok = wait_or_abort(cx, &m.item_full[k & 1], (k >> 1) & 1, 11, k);
        if (!ok) break;
        const Item &item = m.item[k & 1];
        const int seq = item.tile.seq, head = item.head, n_iter = item.n_iter;
        if (seq < 0) break;
        const int halves_last = item.last_live > 64 ? 2 : 1;
        const int nt1 = item.nt[1], nt0 = item.nt[0], q_row = item.tile.q0 + item.row0;
        const int key0 = item.tile.k0 + item.i0 * kKeys;
        const bool clean = (item.last_live & 63) != 0;
        auto load_q = [&](int t) {
          // the item before has read its queries
          if (q_loads[t] > 0) ok = wait_or_abort(cx, &m.q_free[t], (q_loads[t] - 1) & 1, 12, k);
          if (!ok) return;
          ++q_loads[t];
          mbar_arrive_expect_tx(&m.q_full[t], KB * kQTile);
          for (int kb = 0; kb < KB; ++kb)
            tma_load_3d_u(base + (t * KB + kb) * kQTile, &map_q, &m.q_full[t], 64 * kb, head,
                          q_row + 128 * t);
        };
        if (nt0 > 0) load_q(0);
        if (n_iter == 0) mbar_arrive(&m.want);
        for (int i = 0; ok && i < n_iter; ++i) {
          // early enough for the next item's queries to follow this one's last keys
          if (i == max(0, n_iter - kAhead)) mbar_arrive(&m.want);
          const int key = key0 + i * kKeys;
          if (kTest && k == 0 && i == p.test.tile && p.test.block == (int)blockIdx.x) {
            ok = false;                    // the waits for this tile run out
            break;
          }
          before(KB);
          if (!ok) break;
          uint64_t *bar = &m.full[u % kUnits];
          mbar_arrive_expect_tx(bar, KB * kSlotBytes);
          for (int kb = 0; kb < KB; ++kb) {
            if (kb < 2) tma_load_3d_u(next(), &map_k, bar, 64 * kb, head, key);
            else tma_load_2d(next(), &map_r, bar, 64 * (kb - 2), key);
          }
          ++u;
          if (i == 0 && nt1 > 0) load_q(1);
          if (ok) before(2);
          if (!ok) break;
          const int halves = i + 1 < n_iter ? 2 : halves_last;
          bar = &m.full[u % kUnits];
          mbar_arrive_expect_tx(bar, halves * kSlotBytes);
          for (int hf = 0; hf < 2; ++hf) {
            const uint32_t dst = next();
            if (hf >= halves) continue;
            tma_load_3d_u(dst, &map_v, bar, 0, head, key + 64 * hf);
            tma_load_3d_u(dst + 8192, &map_v, bar, 64, head, key + 64 * hf);
          }
          ++u;
        }
        if (ok && n_iter > 0 && clean) mbar_arrive(&m.clean_req[cleans++ & 1]);
        mbar_arrive(&m.item_free[k & 1]);
      }
      m.loaded = u;
      m.loaded_q[0] = q_loads[0];
      m.loaded_q[1] = q_loads[1];
    } else if (warp == kMmaWarp && elect_one()) {
      // ---- MMA issue, by the elected lane (elect.sync lets the compiler keep the
      // descriptors in uniform registers: 270 us against 441 under lane == 0 with
      // descriptors built for each product, and 311 with the warp converged and a
      // branch per product; 4 x 4096 tokens, 16 heads)
      bool ok = true;
      const Desc ring_k(base + kRing, 16), ring_v(base + kRing, 8192);
      uint32_t u0 = 0, cleans = 0;               // units and cleaned tiles of items before
      int seen[2] = {0, 0}, q_seen[2] = {0, 0};  // key tiles and queries of items before
      uint32_t at = 0;                           // first slot of key tile i
      for (int k = 0; ok; ++k) {
        ok = wait_or_abort(cx, &m.item_full[k & 1], (k >> 1) & 1, 26, k);
        if (!ok || m.item[k & 1].tile.seq < 0) break;
        const int n_iter = m.item[k & 1].n_iter, last_live = m.item[k & 1].last_live;
        const int nt[2] = {m.item[k & 1].nt[0], m.item[k & 1].nt[1]};
        mbar_arrive(&m.item_free[k & 1]);
        const bool last_half = last_live > 64, clean = (last_live & 63) != 0;
        const int last_user = nt[1] > 0 ? 1 : 0;   // releases the units
        auto issue_s = [&](int t, int i, uint32_t at) {  // at: first slot of key tile i
          const Desc a(base + t * KB * kQTile, 16);
          const uint32_t u = u0 + 2 * i;
          ok = wait_or_abort(cx, &m.full[u % kUnits], (u / kUnits) & 1, 20, i);
          if (!ok) return;
#pragma unroll
          for (int kb = 0; kb < KB; ++kb) {
            const uint32_t off = at * kSlotBytes;
            at = at + 1 == S ? 0 : at + 1;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              umma_ss(tm + 128 * t, a.at(kb * kQTile + ks * 32), ring_k.at(off + ks * 32), ID_S,
                      kb + ks > 0);
          }
          if (t == last_user) umma_commit(&m.empty[u % kUnits]);
          umma_commit(&m.s_full[t]);
          if (i + 1 == nt[t]) umma_commit(&m.q_free[t]);
        };
        auto issue_pv = [&](int t, int i, uint32_t at) {  // at: first slot of value tile i
          const uint32_t u = u0 + 2 * i + 1;
          const bool last = i + 1 == n_iter;
          ok = wait_or_abort(cx, &m.full[u % kUnits], (u / kUnits) & 1, 21, i);
          // the last tile's rows past the sequence have been zeroed
          if (ok && last && clean)
            ok = wait_or_abort(cx, &m.clean[cleans & 1], (cleans >> 1) & 1, 22, i);
          ok = ok && wait_or_abort(cx, &m.p_ready[t][0], (seen[t] + i) & 1, 23, i);
          if (!ok) return;
          tc_fence_after();
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)
            umma_ts(tm + 256 + 128 * t, tm + 128 * t + 8 * ks,
                    ring_v.at(at * kSlotBytes + ks * 2048), ID_PV, i + ks > 0);
          at = at + 1 == S ? 0 : at + 1;
          ok = wait_or_abort(cx, &m.p_ready[t][1], (seen[t] + i) & 1, 24, i);
          if (!ok) return;
          tc_fence_after();
          if (!last || last_half) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              umma_ts(tm + 256 + 128 * t, tm + 128 * t + 32 + 8 * ks,
                      ring_v.at(at * kSlotBytes + ks * 2048), ID_PV, 1);
          }
          if (t == last_user) umma_commit(&m.empty[u % kUnits]);
        };
        // S of the first tiles follows the item before's last products, which are read
        // out of O while it runs
#pragma unroll
        for (int t = 0; t < 2; ++t)
          if (ok && nt[t] > 0) {
            ok = wait_or_abort(cx, &m.q_full[t], q_seen[t]++ & 1, 25, t);
            if (ok) issue_s(t, 0, at);
          }
        for (int i = 0; ok && i < n_iter; ++i) {
          const uint32_t at_v = at + KB >= S ? at + KB - S : at + KB;
          const uint32_t at_n = at + PER >= S ? at + PER - S : at + PER;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (!ok || i >= nt[t]) continue;
            issue_pv(t, i, at_v);
            if (!ok) continue;
            if (i + 1 < nt[t]) {
              issue_s(t, i + 1, at_n);
            } else {
              umma_commit(&m.o_full[t]);
            }
          }
          at = at_n;
        }
        u0 += 2 * n_iter;
        seen[0] += nt[0];
        seen[1] += nt[1];
        if (n_iter > 0 && clean) ++cleans;
      }
    } else if (warp == kCleanWarp) {
      // ---- cleaner: value rows past the sequence's end are another sequence's, and
      // may hold anything; zero them (0 * NaN would reach the sum).  The loader asks
      // once the copies of the last tile are under way.  It may ask for the next item
      // too before this one's tile is used, but no further (the item after that is only
      // published when all softmax warps are through with this one): two barriers each.
      int tiles_before = 0, cleans = 0;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        ok = warp_wait_idle(cx, &m.item_full[k & 1], (k >> 1) & 1, 32, k);
        if (!ok || m.item[k & 1].tile.seq < 0) break;
        const int n_iter = m.item[k & 1].n_iter, last_live = m.item[k & 1].last_live;
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.item_free[k & 1]);
        tiles_before += n_iter;
        const int from = last_live & 63;
        if (n_iter == 0 || from == 0) continue;
        const int u = 2 * tiles_before - 1, halves_last = last_live > 64 ? 2 : 1;
        ok = warp_wait_idle(cx, &m.clean_req[cleans & 1], (cleans >> 1) & 1, 30, n_iter);
        ok = ok && warp_wait(cx, &m.full[u % kUnits], (u / kUnits) & 1, 31, n_iter);
        if (!ok) break;
        const uint32_t s = ((uint32_t)(tiles_before - 1) * PER + KB + halves_last - 1) % S;
        const uint32_t dst = base + kRing + s * kSlotBytes + from * 128;
        for (int j = lane; j < (64 - from) * 8; j += 32) {
          st_shared_v4(dst + j * 16, 0, 0, 0, 0);
          st_shared_v4(dst + 8192 + j * 16, 0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&m.clean[cleans & 1]);
        ++cleans;
      }
    }
  } else {
    setmaxnreg_inc<kSoftmaxRegs>();
    // ---- softmax and output: thread = query row
    const int t = warp >> 2, r = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t tm_s = tm + lanes + 128 * t, tm_o = tm + lanes + 256 + 128 * t;
    int done = 0, outs = 0;                              // key tiles and outputs of items before
    bool ok = true;
    for (int k = 0; ok; ++k) {
      ok = warp_wait(cx, &m.item_full[k & 1], (k >> 1) & 1, 42, k);
      const Item &item = m.item[k & 1];                    // read where needed: few registers
      const SeqTile &st = item.tile;
      if (!ok || st.seq < 0) break;
      const int row = item.row0 + 128 * t + r;             // of the sequence
      const int n_t = item.nt[t];
      // keys this row sees, counted from the first of the part
      int limit = st.nk;
      if (p.causal) limit = min(limit, row + st.nk - st.nq + 1);
      limit -= item.i0 * kKeys;
      float ref = kNoRef, l = 0.f;
      for (int i = 0; i < n_t; ++i) {
        ok = warp_wait(cx, &m.s_full[t], (done + i) & 1, 40, i);
        if (!ok) break;
        tc_fence_after();
        uint32_t x[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tm_s + 32 * c, x[c]);
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_wait(x[c]);
        const int seen = limit - i * kKeys;                // columns below it are allowed
        if (__any_sync(0xffffffffu, seen < kKeys)) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (32 * c + j >= seen) x[c][j] = __float_as_uint(-CUDART_INF_F);
        }
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          mx[c] = __uint_as_float(x[c][0]);
#pragma unroll
          for (int j = 1; j < 32; ++j) mx[c] = fmaxf(mx[c], __uint_as_float(x[c][j]));
        }
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale2;
        if (__any_sync(0xffffffffu, top > ref + kSlack)) {
          const float now = fmaxf(ref, top), f = ex2(ref - now);
          ref = now;
          l *= f;
          if (i > 0) {
            // S of this tile was issued after the product of the tile before, so its
            // completion covers that product
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t o[32];
              tmem_ld32(tm_o + 32 * c, o);
              tmem_ld_wait(o);
#pragma unroll
              for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
              tmem_st32(tm_o + 32 * c, o);
            }
          }
        }
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float a = ex2(fmaf(__uint_as_float(x[c][j]), p.scale2, -ref));
            const float b = ex2(fmaf(__uint_as_float(x[c][j + 1]), p.scale2, -ref));
            sum[(j >> 1) & 3] += a + b;
            pk[j / 2] = pack_bf16x2(a, b);
          }
          tmem_st16(tm_s + 16 * c, pk);
          if (c & 1) {  // 64 keys are ready for their product
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&m.p_ready[t][c >> 1]);
          }
        }
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      }
      // ---- output
      if (ok && n_t > 0) ok = warp_wait(cx, &m.o_full[t], outs & 1, 41, n_t);
      if (!ok) break;
      if (n_t > 0) tc_fence_after();
      done += n_t;
      outs += n_t > 0;
      const bool live = row < st.nq;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int64_t at = (int64_t)item.slot * 2 + t;       // of a part
      const int64_t to = (st.q0 + row) * (int64_t)p.H + item.head;
      if (item.parts > 1) {
        p.part_ml[at * 256 + r] = ref;
        p.part_ml[at * 256 + 128 + r] = l;
      } else if (live) {
        p.lse[to] = l == 0.f ? -CUDART_INF_F : (ref + log2f(l)) * kLn2;
      }
      const bool parts = item.parts > 1;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        uint32_t o[32];
        if (n_t > 0) {
          tmem_ld32(tm_o + 32 * c, o);
          tmem_ld_wait(o);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = 0;
        }
        if (parts) {  // four channels of the 32 rows beside one another
          uint4 *w = reinterpret_cast<uint4 *>(p.part_o) + (at * (kLatentD / 4) + 8 * c) * 128 + r;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            w[j * 128] = make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
        } else if (live) {
          uint4 *w = reinterpret_cast<uint4 *>(p.out + to * kLatentD) + 4 * c;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t b[4];
#pragma unroll
            for (int j = 0; j < 4; ++j)
              b[j] = pack_bf16x2(__uint_as_float(o[8 * q + 2 * j]) * inv,
                                 __uint_as_float(o[8 * q + 2 * j + 1]) * inv);
            w[q] = make_uint4(b[0], b[1], b[2], b[3]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&m.item_free[k & 1]);
    }
  }

  __syncwarp();
  __syncthreads();
  if (m.abort) {  // nothing in flight outlives the CTA
    if (tid == 32 * kLoadWarp) {
      const uint32_t u = m.loaded;
      for (uint32_t v = u > kUnits ? u - kUnits : 0; v < u; ++v)
        mbar_wait(&m.full[v % kUnits], (v / kUnits) & 1, kWaitNs);
      for (int t = 0; t < 2; ++t)
        if (m.loaded_q[t] > 0) mbar_wait(&m.q_full[t], (m.loaded_q[t] - 1) & 1, kWaitNs);
    }
    if (warp == kMmaWarp && elect_one()) {  // of the lane that issued the products
      umma_commit(&m.fin);
      mbar_wait(&m.fin, 0, kWaitNs);
    }
    __syncthreads();
  }
  if (warp == kMmaWarp) {
    __syncwarp();
    tmem_dealloc(tm, 512);
  }
}

// Joins the parts of divided items in their order.  Block (x: 32 rows, y: item); a lane
// is a row, a warp 16 channels, four parts in flight: it waits for memory (20 us beside
// the 1,850 of the case above, 8 items in 19 parts each).
__global__ void __launch_bounds__(256) kda_latent_fwd_join_kernel(const Params p) {
  __shared__ Item s_item;
  __shared__ int s_ways;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  if (warp == 0) {
    Item it;
    it.tile.seq = -1;
    it.parts = 1;
    int ways = 1;
    const LaneSeqs seqs(p);
    const int64_t tiles = count_tiles(p, seqs, kTileA);
    if (tiles > 0) {
      const Rounds r(p, tiles * p.H);
      ways = r.ways;
      if ((int)blockIdx.y < r.rest) {
        it.tile = place_item(p, seqs, kTileA, (uint32_t)tiles, (uint32_t)(r.whole + blockIdx.y),
                             &it.head);
        it.parts = parts_of(it.tile, r.ways, p.causal);
      }
    }
    if (lane == 0) {
      s_item = it;
      s_ways = ways;
    }
  }
  __syncthreads();
  const Item it = s_item;
  if (it.tile.seq < 0 || it.parts < 2) return;
  const int t = blockIdx.x >> 2, r = (blockIdx.x & 3) * 32 + lane;
  const int row = first_row(it.tile) + 128 * t + r;
  if (row >= it.tile.nq) return;
  const int64_t slot0 = (int64_t)blockIdx.y * s_ways;
  float ref = kNoRef, l = 0.f, o[16];
#pragma unroll
  for (int c = 0; c < 16; ++c) o[c] = 0.f;
#pragma unroll 4
  for (int i = 0; i < it.parts; ++i) {
    const int64_t at = (slot0 + i) * 2 + t;
    const float4 *x =
        reinterpret_cast<const float4 *>(p.part_o) + (at * (kLatentD / 4) + 4 * warp) * 128 + r;
    float4 v[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = x[c * 128];
    const float m = p.part_ml[at * 256 + r], s = p.part_ml[at * 256 + 128 + r];
    const float now = m > ref || m != m ? m : ref;
    const float a = ex2(ref - now), b = ex2(m - now);
    ref = now;
    l = l * a + s * b;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      o[4 * c] = o[4 * c] * a + v[c].x * b;
      o[4 * c + 1] = o[4 * c + 1] * a + v[c].y * b;
      o[4 * c + 2] = o[4 * c + 2] * a + v[c].z * b;
      o[4 * c + 3] = o[4 * c + 3] * a + v[c].w * b;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t at = (it.tile.q0 + row) * (int64_t)p.H + it.head;
  uint32_t w[8];
#pragma unroll
  for (int c = 0; c < 8; ++c) w[c] = pack_bf16x2(o[2 * c] * inv, o[2 * c + 1] * inv);
  uint4 *to = reinterpret_cast<uint4 *>(p.out + at * kLatentD + 16 * warp);
  to[0] = make_uint4(w[0], w[1], w[2], w[3]);
  to[1] = make_uint4(w[4], w[5], w[6], w[7]);
  if (warp == 0) p.lse[at] = l == 0.f ? -CUDART_INF_F : (ref + log2f(l)) * kLn2;
}

// Whether any item can have keys enough for two parts (lengths are on the device).
bool may_split(int64_t n_k) { return n_k >= (2 * kMinPart - 1) * kKeys + 1; }

template <int DR>
cudaError_t launch(const LatentArgs &a, cudaStream_t stream) {
  CUtensorMap mq, mk, mr, mv;
  const cuuint64_t W = kLatentD + DR, H = a.H;
  const cuuint64_t qd[3] = {W, H, (cuuint64_t)a.n_q}, qs[2] = {W * 2, H * W * 2};
  const cuuint64_t nk = a.n_k > 0 ? a.n_k : 1;
  const cuuint64_t kd[3] = {kLatentD, H, nk};
  const cuuint64_t ks[2] = {(cuuint64_t)a.k_hs * 2, (cuuint64_t)a.k_ts * 2};
  const cuuint64_t vs[2] = {(cuuint64_t)a.v_hs * 2, (cuuint64_t)a.v_ts * 2};
  const cuuint64_t rd[2] = {64, nk}, rs[1] = {128};
  const cuuint32_t b128[3] = {64, 1, 128}, b64[3] = {64, 1, 64}, br[2] = {64, 128};
  memset(&mr, 0, sizeof(mr));
  // without keys nothing is loaded; the maps only need a valid base
  const void *any = a.q;
  if (!make_bf16_map(&mq, a.q, 3, qd, qs, b128) ||
      !make_bf16_map(&mk, a.n_k > 0 ? a.k : any, 3, kd, ks, b128) ||
      !make_bf16_map(&mv, a.n_k > 0 ? a.v : any, 3, kd, vs, b64) ||
      (DR && !make_bf16_map(&mr, a.n_k > 0 ? a.k_rope : any, 2, rd, rs, br)))
    return cudaErrorInvalidValue;
  const bool test = a.test.block >= 0;
  auto kernel = test ? kda_latent_fwd_kernel<DR, true> : kda_latent_fwd_kernel<DR, false>;
  // the register split must not exceed what the block is launched with
  if (!(test ? kernel_ready<kda_latent_fwd_kernel<DR, true>>(smem_bytes<DR>(), kLaunchRegs)
             : kernel_ready<kda_latent_fwd_kernel<DR, false>>(smem_bytes<DR>(), kLaunchRegs)))
    return cudaErrorNotSupported;
  Params p;
  p.cu_q = a.cu_q; p.cu_k = a.cu_k; p.n_seqs = a.n_seqs; p.H = a.H;
  p.sms = max(1, sm_count());
  p.rows[kTileA] = kRows;
  p.by_key[kTileA] = false;
  p.rows[kTileB] = p.rows[kTileC] = 0;
  p.n_q = a.n_q; p.n_k = a.n_k;
  cudaError_t e = launch_latent_plan(p, a.scratch, a.status, stream);
  if (e != cudaSuccess) return e;
  unsigned char *parts = static_cast<unsigned char *>(a.scratch) + latent_plan_bytes(a.n_seqs);
  p.split = may_split(a.n_k) && p.sms > 1;
  p.part_ml = reinterpret_cast<float *>(parts);
  p.part_o = p.part_ml + (int64_t)p.sms * 2 * 256;
  p.scale2 = a.scale * kLog2e; p.causal = a.causal;
  p.out = static_cast<__nv_bfloat16 *>(a.out); p.lse = a.lse; p.status = a.status;
  p.test = a.test;
  // as many items as there can be (one sequence: exactly that many), and the parts
  const int64_t tiles = a.n_seqs == 1 ? (a.n_q + kRows - 1) / kRows : a.n_q / kRows + a.n_seqs;
  const int64_t blocks = tiles * a.H + (p.split ? p.sms : 0);
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  kernel<<<(unsigned)blocks, kThreads, smem_bytes<DR>(), stream>>>(mq, mk, mr, mv, p);
  e = cudaGetLastError();
  if (e != cudaSuccess || !p.split) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kRows / 32, (unsigned)(tiles * a.H < p.sms ? tiles * a.H : p.sms));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kda_latent_fwd_join_kernel, p);
}

}  // namespace

size_t latent_fwd_scratch_bytes(int32_t n_seqs, int64_t n_q, int64_t n_k, int32_t H) {
  (void)H;
  const size_t plan = latent_plan_bytes(n_seqs);
  if (n_q == 0 || !may_split(n_k)) return plan;
  const int sms = sm_count();
  return plan + (size_t)(sms > 1 ? sms : 1) * 2 * (256 + 128 * kLatentD) * sizeof(float);
}

cudaError_t launch_latent_fwd(const LatentArgs &a, cudaStream_t stream) {
  if (a.n_q == 0) return cudaSuccess;
  if (!latent::encode_tiled()) return cudaErrorNotSupported;
  return a.dr ? launch<64>(a, stream) : launch<0>(a, stream);
}

}  // namespace kda
