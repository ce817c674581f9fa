// C ABI of the latent-attention and paged-cache operators: argument validation,
// workspace layout and dispatch.  See include/kda.h for the contract.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <atomic>

#include "../../include/kda.h"
#include "kda_latent.h"

namespace {

using kda::kStatusBytes;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

struct Range {
  const void *p;
  size_t n;
};
bool overlap(const Range &a, const Range &b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && a.n && b.n && x < y + b.n && y < x + a.n;
}
// No output may overlap an input or another output.
template <int NI, int NO>
bool any_overlap(const Range (&in)[NI], const Range (&out)[NO]) {
  for (int i = 0; i < NO; ++i) {
    for (const Range &r : in)
      if (overlap(out[i], r)) return true;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return true;
  }
  return false;
}

int check_sizes(int32_t n_seqs, int64_t n_q, int64_t n_k, int32_t H, int32_t dk, int32_t dr,
                int32_t dv, int dtype) {
  if (n_seqs < 1 || n_q < 0 || n_k < 0 || n_q > 0x7fffffffLL - 128 || n_k > 0x7fffffffLL - 128 ||
      H <= 0 || H > 65535 || dk <= 0 || dv <= 0 || dr < 0)
    return KDA_ERR_INVALID_ARG;
  if (dk != kda::kLatentD || dv != kda::kLatentD || (dr != 0 && dr != kda::kLatentRope) ||
      dtype != KDA_BF16)
    return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

size_t cu_bytes(int32_t n_seqs) { return round_up(sizeof(int32_t) * ((size_t)n_seqs + 1), 256); }
size_t base_bytes(int32_t n_seqs) { return kStatusBytes + 2 * cu_bytes(n_seqs); }

// Rows of a strided [n, H, 128] view: strides in elements, and the bytes from
// its first to its last element.
bool strides_ok(int64_t ts, int64_t hs, int32_t H, int64_t n) {
  if (ts % 8 != 0 || hs % 8 != 0 || ts <= 0 || hs <= 0) return false;
  const int64_t lim = (int64_t)1 << 39;  // tensor-map strides are below 2^40 bytes
  const int64_t reach = (int64_t)1 << 52;  // elements; of tokens, of heads: 64 bits count no more
  if (ts >= lim || hs >= lim || (n > 1 && ts > reach / (n - 1)) || (H > 1 && hs > reach / (H - 1)))
    return false;
  // rows must not overlap one another: heads inside a token or tokens inside a head
  const int64_t d = kda::kLatentD;
  if (H > 1 && hs < d) return false;
  if (n > 1 && ts < d) return false;
  return !(H > 1 && n > 1 && ts < (int64_t)(H - 1) * hs + d && hs < (n - 1) * ts + d);
}
size_t span_bytes(int64_t ts, int64_t hs, int32_t H, int64_t n) {
  return n == 0 ? 0 : (size_t)((n - 1) * ts + (int64_t)(H - 1) * hs + kda::kLatentD) * 2;
}

int cuda_result(cudaError_t e) {
  if (e == cudaSuccess) return KDA_OK;
  cudaGetLastError();
  return e == cudaErrorNotSupported ? KDA_ERR_UNSUPPORTED : KDA_ERR_CUDA;
}

// Whether two such views of equal strides have an element in common: whether their
// distance is, but for less than a row, a number of tokens plus a number of heads that
// both lie within a view.  One stride spans all rows of the other (strides_ok), so that
// two numbers of the longer and, for each, two of the shorter come into question.
bool views_overlap(const void *a, const void *b, int64_t ts, int64_t hs, int32_t H, int64_t n) {
  if (n == 0) return false;
  const int64_t far = (int64_t)1 << 62, d = kda::kLatentD;
  const int64_t dist = (int64_t)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a)) / 2;
  struct Dim {
    int64_t stride, count;
  } x = {n > 1 ? ts : far, n}, y = {H > 1 ? hs : far, H};
  const Dim big = x.stride >= y.stride ? x : y, small = x.stride >= y.stride ? y : x;
  auto down = [](int64_t v, int64_t by) { return v / by - (v % by < 0); };
  for (int64_t i = down(dist, big.stride), i1 = i + 1; i <= i1; ++i) {
    if (i <= -big.count || i >= big.count) continue;
    const int64_t left = dist - i * big.stride;
    for (int64_t j = down(left, small.stride), j1 = j + 1; j <= j1; ++j) {
      if (j <= -small.count || j >= small.count) continue;
      const int64_t off = left - j * small.stride;
      if (off > -d && off < d) return true;
    }
  }
  return false;
}

// Host arrays are validated and taken to `dst` (the caller may write or free them after
// the call, also between replays of a captured one); device arrays are used as they are.
int resolve_cu(const int32_t *cu, int32_t n_seqs, int64_t n, void *dst, cudaStream_t st,
               const int32_t **dev) {
  *dev = nullptr;
  if (!cu) return KDA_OK;  // one sequence
  cudaPointerAttributes attr;
  memset(&attr, 0, sizeof(attr));
  if (cudaPointerGetAttributes(&attr, cu) != cudaSuccess) {
    cudaGetLastError();
    return KDA_ERR_CUDA;
  }
  *dev = cu;
  if (attr.type == cudaMemoryTypeDevice || attr.type == cudaMemoryTypeManaged) return KDA_OK;
  if (cu[0] != 0 || cu[n_seqs] != n) return KDA_ERR_INVALID_ARG;
  for (int32_t s = 0; s < n_seqs; ++s)
    if (cu[s + 1] < cu[s]) return KDA_ERR_INVALID_ARG;
  int32_t *to = static_cast<int32_t *>(dst);
  *dev = to;
  return cuda_result(kda::put_ints(to, cu, (int64_t)n_seqs + 1, st));
}

// Fields, checks and device cu_seqlens shared by both directions.
int prepare(kda::LatentArgs &a, int32_t dk, int32_t dv, int dtype, const int32_t *cu_q,
            const int32_t *cu_k, const float *lse) {
  const int d = check_sizes(a.n_seqs, a.n_q, a.n_k, a.H, dk, a.dr, dv, dtype);
  if (d != KDA_OK) return d;
  if (((!cu_q || !cu_k) && a.n_seqs != 1) || (a.n_q > 0 && (!a.q || !a.out || !lse)) || (a.n_k > 0 && (!a.k || !a.v)) ||
      (a.n_k > 0 && (a.dr > 0) != (a.k_rope != nullptr)))
    return KDA_ERR_INVALID_ARG;
  for (const void *p : {a.q, a.k, a.v, a.k_rope, (const void *)a.out})
    if (!aligned(p, 16)) return KDA_ERR_INVALID_ARG;
  if (!aligned(lse, 4) || !aligned(cu_q, 4) || !aligned(cu_k, 4)) return KDA_ERR_INVALID_ARG;
  if (!(a.scale > 0.f) || isinf(a.scale)) return KDA_ERR_INVALID_ARG;
  if (!strides_ok(a.k_ts, a.k_hs, a.H, a.n_k) || !strides_ok(a.v_ts, a.v_hs, a.H, a.n_k))
    return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

// Resolves both cu_seqlens arrays.  The first kernel clears the status block; a
// call without queries has none.
int begin(kda::LatentArgs &a, const int32_t *cu_q, const int32_t *cu_k, unsigned char *ws,
          cudaStream_t st) {
  int r = a.n_q > 0 ? KDA_OK : cuda_result(cudaMemsetAsync(ws, 0, kStatusBytes, st));
  if (r == KDA_OK) r = resolve_cu(cu_q, a.n_seqs, a.n_q, ws + kStatusBytes, st, &a.cu_q);
  if (r == KDA_OK)
    r = resolve_cu(cu_k, a.n_seqs, a.n_k, ws + kStatusBytes + cu_bytes(a.n_seqs), st, &a.cu_k);
  a.status = reinterpret_cast<kda::DeviceStatus *>(ws);
  return r;
}

}  // namespace

// Test control of the waits: armed for one workspace, taken by the next call with it.
static std::atomic<const void *> g_test_workspace{nullptr};
static kda::WaitTest g_test;
kda::WaitTest kda::take_wait_test(const void *workspace) {
  const void *mine = workspace;
  if (g_test_workspace.load(std::memory_order_relaxed) == workspace &&
      g_test_workspace.compare_exchange_strong(mine, nullptr))
    return g_test;
  return {kda::kWaitNs, -1, -1};
}

extern "C" {

int kda_latent_fwd_workspace_size(int32_t n_seqs, int64_t n_q, int64_t n_k, int32_t H, int32_t dk,
                                  int32_t dr, int32_t dv, int dtype, size_t *bytes) {
  if (!bytes) return KDA_ERR_INVALID_ARG;
  const int d = check_sizes(n_seqs, n_q, n_k, H, dk, dr, dv, dtype);
  if (d != KDA_OK) return d;
  *bytes = base_bytes(n_seqs) + round_up(kda::latent_fwd_scratch_bytes(n_seqs, n_q, n_k, H), 256);
  return KDA_OK;
}

int kda_latent_fwd(const void *q, const void *k, const void *v, const void *k_rope,
                   int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                   int64_t v_head_stride, const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                   int32_t n_seqs, int64_t n_q, int64_t n_k, int32_t H, int32_t dk, int32_t dr,
                   int32_t dv, int dtype, float scale, int causal, void *out, float *lse,
                   void *workspace, size_t workspace_bytes, void *stream) {
  kda::LatentArgs a;
  memset(&a, 0, sizeof(a));
  a.q = q; a.k = k; a.v = v; a.k_rope = k_rope;
  a.k_ts = k_token_stride; a.k_hs = k_head_stride; a.v_ts = v_token_stride; a.v_hs = v_head_stride;
  a.n_seqs = n_seqs; a.n_q = n_q; a.n_k = n_k; a.H = H; a.dr = dr;
  a.scale = scale; a.causal = causal != 0; a.out = out; a.lse = lse;
  const int d = prepare(a, dk, dv, dtype, cu_seqlens_q, cu_seqlens_k, lse);
  if (d != KDA_OK) return d;
  const size_t rows = (size_t)n_q * H;
  const Range in[] = {{q, rows * (dk + dr) * 2},
                      {k, span_bytes(a.k_ts, a.k_hs, H, n_k)},
                      {v, span_bytes(a.v_ts, a.v_hs, H, n_k)},
                      {k_rope, (size_t)n_k * dr * 2}};
  const Range outs[] = {{out, rows * dv * 2}, {lse, rows * 4}};
  if (any_overlap(in, outs)) return KDA_ERR_INVALID_ARG;
  const size_t scratch = round_up(kda::latent_fwd_scratch_bytes(n_seqs, n_q, n_k, H), 256);
  if (!workspace || !aligned(workspace, 16) || workspace_bytes < base_bytes(n_seqs) + scratch)
    return KDA_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  unsigned char *ws = static_cast<unsigned char *>(workspace);
  const int r = begin(a, cu_seqlens_q, cu_seqlens_k, ws, st);
  if (r != KDA_OK) return r;
  a.scratch = ws + base_bytes(n_seqs);
  a.test = kda::take_wait_test(workspace);
  return cuda_result(kda::launch_latent_fwd(a, st));
}

int kda_latent_bwd_workspace_size(int32_t n_seqs, int64_t n_q, int64_t n_k, int32_t H, int32_t dk,
                                  int32_t dr, int32_t dv, int dtype, size_t *bytes) {
  if (!bytes) return KDA_ERR_INVALID_ARG;
  const int d = check_sizes(n_seqs, n_q, n_k, H, dk, dr, dv, dtype);
  if (d != KDA_OK) return d;
  *bytes = base_bytes(n_seqs) + round_up(kda::latent_bwd_scratch_bytes(n_seqs, n_q, n_k, H, dr), 256);
  return KDA_OK;
}

int kda_latent_bwd(const void *q, const void *k, const void *v, const void *k_rope,
                   int64_t k_token_stride, int64_t k_head_stride, int64_t v_token_stride,
                   int64_t v_head_stride, const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k,
                   int32_t n_seqs, int64_t n_q, int64_t n_k, int32_t H, int32_t dk, int32_t dr,
                   int32_t dv, int dtype, float scale, int causal, const void *out,
                   const float *lse, const void *d_out, void *dq, void *d_k, void *d_v,
                   void *d_k_rope, int64_t dk_token_stride, int64_t dk_head_stride,
                   int64_t dv_token_stride, int64_t dv_head_stride, void *workspace,
                   size_t workspace_bytes, void *stream) {
  kda::LatentArgs a;
  memset(&a, 0, sizeof(a));
  a.q = q; a.k = k; a.v = v; a.k_rope = k_rope;
  a.k_ts = k_token_stride; a.k_hs = k_head_stride; a.v_ts = v_token_stride; a.v_hs = v_head_stride;
  a.n_seqs = n_seqs; a.n_q = n_q; a.n_k = n_k; a.H = H; a.dr = dr;
  a.scale = scale; a.causal = causal != 0;
  a.out = const_cast<void *>(out); a.lse = const_cast<float *>(lse);
  a.d_out = d_out; a.dq = dq; a.dk = d_k; a.dv = d_v; a.d_k_rope = d_k_rope;
  a.dk_ts = dk_token_stride; a.dk_hs = dk_head_stride;
  a.dv_ts = dv_token_stride; a.dv_hs = dv_head_stride;
  const int d = prepare(a, dk, dv, dtype, cu_seqlens_q, cu_seqlens_k, lse);
  if (d != KDA_OK) return d;
  if ((n_q > 0 && (!d_out || !dq)) || (n_k > 0 && (!d_k || !d_v)) ||
      (n_k > 0 && (dr > 0) != (d_k_rope != nullptr)))
    return KDA_ERR_INVALID_ARG;
  for (const void *p : {d_out, (const void *)dq, (const void *)d_k, (const void *)d_v,
                        (const void *)d_k_rope})
    if (!aligned(p, 16)) return KDA_ERR_INVALID_ARG;
  if (!strides_ok(a.dk_ts, a.dk_hs, H, n_k) || !strides_ok(a.dv_ts, a.dv_hs, H, n_k))
    return KDA_ERR_INVALID_ARG;
  const size_t rows = (size_t)n_q * H;
  const Range in[] = {{q, rows * (dk + dr) * 2},
                      {k, span_bytes(a.k_ts, a.k_hs, H, n_k)},
                      {v, span_bytes(a.v_ts, a.v_hs, H, n_k)},
                      {k_rope, (size_t)n_k * dr * 2},
                      {out, rows * dv * 2},
                      {lse, rows * 4},
                      {d_out, rows * dv * 2}};
  // d_k and d_v may be two interleaved views of one tensor: their spans are checked
  // against everything but each other, their rows against each other's where the
  // strides are equal, as those of such views are.
  const Range o1[] = {{dq, rows * (dk + dr) * 2}, {d_k_rope, (size_t)n_k * dr * 2},
                      {d_k, span_bytes(a.dk_ts, a.dk_hs, H, n_k)}};
  const Range o2[] = {{dq, rows * (dk + dr) * 2}, {d_k_rope, (size_t)n_k * dr * 2},
                      {d_v, span_bytes(a.dv_ts, a.dv_hs, H, n_k)}};
  const bool alike = (n_k <= 1 || a.dk_ts == a.dv_ts) && (H <= 1 || a.dk_hs == a.dv_hs);
  if (any_overlap(in, o1) || any_overlap(in, o2) || (n_k > 0 && d_k == d_v) ||
      (alike && views_overlap(d_k, d_v, a.dk_ts, a.dk_hs, H, n_k)))
    return KDA_ERR_INVALID_ARG;
  const size_t scratch = round_up(kda::latent_bwd_scratch_bytes(n_seqs, n_q, n_k, H, dr), 256);
  if (!workspace || !aligned(workspace, 16) || workspace_bytes < base_bytes(n_seqs) + scratch)
    return KDA_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  unsigned char *ws = static_cast<unsigned char *>(workspace);
  const int r = begin(a, cu_seqlens_q, cu_seqlens_k, ws, st);
  if (r != KDA_OK) return r;
  a.scratch = ws + base_bytes(n_seqs);
  a.test = kda::take_wait_test(workspace);
  return cuda_result(kda::launch_latent_bwd(a, st));
}

static int check_decode(int32_t B, int32_t T, int32_t H, int32_t dc, int32_t dr, int dtype) {
  if (B < 0 || B > 65535 || T <= 0 || H <= 0 || dc <= 0 || dr < 0 || (int64_t)T * H > (1 << 24) ||
      (int64_t)B * T * H > 0x7fffffffLL)
    return KDA_ERR_INVALID_ARG;
  if (dc != kda::kLatentC || (dr != 0 && dr != kda::kLatentRope) || dtype != KDA_BF16)
    return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

int kda_latent_decode_workspace_size(int32_t B, int32_t T, int32_t H, int32_t dc, int32_t dr,
                                     int dtype, size_t *bytes) {
  if (!bytes) return KDA_ERR_INVALID_ARG;
  const int d = check_decode(B, T, H, dc, dr, dtype);
  if (d != KDA_OK) return d;
  *bytes = kStatusBytes + round_up(kda::latent_decode_scratch_bytes(B, T, H, dr), 256);
  return KDA_OK;
}

int kda_latent_decode(const void *q, const void *cache, const int32_t *block_table,
                      const int32_t *seq_lens, const int64_t *tree_mask, int32_t B, int32_t T,
                      int32_t H, int32_t dc, int32_t dr, int32_t n_pages, int32_t page_size,
                      int32_t max_pages, int dtype, float scale, void *out, float *lse,
                      void *workspace, size_t workspace_bytes, void *stream) {
  const int d = check_decode(B, T, H, dc, dr, dtype);
  if (d != KDA_OK) return d;
  if (n_pages <= 0 || page_size <= 0 || page_size % 16 != 0 || max_pages <= 0 ||
      (int64_t)n_pages * page_size > 0x7fffffffLL || (int64_t)max_pages * page_size > 0x7fffffffLL)
    return KDA_ERR_INVALID_ARG;
  if (tree_mask && T > kda::kTreeMax) return KDA_ERR_INVALID_ARG;
  if (!cache || (B > 0 && (!q || !block_table || !seq_lens || !out))) return KDA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(out, 16) || !aligned(block_table, 4) ||
      !aligned(seq_lens, 4) || !aligned(lse, 4) || !aligned(tree_mask, 8))
    return KDA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || isinf(scale)) return KDA_ERR_INVALID_ARG;
  const size_t rows = (size_t)B * T * H;
  const Range in[] = {{q, rows * (dc + dr) * 2},
                      {cache, (size_t)n_pages * page_size * (dc + dr) * 2},
                      {block_table, (size_t)B * max_pages * 4},
                      {seq_lens, (size_t)B * 4},
                      {tree_mask, (size_t)B * T * 8}};
  const Range outs[] = {{out, rows * dc * 2}, {lse, rows * 4}};
  if (any_overlap(in, outs)) return KDA_ERR_INVALID_ARG;
  const size_t need =
      kStatusBytes + round_up(kda::latent_decode_scratch_bytes(B, T, H, dr), 256);
  if (!workspace || !aligned(workspace, 16) || workspace_bytes < need) return KDA_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  unsigned char *ws = static_cast<unsigned char *>(workspace);
  kda::LatentDecodeArgs a;
  a.q = q; a.cache = cache; a.block_table = block_table; a.seq_lens = seq_lens;
  a.tree_mask = tree_mask; a.B = B; a.T = T; a.H = H; a.dr = dr; a.n_pages = n_pages;
  a.page_size = page_size; a.max_pages = max_pages; a.scale = scale; a.out = out; a.lse = lse;
  a.status = reinterpret_cast<kda::DeviceStatus *>(ws);
  a.scratch = ws + kStatusBytes;
  a.test = kda::take_wait_test(workspace);
  return cuda_result(kda::launch_latent_decode(a, st));
}

int kda_latent_test_timeout(const void *workspace, int32_t block, int32_t tile, uint32_t wait_us) {
  if (!workspace || (block >= 0 && (tile < 0 || wait_us < 1 || wait_us > 2000000)))
    return KDA_ERR_INVALID_ARG;
  g_test_workspace.store(nullptr);
  if (block < 0) return KDA_OK;
  g_test = {1000ull * wait_us, block, tile};
  g_test_workspace.store(workspace);
  return KDA_OK;
}

int kda_cache_write(void *cache, const void *rows, int64_t rows_layer_stride,
                    int64_t rows_seq_stride, int64_t rows_token_stride, const int32_t *block_table,
                    const int32_t *start, const int32_t *path, const int32_t *n_write, int32_t L,
                    int32_t n_pages, int32_t page_size, int64_t row_bytes, int32_t B, int32_t T,
                    int32_t max_pages, int32_t *status, void *stream) {
  if (L < 0 || B < 0 || T <= 0 || T > 1024 || n_pages <= 0 || page_size <= 0 || max_pages <= 0 ||
      row_bytes <= 0 || row_bytes % 16 != 0)
    return KDA_ERR_INVALID_ARG;
  if (!cache || (!rows && !path) || (B > 0 && (!block_table || !start))) return KDA_ERR_INVALID_ARG;
  if (!aligned(cache, 16) || !aligned(rows, 16) || !aligned(block_table, 4) || !aligned(start, 4) ||
      !aligned(path, 4) || !aligned(n_write, 4) || !aligned(status, 4))
    return KDA_ERR_INVALID_ARG;
  if (rows) {
    for (const int64_t s : {rows_layer_stride, rows_seq_stride, rows_token_stride})
      if (s < 0 || s % 16 != 0) return KDA_ERR_INVALID_ARG;
    if (L > 0 && B > 0) {
      const Range r = {rows, (size_t)((L - 1) * rows_layer_stride + (B - 1) * rows_seq_stride +
                                      (T - 1) * rows_token_stride + row_bytes)};
      const Range c = {cache, (size_t)L * n_pages * page_size * row_bytes};
      if (overlap(r, c)) return KDA_ERR_INVALID_ARG;
    }
  }
  kda::CacheWriteArgs a;
  a.cache = cache; a.rows = rows; a.rows_ls = rows_layer_stride; a.rows_bs = rows_seq_stride;
  a.rows_ts = rows_token_stride; a.block_table = block_table; a.start = start; a.path = path;
  a.n_write = n_write; a.L = L; a.n_pages = n_pages; a.page_size = page_size;
  a.row_bytes = row_bytes; a.B = B; a.T = T; a.max_pages = max_pages; a.status = status;
  return cuda_result(kda::launch_cache_write(a, static_cast<cudaStream_t>(stream)));
}

int kda_cache_copy_pages(void *cache, const int32_t *src, const int32_t *dst, int32_t n, int32_t L,
                         int32_t n_pages, int64_t page_bytes, int32_t *status, void *stream) {
  if (n < 0 || L < 0 || n_pages <= 0 || page_bytes <= 0 || page_bytes % 16 != 0)
    return KDA_ERR_INVALID_ARG;
  if (!cache || (n > 0 && (!src || !dst))) return KDA_ERR_INVALID_ARG;
  if (!aligned(cache, 16) || !aligned(src, 4) || !aligned(dst, 4) || !aligned(status, 4))
    return KDA_ERR_INVALID_ARG;
  return cuda_result(kda::launch_cache_copy_pages(cache, src, dst, n, L, n_pages, page_bytes, status,
                                                  static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
