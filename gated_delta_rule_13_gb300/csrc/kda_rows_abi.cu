// C ABI of the operators around a cached latent row: argument validation and dispatch.
// See include/kda.h for the contract.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "../../include/kda.h"
#include "kda_rows.h"

namespace {

using kda::kStatusBytes;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
int cuda_result(cudaError_t e) {
  if (e == cudaSuccess) return KDA_OK;
  cudaGetLastError();
  return e == cudaErrorNotSupported ? KDA_ERR_UNSUPPORTED : KDA_ERR_CUDA;
}

// A strided [n, H, d] view; strides and sizes in elements of esz bytes.
struct View {
  const void *p;
  int64_t ts, hs, n, H, d, esz;
  bool empty() const { return !p || n == 0; }
  uintptr_t begin() const { return reinterpret_cast<uintptr_t>(p); }
  uintptr_t end() const { return begin() + ((n - 1) * ts + (H - 1) * hs + d) * esz; }
};

// What an address reaches, in bytes; larger spans and tensors are refused before 64 bits could
// not count them.
constexpr int64_t kReach = (int64_t)1 << 56;

// Strides that a row can be found with: none negative, and all rows of a view within reach.
bool strides_ok(const View &v) {
  const int64_t lim = (int64_t)1 << 40, reach = kReach / 16;   // elements; of tokens, of heads
  return v.ts >= 0 && v.hs >= 0 && v.ts < lim && v.hs < lim && (v.n <= 1 || v.ts <= reach / (v.n - 1)) &&
         (v.H <= 1 || v.hs <= reach / (v.H - 1));
}
// No two rows of a view that is written may meet.
bool rows_apart(const View &v) {
  if (v.H > 1 && v.hs < v.d) return false;
  if (v.n > 1 && v.ts < v.d) return false;
  return !(v.H > 1 && v.n > 1 && v.ts < (v.H - 1) * v.hs + v.d && v.hs < (v.n - 1) * v.ts + v.d);
}

// Whether views may have an element in common.  Where their spans meet, it is told for
// views whose tokens and heads are equally far apart, one stride spanning all rows of the
// other; other views count as meeting.
bool meet(const View &a, const View &b) {
  if (a.empty() || b.empty() || a.begin() >= b.end() || b.begin() >= a.end()) return false;
  if (a.esz != b.esz || (a.n > 1 && b.n > 1 && a.ts != b.ts) ||
      (a.H > 1 && b.H > 1 && a.hs != b.hs))
    return true;
  const int64_t bytes = (int64_t)(b.begin() - a.begin());
  if (bytes % a.esz != 0) return true;
  const int64_t dist = bytes / a.esz, d = a.d > b.d ? a.d : b.d;
  // A row of a and one of b lie dist - i ts - j hs apart, by the differences i and j of
  // their tokens and heads.
  struct Dim {
    int64_t stride, least, most;
  };
  const int64_t far = (int64_t)1 << 62;
  const Dim x = {a.n > 1 ? a.ts : b.n > 1 ? b.ts : far, -(b.n - 1), a.n - 1};
  const Dim y = {a.H > 1 ? a.hs : b.H > 1 ? b.hs : far, -(b.H - 1), a.H - 1};
  const Dim big = x.stride >= y.stride ? x : y, small = x.stride >= y.stride ? y : x;
  const int64_t reach = small.most > -small.least ? small.most : -small.least;
  if (small.stride < d || (small.stride < far && big.stride < far &&
                           big.stride < reach * small.stride + d))
    return true;
  const auto down = [](int64_t v, int64_t by) { return v / by - (v % by < 0); };
  for (int64_t i = down(dist, big.stride) - 1, n = 0; n < 3; ++n, ++i) {
    if (i < big.least || i > big.most) continue;
    const int64_t left = dist - i * big.stride;
    for (int64_t j = down(left, small.stride) - 1, m = 0; m < 3; ++m, ++j) {
      if (j < small.least || j > small.most) continue;
      const int64_t off = left - j * small.stride;
      if (off < a.d && -off < b.d) return true;
    }
  }
  return false;
}
bool same(const View &a, const View &b) {
  return a.p == b.p && (a.n <= 1 || a.ts == b.ts) && (a.H <= 1 || a.hs == b.hs);
}
View flat(const void *p, int64_t n, int64_t esz) { return {p, n, n, 1, 1, n, esz}; }
// An output against an input it may be (in place) or must be apart from.
bool clash(const View &out, const View &in) { return !same(out, in) && meet(out, in); }

bool finite(float x) { return x - x == 0.f; }

}  // namespace

extern "C" {

int kda_rope(const void *x, int64_t x_token_stride, int64_t x_head_stride, void *out,
             int64_t out_token_stride, int64_t out_head_stride, const void *k,
             int64_t k_token_stride, void *k_out, int64_t k_out_token_stride,
             const int32_t *positions, const double *inv_freq, int64_t n_tokens, int32_t H,
             int32_t dr, int interleaved, float scale, int transpose, int dtype, void *stream) {
  if (n_tokens < 0 || n_tokens > 0x7fffffffLL || H <= 0 || H > 65535 || dr <= 0 || dr % 2 != 0)
    return KDA_ERR_INVALID_ARG;
  if (dr > kda::kRopeMax || (dtype != KDA_F32 && dtype != KDA_BF16)) return KDA_ERR_UNSUPPORTED;
  if ((k != nullptr) != (k_out != nullptr) || !finite(scale)) return KDA_ERR_INVALID_ARG;
  if (n_tokens > 0 && (!x || !out || !positions || !inv_freq)) return KDA_ERR_INVALID_ARG;
  const int64_t esz = dtype == KDA_BF16 ? 2 : 4;
  for (const void *p : {x, (const void *)out, k, (const void *)k_out})
    if (!aligned(p, esz)) return KDA_ERR_INVALID_ARG;
  if (!aligned(positions, 4) || !aligned(inv_freq, 8)) return KDA_ERR_INVALID_ARG;
  const View vx = {x, x_token_stride, x_head_stride, n_tokens, H, dr, esz};
  const View vo = {out, out_token_stride, out_head_stride, n_tokens, H, dr, esz};
  const View vk = {k, k_token_stride, 0, n_tokens, 1, dr, esz};
  const View vko = {k_out, k_out_token_stride, 0, n_tokens, 1, dr, esz};
  for (const View &v : {vx, vo, vk, vko})
    if (!strides_ok(v)) return KDA_ERR_INVALID_ARG;
  if (!rows_apart(vo) || (k && !rows_apart(vko))) return KDA_ERR_INVALID_ARG;
  if (clash(vo, vx) || meet(vo, vk) || meet(vo, vko) || clash(vko, vk) || meet(vko, vx))
    return KDA_ERR_INVALID_ARG;
  for (const View &o : {vo, vko})
    if (meet(o, flat(positions, n_tokens * 4, 1)) || meet(o, flat(inv_freq, dr / 2 * 8, 1)))
      return KDA_ERR_INVALID_ARG;
  kda::RopeArgs a;
  a.x = x; a.out = out; a.x_ts = x_token_stride; a.x_hs = x_head_stride;
  a.o_ts = out_token_stride; a.o_hs = out_head_stride;
  a.k = k; a.k_out = k_out; a.k_ts = k_token_stride; a.ko_ts = k_out_token_stride;
  a.positions = positions; a.inv_freq = inv_freq; a.n = n_tokens; a.H = H; a.dr = dr;
  a.interleaved = interleaved != 0; a.transpose = transpose != 0; a.bf16 = dtype == KDA_BF16;
  a.scale = scale;
  return cuda_result(kda::launch_rope(a, static_cast<cudaStream_t>(stream)));
}

static int check_norm(int64_t n, int32_t W, int dtype) {
  if (n < 0 || n > 0x7fffffffLL || W <= 0) return KDA_ERR_INVALID_ARG;
  if (W > kda::kNormMax || (dtype != KDA_F32 && dtype != KDA_BF16)) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

int kda_norm_fwd(const void *x, int64_t x_row_stride, const float *weight, const float *bias,
                 int64_t n, int32_t W, int dtype, int center, float eps, void *out,
                 int64_t out_row_stride, float *mean, float *rstd, void *stream) {
  const int d = check_norm(n, W, dtype);
  if (d != KDA_OK) return d;
  if ((n > 0 && (!x || !out)) || (!center && mean) || !(eps > 0.f) || !finite(eps))
    return KDA_ERR_INVALID_ARG;
  const int64_t esz = dtype == KDA_BF16 ? 2 : 4;
  if (!aligned(x, esz) || !aligned(out, esz) || !aligned(weight, 4) || !aligned(bias, 4) ||
      !aligned(mean, 4) || !aligned(rstd, 4))
    return KDA_ERR_INVALID_ARG;
  const View vx = {x, x_row_stride, 0, n, 1, W, esz}, vo = {out, out_row_stride, 0, n, 1, W, esz};
  if (!strides_ok(vx) || !strides_ok(vo) || !rows_apart(vo) || clash(vo, vx))
    return KDA_ERR_INVALID_ARG;
  const View vm = flat(mean, n * 4, 1), vr = flat(rstd, n * 4, 1);
  const View vw = flat(weight, (int64_t)W * 4, 1), vb = flat(bias, (int64_t)W * 4, 1);
  for (const View &o : {vo, vm, vr})
    if (meet(o, vw) || meet(o, vb)) return KDA_ERR_INVALID_ARG;
  if (meet(vm, vr)) return KDA_ERR_INVALID_ARG;
  for (const View &o : {vm, vr})
    if (meet(o, vo) || meet(o, vx)) return KDA_ERR_INVALID_ARG;
  kda::NormArgs a;
  memset(&a, 0, sizeof(a));
  a.x = x; a.x_rs = x_row_stride; a.n = n; a.weight = weight; a.bias = bias; a.W = W;
  a.bf16 = dtype == KDA_BF16; a.center = center != 0; a.eps = eps; a.out = out;
  a.out_rs = out_row_stride; a.mean = mean; a.rstd = rstd;
  return cuda_result(kda::launch_norm_fwd(a, static_cast<cudaStream_t>(stream)));
}

int kda_norm_bwd_workspace_size(int64_t n, int32_t W, int dtype, size_t *bytes) {
  if (!bytes) return KDA_ERR_INVALID_ARG;
  const int d = check_norm(n, W, dtype);
  if (d != KDA_OK) return d;
  *bytes = kda::norm_bwd_scratch_bytes(n, W, dtype == KDA_BF16);
  return KDA_OK;
}

int kda_norm_bwd(const void *d_out, int64_t d_out_row_stride, const void *x, int64_t x_row_stride,
                 const float *weight, const float *mean, const float *rstd, int64_t n, int32_t W,
                 int dtype, void *d_x, int64_t d_x_row_stride, float *d_weight, float *d_bias,
                 void *workspace, size_t workspace_bytes, void *stream) {
  const int d = check_norm(n, W, dtype);
  if (d != KDA_OK) return d;
  if (n > 0 && (!d_out || !x || !rstd || !d_x)) return KDA_ERR_INVALID_ARG;
  const int64_t esz = dtype == KDA_BF16 ? 2 : 4;
  for (const void *p : {d_out, x, (const void *)d_x})
    if (!aligned(p, esz)) return KDA_ERR_INVALID_ARG;
  for (const float *p : {weight, mean, rstd, (const float *)d_weight, (const float *)d_bias})
    if (!aligned(p, 4)) return KDA_ERR_INVALID_ARG;
  const View vg = {d_out, d_out_row_stride, 0, n, 1, W, esz}, vx = {x, x_row_stride, 0, n, 1, W, esz};
  const View vd = {d_x, d_x_row_stride, 0, n, 1, W, esz};
  for (const View &v : {vg, vx, vd})
    if (!strides_ok(v)) return KDA_ERR_INVALID_ARG;
  if (!rows_apart(vd) || clash(vd, vg) || clash(vd, vx)) return KDA_ERR_INVALID_ARG;
  const View ins[] = {flat(weight, (int64_t)W * 4, 1), flat(mean, n * 4, 1), flat(rstd, n * 4, 1)};
  const View sums[] = {flat(d_weight, (int64_t)W * 4, 1), flat(d_bias, (int64_t)W * 4, 1)};
  for (const View &i : ins)
    if (meet(vd, i) || meet(sums[0], i) || meet(sums[1], i)) return KDA_ERR_INVALID_ARG;
  for (const View &o : sums)
    if (meet(o, vg) || meet(o, vx) || meet(o, vd)) return KDA_ERR_INVALID_ARG;
  if (meet(sums[0], sums[1])) return KDA_ERR_INVALID_ARG;
  const bool partial = d_weight || d_bias;
  const size_t need = partial ? kda::norm_bwd_scratch_bytes(n, W, dtype == KDA_BF16) : 0;
  if (need > 0 && (!workspace || !aligned(workspace, 16) || workspace_bytes < need))
    return KDA_ERR_WORKSPACE;
  kda::NormArgs a;
  memset(&a, 0, sizeof(a));
  a.x = x; a.x_rs = x_row_stride; a.n = n; a.weight = weight; a.W = W; a.bf16 = dtype == KDA_BF16;
  a.center = mean != nullptr; a.mean = const_cast<float *>(mean); a.rstd = const_cast<float *>(rstd);
  a.d_out = d_out; a.do_rs = d_out_row_stride; a.d_x = d_x; a.dx_rs = d_x_row_stride;
  a.d_weight = d_weight; a.d_bias = d_bias;
  a.partial = partial ? static_cast<float *>(workspace) : nullptr;
  return cuda_result(kda::launch_norm_bwd(a, static_cast<cudaStream_t>(stream)));
}

static int check_weights(int32_t B, int32_t T, int32_t H, int32_t dc, int32_t dr, int dtype) {
  if (B < 0 || B > 65535 || T <= 0 || H <= 0 || dc <= 0 || dr < 0 || (int64_t)T * H > (1 << 24) ||
      (int64_t)B * T * H > 0x7fffffffLL)
    return KDA_ERR_INVALID_ARG;
  if (dc != kda::kLatentC || (dr != 0 && dr != kda::kLatentRope) || dtype != KDA_BF16)
    return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

int kda_latent_weights_workspace_size(int32_t B, int32_t T, int32_t H, int32_t dc, int32_t dr,
                                      int dtype, size_t *bytes) {
  if (!bytes) return KDA_ERR_INVALID_ARG;
  const int d = check_weights(B, T, H, dc, dr, dtype);
  if (d != KDA_OK) return d;
  *bytes = kStatusBytes + round_up(kda::latent_weights_scratch_bytes(B, T, H, dr), 256);
  return KDA_OK;
}

int kda_latent_weights(const void *q, const void *cache, const int32_t *block_table,
                       const int32_t *seq_lens, const int64_t *tree_mask, const float *lse,
                       int32_t B, int32_t T, int32_t H, int32_t dc, int32_t dr, int32_t n_pages,
                       int32_t page_size, int32_t max_pages, int dtype, float scale, float decay,
                       float *weights, void *workspace, size_t workspace_bytes, void *stream) {
  const int d = check_weights(B, T, H, dc, dr, dtype);
  if (d != KDA_OK) return d;
  if (n_pages <= 0 || page_size <= 0 || page_size % 16 != 0 || max_pages <= 0 ||
      (int64_t)n_pages * page_size > 0x7fffffffLL || (int64_t)max_pages * page_size > (1 << 30))
    return KDA_ERR_INVALID_ARG;
  if (tree_mask && T > kda::kTreeMax) return KDA_ERR_INVALID_ARG;
  if (!cache || (B > 0 && (!q || !block_table || !seq_lens || !lse || !weights)))
    return KDA_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(cache, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(lse, 4) || !aligned(weights, 4) || !aligned(tree_mask, 8))
    return KDA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !finite(scale) || !(decay >= 0.f) || !finite(decay))
    return KDA_ERR_INVALID_ARG;
  const int64_t rows = (int64_t)B * T * H, cap = (int64_t)max_pages * page_size;
  const View out = flat(weights, B * cap * 4, 1);
  const View in[] = {flat(q, rows * (dc + dr) * 2, 1),
                     flat(cache, (int64_t)n_pages * page_size * (dc + dr) * 2, 1),
                     flat(block_table, (int64_t)B * max_pages * 4, 1),
                     flat(seq_lens, (int64_t)B * 4, 1), flat(lse, rows * 4, 1),
                     flat(tree_mask, (int64_t)B * T * 8, 1)};
  for (const View &v : in)
    if (meet(out, v)) return KDA_ERR_INVALID_ARG;
  const size_t need = kStatusBytes + round_up(kda::latent_weights_scratch_bytes(B, T, H, dr), 256);
  if (!workspace || !aligned(workspace, 16) || workspace_bytes < need) return KDA_ERR_WORKSPACE;
  unsigned char *ws = static_cast<unsigned char *>(workspace);
  kda::LatentWeightsArgs a;
  a.q = q; a.cache = cache; a.block_table = block_table; a.seq_lens = seq_lens;
  a.tree_mask = tree_mask; a.lse = lse; a.B = B; a.T = T; a.H = H; a.dr = dr; a.n_pages = n_pages;
  a.page_size = page_size; a.max_pages = max_pages; a.scale = scale; a.decay = decay;
  a.weights = weights;
  a.status = reinterpret_cast<kda::DeviceStatus *>(ws);
  a.scratch = ws + kStatusBytes;
  a.test = kda::take_wait_test(workspace);
  return cuda_result(kda::launch_latent_weights(a, static_cast<cudaStream_t>(stream)));
}

static int check_evict(int32_t L, int32_t B, int32_t budget) {
  return L < 1 || B < 0 || budget < 1 || budget > (1 << 30) || (int64_t)L * B > 0x7fffffffLL ||
                 (int64_t)L * B * budget > kReach / 16      // 12 bytes each in the workspace
             ? KDA_ERR_INVALID_ARG : KDA_OK;
}

int kda_cache_evict_workspace_size(int32_t L, int32_t B, int32_t budget, size_t *bytes) {
  if (!bytes) return KDA_ERR_INVALID_ARG;
  const int d = check_evict(L, B, budget);
  if (d != KDA_OK) return d;
  *bytes = kda::cache_evict_scratch_bytes(L, B, budget);
  return KDA_OK;
}

int kda_cache_evict(void *cache, const int32_t *block_table, const int32_t *seq_lens,
                    const float *weights, float *weights_out, int32_t L, int32_t n_pages,
                    int32_t page_size, int64_t row_bytes, int32_t B, int32_t max_pages,
                    int32_t budget, int32_t first, int32_t recent, int32_t *new_lens,
                    int32_t *origin, void *workspace, size_t workspace_bytes, int32_t *status,
                    void *stream) {
  const int d = check_evict(L, B, budget);
  if (d != KDA_OK) return d;
  if (n_pages <= 0 || page_size <= 0 || max_pages <= 0 || row_bytes <= 0 || row_bytes % 16 != 0 ||
      row_bytes > (1 << 30) || (int64_t)max_pages * page_size > (1 << 30) ||
      (int64_t)n_pages * page_size > 0x7fffffffLL || first < 0 ||
      recent < 0 || (int64_t)first + recent > budget)
    return KDA_ERR_INVALID_ARG;
  if (!cache || (B > 0 && (!block_table || !seq_lens || !weights || !weights_out || !new_lens ||
                           !origin)))
    return KDA_ERR_INVALID_ARG;
  if (!aligned(cache, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) ||
      !aligned(weights, 4) || !aligned(weights_out, 4) || !aligned(new_lens, 4) ||
      !aligned(origin, 4) || !aligned(status, 4))
    return KDA_ERR_INVALID_ARG;
  const int64_t all = (int64_t)L * B, cap = (int64_t)max_pages * page_size;
  const int64_t layer = (int64_t)n_pages * page_size * row_bytes;   // at most 2^61
  if (layer > kReach / L) return KDA_ERR_INVALID_ARG;
  const View vw = flat(weights, all * cap * 4, 1), vwo = flat(weights_out, all * cap * 4, 1);
  const View outs[] = {flat(cache, L * layer, 1), vwo,
                       flat(new_lens, (int64_t)B * 4, 1), flat(origin, all * budget * 4, 1)};
  const View in[] = {flat(block_table, (int64_t)B * max_pages * 4, 1),
                     flat(seq_lens, (int64_t)B * 4, 1), vw};
  for (int i = 0; i < 4; ++i) {
    for (const View &v : in)
      if (!(i == 1 && weights == weights_out && v.p == weights) && meet(outs[i], v))
        return KDA_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (meet(outs[i], outs[j])) return KDA_ERR_INVALID_ARG;
  }
  if (!workspace || !aligned(workspace, 16) ||
      workspace_bytes < kda::cache_evict_scratch_bytes(L, B, budget))
    return KDA_ERR_WORKSPACE;
  kda::CacheEvictArgs a;
  a.cache = cache; a.block_table = block_table; a.seq_lens = seq_lens; a.weights = weights;
  a.weights_out = weights_out; a.L = L; a.n_pages = n_pages; a.page_size = page_size; a.B = B;
  a.max_pages = max_pages; a.budget = budget; a.first = first; a.recent = recent;
  a.row_bytes = row_bytes; a.new_lens = new_lens; a.origin = origin;
  a.moves = static_cast<int32_t *>(workspace); a.status = status;
  return cuda_result(kda::launch_cache_evict(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
