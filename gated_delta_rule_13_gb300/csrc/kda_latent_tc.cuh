// What the tensor-core kernels of latent attention share: bounded waits with an
// abort flag, tiled copies, clusters, taking over blocks and tensor maps.
#pragma once

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "../../include/kda.h"
#include "kda_latent.h"
#include "kda_sm100.cuh"

namespace kda {
namespace latent {

using namespace sm100;

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// What makes up for the tensor cores' way to add, by which scores are multiplied.  They cut sums
// off: each of W / 16 steps loses half a unit in the last place on average, of a partial sum that
// on average is about half the whole.  A score of one sum of 512 or 576 channels comes out 7 to 10
// times 2^-24 of itself too near to zero (measured), and half as much where it is added up from
// `parts` = 2 sums of half the channels each.
inline double cut_off(int W, int parts) { return 1.0 + W / 16 * 0x1p-26 / parts; }
// Reference of a softmax row that has met no key yet: finite, so that masked
// scores (-inf) stay -inf against it, and below every real score.
constexpr float kNoRef = -3.0e38f;

// Thread-block clusters: an address of another CTA's shared memory, 16 bytes stored
// there asynchronously (counted by a barrier of the receiver), and an arrival on a
// barrier there.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
  return r;
}
__device__ __forceinline__ void st_async_v4(uint32_t dst, uint32_t a, uint32_t b, uint32_t c,
                                            uint32_t d, uint32_t bar) {
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, "
      "[%5];" ::"r"(dst),
      "r"(a), "r"(b), "r"(c), "r"(d), "r"(bar)
      : "memory");
}
// Without a release: what precedes it in the other direction must already have
// reached registers (a release at cluster scope takes about 1,700 cycles).
__device__ __forceinline__ void remote_arrive_relaxed(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar)
               : "memory");
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile(
      "barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
          : "memory");
}
// Work for a block that is done: a block of this grid that has not started is taken
// out of the launch.  take_block asks (16 bytes at dst, counted by the barrier);
// taken_block reads the answer, -1 when no block was left, after which there is no
// asking again.
__device__ __forceinline__ void take_block(uint32_t dst, uint64_t *bar) {
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 "
      "[%0], [%1];" ::"r"(dst),
      "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ int64_t taken_block(uint32_t src) {
  uint32_t any, x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b128 h;\n\tld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %0, 1, 0, p;\n\tmov.u32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, h;\n\t}"
      : "=r"(any), "=r"(x)
      : "r"(src)
      : "memory");
  return any ? (int64_t)x : -1;
}

__device__ __forceinline__ void mbar_inval(uint64_t *bar) {
  asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Where a wait gave up: the abort flag in shared memory ends every other wait of
// the block, so that each role leaves its loop.
struct WaitCtx {
  volatile int *abort;
  DeviceStatus *status;
  int chain;
  uint64_t wait_ns;
};
// kTimes: limits it waits.  A wait as long as a work item takes (kLongWaits) leaves it to
// those it waits for to give up first.
constexpr int kLongWaits = 32;
template <int kTimes = 1>
__device__ __forceinline__ bool wait_or_abort(const WaitCtx &cx, uint64_t *bar, uint32_t parity,
                                              int where, int step) {
  if (mbar_test_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 16; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*cx.abort) return false;
    if (global_timer_ns() - t0 > kTimes * cx.wait_ns) {
      record_device_status(cx.status, KDA_ERR_TIMEOUT, where, cx.chain, step);
      *cx.abort = 1;
      return false;
    }
  }
}

// The same by a converged warp, whose lanes leave together.
template <int kTimes = 1>
__device__ __forceinline__ bool warp_wait(const WaitCtx &cx, uint64_t *bar, uint32_t parity,
                                          int where, int step) {
  if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, wait_or_abort<kTimes>(cx, bar, parity, where, step)) != 0;
}

// For waits as long as a work item takes, by a warp that is in no hurry: it sleeps
// between looks.
__device__ __forceinline__ bool warp_wait_idle(const WaitCtx &cx, uint64_t *bar, uint32_t parity,
                                               int where, int step) {
  const uint64_t t0 = global_timer_ns();
  while (!__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) {
    if (__any_sync(0xffffffffu, *cx.abort)) return false;
    if (__any_sync(0xffffffffu, global_timer_ns() - t0 > kLongWaits * cx.wait_ns)) {
      record_device_status(cx.status, KDA_ERR_TIMEOUT, where, cx.chain, step);
      *cx.abort = 1;
      return false;
    }
    __nanosleep(200);
  }
  return true;
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const CUtensorMap *map, uint64_t *bar,
                                            int32_t c0, int32_t c1) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1)
      : "memory");
}
__device__ __forceinline__ void tma_load_3d_u(uint32_t dst, const CUtensorMap *map, uint64_t *bar,
                                              int32_t c0, int32_t c1, int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

// A shared-memory matrix descriptor (128-byte swizzle) as its two words, so that
// stepping along an operand is one 32-bit addition: the address sits in the low
// word in units of 16 bytes.
struct Desc {
  uint32_t lo, hi;
  __device__ __forceinline__ Desc(uint32_t addr, uint32_t lbo) {
    const uint64_t d = sdesc_sw128(addr, lbo, 1024);
    lo = (uint32_t)d;
    hi = (uint32_t)(d >> 32);
  }
  __device__ __forceinline__ uint64_t at(uint32_t bytes) const {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo + (bytes >> 4)), "r"(hi));
    return d;
  }
};

// A lane holds 64 bytes of row `lane` of 32 rows; they are stored at dst + row * stride
// (bytes), rows >= n_rows left out.  Four lanes exchange their pieces first, so that a
// store covers 64 consecutive bytes of eight rows and not 16 of each of the 32.
__device__ __forceinline__ uint4 shfl_xor(uint4 v, int mask) {
  v.x = __shfl_xor_sync(0xffffffffu, v.x, mask);
  v.y = __shfl_xor_sync(0xffffffffu, v.y, mask);
  v.z = __shfl_xor_sync(0xffffffffu, v.z, mask);
  v.w = __shfl_xor_sync(0xffffffffu, v.w, mask);
  return v;
}
__device__ __forceinline__ void store_rows(uint4 (&v)[4], void *dst, int64_t stride, int n_rows,
                                           int lane) {
#pragma unroll
  for (int b = 1; b < 4; b *= 2) {
    const bool high = lane & b;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j & b) continue;
      const uint4 got = shfl_xor(high ? v[j] : v[j + b], b);
      if (high) v[j] = got;
      else v[j + b] = got;
    }
  }
  unsigned char *to = static_cast<unsigned char *>(dst) + 16 * (lane & 3);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int row = (lane & ~3) + j;
    if (row < n_rows) *reinterpret_cast<uint4 *>(to + row * stride) = v[j];
  }
}

// Programmatic launch: the next kernel's blocks may start; wait for the previous grid.
__device__ __forceinline__ void pdl_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ uint32_t round_up_1k(uint32_t x) { return (x + 1023u) & ~1023u; }

inline PFN_cuTensorMapEncodeTiled_v12000 encode_tiled() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    cudaGetLastError();
    return static_cast<PFN_cuTensorMapEncodeTiled_v12000>(nullptr);
  }();
  return fn;
}

// bf16 map of `rank` dimensions (innermost first), strides in bytes of dimensions
// 1 .., 128-byte swizzle, zeros outside.
inline bool make_bf16_map(CUtensorMap *map, const void *base, uint32_t rank,
                          const cuuint64_t *dims, const cuuint64_t *strides,
                          const cuuint32_t *box) {
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  auto fn = encode_tiled();
  return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), dims,
                  strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// What the host asks of a device is asked once for each (a launch takes a few
// microseconds, and each of these calls one): value(device) for the current device.
constexpr int kMaxDevices = 64;
template <class F>
inline int per_device(std::atomic<int> (&cache)[kMaxDevices], F value) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (dev < 0 || dev >= kMaxDevices) return value(dev);
  int v = cache[dev].load(std::memory_order_relaxed);
  if (v == 0) {
    v = value(dev);
    cache[dev].store(v, std::memory_order_relaxed);
  }
  return v;
}

inline int sm_count() {
  static std::atomic<int> cache[kMaxDevices];
  return per_device(cache, [](int dev) {
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      sms = 0;
    }
    return sms;
  });
}

// The kernel may use `bytes` of dynamic shared memory and is launched with `regs`
// registers a thread at least (0: any).
template <auto kKernel>
inline bool kernel_ready(int bytes, int regs) {
  static std::atomic<int> cache[kMaxDevices];
  return per_device(cache, [=](int) {
    cudaFuncAttributes fa;
    if (cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) !=
            cudaSuccess ||
        cudaFuncGetAttributes(&fa, kKernel) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    return fa.numRegs >= regs ? 1 : 0;
  }) == 1;
}

}  // namespace latent
}  // namespace kda
