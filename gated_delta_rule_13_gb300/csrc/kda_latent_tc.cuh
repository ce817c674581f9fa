// What the tensor-core kernels of latent attention share: bounded waits with an
// abort flag, tiled copies, block reductions and tensor maps.
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

constexpr uint64_t kWaitNs = 2000000000ull;  // limit of any wait in these kernels
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
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
// Where a wait gave up: the abort flag in shared memory ends every other wait of
// the block, so that each role leaves its loop.
struct WaitCtx {
  volatile int *abort;
  DeviceStatus *status;
  int chain;
};
__device__ __forceinline__ bool wait_or_abort(const WaitCtx &cx, uint64_t *bar, uint32_t parity,
                                              int where, int step) {
  if (mbar_test_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 16; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*cx.abort) return false;
    if (global_timer_ns() - t0 > kWaitNs) {
      record_device_status(cx.status, KDA_ERR_TIMEOUT, where, cx.chain, step);
      *cx.abort = 1;
      return false;
    }
  }
}

// The same by a converged warp, whose lanes leave together.
__device__ __forceinline__ bool warp_wait(const WaitCtx &cx, uint64_t *bar, uint32_t parity,
                                          int where, int step) {
  if (__all_sync(0xffffffffu, mbar_test_wait(bar, parity))) return true;
  return __all_sync(0xffffffffu, wait_or_abort(cx, bar, parity, where, step)) != 0;
}

// Barrier `id` over nthreads (a multiple of 32); returns whether any of them passed true.
__device__ __forceinline__ bool bar_any(uint32_t id, uint32_t nthreads, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\t"
      "barrier.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(nthreads), "r"((uint32_t)pred)
      : "memory");
  return r != 0;
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

// Programmatic launch: the next kernel's blocks may start; wait for the previous grid.
__device__ __forceinline__ void pdl_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ uint32_t round_up_1k(uint32_t x) { return (x + 1023u) & ~1023u; }

// A float as an integer of the same order (NaN with a clear sign above +inf).
__device__ __forceinline__ int ordered(float x) {
  const int b = __float_as_int(x);
  return b >= 0 ? b : b ^ 0x7fffffff;
}
__device__ __forceinline__ float unordered(int b) {
  return __int_as_float(b >= 0 ? b : b ^ 0x7fffffff);
}

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
