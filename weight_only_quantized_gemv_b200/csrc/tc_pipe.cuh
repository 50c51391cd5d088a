// What the tcgen05 products of the fused layers and of the 8-bit floating-point layers share:
// bounded waits, split sums, meeting points of a CTA or pair, the tensor map encoder.
#pragma once
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "tc.cuh"

// How the wait that outlasts its first suspension is compiled.  A source whose kernels divide the
// registers among their warps (setmaxnreg) asks for __forceinline__: its epilogue's sums leave no
// room for a call's registers.
#ifndef QTC_WAIT_SLOW
#define QTC_WAIT_SLOW __noinline__
#endif

namespace qtc {

__device__ __forceinline__ long long run_begin(int w, long long U, int W) { return w * U / W; }
__device__ __forceinline__ int worker_of(long long u, long long U, int W) {
  return (int)(((u + 1) * W - 1) / U);
}

// ---------------------------------------------------------------------------
// bounded waits

struct WaitCtx {
  uint32_t abort;  // shared-memory address of the CTA's abort flag
  uint32_t* err;   // global memory
  uint32_t limit_us;
};

// Suspends the thread until the phase completes, or for up to kSuspendNs; whether it completed.
// (Polling instead took as many issue slots as the decoding.)
constexpr uint32_t kSuspendNs = 20000;
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity, bool cluster) {
  uint32_t done;
  if (cluster)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(kSuspendNs)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(kSuspendNs)
        : "memory");
  return done != 0;
}

// The phase has not completed within one suspension: keep waiting up to the limit, or until
// another role has given up; then set the flag.
static __device__ QTC_WAIT_SLOW bool wait_slow(uint32_t bar, uint32_t parity, uint32_t abort,
                                               uint32_t* err, uint32_t limit_us, uint32_t bit,
                                               bool honor_abort, bool cluster) {
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    if (try_wait(bar, parity, cluster)) return true;
    if (honor_abort) {
      uint32_t a;
      asm volatile("ld.volatile.shared.u32 %0, [%1];" : "=r"(a) : "r"(abort) : "memory");
      if (a) break;
    }
    if (globaltimer_ns() - t0 > 1000ull * limit_us) break;
  }
  atomicOr(err, bit);
  asm volatile("st.volatile.shared.u32 [%0], %1;" ::"r"(abort), "r"(1u) : "memory");
  return false;
}

// Waking up from a suspended wait takes hundreds of cycles; polling takes issue slots.  So the
// waits between the pipeline's roles (SPIN > 0) poll SPIN times first where the MMAs set the pace
// (256-token tiles: 190 against 290 us on 1024 x 4096 x 28672 backward) and suspend at once where
// the decoding does (32 rows, 8192 x 18944: 35.1 against 37.6 us).
// CLUSTER: some of the arrivals come from the pair's other CTA (acquire at cluster scope).

// One thread.
template <int SPIN>
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, const WaitCtx& w, uint32_t bit,
                                     bool honor_abort = true) {
#pragma unroll 1
  for (int i = 0; i < SPIN; ++i)
    if (mbar_ready(bar, parity, false)) return true;
  return try_wait(bar, parity, false) ||
         wait_slow(bar, parity, w.abort, w.err, w.limit_us, bit, honor_abort, false);
}

// A whole warp: every lane sees the phase complete (the usual case), or one lane waits on.
template <int SPIN, bool CLUSTER = false>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, const WaitCtx& w,
                                          uint32_t bit, int lane, bool honor_abort = true) {
#pragma unroll 1
  for (int i = 0; i < SPIN; ++i)
    if (__all_sync(0xffffffffu, mbar_ready(bar, parity, CLUSTER))) return true;
  if (__all_sync(0xffffffffu, try_wait(bar, parity, CLUSTER))) return true;
  bool ok = true;
  if (lane == 0)
    ok = wait_slow(bar, parity, w.abort, w.err, w.limit_us, bit, honor_abort, CLUSTER);
  return __shfl_sync(0xffffffffu, ok, 0);
}

// A role that gave up: what it has sent to the pair's other CTA, or has that CTA's barriers count,
// arrives long before this ends (nothing is left to wait on).
constexpr uint32_t kSettleUs = 20000;

// Split-sum arrival with a weight; the count before it.
__device__ __forceinline__ uint32_t arrive_weight(uint32_t* counter, uint32_t weight) {
  uint32_t old;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;"
               : "=r"(old)
               : "l"(counter), "r"(weight)
               : "memory");
  return old;
}

// Every thread of the CTA (PAIR: of both CTAs).  The roles leave their warps divergent, so the
// lanes meet first, and the cluster barrier is the form that does not ask for it.
template <bool PAIR>
__device__ __forceinline__ void sync_all() {
  __syncwarp();
  if constexpr (PAIR)
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
  else
    __syncthreads();
  __syncwarp();
}

// One lane of the warp, the same every time.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// ---------------------------------------------------------------------------
// host side

inline PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> fn{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 f = fn.load(std::memory_order_acquire);
  if (f) return f;
  void* p = nullptr;
  cudaDriverEntryPointQueryResult q;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                       &q) == cudaSuccess &&
      q == cudaDriverEntryPointSuccess)
    f = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  fn.store(f, std::memory_order_release);
  return f;
}

}  // namespace qtc
