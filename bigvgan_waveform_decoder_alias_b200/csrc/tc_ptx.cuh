// Inline-PTX building blocks of the tensor-core kernels (tcgen05, TMA,
// mbarriers) and the TMA descriptor encoder.
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace bv {

constexpr long long DRAIN_LIMIT = 1ll << 22;  // polls for in-flight copies when unwinding

__device__ __forceinline__ unsigned smem_u32(const void *p) {
  return (unsigned)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ void mbar_init(unsigned bar, unsigned count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_arrive(unsigned bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mbar_arrive_tx(unsigned bar, unsigned bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ bool mbar_try_wait(unsigned bar, unsigned parity) {
  unsigned ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

// Non-blocking probe of an mbarrier phase: cheaper than try_wait when the
// phase has already completed (measured on B200: ~160 against ~280 cycles in
// the MMA issuer's wait for a weight chunk that had landed long before).
__device__ __forceinline__ bool mbar_test(unsigned bar, unsigned parity) {
  unsigned ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}

struct Ctl {
  int abort;      // a bounded wait gave up somewhere in the CTA (or its pair)
  unsigned tmem;  // TMEM base address from tcgen05.alloc
};

// How a CTA reports a wait that ran out: its own Ctl, the shared::cluster
// address of its pair peer's abort flag (0 for a lone CTA), the device status
// word and the poll limit.
struct WaitCtx {
  volatile Ctl *ctl;
  unsigned peer_abort;
  int *status;
  long long limit;
};

__device__ __forceinline__ void raise_abort(const WaitCtx &w, int code) {
  w.ctl->abort = 1;
  if (w.peer_abort)
    asm volatile("st.shared::cluster.u32 [%0], %1;\n" ::"r"(w.peer_abort), "r"(1) : "memory");
  if (w.status) atomicExch(w.status, code);
}

// Bounded wait on an mbarrier phase: true once the phase has completed;
// false after w.limit polls (the CTA and its peer are then marked aborted and
// the failure recorded in the device status word) or once an abort raised
// elsewhere in the pair is seen.  A role stops issuing work at its first
// false.
__device__ __forceinline__ bool mbar_wait(unsigned bar, unsigned parity, const WaitCtx &w,
                                          int code) {
  if (mbar_test(bar, parity)) return true;
  for (long long it = 0; it < w.limit; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 255) == 255 && w.ctl->abort) return false;
  }
  raise_abort(w, code);
  return false;
}

// Wait with a fixed bound that does not return early on abort: used to let
// the copies and MMAs a role issued finish before the CTA frees TMEM or exits.
__device__ __forceinline__ void mbar_drain(unsigned bar, unsigned parity) {
  for (long long it = 0; it < DRAIN_LIMIT; ++it)
    if (mbar_try_wait(bar, parity)) return;
}

// Converter-side wait: lane 0 polls the barrier, the warp follows it, so the
// polling does not compete with the conversion for shared-memory bandwidth;
// the outcome is the same for every lane.
__device__ __forceinline__ bool warp_wait(unsigned bar, unsigned parity, const WaitCtx &w,
                                          int code) {
  int ok = 1;
  if ((threadIdx.x & 31) == 0) ok = mbar_wait(bar, parity, w, code) ? 1 : 0;
  return __shfl_sync(0xffffffffu, ok, 0) != 0;
}

// Shared-memory matrix descriptor: K-major, 128-byte swizzle, 8-row groups
// 1024 bytes apart (stride byte offset), descriptor version 1.
__device__ __forceinline__ uint64_t sw128_desc(unsigned addr) {
  return (uint64_t)((addr >> 4) & 0x3FFF) | ((uint64_t)1 << 16) | ((uint64_t)(1024 >> 4) << 32) |
         ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

__device__ __forceinline__ void mma_commit(unsigned bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n" ::"r"(bar)
      : "memory");
}

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;\n" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::
                   : "memory");
}
// Shared::cluster address of the same variable in CTA `rank` of the cluster.
__device__ __forceinline__ unsigned map_to_rank(unsigned addr, unsigned rank) {
  unsigned r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// TMA loads of the pair: the destination is this CTA's shared memory, the
// completion goes to the even CTA's barrier (peer bit cleared).
constexpr unsigned kPeerBitMask = 0xFEFFFFFFu;
__device__ __forceinline__ void tma_load_2d_pair(unsigned dst, const CUtensorMap *map, int c0, int c1,
                                                 unsigned bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];\n" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar & kPeerBitMask)
      : "memory");
}
// `bytes` (a multiple of 16) from global `src` (16-byte aligned) to this CTA's
// shared memory, counted by the barrier.
__device__ __forceinline__ void bulk_load(unsigned dst, uintptr_t src, unsigned bytes, unsigned bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n" ::"r"(
          dst),
      "l"((uint64_t)src), "r"(bytes), "r"(bar)
      : "memory");
}
// Arrive on the barrier at this offset in both CTAs once the MMAs issued so
// far have completed.
__device__ __forceinline__ void mma_commit_pair(unsigned bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;\n" ::"r"(bar),
      "h"((unsigned short)3)
      : "memory");
}

// cuTensorMapEncodeTiled through the runtime's driver entry point (no
// link-time dependency on libcuda).
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// (The first callers may come from several threads: a static's initialisation
// runs once and all of them wait for it.)
inline EncodeTiledFn encode_fn() {
  static const EncodeTiledFn fn = []() -> EncodeTiledFn {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<EncodeTiledFn>(p);
    cudaGetLastError();
    return nullptr;
  }();
  return fn;
}

}  // namespace bv
