// decode.cuh -- what the paged decode kernels share (include/dsa_decode.h).
//
// A cache page holds page_size tokens = ppp pools, so the physical pool of a
// row's pool p is  table[p / ppp] * ppp + p % ppp.  ppp is any number >= 1
// known at launch: the division is a multiplication by a precomputed
// reciprocal (Granlund and Montgomery, "Division by invariant integers using
// multiplication"): with s = ceil(log2 ppp) and m = floor(2^(29+s) / ppp) + 1,
// p / ppp = (p * m) >> (29 + s) for every p < 2^29, since 2^(29+s) < m * ppp
// <= 2^(29+s) + 2^s.  Capacities are below 2^31 tokens, so p < 2^29 holds and
// the product stays below 2^60.
#pragma once

#include "common.cuh"
#include "decode.h"

namespace dsa {

// Load of what the kernel before this one on the stream may have written while
// this one was resident (chain_wait below): a plain one.  The non-coherent path
// (__ldg, or a const __restrict__ pointer) is for data that nobody writes in a
// kernel's life.
template <typename T>
__device__ __forceinline__ T ld_live(const T* p) {
  return *p;
}

__device__ __forceinline__ int page_of_pool(const PagedView& pv, int p) {
  return (int)(((uint64_t)(uint32_t)p * pv.div_mul) >> pv.div_shift);
}

// Length of row b, 0 (idle) when it lies outside 0..capacity.
__device__ __forceinline__ int row_length(const PagedView& pv, int64_t b, bool& bad) {
  const int n = ld_live(pv.lens + b);
  if (n < 0 || n > pv.capacity) {
    bad = true;
    return 0;
  }
  return n;
}

// Physical pool of pool p of the row whose block-table row is `trow`, given
// its page entry (trow[page_of_pool(p)], loaded earlier by the caller); -1
// for a page outside the cache.
__device__ __forceinline__ int phys_pool(const PagedView& pv, int p, int col, int page, bool& bad) {
  if ((uint32_t)page >= (uint32_t)pv.num_pages) {
    bad = true;
    return -1;
  }
  return page * pv.ppp + (p - col * pv.ppp);
}

// 16-byte global->shared copy of a row that is there (cp_async16 of common.cuh
// without the size operand).
__device__ __forceinline__ void cp_async16_full(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(dst), "l"(src) : "memory");
}

// Programmatic dependent launch: a kernel launched by launch_chained
// (decode.h) may become resident while its predecessor on the stream still
// runs.  chain_wait() returns when the predecessor has finished and its writes
// are visible; nothing is read or written before it.  chain_release(), by
// every CTA (or its end), lets the successor become resident.
__device__ __forceinline__ void chain_wait() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
__device__ __forceinline__ void chain_release() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }

// Thread-block clusters: barrier over all threads of the cluster (release /
// acquire of shared memory), and accesses to another CTA's shared memory (only
// between two barriers: after one the CTA is known to run, until the next it
// does not leave).
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
__device__ __forceinline__ uint32_t cluster_map(uint32_t saddr, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;\n" : "=r"(a) : "r"(saddr), "r"(rank));
  return a;
}
__device__ __forceinline__ void cluster_st4(uint32_t addr, float4 v) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};\n" ::"r"(addr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
               : "memory");
}
__device__ __forceinline__ void cluster_st_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;\n" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_st2(uint32_t addr, float2 v) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};\n" ::"r"(addr), "f"(v.x), "f"(v.y) : "memory");
}

}  // namespace dsa
