// What the tree operators share: a row's tree, where its columns are, clusters (sm_103a).
#pragma once

#include "common.cuh"

namespace specdec {

constexpr int kMaxTree = SPECDEC_MAX_TREE;
constexpr int kUnusedNode = -2;

// The bit set of node i and its ancestors (bit 0 is the root); 0 for an unused node.  `par` is
// the row's parents in shared memory, or nullptr for a chain.  Sets `bad` where a parent is out
// of range or an ancestor unused.  Parents lie below their children, so the walk ends.
__device__ __forceinline__ unsigned long long tree_ancestors(const int* par, int i, bool& bad) {
  if (par == nullptr) return ~0ull >> (63 - i);
  int p = par[i];
  if (p == kUnusedNode) return 0ull;
  unsigned long long m = 1ull << i;
  while (i > 0) {
    if (p < 0 || p >= i) {
      bad = true;
      return 0ull;
    }
    m |= 1ull << p;
    i = p;
    p = par[i];
  }
  if (p != -1) {  // a used root has parent -1
    bad = true;
    return 0ull;
  }
  return m;
}

// 16-byte asynchronous copy global -> shared; zero-fills where `take` is false.
__device__ __forceinline__ void cp_async16(void* dst, const void* src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
               ::"r"(smem_addr(dst)), "l"(src), "r"(take ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Cluster barrier, and the address of this CTA's shared-memory location in the CTA of `rank`.
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_map(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  return a;
}
// Stores to a CTA of the cluster that count their bytes on a barrier there when they have landed
// (addresses by cluster_map): data and signal in one, where a cluster barrier would be a second
// trip.
__device__ __forceinline__ void cluster_send(uint32_t a, unsigned long long v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.u64 [%0], %1, [%2];"
               ::"r"(a), "l"(v), "r"(bar) : "memory");
}
__device__ __forceinline__ void cluster_send4(uint32_t a, float4 v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];"
               ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar) : "memory");
}

}  // namespace specdec
