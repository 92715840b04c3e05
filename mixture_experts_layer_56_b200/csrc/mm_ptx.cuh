// What the training operators' matrix products use beside sm100_ptx.cuh:
// MN-major shared-memory operands and a cluster-wide release on an mbarrier.
#pragma once

#include "sm100_ptx.cuh"

namespace moe {
namespace sm100 {

// mbar_arrive_cluster, releasing this thread's earlier writes to the cluster
__device__ __forceinline__ void mbar_arrive_cluster_release(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}

// One lane of a converged warp.  The issuing warps run their loops with all
// lanes and pick one for the TMA and MMA instructions only: those take their
// operands from uniform registers, and inside a branch on the lane number the
// compiler cannot tell that a value is uniform (MMA issue then bounds the
// kernel: with it, 0.45 us per 64-wide k-block).
__device__ __forceinline__ bool elect_lane() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// Shared-memory matrix descriptor for an MN-major operand tile written by TMA
// with 128-byte swizzling: slices of 64 m (or n) values in k rows of 128
// bytes, groups of 8 k rows 1024 B apart, the next slice `slice_bytes` on.
//   bits 16-29  leading byte offset >> 4: from one 64-value slice to the next
//   bits 32-45  stride byte offset >> 4: from one group of 8 k rows to the next
// (the other fields as in desc_kmajor_sw128)
__device__ __forceinline__ uint64_t desc_mnmajor_sw128(uint32_t saddr, uint32_t slice_bytes) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(slice_bytes >> 4) << 16;
  d |= static_cast<uint64_t>(1024u >> 4) << 32;
  d |= static_cast<uint64_t>(1u) << 46;
  d |= static_cast<uint64_t>(2u) << 61;
  return d;
}

// Instruction descriptor of kind::f16 with fp16 (formats 0) or bf16 (1)
// operands, both the same, fp32 D, either operand K- or MN-major.
__host__ __device__ constexpr uint32_t idesc_16bit_f32(int M, int N, bool fp16, bool a_mn,
                                                       bool b_mn) {
  return (1u << 4) | (fp16 ? 0u : (1u << 7) | (1u << 10)) | (a_mn ? 1u << 15 : 0u) |
         (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

}  // namespace sm100
}  // namespace moe
