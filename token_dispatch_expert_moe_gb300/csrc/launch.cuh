// Launch helpers of the operators around the layer: programmatic dependent
// launch, the SM count, byte-range overlap.
#pragma once
#include "common.cuh"

namespace moe {

// A kernel launched with launch_pdl is brought up while its predecessor on the
// stream still runs. It reads nothing that the predecessor writes, and writes
// nothing to memory, before pdl_wait() has returned (the predecessor has
// completed and its writes are visible). Every thread of every CTA waits, so
// that this kernel's end means the end of all before it.
// Within one operator a kernel may let only those threads wait that use the
// predecessor's results, and its last CTA at the end, which keeps that meaning: if
// the predecessor triggers after a wait of its own, or likewise knows that all
// before it has completed, and neither writes what the other touches.
// The norm, the balance loss, the permutation and the gradients' kernels do not
// trigger their successor early: measured, that gained nothing (norm of 16384 x
// 6144: 131 us with or without, 133 us without this launch) and cost up to 1 us
// where the successor's CTAs took the place of work. The adapters' kernels do
// (pdl_trigger): theirs are chains of short kernels, each of which has
// microseconds to set up.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Lets the successor be brought up as soon as every CTA of this grid has come
// here. After pdl_wait() a successor that has been brought up knows that all before
// this kernel has completed; one that could rely on that is launched only behind
// kernels that trigger so, or that were themselves brought up so.
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_clusters(void (*k)(KArgs...), dim3 grid, dim3 block, int cluster, size_t smem,
                                cudaStream_t s, Args... args) {
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = (unsigned)cluster;
  attrs[1].val.clusterDim.y = 1;
  attrs[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attrs;
  cfg.numAttrs = cluster > 0 ? 2 : 1;   // 0: what the kernel itself says
  return cudaLaunchKernelEx(&cfg, k, static_cast<KArgs>(args)...);
}

template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*k)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                       Args... args) {
  return launch_pdl_clusters(k, grid, block, 0, smem, s, args...);
}

inline int sm_count() {
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms > 0 ? sms : 1;
}

}  // namespace moe
