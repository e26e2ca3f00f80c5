// Bounded waits of the single-token kernels.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

#include "wave_sync.cuh"

namespace wavei {

// wait_bar with the first test in line, for threads whose time between waits is
// what a loop is bound by. A try_wait may suspend for longer than a short bound
// and then succeed, so with bounds under a millisecond (which a test sets to
// make a wait run out) the clock decides after a success too.
__device__ __forceinline__ bool wait_within(uint32_t bar, uint32_t parity, const Ctl& ctl, int code) {
  if (ctl.timeout_ns >= kLongWaitNs) {
    if (wptx::mbar_try_wait(bar, parity)) return true;
    return wait_bar(bar, parity, ctl, code);
  }
  const uint64_t t0 = wptx::globaltimer_ns();
  if (!wait_bar(bar, parity, ctl, code)) return false;
  if (wptx::globaltimer_ns() - t0 <= ctl.timeout_ns) return true;
  *ctl.abort_flag = 1;
  atomicCAS(ctl.status, 0, code);
  return false;
}

// Programmatic dependent launch. A kernel launched by launch_chained may start while
// the kernel before it in the stream still runs: `chain_begin` lets the next one do
// so, and nothing of global memory is read or written before `chain_wait`, which
// returns when the kernel before has ended and its writes are visible (to plain
// loads and TMA: .nc loads ask for data that nothing writes while the kernel runs,
// and the kernel before may). One exception: token_rows_kernel sends for weights into L2
// ahead of the wait, where every SM's reads and writes meet, so that what the kernel
// before still writes is written there. A kernel with tensor memory calls chain_begin
// when it has its columns: the next one's allocation then waits for this one's end,
// never this one's for the next. What is saved is a launch's latency and a prologue per
// kernel of a token's step.
__device__ __forceinline__ void chain_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void chain_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// All threads of a cluster, whose writes to each other's shared memory are then seen. By
// whole warps.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A launch whose kernel begins with chain_begin and chain_wait; cluster: CTAs per
// cluster (1: none).
template <class K, class... A>
cudaError_t launch_chained(K kernel, dim3 grid, unsigned threads, size_t shared, cudaStream_t stream, unsigned cluster,
                           const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = shared;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) cudaGetLastError();
  return e;
}

}  // namespace wavei
