// What the kernels of the operators around the block share: dependent launches, and a bounded wait that
// lets the hardware hold the thread.
#pragma once

#include "fp8q_common.cuh"

namespace fp8q {

// A launch whose blocks may become resident as soon as every block of the kernel before it on the stream has called
// start_dependents() or exited; they call wait_for_previous(), which returns once that kernel is
// complete and its writes are visible, before they touch global memory.  What it hides: the launch, and the
// block's own preparation (barriers, tensor memory, descriptors), about 3 us between two short kernels.
template <class... P, class... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t s, A... args) {
  cudaLaunchConfig_t c{};
  c.gridDim = grid;
  c.blockDim = dim3((unsigned)threads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, static_cast<P>(args)...);
}
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void start_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// mbar_wait with a time for which the hardware may hold the thread at each try (1 ms): a warp that waits for a tile's
// whole main loop, or for a row, then issues next to nothing.  Without it the waiting warps' polling took issue slots and
// shared-memory cycles from the others (head forward, T = 8192, d = 3584, V = 32000: 1054 -> 964 us cold, 1150 ->
// 1081 us at the power cap).  Layer norm's waits are short, and held threads wake later: 40 us against 42 with it, so it
// polls.  Gives up (returns false) after kWaitLimitNs, or soon after *abort is set.
__device__ __forceinline__ bool mbar_try_held(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity), "r"(1000000u)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool mbar_wait_held(uint64_t* bar, uint32_t parity, volatile int* abort) {
  if (mbar_try_held(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    if (mbar_try_held(bar, parity)) return true;
    if (*abort || globaltimer_ns() - t0 > kWaitLimitNs) return false;
  }
}

}  // namespace fp8q
