// How the head's kernels follow one another on a stream, and how the producer and MMA warps
// of its tensor-core kernels wait and issue (gemm_fp8.cuh, linear_ce.cuh, few_tokens.cuh).
#pragma once

#include "gemm_tc2.cuh"

namespace bl {

// The head's kernels are launched with programmatic stream serialisation: a kernel may be
// set up (blocks placed, barriers and TMEM prepared) while the one before it on the stream
// still runs, and waits here, before its first access to global memory, until that one has
// completed and its writes are visible. Every thread calls it.
__device__ __forceinline__ void follow_stream() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// A load of data that a kernel before this one may have written: an ordinary one, ordered by
// follow_stream(), and not through the read-only path, whose data must not change while a
// kernel is resident, waiting included.
template <class T>
__device__ __forceinline__ T ld_plain(const T* p) {
  return *p;
}

// One lane of a converged warp, always the same one. The MMA and producer warps run their
// loops with all 32 lanes and branch on this only around the instructions themselves: from
// such a branch the compiler issues them with descriptors and addresses kept in uniform
// registers, where they take them. Measured (8192 tokens, eight MMAs): 300 cycles to issue;
// 570 by a lane chosen once and a predicate on each instruction, 670 from a branch on that
// lane, which made the issuing warp slower than the tensor cores (11008 -> 2048: 171 us
// against 145).
__device__ __forceinline__ bool elect_one() {
  uint32_t on;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(on));
  return on != 0;
}
// Wait of a whole warp, bounded like mbar_wait. `live` is 0 once a wait has given up, and
// every later wait returns at once; the first to give up raises the pair's abort flags. The
// loops around it do not branch on the outcome (their trip counts stay uniform), they only
// stop issuing. kCluster: acquire at cluster scope, for a barrier that the other CTA's
// threads arrive on after writing what they hand over.
template <bool kCluster>
__device__ __forceinline__ uint32_t wait_live(uint32_t live, uint32_t bar, uint32_t parity, volatile int* abort, uint32_t peer_flag) {
  auto poll = [&]() {
    uint32_t done;
    if (kCluster)
      asm volatile(
          "{\n\t.reg .pred p;\n\t"
          "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
          "selp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(done)
          : "r"(bar), "r"(parity)
          : "memory");
    else done = mbar_try_wait(bar, parity) ? 1u : 0u;
    return __all_sync(0xffffffffu, done != 0) != 0;
  };
  if (poll()) return live;
  if (!live) return 0;
  const uint64_t t0 = global_timer_ns();
  while (!poll())
    if (__any_sync(0xffffffffu, *abort != 0 || global_timer_ns() - t0 > kWaitTimeoutNs)) {
      pair_abort(abort, peer_flag);
      return 0;
    }
  return live;
}

}  // namespace bl
