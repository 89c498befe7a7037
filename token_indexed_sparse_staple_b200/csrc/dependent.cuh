// Programmatic dependent launches: kernels launched by launch_dependent()
// (internal.h) start while the kernel in front of them in the stream drains.
#pragma once

namespace stp {

// Wait until the kernels before this one in the stream have completed and
// their writes are visible.  Every write to memory comes after this, and so does
// every read of what a kernel before it may write.  Inside one call a kernel may read
// earlier what no kernel of the call writes (weights, ids, E), provided that the
// kernel in front released it only after its own wait: all work before the call is
// then complete.
__device__ __forceinline__ void wait_prior_kernels() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Let the next kernel of the stream start, if it was launched as a programmatic
// dependent, as soon as every block of this one has come this far.  Only where
// that kernel is the library's own and part of the same call: another one
// might read before it waits (the decode kernel fetches its weights so), and
// what it reads might be this kernel's output.  After wait_prior_kernels(), so
// that what it does read early is older than both.
__device__ __forceinline__ void release_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace stp
