// kda_pdl.cuh -- programmatic dependent launch.  Not installed.
#pragma once

namespace kda {

// Programmatic dependent launch: the next kernel of the stream may start where this
// one leaves room; and in that kernel, waiting for the end of the one before.
__device__ __forceinline__ void grid_go_on() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace kda
