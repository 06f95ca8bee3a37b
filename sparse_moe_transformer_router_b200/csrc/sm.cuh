// sm.cuh -- the few inline-PTX wrappers of the operators that are compiled in
// files of their own (ptx.cuh, the layer's, defines a kernel and so belongs
// to one translation unit).
#pragma once
#include <cstdint>

namespace l4moe {
namespace op {

// Programmatic dependent launch: wait until the previous kernel of the stream
// has finished, then let the next one start launching.
__device__ __forceinline__ void pdl_enter() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace op
}  // namespace l4moe
