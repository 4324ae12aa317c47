// Places in rings of barriers, and the waits of the warps that widen weights in lanes_kernel. Nothing here needs a
// GPU: the order of the waits is stepped on the host as well.
#pragma once
#include <cuda_runtime.h>
#include <cstdint>

namespace moe {
namespace rows {

// A place in a ring of n barriers: the slot, and the parity of its use. (Divisions
// by the number of slots took a quarter of a widening warp's step.)
struct Ring {
  uint32_t slot = 0, parity = 0;
  __host__ __device__ __forceinline__ void next(uint32_t n) {
    if (++slot == n) {
      slot = 0;
      parity ^= 1;
    }
  }
};

}  // namespace rows

namespace dense {

// Barriers of a slot of lanes_kernel: its copy has landed; the tensor core is done with it.
enum LaneWait { LANE_FULL, LANE_EMPTY };

// What a widening warp waits for before it reads a slot. Two groups of warps take the steps in turn, and a wait by
// parity tells a phase from its neighbour only: who comes to a slot's use before the copy of the use before has
// landed finds the parity of the use before that, and passes. With an odd number of slots the use before is the other
// group's, and copies land in any order. So the warp first waits until the tensor core is done with that use, whose copy
// has landed then; the copy that it waits for next is asked for behind the same barrier.
// Neither wait passes early: two steps ago the warp saw the tensor core done with a later step than the
// slot's use before last, where there are two slots or more. Neither passes too late: the slot's next use waits for
// this step's product, and that for this warp. (To wait for the other group's copies as well would not
// do: their slots can be filled again without this group, whose wait would then find its parity gone.)
// With slots >= stages + 2 the warp knows it already: two steps ago it waited for a place in tensor memory, and so for the
// product of `stages` steps before that one. (32 rows through the int8 block, 4096 x 8192: 37.2 us, with the wait 38.0.)
template <class Wait>
__host__ __device__ __forceinline__ bool landed(const rows::Ring& it, int slots, int stages, Wait wait) {
  return (slots >= stages + 2 || wait(LANE_EMPTY, it.slot, it.parity ^ 1)) && wait(LANE_FULL, it.slot, it.parity);
}

// The step at which a widening group waits for the launch before, or the end where it has no such step: its first that has to
// wait for a place in tensor memory. (Nothing that it does before touches what that launch writes.)
__host__ __device__ __forceinline__ int behind_at(int stages, int group) { return stages + ((stages ^ group) & 1); }

}  // namespace dense
}  // namespace moe
