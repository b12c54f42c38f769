// stage.h -- which phases of a stage's barriers its last copies complete
// (paged_decode.cu).  Plain C++, so that it can be checked without a GPU.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define PI_STAGE_FN __host__ __device__ __forceinline__
#else
#define PI_STAGE_FN inline
#endif

namespace piattn {

// A warp's stage holds one tile of K and one of V, a barrier each; copy n of an
// operand completes phase n of its barrier.  K is refilled for the next tile as
// soon as the scores are done, before the warp waits for V: at that wait K is one
// copy ahead of V.
enum class Stuck : uint32_t {
  kNo = 0,
  kAtK,        // the wait for K of tile `used` ran out: K and V of that tile are under way
  kAtV,        // the wait for V ran out, and there was no next tile
  kAtVAhead    // the wait for V ran out with K of the next tile under way
};

// Parities of the phases that the last copies complete.  used: tiles used up.
struct StagePhases { uint32_t k, v; };
PI_STAGE_FN StagePhases last_phases(uint32_t used, Stuck at) {
  return {(used + (at == Stuck::kAtVAhead ? 1u : 0u)) & 1u, used & 1u};
}

}  // namespace piattn
