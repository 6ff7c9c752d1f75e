// Where loads of 16 bytes a lane go: arithmetic alone, so that it is checked on the host
// as well.
#pragma once
#include <stddef.h>
#include <stdint.h>

namespace moe {

// a lane's offset that is past the end of every buffer, and 4 KB on
constexpr uint32_t kPastEnd = 0xf0000000u;

// Reads `bytes` (a multiple of 16) once from their start on, in rounds of `all` bytes of
// which this lane's 16 begin at `mine`: load(first byte and records of the descriptor,
// lane's offset, scalar offset).  What the last round has too much is past the end by the
// lane's own offset.
template <typename Load>
__host__ __device__ __forceinline__ void read_once(size_t bytes, uint32_t mine, uint32_t all, Load load) {
  constexpr uint32_t kPart = 1u << 30;  // of a descriptor
  for (size_t base = 0; base < bytes; base += kPart) {
    const uint32_t n = static_cast<uint32_t>(bytes - base < kPart ? bytes - base : kPart);
    for (uint32_t o = 0; o < n; o += all) load(base, n, mine + o < n ? mine + o : kPastEnd, 0u);
  }
}

// Where a lane's load of a stage goes: records of the descriptor, the lane's offset and
// the scalar one.  Stages past the sum's last are loaded all the same, as zeros: they have
// a scalar offset of 0, since it may be more than the records and some range checks would
// take it off them.
struct StageLoad {
  uint32_t records, at, step_at;
};

// contiguous rows of `bytes` in all, their stages `stage` bytes apart: `at` is the lane's
// chunk in the first one, `left` is what the stage holds of a row's sum, `from` the chunk's
// first of it
__host__ __device__ __forceinline__ StageLoad load_rows(uint32_t bytes, uint32_t at, int step, int stage, int left,
                                                       int from) {
  return {bytes, from < left ? at : kPastEnd, left > 0 ? static_cast<uint32_t>(step * stage) : 0u};
}

// packed weights, 2 KB a stage of each group
__host__ __device__ __forceinline__ StageLoad load_packed(uint32_t bytes, uint32_t at, int step, int left) {
  return {left > 0 ? bytes : 0u, at, left > 0 ? static_cast<uint32_t>(step * 2048) : 0u};
}

}  // namespace moe
