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

}  // namespace moe
