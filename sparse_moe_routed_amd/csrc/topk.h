// Top-k selection of one token's logits by one wave, shared by the router and
// the few-token layer.
#pragma once

#include "moe_common.h"

namespace moe {

constexpr int kMaxE = 256;  // experts the selection covers: four per lane

// Largest 32-bit unsigned value over the wave, in every lane.  DPP row shifts
// reduce each 16-lane row into its lane 15, two row broadcasts combine the
// rows into lane 63; zero (the identity) fills lanes a shift leaves empty.
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x111, 0xf, 0xf, false)));
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x112, 0xf, 0xf, false)));
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x114, 0xf, 0xf, false)));
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x118, 0xf, 0xf, false)));
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x142, 0xa, 0xf, false)));
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x143, 0xc, 0xf, false)));
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
}

// order-preserving unsigned key of a float (larger float -> larger key; -inf
// maps above 0, which marks an empty slot).  -0 and +0 compare equal as
// floats, so -0 is first made +0 (x + 0 is +0 for x = -0 under round to
// nearest) and both get one key: a tie between them goes to the lower index.
__device__ __forceinline__ uint32_t float_key(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// The k largest of the logits v over the wave (lane l holds experts l + 64 i, i < N;
// key is float_key(v), 0 past E, and is used up): sel_i in order of (logit
// desc, index asc), sel_v their logits.  Each of the k rounds takes the largest
// key over the wave, then the lowest expert index holding it (ballots over the
// slots in index order), and retires that expert.
template <int N>
__device__ __forceinline__ void wave_topk(const float (&v)[N], uint32_t (&key)[N], int k,
                                          float (&sel_v)[8], int (&sel_i)[8]) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    sel_v[j] = 0.f;
    sel_i[j] = 0;
    if (j >= k) continue;
    uint32_t m = key[0];
#pragma unroll
    for (int i = 1; i < N; ++i) m = max(m, key[i]);
    const uint32_t best = wave_umax(m);
    int win = -1;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint64_t b = __ballot(key[i] == best && key[i] != 0u);
      if (win < 0 && b) win = 64 * i + __ffsll(static_cast<unsigned long long>(b)) - 1;
    }
    // the winner's logit, from the lane that holds it
    float wv = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (lane + 64 * i == win) {
        wv = v[i];
        key[i] = 0u;
      }
    sel_v[j] = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, wv), win & 63));
    sel_i[j] = win;
  }
}

}  // namespace moe
