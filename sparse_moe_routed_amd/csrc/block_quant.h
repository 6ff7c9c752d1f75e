// E4M3 codes with one fp32 scale per block of 128 values of a row: device code
// shared by the kernels that make them.
#pragma once
#include <type_traits>

#include "moe_common.h"
#include "moe_internal.h"

namespace moe {

constexpr int kQThreads = 256;

// amax below this makes a zero block: 448 / amax must stay finite
constexpr float kTinyAmax = 7.888609e-31f;  // 2^-100

__device__ __forceinline__ float amax8(u32x4 v) {
  float m = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    m = fmaxf(m, fabsf(__uint_as_float(v[w] << 16)));
    m = fmaxf(m, fabsf(__uint_as_float(v[w] & 0xffff0000u)));
  }
  return m;
}

// codes of v inv for four bf16 values of at most 448 / inv: nothing to clamp, and
// NaN (and infinity, whose block has inv = 0) becomes a NaN code.  The added 0
// makes -0 the code 0 and costs nothing in a multiply-add.
__device__ __forceinline__ uint32_t encode4(uint32_t a, uint32_t b, float inv) {
  const auto low = [&](uint32_t u) { return __builtin_fmaf(__uint_as_float(u << 16), inv, 0.f); };
  const auto high = [&](uint32_t u) { return __builtin_fmaf(__uint_as_float(u & 0xffff0000u), inv, 0.f); };
  const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(low(a), high(a), 0, false);
  return __builtin_amdgcn_cvt_pk_fp8_f32(low(b), high(b), lo, true);
}

__device__ __forceinline__ uint2 encode8(u32x4 v, float inv) {
  return make_uint2(encode4(v[0], v[1], inv), encode4(v[2], v[3], inv));
}

// max of v (0 or more, or NaN as fmaxf takes it) over each 8 lanes, in all of them
__device__ __forceinline__ float row8_max(float v) {
  const auto other = [&](auto how) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), decltype(how)::value,
                                                              0xf, 0xf, true));
  };
  v = fmaxf(v, other(std::integral_constant<int, 0xb1>{}));   // lane ^ 1
  v = fmaxf(v, other(std::integral_constant<int, 0x4e>{}));   // lane ^ 2
  return fmaxf(v, other(std::integral_constant<int, 0x141>{}));  // the other 4 of 8
}

// and over each 16
__device__ __forceinline__ float row16_max(float v) {
  v = row8_max(v);
  return fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), 0x140, 0xf, 0xf,
                                                                     true)));  // lane 15 - i
}

// The part of q's rows that workgroup `group` of `groups` (kQThreads threads each)
// takes: 16 lanes to a block of 128 values, 8 values a lane.
__device__ __forceinline__ void block_quantise(const BlockQuantArgs& q, int group, int groups) {
  const int kb_n = (q.cols + 127) / 128;
  const int l16 = threadIdx.x & 15;
  const int64_t n = static_cast<int64_t>(q.rows) * kb_n;
  const int64_t step = static_cast<int64_t>(groups) * (kQThreads / 16);
  for (int64_t i = static_cast<int64_t>(group) * (kQThreads / 16) + (threadIdx.x >> 4); i < n; i += step) {
    const int r = static_cast<int>(i / kb_n), kb = static_cast<int>(i - static_cast<int64_t>(r) * kb_n);
    const int k = kb * 128 + l16 * 8;
    const size_t at = static_cast<size_t>(r) * q.cols + k;
    u32x4 v = {0u, 0u, 0u, 0u};
    if (k < q.cols) v = *reinterpret_cast<const u32x4*>(q.x + at);
    const float amax = row16_max(amax8(v));
    const bool live = amax >= kTinyAmax;
    if (k < q.cols)
      *reinterpret_cast<uint2*>(q.codes + at) = encode8(v, live ? __fdiv_rn(448.f, amax) : 0.f);
    if (l16 == 0) q.scales[static_cast<size_t>(kb) * q.rows + r] = live ? __fdiv_rn(amax, 448.f) : 0.f;
  }
}

// workgroups for q's rows
inline int block_quant_groups(const BlockQuantArgs& q) {
  const int64_t n = static_cast<int64_t>(q.rows) * ((q.cols + 127) / 128);
  const int64_t g = (n + kQThreads / 16 - 1) / (kQThreads / 16);
  return static_cast<int>(g < 8192 ? g : 8192);
}

}  // namespace moe
