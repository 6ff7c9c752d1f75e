// 8-bit integer codes with one fp32 scale per row: device code shared by the kernels
// that make them.  A row's amax gives s = f32(amax / 127) and codes RNE(v inv) with
// inv = f32(127 / amax), the product exact; amax below 2^-100 makes a zero row.  A row
// that holds a NaN or an infinity has scale NaN and codes 0, so that its results are
// NaN and no others are.
#pragma once
#include "block_quant.h"
#include "moe_common.h"
#include "moe_internal.h"

namespace moe {

struct RowScale {
  float inv, scale;
};

// of the largest magnitude's bf16 bits
__device__ __forceinline__ RowScale row_scale(uint32_t amax_bits) {
  if (amax_bits >= 0x7f80u) return {0.f, __uint_as_float(0x7fc00000u)};
  const float amax = __uint_as_float(amax_bits << 16);
  if (!(amax >= kTinyAmax)) return {0.f, 0.f};
  return {__fdiv_rn(127.f, amax), __fdiv_rn(amax, 127.f)};
}

// codes of four bf16 values.  The sum with 1.5 * 2^23 is the product rounded once to
// an integer (ties to even), which then is the sum's low byte in two's complement;
// NaN, as of infinity times 0, leaves a zero there.
__device__ __forceinline__ uint32_t int8x4(uint32_t a, uint32_t b, float inv) {
  constexpr float kRound = 12582912.f;
  const uint32_t c0 = __float_as_uint(__builtin_fmaf(__uint_as_float(a << 16), inv, kRound));
  const uint32_t c1 = __float_as_uint(__builtin_fmaf(__uint_as_float(a & 0xffff0000u), inv, kRound));
  const uint32_t c2 = __float_as_uint(__builtin_fmaf(__uint_as_float(b << 16), inv, kRound));
  const uint32_t c3 = __float_as_uint(__builtin_fmaf(__uint_as_float(b & 0xffff0000u), inv, kRound));
  return __builtin_amdgcn_perm(c1, c0, 0x0c0c0400u) | __builtin_amdgcn_perm(c3, c2, 0x04000c0cu);
}

__device__ __forceinline__ uint2 int8x8(u32x4 v, float inv) {
  return make_uint2(int8x4(v[0], v[1], inv), int8x4(v[2], v[3], inv));
}

// the largest magnitude of eight bf16 values, as bits
__device__ __forceinline__ uint32_t amax_bits8(u32x4 v) {
  uint32_t m = 0u;
#pragma unroll
  for (int w = 0; w < 4; ++w) m = max(m, max(v[w] & 0x7fffu, (v[w] >> 16) & 0x7fffu));
  return m;
}

__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), o)));
  return v;
}

// One row of `cols` values (a multiple of 8) by one wave: put(k, codes) for every
// eight values, k their first column, and the scale.  Rows of up to kRowHeld values
// are read once.
constexpr int kRowHeld = 4096;
template <typename Put>
__device__ __forceinline__ float quantise_row(const uint16_t* row, int cols, Put put) {
  constexpr int kHeld = kRowHeld / 512;
  const int k0 = (threadIdx.x & 63) * 8;
  const auto at = [&](int k) { return *reinterpret_cast<const u32x4*>(row + k); };
  u32x4 v[kHeld];
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < kHeld; ++i) {
    v[i] = u32x4{0u, 0u, 0u, 0u};
    if (k0 + i * 512 < cols) v[i] = at(k0 + i * 512);
  }
#pragma unroll
  for (int i = 0; i < kHeld; ++i) m = max(m, amax_bits8(v[i]));
  for (int k = k0 + kRowHeld; k < cols; k += 512) m = max(m, amax_bits8(at(k)));
  const RowScale s = row_scale(wave_max_u32(m));
#pragma unroll
  for (int i = 0; i < kHeld; ++i)
    if (k0 + i * 512 < cols) put(k0 + i * 512, int8x8(v[i], s.inv));
  for (int k = k0 + kRowHeld; k < cols; k += 512) put(k, int8x8(at(k), s.inv));
  return s.scale;
}

// The part of q's rows that workgroup `group` of `groups` (kQThreads threads each)
// takes: codes row-major, scales [rows]
__device__ __forceinline__ void row_quantise(const BlockQuantArgs& q, int rows, int group, int groups) {
  for (int64_t r = static_cast<int64_t>(group) * (kQThreads / 64) + (threadIdx.x >> 6); r < rows;
       r += static_cast<int64_t>(groups) * (kQThreads / 64)) {
    uint8_t* const out = q.codes + static_cast<size_t>(r) * q.cols;
    const float s = quantise_row(q.x + static_cast<size_t>(r) * q.cols, q.cols, [&](int k, uint2 codes) {
      *reinterpret_cast<uint2*>(out + k) = codes;
    });
    if ((threadIdx.x & 63) == 0) q.scales[r] = s;
  }
}

// tokens in the format of the bank that takes them
__device__ __forceinline__ void quantise_tokens(const BlockQuantArgs& q, int group, int groups) {
  if (q.int8) row_quantise(q, q.rows, group, groups);
  else block_quantise(q, group, groups);
}

}  // namespace moe
