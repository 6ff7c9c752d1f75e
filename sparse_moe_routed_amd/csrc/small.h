// The products of few rows: dense in 8-bit integers (with the quantisation of the rows
// inside or without) and grouped in bf16.
#pragma once
#include "channel_quant.h"
#include "products.h"

namespace moe {

// ---- few rows: 32 weight rows x 16 G rows per workgroup, the steps of K dealt to 8
// waves; the waves' sums are joined through LDS.  The rows come a line at a time (8 lanes
// to 128 bytes) and are turned into operand order in LDS that belongs to the wave.  With
// QUANT the rows are bf16: the workgroup first takes the maxima of whole rows, then makes
// the codes as the steps go.
// Bound by memory latencies in a row, so 8 waves share K: a wave has 3 steps at K = 2688.
// A step's loads stand before the products of the step before it but do not run beside
// them: chunks past K are made zero where they are loaded, which waits for the step's
// loads, the weights' among them.  A row's maximum is a load and its wait at a time, six at
// K = 2688, after the first step's.  1 x 3712 x 2688 7.0 us with the quantisation inside
// (10 MB of weights, 1.4 TB/s); 77 rows 8.2 us, their quantisation 3.3 before it: past 32
// rows every workgroup would repeat too much of it.
constexpr int kSmallWaves = 8;
constexpr int kSmallN = 32;

template <typename T, int MODE, int G, bool QUANT, bool ONCE>
__global__ __launch_bounds__(kSmallWaves * kWave) void small_kernel(NtArgs g) {
  static_assert(!QUANT || T::kBytes == 1, "codes are 8-bit integers");
  typedef typename T::Acc Acc;
  constexpr int kTurn = 4096, kJoin = G * 1024;
  constexpr int kRaw = QUANT ? 2 : 1;  // 16-byte loads per 16 values
  constexpr int kPolicy = ONCE ? 2 : 0;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kSmallWaves * (kTurn > kJoin ? kTurn : kJoin)];
  __shared__ float inv_of[QUANT ? 16 * G : 1], scale_of[QUANT ? 16 * G : 1];
  NtTile t;
  if (!nt_find<T, MODE, 16 * G, kSmallN>(g, t)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, q = lane >> 4;
  const int row_bytes = g.K * T::kBytes, steps = (row_bytes + 127) / 128;
  const int lr = lane >> 3, ch = lane & 7;  // row of 8 and 16-value chunk this lane loads
  // groups of 16 rows that hold any
  const int live = __builtin_amdgcn_readfirstlane((t.rows + 15) >> 4);

  // two groups of 16 weight rows; what lies past N is past the buffer's end
  const int held = min(kSmallN, g.N - t.n0);
  const uint32_t group_bytes = steps * 2048u;
  const Buffer wb = T::kPacked
                        ? buffer_of(t.w + static_cast<size_t>(t.n0 / 16) * group_bytes, (held > 16 ? 2u : 1u) * group_bytes)
                        : buffer_of(t.w + static_cast<size_t>(t.n0) * row_bytes, held * static_cast<uint32_t>(row_bytes));
  uint32_t wat[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    wat[i] = T::kPacked ? (i == 0 || held > 16 ? lane * 16u + i * group_bytes : kPastEnd)
                        : (i * 16 + c < held ? static_cast<uint32_t>(i * 16 + c) * row_bytes + q * 16u : kPastEnd);
  const uint8_t* xp[G][2];
#pragma unroll
  for (int j = 0; j < G; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      xp[j][h] = g.a + (static_cast<size_t>(t.row0 + min(j * 16 + h * 8 + lr, t.rows - 1)) * row_bytes + ch * 16) * kRaw;

  struct Block {
    u32x4 w[2][2], x[G][2][kRaw];
  };
  const u32x4 zero = {0u, 0u, 0u, 0u};
  const auto load_w = [&](Block& b, int step) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (T::kPacked) {
        b.w[i][0] = __builtin_amdgcn_raw_buffer_load_b128(wb, wat[i], step * 2048, kPolicy);
        b.w[i][1] = __builtin_amdgcn_raw_buffer_load_b128(wb, wat[i] + 1024u, step * 2048, kPolicy);
      } else {  // a lane past K reads zero: what lies there may be no number
        const int left = row_bytes - step * 128;
        b.w[i][0] = __builtin_amdgcn_raw_buffer_load_b128(wb, q * 16 < left ? wat[i] : kPastEnd, step * 128, kPolicy);
        b.w[i][1] = __builtin_amdgcn_raw_buffer_load_b128(wb, q * 16 + 64 < left ? wat[i] + 64u : kPastEnd, step * 128,
                                                          kPolicy);
      }
    }
  };
  const auto load_x = [&](Block& b, int step) {
    const bool in = step * 128 + ch * 16 < row_bytes;  // a last step may be short
    const int at = (in ? step * 128 : -ch * 16) * kRaw;  // the row's first chunk, then made zero
#pragma unroll
    for (int j = 0; j < G; ++j) {
      if (j >= live) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < kRaw; ++i) {
          b.x[j][h][i] = reinterpret_cast<const u32x4*>(xp[j][h] + at)[i];
          if (!in) b.x[j][h][i] = zero;
        }
    }
  };

  Acc acc[2][G];
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int j = 0; j < G; ++j) acc[f][j] = Acc{};
  uint8_t* const mine = lds + wave * kTurn;
  // 16 rows of 128 bytes: chunk x of row r lies at x ^ (r % 8)
  const auto put = [&](int piece, u32x4 a, u32x4 b) {
    u32x4* p = reinterpret_cast<u32x4*>(mine + piece * 2048 + lr * 128 + ((ch ^ lr) << 4));
    wave_lds_order();  // what was there has been read
    p[0] = a;
    p[64] = b;
    wave_lds_order();
  };
  const auto multiply = [&](const Block& b) {
#pragma unroll
    for (int j = 0; j < G; ++j) {
      if (j >= live) continue;
      if constexpr (QUANT) {
        u32x4 code[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float inv = inv_of[j * 16 + h * 8 + lr];
          const uint2 lo = int8x8(b.x[j][h][0], inv), hi = int8x8(b.x[j][h][1], inv);
          code[h] = u32x4{lo.x, lo.y, hi.x, hi.y};
        }
        put(j & 1, code[0], code[1]);
      } else {
        put(j & 1, b.x[j][0][0], b.x[j][1][0]);
      }
      const uint8_t* p = mine + (j & 1) * 2048 + c * 128;
      const u32x4 x0 = *reinterpret_cast<const u32x4*>(p + ((q ^ (c & 7)) << 4));
      const u32x4 x1 = *reinterpret_cast<const u32x4*>(p + (((q + 4) ^ (c & 7)) << 4));
#pragma unroll
      for (int f = 0; f < 2; ++f) {
        acc[f][j] = T::mma(b.w[f][0], x0, acc[f][j]);
        acc[f][j] = T::mma(b.w[f][1], x1, acc[f][j]);
      }
    }
  };
  Block b0, b1;
  if (wave < steps) {
    load_w(b0, wave);
    load_x(b0, wave);
  }
  if constexpr (QUANT) {
    for (int r = wave; r < 16 * G; r += kSmallWaves) {
      uint32_t m = 0u;
      if (r < t.rows) {
        const uint16_t* row = reinterpret_cast<const uint16_t*>(g.a) + static_cast<size_t>(t.row0 + r) * g.K;
        for (int k = lane * 8; k < g.K; k += 512) m = max(m, amax_bits8(*reinterpret_cast<const u32x4*>(row + k)));
      }
      const RowScale s = row_scale(wave_max_u32(m));
      if (lane == 0) {
        inv_of[r] = s.inv;
        scale_of[r] = s.scale;
      }
    }
    __syncthreads();
  }
  for (int step = wave; step < steps; step += 2 * kSmallWaves) {
    if (step + kSmallWaves < steps) {
      load_w(b1, step + kSmallWaves);
      load_x(b1, step + kSmallWaves);
    }
    multiply(b0);
    if (step + kSmallWaves >= steps) break;
    if (step + 2 * kSmallWaves < steps) {
      load_w(b0, step + 2 * kSmallWaves);
      load_x(b0, step + 2 * kSmallWaves);
    }
    multiply(b1);
  }

  // join: wave j adds up group j
#pragma unroll
  for (int f = 0; f < 2; ++f) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < G; ++j)
      if (j < live) reinterpret_cast<Acc*>(lds)[(wave * G + j) * kWave + lane] = acc[f][j];
    __syncthreads();
    if (wave < live) {
      Acc v{};
#pragma unroll
      for (int w = 0; w < kSmallWaves; ++w) v += reinterpret_cast<const Acc*>(lds)[(w * G + wave) * kWave + lane];
      const int r = wave * 16 + c, n = t.n0 + f * 16 + 4 * q;
      if (r < t.rows && n < g.N) {
        float rs = 1.f;
        if constexpr (T::kBytes == 1) rs = QUANT ? scale_of[r] : g.a_s[t.row0 + r];
        const f32x4 cs = nt_cols<T>(g, t, n);
        nt_store_as<T, MODE>(g, g.N, [&](auto f32_c, auto whole_c) __attribute__((always_inline)) {
          nt_store<T, MODE, decltype(f32_c)::value, decltype(whole_c)::value>(
              g, static_cast<size_t>(t.row0 + r) * g.N + n, g.N, n, v, rs, cs, 1.f);
        });
      }
    }
  }
}

template <typename T, int MODE, int G, bool QUANT, bool ONCE = true>
hipError_t launch_small(const NtArgs& g, hipStream_t stream) {
  return launch_tiles(reinterpret_cast<const void*>(&small_kernel<T, MODE, G, QUANT, ONCE>),
                      row_tiles<MODE, 16 * G, kSmallN>(g), kSmallWaves * kWave, g, stream);
}

}  // namespace moe
