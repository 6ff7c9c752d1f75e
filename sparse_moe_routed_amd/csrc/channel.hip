// Products in 8-bit integers with one fp32 scale per token and one per output
// channel,
//   y[m, n] = (sum_k q_x[m, k] q_w[n, k]) s_x[m] s_w[n]
// as a dense product (moe_channel_matmul, moe_channel_linear) and as the grouped
// expert products of an "int8" bank (moe_forward).  The sum is exact in int32 (K is
// at most 65536, so it stays below 2^30.1), whatever order it is taken in; the two
// scales are two fp32 multiplies of its fp32 value, so a result is off by at most
// three fp32 roundings before its own.
#include "channel_quant.h"
#include "nt.h"

namespace moe {

namespace {

__global__ __launch_bounds__(kQThreads) void channel_quant_kernel(BlockQuantArgs q, const int32_t* n_rows) {
  const int rows = n_rows ? min(max(*n_rows, 0), q.rows) : q.rows;
  row_quantise(q, rows, blockIdx.x, gridDim.x);
}

// where the eight codes from column k (a multiple of 8) of weight row n lie in a
// packed matrix of `steps` steps of 128
__device__ __forceinline__ size_t packed_at(int n, int k, int steps) {
  const int ch = (k & 127) >> 4;
  return (static_cast<size_t>(n >> 4) * steps + (k >> 7)) * 2048 + (ch >> 2) * 1024 + ((ch & 3) * 16 + (n & 15)) * 16 +
         (k & 8);
}

// a wave per weight row; rows past N and columns past K become zero
__global__ __launch_bounds__(kQThreads) void channel_pack_kernel(const uint16_t* __restrict__ w, int N, int K,
                                                                 uint8_t* __restrict__ codes,
                                                                 float* __restrict__ scales) {
  const int steps = (K + 127) / 128, n16 = (N + 15) / 16 * 16;
  const int n = blockIdx.x * (kQThreads / 64) + (threadIdx.x >> 6);
  if (n >= n16) return;
  const uint16_t* const row = w + (static_cast<size_t>(blockIdx.y) * N + min(n, N - 1)) * K;
  uint8_t* const out = codes + static_cast<size_t>(blockIdx.y) * n16 * steps * 128;
  const float s = quantise_row(row, K, [&](int k, uint2 c) {
    *reinterpret_cast<uint2*>(out + packed_at(n, k, steps)) = n < N ? c : make_uint2(0u, 0u);
  });
  for (int k = K + (threadIdx.x & 63) * 8; k < steps * 128; k += 512)
    *reinterpret_cast<uint2*>(out + packed_at(n, k, steps)) = make_uint2(0u, 0u);
  if (n < N && (threadIdx.x & 63) == 0) scales[static_cast<size_t>(blockIdx.y) * N + n] = s;
}

// row-major codes [N, K] into the packed order, 8 bytes a thread
__global__ __launch_bounds__(kQThreads) void channel_pack_codes_kernel(const uint8_t* __restrict__ q, int N, int K,
                                                                       uint8_t* __restrict__ codes) {
  const int steps = (K + 127) / 128, n16 = (N + 15) / 16 * 16;
  const int64_t total = static_cast<int64_t>(n16) * steps * 16;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kQThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kQThreads) {
    const int n = static_cast<int>(i / (steps * 16)), k = static_cast<int>(i % (steps * 16)) * 8;
    uint2 v = make_uint2(0u, 0u);
    if (n < N && k < K) v = *reinterpret_cast<const uint2*>(q + static_cast<size_t>(n) * K + k);
    *reinterpret_cast<uint2*>(codes + packed_at(n, k, steps)) = v;
  }
}

// ---- few rows: 32 weight rows x 16 G rows per workgroup, the steps of K dealt to 8
// waves, each one step ahead of its products; the waves' sums are joined through LDS.
// The rows' codes come a line at a time (8 lanes to 128 bytes) and are turned into
// operand order in LDS that belongs to the wave.  With QUANT the rows are bf16: the
// workgroup first takes the maxima of whole rows, while its first weights are on
// their way, then makes the codes as the steps go.
constexpr int kSmallWaves = 8;
constexpr int kSmallN = 32;

template <int G, bool QUANT, bool ONCE>
__global__ __launch_bounds__(kSmallWaves * kWave) void channel_small_kernel(NtArgs g) {
  constexpr int kTurn = 4096, kJoin = G * 1024;
  constexpr int kRaw = QUANT ? 2 : 1;  // 16-byte loads per 16 values
  constexpr int kPolicy = ONCE ? 2 : 0;
  __shared__ __attribute__((aligned(16))) uint8_t lds[kSmallWaves * (kTurn > kJoin ? kTurn : kJoin)];
  __shared__ float inv_of[QUANT ? 16 * G : 1], scale_of[QUANT ? 16 * G : 1];
  NtTile t;
  if (!nt_find<NtInt8, kNtDense, 16 * G, kSmallN>(g, t)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, q = lane >> 4;
  const int K = g.K, steps = (K + 127) / 128;
  const int lr = lane >> 3, ch = lane & 7;  // row of 8 and 16-value chunk this lane loads
  // groups of 16 rows that hold any
  const int live = __builtin_amdgcn_readfirstlane((t.rows + 15) >> 4);

  // two groups of weight rows; the second may lie past N and is then not read
  const uint32_t group_bytes = steps * 2048u;
  const bool two = t.n0 + 16 < g.N;
  const Buffer wb = buffer_of(t.w + static_cast<size_t>(t.n0 / 16) * group_bytes, (two ? 2u : 1u) * group_bytes);
  const uint32_t wat[2] = {lane * 16u, two ? lane * 16u + group_bytes : kPastEnd};
  const uint8_t* xp[G][2];
#pragma unroll
  for (int j = 0; j < G; ++j)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      xp[j][h] = g.a + (static_cast<size_t>(t.row0 + min(j * 16 + h * 8 + lr, t.rows - 1)) * K + ch * 16) * kRaw;

  struct Block {
    u32x4 w[2][2], x[G][2][kRaw];
  };
  const u32x4 zero = {0u, 0u, 0u, 0u};
  const auto load_w = [&](Block& b, int step) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      b.w[i][0] = __builtin_amdgcn_raw_buffer_load_b128(wb, wat[i], step * 2048, kPolicy);
      b.w[i][1] = __builtin_amdgcn_raw_buffer_load_b128(wb, wat[i] + 1024u, step * 2048, kPolicy);
    }
  };
  const auto load_x = [&](Block& b, int step) {
    const bool in = step * 128 + ch * 16 < K;  // a last step may be short
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

  i32x4 acc[2][G];
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int j = 0; j < G; ++j) acc[f][j] = i32x4{0, 0, 0, 0};
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
        acc[f][j] = NtInt8::mma(b.w[f][0], x0, acc[f][j]);
        acc[f][j] = NtInt8::mma(b.w[f][1], x1, acc[f][j]);
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
        const uint16_t* row = reinterpret_cast<const uint16_t*>(g.a) + static_cast<size_t>(t.row0 + r) * K;
        for (int k = lane * 8; k < K; k += 512) m = max(m, amax_bits8(*reinterpret_cast<const u32x4*>(row + k)));
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
      if (j < live) reinterpret_cast<i32x4*>(lds)[(wave * G + j) * kWave + lane] = acc[f][j];
    __syncthreads();
    if (wave < live) {
      i32x4 v = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < kSmallWaves; ++w) v += reinterpret_cast<const i32x4*>(lds)[(w * G + wave) * kWave + lane];
      const int r = wave * 16 + c, n = t.n0 + f * 16 + 4 * q;
      if (r < t.rows && n < g.N)
        nt_store<NtInt8, kNtDense>(g, t.row0 + r, n, v, QUANT ? scale_of[r] : g.a_s[t.row0 + r],
                                   nt_cols<NtInt8>(g, t, n));
    }
  }
}

template <int G, bool QUANT, bool ONCE = true>
hipError_t launch_small(const NtArgs& g, hipStream_t stream) {
  return launch_tiles(reinterpret_cast<const void*>(&channel_small_kernel<G, QUANT, ONCE>),
                      nt_tiles<NtInt8, kNtDense, 16 * G, kSmallN>(g), kSmallWaves * kWave, g, stream);
}

}  // namespace

hipError_t launch_channel_experts(int stage, const NtArgs& g, hipStream_t stream, const KernelEvents& ev) {
  if (g.M < (16 * g.E > 256 ? 16 * g.E : 256))
    return stage == 0 ? launch_nt<NtInt8, kNtUp, 32, 64, 1, 4, 4, 4, true>(g, stream, ev)
                      : launch_nt<NtInt8, kNtDown, 32, 64, 1, 4, 4, 4, true>(g, stream, ev);
  return stage == 0 ? launch_nt<NtInt8, kNtUp, 128, 128, 2, 2, 4, 2>(g, stream, ev)
                    : launch_nt<NtInt8, kNtDown, 128, 128, 2, 2, 4, 2>(g, stream, ev);
}

constexpr int kFill = 200;  // tiles that fill the chip
hipError_t launch_channel_dense(const NtArgs& g, hipStream_t stream) {
  if (g.M <= 16) return launch_small<1, false>(g, stream);
  if (g.M <= 32) return launch_small<2, false>(g, stream);
  if (g.M <= 64) return launch_small<4, false>(g, stream);
  if (g.M <= 128) return launch_small<4, false, false>(g, stream);  // two row tiles
  const auto fills = [&](long long bm, long long bn) {
    return ((g.M + bm - 1) / bm) * ((g.N + bn - 1) / bn) >= kFill;
  };
  if (fills(256, 256)) return launch_nt<NtInt8, kNtDense, 256, 256, 2, 4, 4, 2>(g, stream);
  if (fills(128, 256)) return launch_nt<NtInt8, kNtDense, 128, 256, 1, 8, 4, 2>(g, stream);
  if (fills(128, 128)) return launch_nt<NtInt8, kNtDense, 128, 128, 2, 4, 4, 2>(g, stream);
  if (fills(64, 128)) return launch_nt<NtInt8, kNtDense, 64, 128, 2, 4, 4, 2>(g, stream);
  return launch_nt<NtInt8, kNtDense, 64, 64, 2, 4, 4, 4>(g, stream);
}

// at most kChannelFewRows bf16 rows, quantised by every workgroup that takes them
hipError_t launch_channel_few_linear(const NtArgs& g, hipStream_t stream) {
  return g.M <= 16 ? launch_small<1, true>(g, stream) : launch_small<2, true>(g, stream);
}

hipError_t launch_channel_quant(const BlockQuantArgs& q, const int32_t* n_rows, hipStream_t stream) {
  if (q.rows <= 0) return hipSuccess;
  hipLaunchKernelGGL(channel_quant_kernel, dim3(quant_groups(q)), dim3(kQThreads), 0, stream, q, n_rows);
  return hipGetLastError();
}

hipError_t launch_channel_pack_codes(const uint8_t* q, int N, int K, uint8_t* codes, hipStream_t stream) {
  const int64_t n = static_cast<int64_t>((N + 15) / 16 * 16) * ((K + 127) / 128) * 16;
  const int64_t blocks = (n + kQThreads - 1) / kQThreads;
  hipLaunchKernelGGL(channel_pack_codes_kernel, dim3(static_cast<unsigned>(blocks < 8192 ? blocks : 8192)),
                     dim3(kQThreads), 0, stream, q, N, K, codes);
  return hipGetLastError();
}

hipError_t launch_channel_pack(const uint16_t* w, int E, int N, int K, uint8_t* codes, float* scales,
                               hipStream_t stream) {
  const int n16 = (N + 15) / 16 * 16;
  hipLaunchKernelGGL(channel_pack_kernel, dim3((n16 + kQThreads / 64 - 1) / (kQThreads / 64), E), dim3(kQThreads), 0,
                     stream, w, N, K, codes, scales);
  return hipGetLastError();
}

}  // namespace moe
