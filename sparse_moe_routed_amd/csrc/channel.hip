// Products in 8-bit integers with one fp32 scale per token and one per output
// channel,
//   y[m, n] = (sum_k q_x[m, k] q_w[n, k]) s_x[m] s_w[n]
// as a dense product (moe_channel_matmul, moe_channel_linear) and as the grouped
// expert products of an "int8" bank (moe_forward).  The sum is exact in int32 (K is
// at most 65536, so it stays below 2^30.1), whatever order it is taken in; the two
// scales are two fp32 multiplies of its fp32 value, so a result is off by at most
// three fp32 roundings before its own.
#include "channel_quant.h"
#include "products.h"
#include "small.h"
#include "tile_gemm.h"

namespace moe {

namespace {

// a wave per row, read once: 4096 x 2688 8.5 us, 33 MB at 3.9 TB/s
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

// a wave per weight row; rows past N and columns past K become zero.  128 x 2688 x 1856
// 570 us, 1.9 GB at 3.4 TB/s: done once, when weights are loaded
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

// Tiles of BM rows x BN weight rows in WM x WN waves, 128 bytes of K a step.  The
// rows go from memory straight into LDS (4 buffers, 3 steps under way);
// the weights straight into registers (WBUF operands per wave and group, WBUF - 1
// steps under way): a weight is read by the WM waves of a column and no other, while a
// row serves all WN.  ONCE: weights non-temporal, where one workgroup reads them
// (as with experts of up to 32 rows; a single expert of 255 has them read eight times).
// Bound by the weights: at 2688 x 1856 and 107 experts of 3.6 rows tiles of 32 x 64 read
// them at 6.2 to 6.5 TB/s (82 and 86 us).  With 192 rows an expert tiles of 128 x 128 move 4.3
// and 4.1 TB/s of weights, rows and results (216 and 247 us), the matrix unit 31 and 25 %
// busy: neither is full.
template <int MODE, int BM, int BN, int WM, int WN, int WBUF, bool ONCE>
__global__ __launch_bounds__(WM* WN * 64) void channel_tile_kernel(NtArgs g) {
  typedef NtInt8 T;
  typedef T::Acc Acc;
  constexpr int NW = WM * WN;
  constexpr int WTM = BM / WM, WTN = BN / WN;
  constexpr int MS = WTM / 16, NS = WTN / 16;  // 16 x 16 products of a wave
  constexpr int QA = BM / 8 / NW;              // loads of 8 rows per wave and step
  constexpr int kRowsAhead = 2 * QA;  // loads that may be under way when a step's rows are there:
  // of rows, and of weights those of steps from this one on issued after its rows.  Loads
  // are spread between the products where rows and weights are both ahead of time;
  // otherwise all at once, rows first.
  constexpr bool kSpread = !ONCE;
  constexpr int kAhead = kRowsAhead + (kSpread ? WBUF / 2 : WBUF - 1) * 2 * NS;
  constexpr int BUF = BM * 128;
  static_assert(QA * 8 * NW == BM, "tile");
  static_assert((WBUF == 2 || WBUF == 4) && kAhead < 64, "buffers");
  __shared__ __attribute__((aligned(1024))) uint8_t lds0[BUF];
  __shared__ __attribute__((aligned(1024))) uint8_t lds1[BUF];
  __shared__ __attribute__((aligned(1024))) uint8_t lds2[BUF];
  __shared__ __attribute__((aligned(1024))) uint8_t lds3[BUF];
  NtTile t;
  if (!nt_find<T, MODE, BM, BN>(g, t)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int c = lane & 15, q = lane >> 4;
  const int row_bytes = g.K, steps = (row_bytes + 127) / 128, chunks = row_bytes / 16;

  // Rows: gathered ones are addressed from the first row (fewer than 2^32 bytes,
  // checked by the caller), others from the tile's first.
  const bool gather = MODE == kNtUp;
  const size_t first = gather ? 0 : static_cast<size_t>(t.row0);
  const uint32_t a_bytes = static_cast<uint32_t>(static_cast<size_t>(gather ? g.a_rows : t.rows) * row_bytes);
  const uint8_t* const a = g.a + first * row_bytes;
  uint32_t ar[QA];
#pragma unroll
  for (int i = 0; i < QA; ++i) {
    const int r = (wave * QA + i) * 8 + (lane >> 3);
    const uint32_t row = static_cast<uint32_t>(nt_source<MODE>(g, t.row0 + min(r, t.rows - 1)) - first);
    ar[i] = row * row_bytes + ((lane & 7) ^ swz(r)) * 16;
  }
  const auto load_row = [&](int step, uint8_t* buf, int i) __attribute__((always_inline)) {
    const bool in = step < steps;
    const Buffer b = buffer_of(a, in ? a_bytes : 0u);
    const int ch = (lane & 7) ^ swz((wave * QA + i) * 8 + (lane >> 3));
    load16_to_lds(b, ch < chunks - step * 8 ? ar[i] : kPastEnd, in ? step * 128 : 0, buf + (wave * QA + i) * 1024);
    __builtin_amdgcn_sched_barrier(0);  // the order of the loads is what the waits count on
  };
  const auto load_rows = [&](int step, uint8_t* buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < QA; ++i) load_row(step, buf, i);
  };
  // weights: the wave's groups of 16 rows; the last one stands in for those past N
  const int nw0 = wn * WTN;
  const int groups = (g.N - t.n0 - nw0 + 15) / 16;
  const uint8_t* const w_at = t.w + static_cast<size_t>(t.n0 + nw0) / 16 * steps * 2048;
  const uint32_t w_bytes = static_cast<uint32_t>(groups <= 0 ? 0 : (groups < NS ? groups : NS)) * steps * 2048u;
  typedef u32x4 Weights[NS][2];
  constexpr int kPolicy = ONCE ? 2 : 0;
  const auto load_w1 = [&](Weights& w, int step, int i) __attribute__((always_inline)) {
    const bool in = step < steps;
    const Buffer b = buffer_of(w_at, in ? w_bytes : 0u);
    const uint32_t at = lane * 16u + max(min(i, groups - 1), 0) * steps * 2048u;
    w[i][0] = __builtin_amdgcn_raw_buffer_load_b128(b, at, in ? step * 2048 : 0, kPolicy);
    w[i][1] = __builtin_amdgcn_raw_buffer_load_b128(b, at + 1024u, in ? step * 2048 : 0, kPolicy);
    __builtin_amdgcn_sched_barrier(0);
  };
  const auto load_w = [&](Weights& w, int step) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NS; ++i) load_w1(w, step, i);
  };

  // Row groups of 16 go round the WM waves, so that a ragged tile's are shared out:
  // group j of this wave is j WM + wm.  `live` of them hold rows (the first is
  // multiplied in any case).
  const int live = __builtin_amdgcn_readfirstlane(min(MS, (((t.rows + 15) >> 4) - wm + WM - 1) / WM));
  Acc acc[NS][MS];
#pragma unroll
  for (int i = 0; i < NS; ++i)
#pragma unroll
    for (int j = 0; j < MS; ++j) acc[i][j] = Acc{};
  // this lane's chunk of row c of a 16-row group in either half (groups are 2 KB
  // apart, and a group's first row is a multiple of 16, so its swizzle is c's)
  const int off0 = c * 128 + ((q ^ swz(c)) << 4), off1 = c * 128 + (((q + 4) ^ swz(c)) << 4);
  const auto compute = [&](const uint8_t* buf, const Weights& w, auto live_c, auto issue)
                           __attribute__((always_inline)) {
    constexpr int ML = decltype(live_c)::value;
    const uint8_t* const xrow = buf + wm * 2048;
    u32x4 x[2][2];
    const auto read = [&](u32x4 (&to)[2], int j) __attribute__((always_inline)) {
      to[0] = *reinterpret_cast<const u32x4*>(xrow + j * WM * 2048 + off0);
      to[1] = *reinterpret_cast<const u32x4*>(xrow + j * WM * 2048 + off1);
    };
    read(x[0], 0);
#pragma unroll
    for (int j = 0; j < ML; ++j) {
      if (j + 1 < ML) read(x[(j + 1) & 1], j + 1);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          acc[i][j] = T::mma(w[i][h], x[j & 1][h], acc[i][j]);
          if (h == 1) issue(j * NS + i);
        }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // One step: its rows have arrived (this wave's, then at the barrier everyone's),
  // those of step + 3 start into the buffer that everyone has read, the
  // weights of step + WBUF - 1 into the registers of step - 1, then the products.
  // The last steps of all (TAIL, fewer than 4) wait for all that is under way.
  const auto body = [&](int step, const uint8_t* cur, uint8_t* ahead, const Weights& now, Weights& next,
                        auto live_c, auto tail_c) __attribute__((always_inline)) {
    constexpr bool TAIL = decltype(tail_c)::value;
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(TAIL ? 0 : kAhead));
    __asm__ volatile("s_barrier" ::: "memory");
    if constexpr (!TAIL && kSpread) {
      constexpr int kLoads = QA + NS, kProducts = decltype(live_c)::value * NS;
      compute(cur, now, live_c, [&](int u) __attribute__((always_inline)) {
#pragma unroll
        for (int l = 0; l < kLoads; ++l) {
          if (l * kProducts / kLoads != u) continue;
          if (l < NS) load_w1(next, step + WBUF - 1, l);
          else load_row(step + 3, ahead, l - NS);
        }
      });
    } else {
      if (!TAIL) load_rows(step + 3, ahead);
      if (!TAIL || WBUF == 2) load_w(next, step + WBUF - 1);
      compute(cur, now, live_c, [](int) {});
    }
  };
  const auto run = [&](auto live_c) __attribute__((always_inline)) {
    Weights w0, w1, w2, w3;
    load_rows(0, lds0);
    load_rows(1, lds1);
    load_rows(2, lds2);
    load_w(w0, 0);
    if (WBUF == 4) {
      load_w(w1, 1);
      load_w(w2, 2);
    }
    // (the buffers' and operands' places are fixed in the code, so that the
    // compiler sees which loads each step has to wait for)
    int step = 0;
    const auto one = [&](auto k_c, auto tail_c) __attribute__((always_inline)) {
      constexpr int n = decltype(k_c)::value, ah = (n + 3) % 4;
      constexpr int v = n % WBUF, y = (n + WBUF - 1) % WBUF;
      const uint8_t* const cur = n == 0 ? lds0 : (n == 1 ? lds1 : (n == 2 ? lds2 : lds3));
      uint8_t* const ahead = ah == 0 ? lds0 : (ah == 1 ? lds1 : (ah == 2 ? lds2 : lds3));
      Weights& now = v == 0 ? w0 : (v == 1 ? w1 : (v == 2 ? w2 : w3));
      Weights& next = y == 0 ? w0 : (y == 1 ? w1 : (y == 2 ? w2 : w3));
      body(step + n, cur, ahead, now, next, live_c, tail_c);
    };
    constexpr std::integral_constant<int, 0> k0{};
    constexpr std::integral_constant<int, 1> k1{};
    constexpr std::integral_constant<int, 2> k2{};
    constexpr std::integral_constant<int, 3> k3{};
    for (; step + 4 <= steps; step += 4) {
      one(k0, std::false_type{});
      one(k1, std::false_type{});
      one(k2, std::false_type{});
      one(k3, std::false_type{});
    }
    if (step >= steps) return;
    one(k0, std::true_type{});
    if (step + 1 >= steps) return;
    one(k1, std::true_type{});
    if (step + 2 >= steps) return;
    one(k2, std::true_type{});
  };
  // products of the row groups that hold rows, in quarters of the tile
  constexpr int kQuarter = MS < 4 ? 1 : MS / 4;
  if (live <= kQuarter) run(std::integral_constant<int, kQuarter>{});
  else if (MS > 2 && live <= MS / 2) run(std::integral_constant<int, MS / 2>{});
  else if (MS > 2 && live <= MS / 2 + kQuarter) run(std::integral_constant<int, MS / 2 + kQuarter>{});
  else run(std::integral_constant<int, MS>{});
  __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));  // nothing is under way into LDS when the workgroup ends
  if constexpr (BN >= 128 && BUF >= 16 * WM * BN * 4) {
    const int cols = min(BN, g.N - t.n0);
    const StoreAt to{t.row0, t.rows, t.n0, cols, g.N, static_cast<size_t>(t.row0) * g.N + t.n0, t.w_s};
    const auto buffers = [&](int b) __attribute__((always_inline)) {
      return b == 0 ? (Lds)lds0 : (b == 1 ? (Lds)lds1 : (b == 2 ? (Lds)lds2 : (Lds)lds3));
    };
    store_tile<T, MODE, BM, BN, WM, WN, 4, BUF>(g, to, buffers, acc);
    return;
  }
  float rs[MS], gate[MS];  // all loads at once
  size_t source[MS];
#pragma unroll
  for (int j = 0; j < MS; ++j) {
    const int r = t.row0 + min((j * WM + wm) * 16 + c, t.rows - 1);
    source[j] = nt_source<MODE>(g, r);
    gate[j] = MODE == kNtDown ? g.row_gate[r] : 1.f;
  }
#pragma unroll
  for (int j = 0; j < MS; ++j) rs[j] = g.a_s[source[j]];
  nt_store_as<T, MODE>(g, g.N, [&](auto f32_c, auto whole_c) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int n = t.n0 + nw0 + i * 16 + 4 * q;
      if (n >= g.N) continue;
      const f32x4 cs = nt_cols<T>(g, t, n);
#pragma unroll
      for (int j = 0; j < MS; ++j) {
        const int r = (j * WM + wm) * 16 + c;
        if (r >= t.rows) continue;
        nt_store<T, MODE, decltype(f32_c)::value, decltype(whole_c)::value>(
            g, static_cast<size_t>(t.row0 + r) * g.N + n, g.N, n, acc[i][j], rs[j], cs, gate[j]);
      }
    }
  });
}

template <int MODE, int BM, int BN, int WM, int WN, int WBUF, bool ONCE = false>
hipError_t launch_channel_tile(const NtArgs& g, hipStream_t stream, const KernelEvents& ev = KernelEvents{}) {
  return launch_tiles(reinterpret_cast<const void*>(&channel_tile_kernel<MODE, BM, BN, WM, WN, WBUF, ONCE>),
                      row_tiles<MODE, BM, BN>(g), WM * WN * 64, g, stream, ev);
}

}  // namespace

// Few rows an expert: small tiles, so that many workgroups share the streaming of the
// weights; many: larger ones, which read them fewer times.  The layer of 128 experts,
// 2688 x 1856, 6 a token, us with tiles of 32 x 64 and of 128 x 128: 384 rows 195 and 240;
// 2400 rows 260 and 286; 3600 rows 319 and 306; 24576 rows 1161 and 614 (64 x 128 lie
// between: 238, 284, 303 and 648).  A single expert of every token takes the same tiles,
// which are few for the chip: 2688 -> 3712 -> 2688 of 64 tokens 29 us, 255 39, 1024 53, 4096
// 155; two dense products with their quantisations 27, 27, 41 and 100.
hipError_t launch_channel_experts(int stage, const NtArgs& g, hipStream_t stream, const KernelEvents& ev) {
  if (g.M < (24 * g.E > 256 ? 24 * g.E : 256))
    return stage == 0 ? launch_channel_tile<kNtUp, 32, 64, 1, 4, 4, true>(g, stream, ev)
                      : launch_channel_tile<kNtDown, 32, 64, 1, 4, 4, true>(g, stream, ev);
  return stage == 0 ? launch_channel_tile<kNtUp, 128, 128, 1, 4, 4>(g, stream, ev)
                    : launch_channel_tile<kNtDown, 128, 128, 1, 4, 4>(g, stream, ev);
}

// Tiles by size, us measured at N x K:
//   - few rows: 32 columns a workgroup and the sum dealt to its waves, for up to 32 rows
//     (14336 x 4096, 1 row 10.1, in tiles of 64 x 64 11.7) and, while one round of
//     workgroups covers the columns, up to 128 (3712 x 2688, 100 rows 7.3 and 8.6; but
//     14336 x 4096 32 and 18);
//   - then the largest tile of which there are kFill, which reads least from the caches
//     for each product.  2688 x 1856: 1024 rows 10.6 in the 168 tiles of 128 x 128, 15.6
//     in 64 x 128; 1500 rows 11.7 in 128 x 128, 15.7 in the 132 of 128 x 256; 2048 rows
//     16.3 in 176 of those and 19.2; 4096 rows 28.5 in 176 of 256 x 256, 32 in 128 x 256.
constexpr int kFill = 140;
hipError_t launch_channel_dense(const NtArgs& g, hipStream_t stream) {
  if (g.M <= 16) return launch_small<NtInt8, kNtDense, 1, false>(g, stream);
  if (g.M <= 32) return launch_small<NtInt8, kNtDense, 2, false>(g, stream);
  if (g.N <= 256 * kSmallN) {
    if (g.M <= 64) return launch_small<NtInt8, kNtDense, 4, false>(g, stream);
    if (g.M <= 128) return launch_small<NtInt8, kNtDense, 4, false, false>(g, stream);  // two row tiles
  }
  const auto fills = [&](long long bm, long long bn) {
    return ((g.M + bm - 1) / bm) * ((g.N + bn - 1) / bn) >= kFill;
  };
  if (fills(256, 256)) return launch_tile<NtInt8, kNtDense, 256, 256, 2, 4, 2, 2>(g, stream);
  if (fills(128, 256)) return launch_channel_tile<kNtDense, 128, 256, 1, 8, 2>(g, stream);
  if (fills(128, 128)) return launch_channel_tile<kNtDense, 128, 128, 2, 4, 2>(g, stream);
  if (fills(64, 128)) return launch_channel_tile<kNtDense, 64, 128, 2, 4, 2>(g, stream);
  return launch_channel_tile<kNtDense, 64, 64, 2, 4, 4>(g, stream);
}

// at most kChannelFewRows bf16 rows, quantised by every workgroup that takes them
hipError_t launch_channel_few_linear(const NtArgs& g, hipStream_t stream) {
  return g.M <= 16 ? launch_small<NtInt8, kNtDense, 1, true>(g, stream) : launch_small<NtInt8, kNtDense, 2, true>(g, stream);
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
