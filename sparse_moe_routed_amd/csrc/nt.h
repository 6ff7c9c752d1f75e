// Products of rows with weight rows, both with K contiguous:
//   out[m, n] = sum_k a[m, k] w[n, k]
// over one matrix or over groups of rows with a matrix each, in bf16 or in 8-bit
// integers.  Sums are fp32 of exact products, or exact int32.
//
// Both types take the same path because a step of K is 128 bytes of a row in both:
// 64 bf16 or 128 integers, two instructions of 16 x 16 results whose operands are
// one 16-byte chunk per lane (row lane % 16, chunk lane / 16 of four).
#pragma once
#include <hip/hip_runtime.h>
#include <type_traits>

#include "moe_common.h"
#include "moe_internal.h"
#include "tile.h"

namespace moe {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

// Element types.  kPacked: weights in operand order, for each 16 rows and 128 bytes
// of K 2 KB, [half][lane][16 bytes] = row lane % 16, chunk 4 half + lane / 16 of the
// step; zeros past N and K.  Otherwise row-major.
struct NtBf16 {
  typedef f32x4 Acc;
  static constexpr int kBytes = 2;
  static constexpr bool kPacked = false;
  static __device__ __forceinline__ Acc mma(u32x4 w, u32x4 x, Acc c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w), __builtin_bit_cast(bf16x8, x), c,
                                                   0, 0, 0);
  }
};
struct NtInt8 {
  typedef i32x4 Acc;
  static constexpr int kBytes = 1;
  static constexpr bool kPacked = true;
  static __device__ __forceinline__ Acc mma(u32x4 w, u32x4 x, Acc c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, w), __builtin_bit_cast(i32x4, x), c, 0, 0,
                                                 0);
  }
};

// what becomes of the sums
enum NtMode {
  kNtDense = 0,   // one matrix: out = sum (times the two scales), bf16 or fp32
  kNtGroups = 1,  // groups of consecutive rows: the same
  kNtUp = 2,      // experts, rows gathered through sorted_src: bf16(relu(h)^2)
  kNtDown = 3     // experts: fp32 gate * h
};

struct NtTile {
  int row0, rows, n0;
  const uint8_t* w;    // the matrix
  const float* w_s;
};

// bytes of a matrix of N weight rows
template <typename T>
__host__ __device__ __forceinline__ size_t nt_matrix_bytes(int N, int K) {
  return T::kPacked ? static_cast<size_t>((N + 15) / 16) * ((K * T::kBytes + 127) / 128) * 2048
                    : static_cast<size_t>(N) * K * T::kBytes;
}

template <typename T, int MODE, int BM, int BN>
__device__ __forceinline__ bool nt_find(const NtArgs& g, NtTile& t) {
  const int n_nt = (g.N + BN - 1) / BN;
  int e = 0, nt;
  if constexpr (MODE == kNtDense) {
    const int n_mt = (g.M + BM - 1) / BM, total = n_nt * n_mt, per_xcd = (total + 7) >> 3;
    const int local = blockIdx.x >> 3;
    const int logical = (blockIdx.x & 7) * per_xcd + local;
    if (local >= per_xcd || logical >= total) return false;
    nt = logical / n_mt;
    const int mt = logical - nt * n_mt;
    t.row0 = mt * BM;
    t.rows = min(BM, g.M - t.row0);
  } else {
    GroupTile p;
    if (!find_group_tile<BM>(g.offsets, g.E, g.M, n_nt, p)) return false;
    e = p.e;
    nt = p.nt;
    t.row0 = p.row0;
    t.rows = p.rows;
  }
  t.n0 = nt * BN;
  const int ew = MODE != kNtDense && g.w_slot ? g.w_slot[e] : e;
  t.w = g.w + static_cast<size_t>(ew) * nt_matrix_bytes<T>(g.N, g.K);
  t.w_s = T::kBytes == 1 ? g.w_s + static_cast<size_t>(e) * g.N : nullptr;
  return true;
}

// row of a behind row r
template <int MODE>
__device__ __forceinline__ size_t nt_source(const NtArgs& g, int r) {
  return MODE == kNtUp ? static_cast<size_t>(g.sorted_src[r] / g.top_k) : static_cast<size_t>(r);
}

// the scaled sum; a zero sum stays 0 whatever finite scales multiply to
__device__ __forceinline__ float nt_value(float v, float, float) { return v; }
__device__ __forceinline__ float nt_value(int32_t v, float row, float col) {
  return static_cast<float>(v) * row * col;
}

// the scales of weight rows n .. n + 3 (1 for bf16)
template <typename T>
__device__ __forceinline__ f32x4 nt_cols(const NtArgs& g, const NtTile& t, int n) {
  f32x4 s = {1.f, 1.f, 1.f, 1.f};
  if constexpr (T::kBytes == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = t.w_s[min(n + i, g.N - 1)];
  }
  return s;
}

// four results of row `row` (of all rows): weight rows n .. n + 3
template <typename T, int MODE>
__device__ __forceinline__ void nt_store(const NtArgs& g, int row, int n, typename T::Acc v, float rs, f32x4 cs) {
  f32x4 h;
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = nt_value(v[i], rs, cs[i]);
  const size_t at = static_cast<size_t>(row) * g.N + n;
  const bool whole = g.N % 4 == 0;  // rows of whole quads, and quads aligned
  if (MODE == kNtDown || (MODE != kNtUp && g.out_f32)) {
    float* const o = static_cast<float*>(g.out) + at;
    if constexpr (MODE == kNtDown) {
      const float gate = g.row_gate[row];
#pragma unroll
      for (int i = 0; i < 4; ++i) h[i] *= gate;
    }
    if (whole) {
      *reinterpret_cast<f32x4*>(o) = h;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < g.N) o[i] = h[i];
    }
  } else {
    uint16_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = MODE == kNtUp ? relu_sq_bf16(h[i]) : f32_to_bf16(h[i]);
    uint16_t* const o = static_cast<uint16_t*>(g.out) + at;
    if (whole) {
      *reinterpret_cast<uint2*>(o) = make_uint2(b[0] | (static_cast<uint32_t>(b[1]) << 16),
                                                b[2] | (static_cast<uint32_t>(b[3]) << 16));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < g.N) o[i] = b[i];
    }
  }
}

// Tiles of BM rows x BN weight rows in WM x WN waves, 128 bytes of K a step.  The
// rows go from memory straight into LDS (NBUF buffers, NBUF - 1 steps under way);
// the weights straight into registers (WBUF operands per wave and group, WBUF - 1
// steps under way): a weight is read by the WM waves of a column and no other, while a
// row serves all WN.  ONCE: weights non-temporal, where one workgroup reads them.
template <typename T, int MODE, int BM, int BN, int WM, int WN, int NBUF, int WBUF, bool ONCE>
__global__ __launch_bounds__(WM* WN * 64) void nt_kernel(NtArgs g) {
  typedef typename T::Acc Acc;
  constexpr int NW = WM * WN;
  constexpr int WTM = BM / WM, WTN = BN / WN;
  constexpr int MS = WTM / 16, NS = WTN / 16;  // 16 x 16 products of a wave
  constexpr int QA = BM / 8 / NW;              // loads of 8 rows per wave and step
  constexpr int kRowsAhead = (NBUF - 2) * QA;  // loads that may be under way when a step's rows are there:
  // of rows, and of weights those of steps from this one on issued after its rows.  Loads
  // are spread between the products where rows and weights are both ahead of time;
  // otherwise all at once, rows first.
  constexpr bool kSpread = NBUF == 4 && !ONCE;
  constexpr int kAhead = kRowsAhead + (kSpread ? WBUF / 2 : WBUF - 1) * 2 * NS;
  constexpr int BUF = BM * 128;
  static_assert(QA * 8 * NW == BM, "tile");
  static_assert((NBUF == 2 || NBUF == 4) && (WBUF == 2 || WBUF == 4) && kAhead < 64, "buffers");
  __shared__ __attribute__((aligned(1024))) uint8_t lds0[BUF];
  __shared__ __attribute__((aligned(1024))) uint8_t lds1[BUF];
  __shared__ __attribute__((aligned(1024))) uint8_t lds2[NBUF == 4 ? BUF : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t lds3[NBUF == 4 ? BUF : 16];
  NtTile t;
  if (!nt_find<T, MODE, BM, BN>(g, t)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int c = lane & 15, q = lane >> 4;
  const int row_bytes = g.K * T::kBytes, steps = (row_bytes + 127) / 128, chunks = row_bytes / 16;

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
  // Weights: the wave's groups of 16 rows; the last group stands in for those past
  // N.  A row-major lane past K reads zero (what lies there may be no number).
  const int m0 = wm * WTM, nw0 = wn * WTN;
  const int groups = (g.N - t.n0 - nw0 + 15) / 16;
  const uint8_t* const w_at = T::kPacked ? t.w + static_cast<size_t>(t.n0 + nw0) / 16 * steps * 2048
                                         : t.w + static_cast<size_t>(min(t.n0 + nw0, g.N - 1)) * row_bytes;
  const int held = groups <= 0 ? 0 : (groups < NS ? groups : NS);
  const uint32_t w_bytes = T::kPacked ? static_cast<uint32_t>(held) * steps * 2048u
                                      : static_cast<uint32_t>(max(min(WTN, g.N - t.n0 - nw0), 0)) * row_bytes;
  uint32_t wr[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i)
    wr[i] = T::kPacked ? lane * 16u + max(min(i, groups - 1), 0) * steps * 2048u
                       : static_cast<uint32_t>(max(min(i * 16 + c, g.N - 1 - t.n0 - nw0), 0)) * row_bytes + q * 16u;
  typedef u32x4 Weights[NS][2];
  constexpr int kPolicy = ONCE ? 2 : 0;
  const auto load_w1 = [&](Weights& w, int step, int i) __attribute__((always_inline)) {
    const bool in = step < steps;
    const Buffer b = buffer_of(w_at, in ? w_bytes : 0u);
    if constexpr (T::kPacked) {
      w[i][0] = __builtin_amdgcn_raw_buffer_load_b128(b, wr[i], in ? step * 2048 : 0, kPolicy);
      w[i][1] = __builtin_amdgcn_raw_buffer_load_b128(b, wr[i] + 1024u, in ? step * 2048 : 0, kPolicy);
    } else {
      const int left = chunks - step * 8;
      w[i][0] = __builtin_amdgcn_raw_buffer_load_b128(b, q < left ? wr[i] : kPastEnd, in ? step * 128 : 0, kPolicy);
      w[i][1] = __builtin_amdgcn_raw_buffer_load_b128(b, q + 4 < left ? wr[i] + 64u : kPastEnd, in ? step * 128 : 0,
                                                      kPolicy);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  const auto load_w = [&](Weights& w, int step) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NS; ++i) load_w1(w, step, i);
  };

  // 16-row groups of this wave that hold rows; a wave whose columns all lie past
  // N multiplies nothing
  int live_raw = (t.rows - m0 + 15) >> 4;
  if (groups <= 0) live_raw = 0;
  const int live = __builtin_amdgcn_readfirstlane(live_raw < 0 ? 0 : (live_raw > MS ? MS : live_raw));
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
    const uint8_t* const xrow = buf + m0 * 128;
    u32x4 x[2][2];
    const auto read = [&](u32x4 (&to)[2], int j) __attribute__((always_inline)) {
      to[0] = *reinterpret_cast<const u32x4*>(xrow + j * 2048 + off0);
      to[1] = *reinterpret_cast<const u32x4*>(xrow + j * 2048 + off1);
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
  // those of step + NBUF - 1 start into the buffer that everyone has read, the
  // weights of step + WBUF - 1 into the registers of step - 1, then the products.  A
  // load that nothing uses is not there to be counted, the compiler drops it: a wave
  // without products loads no weights and counts none, and the last steps of all
  // (TAIL, fewer than 4) wait for all that is under way.
  const auto body = [&](int step, const uint8_t* cur, uint8_t* ahead, const Weights& now, Weights& next,
                        auto live_c, auto tail_c) __attribute__((always_inline)) {
    constexpr bool TAIL = decltype(tail_c)::value, kAny = decltype(live_c)::value > 0;
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(TAIL ? 0 : (kAny ? kAhead : kRowsAhead)));
    __asm__ volatile("s_barrier" ::: "memory");
    if constexpr (kAny && !TAIL && kSpread) {
      constexpr int kLoads = QA + NS, kProducts = decltype(live_c)::value * NS;
      const auto issue = [&](int u) __attribute__((always_inline)) {
#pragma unroll
        for (int l = 0; l < kLoads; ++l) {
          if (l * kProducts / kLoads != u) continue;
          if (l < NS) load_w1(next, step + WBUF - 1, l);
          else load_row(step + NBUF - 1, ahead, l - NS);
        }
      };
      compute(cur, now, live_c, issue);
    } else {
      if (!TAIL || NBUF == 2) load_rows(step + NBUF - 1, ahead);
      if (kAny && (!TAIL || WBUF == 2)) load_w(next, step + WBUF - 1);
      if constexpr (kAny) compute(cur, now, live_c, [](int) {});
    }
  };
  const auto run = [&](auto live_c) __attribute__((always_inline)) {
    constexpr bool kAny = decltype(live_c)::value > 0;
    Weights w0, w1, w2, w3;
    load_rows(0, lds0);
    if (NBUF == 4) {
      load_rows(1, lds1);
      load_rows(2, lds2);
    }
    if (kAny) load_w(w0, 0);
    if (kAny && WBUF == 4) {
      load_w(w1, 1);
      load_w(w2, 2);
    }
    // (the buffers' and operands' places are fixed in the code, so that the
    // compiler sees which loads each step has to wait for)
    int step = 0;
    const auto one = [&](auto k_c, auto tail_c) __attribute__((always_inline)) {
      constexpr int k = decltype(k_c)::value, n = k % NBUF, ah = (k + NBUF - 1) % NBUF;
      constexpr int v = k % WBUF, y = (k + WBUF - 1) % WBUF;
      const uint8_t* const cur = n == 0 ? lds0 : (n == 1 ? lds1 : (n == 2 ? lds2 : lds3));
      uint8_t* const ahead = ah == 0 ? lds0 : (ah == 1 ? lds1 : (ah == 2 ? lds2 : lds3));
      Weights& now = v == 0 ? w0 : (v == 1 ? w1 : (v == 2 ? w2 : w3));
      Weights& next = y == 0 ? w0 : (y == 1 ? w1 : (y == 2 ? w2 : w3));
      body(step + k, cur, ahead, now, next, live_c, tail_c);
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
  static_assert(MS == 2 || MS == 4 || MS == 8, "live groups");
  // a ragged group's last rows: products of the 16-row groups that hold rows only
  if (live == 0) run(std::integral_constant<int, 0>{});
  else if (MODE != kNtDense && live <= MS / 2) run(std::integral_constant<int, MS / 2>{});
  else run(std::integral_constant<int, MS>{});
  __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));  // nothing is under way into LDS when the workgroup ends
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const int n = t.n0 + nw0 + i * 16 + 4 * q;
    if (n >= g.N) continue;
    const f32x4 cs = nt_cols<T>(g, t, n);
#pragma unroll
    for (int j = 0; j < MS; ++j) {
      const int r = m0 + j * 16 + c;
      if (j >= live || r >= t.rows) continue;
      float rs = 1.f;
      if constexpr (T::kBytes == 1) rs = g.a_s[nt_source<MODE>(g, t.row0 + r)];
      nt_store<T, MODE>(g, t.row0 + r, n, acc[i][j], rs, cs);
    }
  }
}

template <typename T, int MODE, int BM, int BN>
long long nt_tiles(const NtArgs& g) {
  const long long n_nt = (g.N + BN - 1) / BN;
  if (MODE != kNtDense) return group_tiles(g.M, g.E, BM, n_nt);
  return (n_nt * ((g.M + BM - 1) / BM) + 7) / 8 * 8;
}

// with timing events the kernel's own start and end are stamped
template <typename Args>
hipError_t launch_tiles(const void* kernel, long long blocks, int threads, const Args& g, hipStream_t stream,
                        const KernelEvents& ev = KernelEvents{}) {
  Args a = g;
  void* args[] = {&a};
  const dim3 grid(static_cast<unsigned>(blocks)), block(threads);
  if (ev.start || ev.stop)
    return hipExtLaunchKernel(kernel, grid, block, args, 0, stream, ev.start, ev.stop, 0);
  return hipLaunchKernel(kernel, grid, block, args, 0, stream);
}

template <typename T, int MODE, int BM, int BN, int WM, int WN, int NBUF, int WBUF, bool ONCE = false>
hipError_t launch_nt(const NtArgs& g, hipStream_t stream, const KernelEvents& ev = KernelEvents{}) {
  return launch_tiles(reinterpret_cast<const void*>(&nt_kernel<T, MODE, BM, BN, WM, WN, NBUF, WBUF, ONCE>),
                      nt_tiles<T, MODE, BM, BN>(g), WM * WN * 64, g, stream, ev);
}

}  // namespace moe
