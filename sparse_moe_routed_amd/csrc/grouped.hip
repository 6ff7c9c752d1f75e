// Products of bf16 rows grouped by expert, with both gradients:
//   y[r, n]      = sum_k x[r, k] w[e, n, k]         rows r of expert e
//   dx[r, k]     = sum_n dy[r, n] w[e, n, k]
//   dw[e, n, k] (+)= sum_{r of e} dy[r, n] x[r, k]
// Sums are fp32 of exact products; results are rounded once.
//
// The first has both operands contiguous along the sum and is nt.h's kernel.  In the
// others the sum runs over the rows of a matrix: of w for dx, of dy and x for dw.
// Such an operand goes into LDS as it lies in memory, 64 rows a step, and is turned
// on its way into registers: ds_read_b64_tr_b16 hands lane i of 16 column i of four
// rows, so two of them are the 8 values of the sum that a lane of
// v_mfma_f32_16x16x32_bf16 takes.
#include "nt.h"

namespace moe {

namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));

struct TrArgs {
  int R, N, K;          // rows of all groups, rows and columns of a weight
  const uint16_t* rows; // dy
  const uint16_t* cols; // dx: w [E, N, K]; dw: x [R, K]
  void* out;            // dx [R, K]; dw [E, N, K]
  int out_f32, accumulate;
  int E;
  const int32_t* offsets;
};

struct TrTile {
  int rows, cols;         // of the output tile: valid rows and columns
  int steps;              // of 64 along the sum
  int length;             // of the sum
  const uint8_t* a;       // rows operand at the tile
  const uint8_t* b;       // columns operand at the tile
  uint32_t a_stride, b_stride;  // bytes between rows of memory
  size_t out;             // first value of the output tile
};

// what a reduction row's 32-byte pairs of 16-byte chunks are moved by: the rows that
// the lanes of half a wave read at once (k % 32 in 0..3 and 8..11, then 16..19 and
// 24..27, each then 4 on) lie on distinct banks
__device__ __forceinline__ int tr_swz(int k) { return (k & 3) | ((k >> 3) & 1) << 2; }

// Output tiles of BM x BN in WM x WN waves.  kDw: both operands turned; otherwise the
// rows are contiguous along the sum.  NBUF buffers of 64 values of the sum, NBUF - 1
// steps under way.
template <bool kDw, int BM, int BN, int WM, int WN, int NBUF>
__global__ __launch_bounds__(WM* WN * 64) void tr_kernel(TrArgs g) {
  constexpr int NW = WM * WN, WTM = BM / WM, WTN = BN / WN, MS = WTM / 16, NS = WTN / 16;
  constexpr int ABYTES = BM * 128, BBYTES = BN * 128, BUF = ABYTES + BBYTES;
  constexpr int QA = ABYTES / 1024 / NW, QB = BBYTES / 1024 / NW;  // loads per wave and step
  constexpr int kAhead = (NBUF - 2) * (QA + QB);
  static_assert(QA * NW * 1024 == ABYTES && QB * NW * 1024 == BBYTES, "tile");
  static_assert(BN >= 128 && (!kDw || BM >= 128), "a row of a turned operand covers the banks");
  static_assert(NBUF >= 2 && NBUF <= 4 && kAhead < 64, "buffers");
  __shared__ __attribute__((aligned(1024))) uint8_t lds0[BUF];
  __shared__ __attribute__((aligned(1024))) uint8_t lds1[BUF];
  __shared__ __attribute__((aligned(1024))) uint8_t lds2[NBUF > 2 ? BUF : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t lds3[NBUF > 3 ? BUF : 16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int c = lane & 15, q = lane >> 4;

  TrTile t;
  const int n_ct = (g.K + BN - 1) / BN;
  if constexpr (kDw) {
    // a row of tiles of one expert is one XCD's, the rows of tiles go round: experts
    // of many rows are then shared by all
    const int n_rt = (g.N + BM - 1) / BM;
    const int l = blockIdx.x >> 3, panel = l / n_ct * 8 + (blockIdx.x & 7), ct = l % n_ct;
    if (panel >= g.E * n_rt) return;
    const int e = panel / n_rt, rt = panel - e * n_rt;
    const int lo = min(max(g.offsets[e], 0), g.R), hi = min(max(g.offsets[e + 1], 0), g.R);
    t.length = __builtin_amdgcn_readfirstlane(max(hi - lo, 0));
    if (t.length == 0 && g.accumulate) return;
    t.rows = min(BM, g.N - rt * BM);
    t.cols = min(BN, g.K - ct * BN);
    t.a_stride = g.N * 2u;
    t.b_stride = g.K * 2u;
    const size_t first = __builtin_amdgcn_readfirstlane(lo);
    t.a = reinterpret_cast<const uint8_t*>(g.rows) + first * t.a_stride + rt * BM * 2;
    t.b = reinterpret_cast<const uint8_t*>(g.cols) + first * t.b_stride + ct * BN * 2;
    t.out = (static_cast<size_t>(e) * g.N + rt * BM) * g.K + ct * BN;
  } else {
    GroupTile p;
    if (!find_group_tile<BM>(g.offsets, g.E, g.R, n_ct, p)) return;
    t.length = g.N;
    t.rows = p.rows;
    t.cols = min(BN, g.K - p.nt * BN);
    t.a_stride = g.N * 2u;
    t.b_stride = g.K * 2u;
    t.a = reinterpret_cast<const uint8_t*>(g.rows) + static_cast<size_t>(p.row0) * t.a_stride;
    t.b = reinterpret_cast<const uint8_t*>(g.cols) + (static_cast<size_t>(p.e) * g.N * g.K + p.nt * BN) * 2;
    t.out = static_cast<size_t>(p.row0) * g.K + p.nt * BN;
  }
  t.steps = (t.length + 63) / 64;

  // Turned operands: the descriptor of a step starts at its first row of memory and
  // ends behind its last, so rows past the sum read zero; columns past the matrix are
  // past the end by the lane's offset.  Row k of the step lies at k * width, its pair
  // p of chunks at p ^ tr_swz(k).
  const auto turned_at = [&](int piece, int width_bytes, uint32_t stride, int valid) __attribute__((always_inline)) {
    const int at = piece * 1024 + lane * 16, k = at / width_bytes, ch = at % width_bytes / 16;
    const int col = (((ch >> 1) ^ tr_swz(k)) << 4) + ((ch & 1) << 3);  // first of 8 columns
    return col < valid ? k * stride + col * 2u : kPastEnd;
  };
  uint32_t aa[QA], ba[QB];
#pragma unroll
  for (int i = 0; i < QA; ++i) {
    const int piece = wave * QA + i;
    if constexpr (kDw) {
      aa[i] = turned_at(piece, BM * 2, t.a_stride, t.rows);
    } else {
      const int r = piece * 8 + (lane >> 3);
      aa[i] = static_cast<uint32_t>(min(r, t.rows - 1)) * t.a_stride + ((lane & 7) ^ swz(r)) * 16;
    }
  }
#pragma unroll
  for (int i = 0; i < QB; ++i) ba[i] = turned_at(wave * QB + i, BN * 2, t.b_stride, t.cols);
  const uint32_t a_span = static_cast<uint32_t>(kDw ? 0 : t.rows) * t.a_stride;
  const auto load = [&](int step, uint8_t* buf) __attribute__((always_inline)) {
    const int left = min(t.length - step * 64, 64);  // of the sum's values
    const size_t at = static_cast<size_t>(step) * 64;
    const Buffer bb = buffer_of(t.b + at * t.b_stride, left * t.b_stride);
    if constexpr (kDw) {
      const Buffer ab = buffer_of(t.a + at * t.a_stride, left * t.a_stride);
#pragma unroll
      for (int i = 0; i < QA; ++i) load16_to_lds(ab, aa[i], 0, buf + (wave * QA + i) * 1024);
    } else {
      const Buffer ab = buffer_of(t.a, a_span);
#pragma unroll
      for (int i = 0; i < QA; ++i) {
        const int ch = (lane & 7) ^ swz((wave * QA + i) * 8 + (lane >> 3));
        load16_to_lds(ab, ch * 8 < left ? aa[i] : kPastEnd, step * 128, buf + (wave * QA + i) * 1024);
      }
    }
#pragma unroll
    for (int i = 0; i < QB; ++i) load16_to_lds(bb, ba[i], 0, buf + ABYTES + (wave * QB + i) * 1024);
  };

  const int m0 = wm * WTM, n0 = wn * WTN;
  int live_raw = n0 < t.cols ? (t.rows - m0 + 15) >> 4 : 0;
  const int live = __builtin_amdgcn_readfirstlane(live_raw < 0 ? 0 : (live_raw > MS ? MS : live_raw));
  f32x4 acc[NS][MS];
#pragma unroll
  for (int i = 0; i < NS; ++i)
#pragma unroll
    for (int j = 0; j < MS; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  // a lane's place in a turned operand: row 8 q + c / 4 of 32, column 4 (c % 4) of a pair
  const int tr_row = 8 * q + (c >> 2), f = tr_swz(tr_row);
  const auto turned = [&](const uint8_t* tile, int width_bytes, int pair, int h) __attribute__((always_inline)) {
    const uint8_t* p = tile + (h * 32 + tr_row) * width_bytes + ((pair ^ f) << 5) + ((c & 3) << 3);
    typedef __attribute__((address_space(3))) s16x4* Lds;
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(p));
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Lds)(p + 4 * width_bytes));
    return __builtin_bit_cast(
        bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  };
  const auto compute = [&](const uint8_t* buf, auto live_c) __attribute__((always_inline)) {
    constexpr int ML = decltype(live_c)::value;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      bf16x8 w[NS], x[ML];
#pragma unroll
      for (int i = 0; i < NS; ++i) w[i] = turned(buf + ABYTES, BN * 2, n0 / 16 + i, h);
#pragma unroll
      for (int j = 0; j < ML; ++j) {
        if constexpr (kDw) {
          x[j] = turned(buf, BM * 2, m0 / 16 + j, h);
        } else {
          const int ch = (q + 4 * h) ^ swz(c);
          x[j] = *reinterpret_cast<const bf16x8*>(buf + (m0 + j * 16 + c) * 128 + (ch << 4));
        }
      }
#pragma unroll
      for (int j = 0; j < ML; ++j)
#pragma unroll
        for (int i = 0; i < NS; ++i)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[i], x[j], acc[i][j], 0, 0, 0);
    }
    __builtin_amdgcn_sched_barrier(0);  // what was read has been read before the next barrier
  };
  const auto run = [&](auto live_c) __attribute__((always_inline)) {
    constexpr bool kAny = decltype(live_c)::value > 0;
    if (t.steps > 0) load(0, lds0);
    if (NBUF > 2 && t.steps > 1) load(1, lds1);
    if (NBUF > 3 && t.steps > 2) load(2, lds2);
    int step = 0;
    const auto one = [&](auto k_c) __attribute__((always_inline)) {
      constexpr int k = decltype(k_c)::value, n = k % NBUF, ah = (k + NBUF - 1) % NBUF;
      const uint8_t* const cur = n == 0 ? lds0 : (n == 1 ? lds1 : (n == 2 ? lds2 : lds3));
      uint8_t* const ahead = ah == 0 ? lds0 : (ah == 1 ? lds1 : (ah == 2 ? lds2 : lds3));
      // this step's have arrived (this wave's, then at the barrier everyone's); at
      // the end fewer are under way
      if (step + k + NBUF - 2 < t.steps) __builtin_amdgcn_s_waitcnt(vmcnt_imm(kAhead));
      else __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
      __asm__ volatile("s_barrier" ::: "memory");
      if (step + k + NBUF - 1 < t.steps) load(step + k + NBUF - 1, ahead);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (kAny) compute(cur, live_c);
    };
    constexpr std::integral_constant<int, 0> k0{};
    constexpr std::integral_constant<int, 1> k1{};
    constexpr std::integral_constant<int, 2> k2{};
    constexpr std::integral_constant<int, 3> k3{};
    while (true) {
      if (step >= t.steps) break;
      one(k0);
      if (step + 1 >= t.steps) break;
      one(k1);
      if (NBUF > 2) {
        if (step + 2 >= t.steps) break;
        one(k2);
      }
      if (NBUF > 3) {
        if (step + 3 >= t.steps) break;
        one(k3);
      }
      step += NBUF;
    }
  };
  if (live == 0) run(std::integral_constant<int, 0>{});
  else if (MS > 1 && live <= MS / 2) run(std::integral_constant<int, MS / 2>{});
  else run(std::integral_constant<int, MS>{});

#pragma unroll
  for (int j = 0; j < MS; ++j) {
    const int r = m0 + j * 16 + c;
    if (j >= live || r >= t.rows) continue;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int n = n0 + i * 16 + 4 * q;
      if (n >= t.cols) continue;  // columns come in eights, so a quad is whole
      const size_t at = t.out + static_cast<size_t>(r) * g.K + n;
      f32x4 v = acc[i][j];
      if (g.out_f32) {
        f32x4* const o = reinterpret_cast<f32x4*>(static_cast<float*>(g.out) + at);
        if (kDw && g.accumulate) v += *o;
        *o = v;
      } else {
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(g.out) + at) =
            make_uint2(f32_to_bf16(v[0]) | (static_cast<uint32_t>(f32_to_bf16(v[1])) << 16),
                       f32_to_bf16(v[2]) | (static_cast<uint32_t>(f32_to_bf16(v[3])) << 16));
      }
    }
  }
}

// rows of no expert, [offsets[E], R), set to zero: 16 bytes a thread
__global__ __launch_bounds__(256) void zero_rest_kernel(const int32_t* __restrict__ offsets, int E, int R,
                                                        size_t row_bytes, uint8_t* __restrict__ out) {
  const int from = min(max(offsets[E], 0), R);
  const size_t end = static_cast<size_t>(R) * row_bytes;
  const u32x4 zero = {0u, 0u, 0u, 0u};
  for (size_t i = static_cast<size_t>(from) * row_bytes + (static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x) * 16;
       i < end; i += static_cast<size_t>(gridDim.x) * 256 * 16)
    *reinterpret_cast<u32x4*>(out + i) = zero;
}

template <bool kDw, int BM, int BN, int WM, int WN, int NBUF>
hipError_t launch_tr(const TrArgs& g, hipStream_t stream) {
  const long long n_ct = (g.K + BN - 1) / BN, n_rt = (g.N + BM - 1) / BM;
  const long long blocks = kDw ? (g.E * n_rt + 7) / 8 * 8 * n_ct : group_tiles(g.R, g.E, BM, n_ct);
  return launch_tiles(reinterpret_cast<const void*>(&tr_kernel<kDw, BM, BN, WM, WN, NBUF>), blocks,
                      WM * WN * 64, g, stream);
}

hipError_t launch_zero_rest(const GroupedArgs& g, int width, hipStream_t stream) {
  hipLaunchKernelGGL(zero_rest_kernel, dim3(256), dim3(256), 0, stream, g.offsets, g.E, g.R,
                     static_cast<size_t>(width) * (g.out_f32 ? 4 : 2), static_cast<uint8_t*>(g.out));
  return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_matmul(const GroupedArgs& g, hipStream_t stream) {
  NtArgs a{};
  a.M = a.a_rows = g.R;
  a.N = g.N;
  a.K = g.K;
  a.a = static_cast<const uint8_t*>(g.x);
  a.w = static_cast<const uint8_t*>(g.w);
  a.out = g.out;
  a.out_f32 = g.out_f32;
  a.E = g.E;
  a.offsets = g.offsets;
  const hipError_t err = g.R < 16 * g.E ? launch_nt<NtBf16, kNtGroups, 32, 64, 1, 4, 4, 4, true>(a, stream)
                                        : launch_nt<NtBf16, kNtGroups, 128, 128, 2, 2, 4, 2>(a, stream);
  return err == hipSuccess && g.zero_rest ? launch_zero_rest(g, g.N, stream) : err;
}

hipError_t launch_grouped_input_grad(const GroupedArgs& g, hipStream_t stream) {
  const TrArgs a{g.R, g.N, g.K, static_cast<const uint16_t*>(g.dy), static_cast<const uint16_t*>(g.w), g.out,
                 g.out_f32, 0, g.E, g.offsets};
  const hipError_t err = g.R < 16 * g.E ? launch_tr<false, 32, 128, 1, 4, 4>(a, stream)
                                        : launch_tr<false, 128, 128, 2, 2, 2>(a, stream);
  return err == hipSuccess && g.zero_rest ? launch_zero_rest(g, g.K, stream) : err;
}

hipError_t launch_grouped_weight_grad(const GroupedArgs& g, hipStream_t stream) {
  const TrArgs a{g.R, g.N, g.K, static_cast<const uint16_t*>(g.dy), static_cast<const uint16_t*>(g.x), g.out,
                 g.out_f32, g.accumulate, g.E, g.offsets};
  return launch_tr<true, 128, 128, 2, 2, 2>(a, stream);
}

}  // namespace moe
