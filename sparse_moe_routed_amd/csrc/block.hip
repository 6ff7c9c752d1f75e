// E4M3 products with one fp32 scale per block of 128: of the activations one
// for every 128 values of a row, of the weights one for every 128 x 128 block,
//   y[m, n] = sum_kb s_a[m, kb] s_w[n / 128, kb] sum_{k in kb} q_a[m, k] q_w[n, k]
// as a dense product (moe_block_matmul, moe_block_linear) and as the grouped
// expert products of an "fp8_block" bank (moe_forward).
//
// One v_mfma_f32_16x16x128_f8f6f4 multiplies exactly one K block, so its result
// times the two scales is one fp32 multiply-add into the running sum.  Weights
// are the rows and tokens the columns of the product: a lane's four results
// belong to one token, and s_a s_w is one value per lane.  The instruction sums
// its 128 products with a short significand: against exact sums of E4M3 data
// its result is off by 1.5e-5 of its own size (rms; 6e-5 where one value of a
// row is 100 times the others), far below the bf16 rounding of y (1.7e-3), and
// sums across blocks are fp32.
//
// Codes are stored row-major; K is a multiple of 16.  Scales of activations lie
// block by block, [ceil(K / 128), rows], so that the tokens of one MFMA read
// consecutive words; weight scales are [ceil(N / 128), ceil(K / 128)].
#include <hip/hip_ext.h>

#include "moe_common.h"
#include "moe_internal.h"

namespace moe {

namespace {

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

__device__ __forceinline__ uint2 encode8(u32x4 v, float inv) {
  uint32_t c[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t a = v[2 * h], b = v[2 * h + 1];
    c[h] = e4m3_encode4(__uint_as_float(a << 16) * inv, __uint_as_float(a & 0xffff0000u) * inv,
                        __uint_as_float(b << 16) * inv, __uint_as_float(b & 0xffff0000u) * inv);
  }
  return make_uint2(c[0], c[1]);
}

// max over each row of 16 lanes, in all of them
__device__ __forceinline__ float row16_max(float v) {
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}

// ---- activations: 16 lanes take one block of 128 values, 8 values each
__global__ __launch_bounds__(kQThreads) void block_quant_kernel(
    const uint16_t* __restrict__ x, const int32_t* n_rows_dev, int rows, int cols, int row_stride,
    uint8_t* __restrict__ codes, float* __restrict__ scales) {
  const int nr = n_rows_dev ? min(*n_rows_dev, rows) : rows;
  const int kb_n = (cols + 127) / 128;
  const int l16 = threadIdx.x & 15;
  const int64_t n = static_cast<int64_t>(nr) * kb_n;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kQThreads / 16);
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * (kQThreads / 16) + (threadIdx.x >> 4); i < n;
       i += step) {
    const int r = static_cast<int>(i / kb_n), kb = static_cast<int>(i - static_cast<int64_t>(r) * kb_n);
    const int k = kb * 128 + l16 * 8;
    const size_t at = static_cast<size_t>(r) * cols + k;
    u32x4 v = {0u, 0u, 0u, 0u};
    if (k < cols) v = *reinterpret_cast<const u32x4*>(x + at);
    const float amax = row16_max(amax8(v));
    const bool live = amax >= kTinyAmax;
    if (k < cols)
      *reinterpret_cast<uint2*>(codes + at) = encode8(v, live ? __fdiv_rn(448.f, amax) : 0.f);
    if (l16 == 0)
      scales[static_cast<size_t>(kb) * row_stride + r] = live ? __fdiv_rn(amax, 448.f) : 0.f;
  }
}

// ---- weights: a workgroup per 128 x 128 block; rows of 16 lanes
__global__ __launch_bounds__(kQThreads) void block_pack_kernel(const uint16_t* __restrict__ w, int N,
                                                               int K, uint8_t* __restrict__ codes,
                                                               float* __restrict__ scales) {
  __shared__ float part[kQThreads / 64];
  const int kb = blockIdx.x, nb = blockIdx.y;
  const size_t base = static_cast<size_t>(blockIdx.z) * N * K;
  const int r0 = threadIdx.x >> 4, k = kb * 128 + (threadIdx.x & 15) * 8;
  u32x4 v[8];
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int n = nb * 128 + r0 + 16 * j;
    v[j] = u32x4{0u, 0u, 0u, 0u};
    if (n < N && k < K) v[j] = *reinterpret_cast<const u32x4*>(w + base + static_cast<size_t>(n) * K + k);
    m = fmaxf(m, amax8(v[j]));
  }
  m = wave_max(m);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
  __syncthreads();
  m = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
  const bool live = m >= kTinyAmax;
  const float inv = live ? __fdiv_rn(448.f, m) : 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int n = nb * 128 + r0 + 16 * j;
    if (n < N && k < K)
      *reinterpret_cast<uint2*>(codes + base + static_cast<size_t>(n) * K + k) = encode8(v[j], inv);
  }
  if (threadIdx.x == 0)
    scales[(static_cast<size_t>(blockIdx.z) * gridDim.y + nb) * gridDim.x + kb] =
        live ? __fdiv_rn(m, 448.f) : 0.f;
}

// ---- products
// the tile's expert for grouped products: the largest e with
// tile_off[e] * n_ntiles <= logical (tile_off is nondecreasing from 0)
__device__ __forceinline__ int owner_expert(const int32_t* __restrict__ tile_off, int E,
                                            int n_ntiles, int logical) {
  const int lane = threadIdx.x & 63;
  int cnt = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int e = 1 + lane + 64 * q;
    cnt += __popcll(__ballot(e < E && tile_off[e < E ? e : 0] * n_ntiles <= logical));
  }
  return __builtin_amdgcn_readfirstlane(cnt);
}

struct TileAt {
  int row0, rows;  // first row (of M, or of the sorted rows) and valid rows
  int n0;          // first weight row
  size_t w_row;    // weight rows before it: the matrix's, then n0
  size_t w_blk;    // 128 x 128 scale rows before the matrix's
};

// The tile of this workgroup, false for a surplus one.  Workgroups go round
// robin to the 8 XCDs; each XCD takes a contiguous eighth of the logical tiles
// (grouped: expert, column tile, row tile), so that sharers of a weight panel
// share an L2.
template <int MODE>
__device__ __forceinline__ bool find_tile(const BlockArgs& g, int bm, int bn, TileAt& t) {
  const int n_nt = (g.N + bn - 1) / bn;
  const int n_mt = MODE == kBlockDense ? (g.M + bm - 1) / bm : g.tile_off[g.E];
  const int total = n_nt * n_mt;
  const int per_xcd = (total + 7) >> 3;
  const int local = blockIdx.x >> 3;
  const int logical = (blockIdx.x & 7) * per_xcd + local;
  if (local >= per_xcd || logical >= total) return false;
  int e = 0, mt, nt;
  if constexpr (MODE == kBlockDense) {
    nt = logical / n_mt;
    mt = logical - nt * n_mt;
    t.row0 = mt * bm;
    t.rows = min(bm, g.M - t.row0);
  } else {
    e = owner_expert(g.tile_off, g.E, n_nt, logical);
    const int te = g.tile_off[e + 1] - g.tile_off[e];
    const int loc = logical - g.tile_off[e] * n_nt;
    nt = loc / te;
    mt = loc - nt * te;
    t.row0 = g.offsets[e] + mt * bm;
    t.rows = min(bm, g.offsets[e + 1] - t.row0);
  }
  t.n0 = nt * bn;
  const int ew = MODE != kBlockDense && g.w_slot ? g.w_slot[e] : e;
  t.w_row = static_cast<size_t>(ew) * g.N + t.n0;
  t.w_blk = static_cast<size_t>(e) * ((g.N + 127) / 128);
  return true;
}

// row of the activations behind row r of a tile
template <int MODE>
__device__ __forceinline__ size_t source_row(const BlockArgs& g, int r) {
  return MODE == kBlockUp ? static_cast<size_t>(g.sorted_src[r] / g.top_k) : static_cast<size_t>(r);
}

__device__ __forceinline__ f32x4 mma128(i32x8 w, i32x8 x) {
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, zero, 0, 0, 0, 127, 0, 127);
}

__device__ __forceinline__ i32x8 join(u32x4 a, u32x4 b) {
  return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// four results of one row: weight rows n .. n + 3 of row `row`
template <int MODE>
__device__ __forceinline__ void store4(const BlockArgs& g, int row, int n, f32x4 v) {
  if constexpr (MODE == kBlockDown) {
    const float gate = g.row_gate[row];
    *reinterpret_cast<f32x4*>(static_cast<float*>(g.out) + static_cast<size_t>(row) * g.N + n) =
        f32x4{gate * v[0], gate * v[1], gate * v[2], gate * v[3]};
  } else {
    uint16_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = MODE == kBlockUp ? relu_sq_bf16(v[i]) : f32_to_bf16(v[i]);
    uint16_t* o = static_cast<uint16_t*>(g.out) + static_cast<size_t>(row) * g.N + n;
    if (MODE == kBlockUp || g.N % 4 == 0) {
      *reinterpret_cast<uint2*>(o) = make_uint2(b[0] | (static_cast<uint32_t>(b[1]) << 16),
                                                b[2] | (static_cast<uint32_t>(b[3]) << 16));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < g.N) o[i] = b[i];
    }
  }
}

// ---- few rows (a decode batch, or a ragged expert's rows): 32 weight rows x 16 G
// rows per workgroup, the K blocks dealt to 8 waves, each streaming its blocks
// from memory into registers one block ahead.  Bound by the weights' bytes; the
// waves' sums are joined through LDS in wave order.  Lines are loaded whole (8
// lanes to a row's 128 bytes) and turned into operand order in 2 KB pieces of
// LDS that belong to the wave.
constexpr int kSmallWaves = 8;
constexpr int kSmallN = 32;

template <int MODE, int G>
__global__ __launch_bounds__(kSmallWaves * kWave) void block_small_kernel(BlockArgs g) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[kSmallWaves][8192];
  TileAt t;
  if (!find_tile<MODE>(g, 16 * G, kSmallN, t)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = lane & 15, q = lane >> 4;
  const int K = g.K, blocks = (K + 127) / 128;
  const int lr = lane >> 3, ch = lane & 7;  // row of 8 and 16-byte chunk this lane loads
  // groups of 16 rows that hold any
  const int live = __builtin_amdgcn_readfirstlane((t.rows + 15) >> 4);

  const uint8_t* wp[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    wp[i] = g.w + (t.w_row - t.n0 + min(t.n0 + i * 8 + lr, g.N - 1)) * K + ch * 16;
  const uint8_t* xp[G][2];
  size_t sp[G];
#pragma unroll
  for (int j = 0; j < G; ++j) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      xp[j][h] = g.a + source_row<MODE>(g, t.row0 + min(j * 16 + h * 8 + lr, t.rows - 1)) * K + ch * 16;
    sp[j] = source_row<MODE>(g, t.row0 + min(j * 16 + c, t.rows - 1));
  }
  const float* ws = g.w_s + (t.w_blk + t.n0 / 128) * blocks;

  struct Block {
    u32x4 w[4], x[G][2];
    float s[G];
  };
  const u32x4 zero = {0u, 0u, 0u, 0u};
  const auto load = [&](Block& b, int kb) {
    const bool in = kb * 128 + ch * 16 < K;  // a last block may be short
    const int at = in ? kb * 128 : -ch * 16;  // the row's first chunk, then made zero
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      b.w[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(wp[i] + at));
      if (!in) b.w[i] = zero;
    }
    const float sw = ws[kb];
#pragma unroll
    for (int j = 0; j < G; ++j) {
      if (j >= live) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        b.x[j][h] = *reinterpret_cast<const u32x4*>(xp[j][h] + at);
        if (!in) b.x[j][h] = zero;
      }
      b.s[j] = g.a_s[static_cast<size_t>(kb) * g.a_rows + sp[j]] * sw;
    }
  };

  f32x4 acc[2][G];
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int j = 0; j < G; ++j) acc[f][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  uint8_t* const mine = lds[wave];
  // 16 rows of 128 bytes: chunk x of row r lies at x ^ (r % 8)
  const auto put = [&](int piece, u32x4 a, u32x4 b) {
    u32x4* p = reinterpret_cast<u32x4*>(mine + piece * 2048 + lr * 128 + ((ch ^ lr) << 4));
    p[0] = a;
    p[64] = b;
  };
  const auto get = [&](int piece) {
    const uint8_t* p = mine + piece * 2048 + c * 128;
    return join(*reinterpret_cast<const u32x4*>(p + (((2 * q) ^ (c & 7)) << 4)),
                *reinterpret_cast<const u32x4*>(p + (((2 * q + 1) ^ (c & 7)) << 4)));
  };
  const auto multiply = [&](const Block& b) {
    put(0, b.w[0], b.w[1]);
    put(1, b.w[2], b.w[3]);
    const i32x8 w0 = get(0), w1 = get(1);
#pragma unroll
    for (int j = 0; j < G; ++j) {
      if (j >= live) continue;
      put(2 + (j & 1), b.x[j][0], b.x[j][1]);
      const i32x8 x = get(2 + (j & 1));
      const f32x4 p0 = mma128(w0, x), p1 = mma128(w1, x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[0][j][i] += b.s[j] * p0[i];
        acc[1][j][i] += b.s[j] * p1[i];
      }
    }
  };
  Block b0, b1;
  if (wave < blocks) load(b0, wave);
  for (int kb = wave; kb < blocks; kb += 2 * kSmallWaves) {
    if (kb + kSmallWaves < blocks) load(b1, kb + kSmallWaves);
    multiply(b0);
    if (kb + kSmallWaves >= blocks) break;
    if (kb + 2 * kSmallWaves < blocks) load(b0, kb + 2 * kSmallWaves);
    multiply(b1);
  }

  // join: wave j adds up group j
#pragma unroll
  for (int f = 0; f < 2; ++f) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < G; ++j)
      if (j < live) reinterpret_cast<f32x4*>(&lds[0][0])[(wave * G + j) * kWave + lane] = acc[f][j];
    __syncthreads();
    if (wave < live) {
      f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kSmallWaves; ++w)
        v += reinterpret_cast<const f32x4*>(&lds[0][0])[(w * G + wave) * kWave + lane];
      const int r = wave * 16 + c, n = t.n0 + f * 16 + 4 * q;
      if (r < t.rows && n < g.N) store4<MODE>(g, t.row0 + r, n, v);
    }
  }
}

// ---- many rows: BM x BN tiles, both operands from memory straight into LDS
// (global_load_lds_dwordx4), one K block per step, two buffers.  Rows are 128
// bytes; chunk x of row r lies at x ^ ((r / 2) % 8), so that the 16 rows of an
// operand read fall on distinct banks.  WM x WN waves (rows x weight rows).
__device__ __attribute__((aligned(16))) uint32_t zeros[4];  // what lies past K

// 16 bytes a lane from p straight into LDS at `to` + 16 * lane
__device__ __forceinline__ void load_to_lds(const uint8_t* p, uint8_t* to) {
  __builtin_amdgcn_global_load_lds(p, (__attribute__((address_space(3))) void*)to, 16, 0, 0);
}

__device__ __forceinline__ int swz(int r) { return (r >> 1) & 7; }

template <int MODE, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM* WN * 64) void block_gemm_kernel(BlockArgs g) {
  constexpr int NW = WM * WN;
  constexpr int WTM = BM / WM, WTN = BN / WN;
  constexpr int MS = WTM / 16, NS = WTN / 16;  // 16 x 16 products of a wave
  constexpr int QA = BM / 8 / NW, QB = BN / 8 / NW;  // loads (8 rows) per wave and step
  constexpr int BUF = (BM + BN) * 128;
  static_assert(QA * 8 * NW == BM && QB * 8 * NW == BN && 128 % WTN == 0, "tile");
  __shared__ __attribute__((aligned(1024))) uint8_t lds0[BUF];
  __shared__ __attribute__((aligned(1024))) uint8_t lds1[BUF];
  TileAt t;
  if (!find_tile<MODE>(g, BM, BN, t)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wm = wave / WN, wn = wave % WN;
  const int c = lane & 15, q = lane >> 4;
  const int K = g.K, steps = (K + 127) / 128;

  const uint8_t *ap[QA], *bp[QB];
  int ach[QA], bch[QB];
#pragma unroll
  for (int i = 0; i < QA; ++i) {
    const int r = (wave * QA + i) * 8 + (lane >> 3);
    ach[i] = ((lane & 7) ^ swz(r)) * 16;
    ap[i] = g.a + source_row<MODE>(g, t.row0 + min(r, t.rows - 1)) * K + ach[i];
  }
#pragma unroll
  for (int i = 0; i < QB; ++i) {
    const int r = (wave * QB + i) * 8 + (lane >> 3);
    bch[i] = ((lane & 7) ^ swz(r)) * 16;
    bp[i] = g.w + (t.w_row - t.n0 + min(t.n0 + r, g.N - 1)) * K + bch[i];
  }
  const uint8_t* const past = reinterpret_cast<const uint8_t*>(zeros);
  const auto dma = [&](int step, uint8_t* buf) {
    const int kb = step * 128;
    const bool whole = kb + 128 <= K;
#pragma unroll
    for (int i = 0; i < QA; ++i)
      load_to_lds(whole || kb + ach[i] < K ? ap[i] + kb : past, buf + (wave * QA + i) * 1024);
#pragma unroll
    for (int i = 0; i < QB; ++i)
      load_to_lds(whole || kb + bch[i] < K ? bp[i] + kb : past,
                  buf + BM * 128 + (wave * QB + i) * 1024);
  };

  // 16-row groups of this wave that hold rows; columns past N are not skipped
  // but for whole waves
  const int m0 = wm * WTM, nw0 = wn * WTN;
  const bool idle = m0 >= t.rows || t.n0 + nw0 >= g.N;
  size_t src[MS];
#pragma unroll
  for (int j = 0; j < MS; ++j) src[j] = source_row<MODE>(g, t.row0 + min(m0 + j * 16 + c, t.rows - 1));
  const float* ws = g.w_s + (t.w_blk + min(t.n0 + nw0, g.N - 1) / 128) * steps;

  f32x4 acc[NS][MS];
#pragma unroll
  for (int i = 0; i < NS; ++i)
#pragma unroll
    for (int j = 0; j < MS; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  float s[MS];
  const auto load_scales = [&](int step) {
    const float sw = ws[step];
#pragma unroll
    for (int j = 0; j < MS; ++j) s[j] = g.a_s[static_cast<size_t>(step) * g.a_rows + src[j]] * sw;
  };
  const auto frag = [&](const uint8_t* rows, int r) {
    const uint8_t* p = rows + r * 128;
    return join(*reinterpret_cast<const u32x4*>(p + (((2 * q) ^ swz(r)) << 4)),
                *reinterpret_cast<const u32x4*>(p + (((2 * q + 1) ^ swz(r)) << 4)));
  };
  const auto compute = [&](const uint8_t* buf) {
    i32x8 w[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) w[i] = frag(buf + BM * 128, nw0 + i * 16 + c);
#pragma unroll
    for (int j = 0; j < MS; ++j) {
      const i32x8 x = frag(buf, m0 + j * 16 + c);
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const f32x4 p = mma128(w[i], x);
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] += s[j] * p[r];
      }
    }
  };
  const auto body = [&](int step, const uint8_t* cur, uint8_t* ahead) {
    if (step >= steps) return;
    load_scales(step);
    __builtin_amdgcn_s_waitcnt(0);  // this wave's loads of the step
    __asm__ volatile("s_barrier" ::: "memory");
    if (step + 1 < steps) dma(step + 1, ahead);
    if (!idle) compute(cur);
  };
  dma(0, lds0);
  for (int step = 0; step < steps; step += 2) {
    body(step, lds0, lds1);
    body(step + 1, lds1, lds0);
  }
  if (idle) return;
#pragma unroll
  for (int j = 0; j < MS; ++j) {
    const int r = m0 + j * 16 + c;
    if (r >= t.rows) continue;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int n = t.n0 + nw0 + i * 16 + 4 * q;
      if (n < g.N) store4<MODE>(g, t.row0 + r, n, acc[i][j]);
    }
  }
}

long long tiles_of(const BlockArgs& g, int mode, int bm, int bn) {
  const long long n_nt = (g.N + bn - 1) / bn;
  const long long n_mt = mode == kBlockDense ? (g.M + bm - 1) / bm : g.max_tiles;
  return (n_nt * n_mt + 7) / 8 * 8;
}

// with timing events the kernel's own start and end are stamped (see GemmArgs'
// launches)
hipError_t dispatch(const void* kernel, long long blocks, int threads, const BlockArgs& g,
                    hipStream_t stream, const KernelEvents& ev) {
  BlockArgs a = g;
  void* args[] = {&a};
  const dim3 grid(static_cast<unsigned>(blocks)), block(threads);
  if (ev.start || ev.stop)
    return hipExtLaunchKernel(kernel, grid, block, args, 0, stream, ev.start, ev.stop, 0);
  return hipLaunchKernel(kernel, grid, block, args, 0, stream);
}

template <int MODE, int G>
hipError_t launch_small(const BlockArgs& g, hipStream_t stream, const KernelEvents& ev = KernelEvents{}) {
  return dispatch(reinterpret_cast<const void*>(&block_small_kernel<MODE, G>),
                  tiles_of(g, MODE, 16 * G, kSmallN), kSmallWaves * kWave, g, stream, ev);
}

template <int MODE, int BM, int BN, int WM, int WN>
hipError_t launch_large(const BlockArgs& g, hipStream_t stream, const KernelEvents& ev = KernelEvents{}) {
  return dispatch(reinterpret_cast<const void*>(&block_gemm_kernel<MODE, BM, BN, WM, WN>),
                  tiles_of(g, MODE, BM, BN), WM * WN * 64, g, stream, ev);
}

}  // namespace

int block_tile_rows(int T) { return T < kBlockDecodeMaxT ? 32 : 128; }

hipError_t launch_block_experts(int stage, int T, const BlockArgs& g, hipStream_t stream,
                                const KernelEvents& ev) {
  if (T < kBlockDecodeMaxT)
    return stage == 0 ? launch_small<kBlockUp, 2>(g, stream, ev) : launch_small<kBlockDown, 2>(g, stream, ev);
  return stage == 0 ? launch_large<kBlockUp, 128, 128, 2, 2>(g, stream, ev)
                    : launch_large<kBlockDown, 128, 128, 2, 2>(g, stream, ev);
}

hipError_t launch_block_dense(const BlockArgs& g, hipStream_t stream) {
  if (g.M <= 16) return launch_small<kBlockDense, 1>(g, stream);
  if (g.M <= 32) return launch_small<kBlockDense, 2>(g, stream);
  if (g.M <= 128) return launch_small<kBlockDense, 4>(g, stream);
  if (tiles_of(g, kBlockDense, 256, 256) >= 128) return launch_large<kBlockDense, 256, 256, 2, 4>(g, stream);
  return launch_large<kBlockDense, 128, 128, 2, 2>(g, stream);
}

hipError_t launch_block_quant(const uint16_t* x, const int32_t* n_rows_dev, int rows, int cols,
                              uint8_t* codes, float* scales, hipStream_t stream) {
  if (rows <= 0) return hipSuccess;
  const int64_t n = static_cast<int64_t>(rows) * ((cols + 127) / 128);
  int64_t blocks = (n + kQThreads / 16 - 1) / (kQThreads / 16);
  if (blocks > 8192) blocks = 8192;
  hipLaunchKernelGGL(block_quant_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kQThreads), 0,
                     stream, x, n_rows_dev, rows, cols, rows, codes, scales);
  return hipGetLastError();
}

hipError_t launch_block_pack(const uint16_t* w, int E, int N, int K, uint8_t* codes, float* scales,
                             hipStream_t stream) {
  hipLaunchKernelGGL(block_pack_kernel, dim3((K + 127) / 128, (N + 127) / 128, E), dim3(kQThreads), 0,
                     stream, w, N, K, codes, scales);
  return hipGetLastError();
}

}  // namespace moe
