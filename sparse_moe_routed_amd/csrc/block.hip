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
// sums across blocks are fp32.  What it drops lies some 13 bits below the block's
// largest product, at most 128 times: 2^-6 of that product where products cancel,
// below the half step (2^-4) by which its own codes may be off.
//
// The experts' up projection is the exception: its sums become codes again, and
// there a sum that is cut short moves a whole E4M3 step, or a block's scale.  Its
// products are exact: both operands' codes become fp16 in registers, and four
// 16x16x32 products in fp32 take the place of the one.  Against exact sums the
// layer's bf16 output is then off by 1.7e-3, its own rounding (with the short sums
// 2.0e-3 to 2.9e-3).  Batches that read weights from memory do not notice (T = 5
// 54 us, T = 64 157); at T = 4096 the up projection takes 341 us instead of 226.
//
// Weight codes are packed in operand order: for each group of 16 rows and each
// K block 2 KB, [half h][lane l][16 bytes] = row l % 16, values 32 (l / 16) + 16 h
// and on, zeros past N and K.  A wave reads its operand with two contiguous 1 KB
// loads straight into registers: weights need no LDS and no masks, and a weight
// stream is one contiguous run per 16 rows whatever K is.  Activation codes are
// row-major (their rows are gathered) and go through LDS.  Scales of activations
// lie block by block, [ceil(K / 128), rows], so that the tokens of one MFMA read
// consecutive words; weight scales are [ceil(N / 128), ceil(K / 128)].
#include <hip/hip_ext.h>
#include <type_traits>

#include "block_quant.h"
#include "moe_common.h"
#include "moe_internal.h"
#include "tile.h"

namespace moe {

namespace {

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// ---- activations: HBM bound, one pass (4096 x 2688: 34 MB in 8.0 us, 4.2 TB/s)
__global__ __launch_bounds__(kQThreads) void block_quant_kernel(BlockQuantArgs q) {
  block_quantise(q, blockIdx.x, gridDim.x);
}

// where value k of weight row n lies in a packed matrix of kb_n K blocks
__device__ __forceinline__ size_t packed_at(int n, int k, int kb_n) {
  const int in = k & 127;
  return (static_cast<size_t>(n >> 4) * kb_n + (k >> 7)) * 2048 + ((in >> 4) & 1) * 1024 +
         ((in >> 5) * 16 + (n & 15)) * 16 + (k & 15);
}

// bf16 pairs with infinities turned into NaN: a NaN is no part of a block's
// amax, so the block's other values keep their codes
__device__ __forceinline__ u32x4 inf_to_nan(u32x4 v) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if ((v[w] & 0x7fffu) == 0x7f80u) v[w] |= 0x40u;
    if ((v[w] & 0x7fff0000u) == 0x7f800000u) v[w] |= 0x400000u;
  }
  return v;
}

// ---- weights: a workgroup per 128 x 128 block; rows of 16 lanes
__global__ __launch_bounds__(kQThreads) void block_pack_kernel(const uint16_t* __restrict__ w, int N,
                                                               int K, uint8_t* __restrict__ codes,
                                                               float* __restrict__ scales) {
  __shared__ float part[kQThreads / 64];
  const int kb = blockIdx.x, nb = blockIdx.y;
  const int n16 = (N + 15) / 16 * 16;
  const uint16_t* const src = w + static_cast<size_t>(blockIdx.z) * N * K;
  uint8_t* const dst = codes + static_cast<size_t>(blockIdx.z) * n16 * gridDim.x * 128;
  const int r0 = threadIdx.x >> 4, k = kb * 128 + (threadIdx.x & 15) * 8;
  u32x4 v[8];
  float m = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int n = nb * 128 + r0 + 16 * j;
    v[j] = u32x4{0u, 0u, 0u, 0u};
    if (n < N && k < K) v[j] = inf_to_nan(*reinterpret_cast<const u32x4*>(src + static_cast<size_t>(n) * K + k));
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
    if (n < n16) *reinterpret_cast<uint2*>(dst + packed_at(n, k, gridDim.x)) = encode8(v[j], inv);
  }
  if (threadIdx.x == 0)
    scales[(static_cast<size_t>(blockIdx.z) * gridDim.y + nb) * gridDim.x + kb] =
        live ? __fdiv_rn(m, 448.f) : 0.f;
}

// row-major codes [N, K] into the packed order, 16 bytes a thread
__global__ __launch_bounds__(kQThreads) void block_pack_codes_kernel(const uint8_t* __restrict__ q, int N,
                                                                     int K, uint8_t* __restrict__ codes) {
  const int kb_n = (K + 127) / 128, n16 = (N + 15) / 16 * 16;
  const int64_t total = static_cast<int64_t>(n16) * kb_n * 8;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kQThreads + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * kQThreads) {
    const int n = static_cast<int>(i / (kb_n * 8)), k = static_cast<int>(i % (kb_n * 8)) * 16;
    u32x4 v = {0u, 0u, 0u, 0u};
    if (n < N && k < K) v = *reinterpret_cast<const u32x4*>(q + static_cast<size_t>(n) * K + k);
    *reinterpret_cast<u32x4*>(codes + packed_at(n, k, kb_n)) = v;
  }
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
  const uint8_t* w;  // the matrix's codes
  size_t w_blk;      // 128 x 128 scale rows before the matrix's
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
  t.w = g.w + static_cast<size_t>(ew) * ((g.N + 15) / 16 * 16) * ((g.K + 127) / 128 * 128);
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
    for (int i = 0; i < 4; ++i) b[i] = f32_to_bf16(v[i]);
    uint16_t* o = static_cast<uint16_t*>(g.out) + static_cast<size_t>(row) * g.N + n;
    if (g.N % 4 == 0) {
      *reinterpret_cast<uint2*>(o) = make_uint2(b[0] | (static_cast<uint32_t>(b[1]) << 16),
                                                b[2] | (static_cast<uint32_t>(b[3]) << 16));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < g.N) o[i] = b[i];
    }
  }
}

// the operand of 16 weight rows and one K block: `at` is the lane's offset of the
// rows' first block, kPastEnd for rows past N
// ONCE: non-temporal, for weights that one workgroup reads (dense, up to 64 rows:
// 3712 x 2688 from memory, M = 16 5.9 us, cached 6.2; with a second row tile M = 77
// 9.6, cached 8.6), and for the experts' 32-row tiles, where the few weights that
// several tiles of a popular expert share are cheaper to read again than to keep
// (full layer, uneven use: T = 64 156.6 us, cached 178; T = 256 244 and 261).
template <bool ONCE>
__device__ __forceinline__ void load_weights(u32x4 (&w)[2], Buffer b, uint32_t at, uint32_t block_at) {
  constexpr int kPolicy = ONCE ? 2 : 0;
  w[0] = __builtin_amdgcn_raw_buffer_load_b128(b, at, block_at, kPolicy);
  w[1] = __builtin_amdgcn_raw_buffer_load_b128(b, at + 1024u, block_at, kPolicy);
}

// ---- few rows: 32 weight rows x 16 G rows per workgroup, the K blocks dealt to 8
// waves, each one block ahead of its products.  Bound by the weights' bytes and
// the latency of a few blocks: a wave of M = 1 and K = 2688 has three of them, one
// load's latency and the join (4.5 us; 8192 x 8192, M = 4 13 us, 5.2 TB/s).  The
// waves' sums are joined through LDS in wave order.  The rows' codes come a line at a time (8 lanes to 128 bytes) and are
// turned into operand order in 2 KB of LDS that belong to the wave.  With QUANT
// the rows are bf16 and become codes on their way into that LDS.
constexpr int kSmallWaves = 8;
constexpr int kSmallN = 32;

template <int G, bool QUANT, bool ONCE>
__global__ __launch_bounds__(kSmallWaves * kWave) void block_small_kernel(BlockArgs g) {
  constexpr int kTurn = 4096, kJoin = G * 1024;
  constexpr int kRaw = QUANT ? 2 : 1;  // 16-byte loads per 16 values
  __shared__ __attribute__((aligned(16))) uint8_t lds[kSmallWaves * (kTurn > kJoin ? kTurn : kJoin)];
  TileAt t;
  if (!find_tile<kBlockDense>(g, 16 * G, kSmallN, t)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, q = lane >> 4;
  const int K = g.K, blocks = (K + 127) / 128;
  const int lr = lane >> 3, ch = lane & 7;  // row of 8 and 16-byte chunk this lane loads
  // groups of 16 rows that hold any
  const int live = __builtin_amdgcn_readfirstlane((t.rows + 15) >> 4);

  // two groups of weight rows; the second may lie past N and is then not read
  const Buffer wb = buffer_of(t.w + static_cast<size_t>(t.n0 / 16) * blocks * 2048,
                              (t.n0 + 16 < g.N ? 2u : 1u) * blocks * 2048);
  const uint32_t wat[2] = {lane * 16u, t.n0 + 16 < g.N ? lane * 16u + blocks * 2048u : kPastEnd};
  const uint8_t* xp[G][2];
  size_t sp[G];
#pragma unroll
  for (int j = 0; j < G; ++j) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      xp[j][h] = g.a + (static_cast<size_t>(t.row0 + min(j * 16 + h * 8 + lr, t.rows - 1)) * K + ch * 16) * kRaw;
    sp[j] = t.row0 + min(j * 16 + c, t.rows - 1);
  }
  const float* ws = g.w_s + (t.w_blk + t.n0 / 128) * blocks;

  struct Block {
    u32x4 w[2][2], x[G][2][kRaw];
    float s[G];  // QUANT: of the weights alone
  };
  const u32x4 zero = {0u, 0u, 0u, 0u};
  const auto load = [&](Block& b, int kb) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      load_weights<ONCE>(b.w[i], wb, wat[i], kb * 2048);
    const bool in = kb * 128 + ch * 16 < K;  // a last block may be short
    const int at = (in ? kb * 128 : -ch * 16) * kRaw;  // the row's first chunk, then made zero
    const float sw = ws[kb];
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
      b.s[j] = QUANT ? sw : g.a_s[static_cast<size_t>(kb) * g.a_rows + sp[j]] * sw;
    }
  };

  f32x4 acc[2][G];
#pragma unroll
  for (int f = 0; f < 2; ++f)
#pragma unroll
    for (int j = 0; j < G; ++j) acc[f][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  uint8_t* const mine = lds + wave * kTurn;
  // 16 rows of 128 bytes: chunk x of row r lies at x ^ (r % 8)
  const auto put = [&](int piece, u32x4 a, u32x4 b) {
    u32x4* p = reinterpret_cast<u32x4*>(mine + piece * 2048 + lr * 128 + ((ch ^ lr) << 4));
    wave_lds_order();  // what was there has been read
    p[0] = a;
    p[64] = b;
    wave_lds_order();
  };
  const auto get = [&](int piece) {
    const uint8_t* p = mine + piece * 2048 + c * 128;
    return join(*reinterpret_cast<const u32x4*>(p + (((2 * q) ^ (c & 7)) << 4)),
                *reinterpret_cast<const u32x4*>(p + (((2 * q + 1) ^ (c & 7)) << 4)));
  };
  const auto multiply = [&](const Block& b) {
    const i32x8 w0 = join(b.w[0][0], b.w[0][1]), w1 = join(b.w[1][0], b.w[1][1]);
#pragma unroll
    for (int j = 0; j < G; ++j) {
      if (j >= live) continue;
      float s = b.s[j];
      if constexpr (QUANT) {  // as block_quant_kernel: 8 lanes hold a row's block
        u32x4 code[2];
        float scale[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (h == 1 && t.rows <= j * 16 + 8) {  // rows that are not there
            code[1] = code[0];
            scale[1] = scale[0];
            continue;
          }
          const u32x4 lo = b.x[j][h][0], hi = b.x[j][h][1];
          const float amax = row8_max(fmaxf(amax8(lo), amax8(hi)));
          const bool any = amax >= kTinyAmax;
          const float inv = any ? __fdiv_rn(448.f, amax) : 0.f;
          scale[h] = any ? __fdiv_rn(amax, 448.f) : 0.f;
          const uint2 a = encode8(lo, inv), z = encode8(hi, inv);
          code[h] = u32x4{a.x, a.y, z.x, z.y};
        }
        put(j & 1, code[0], code[1]);
        // row c's scale lies with the lanes that hold row c
        const float s0 = __shfl(scale[0], (c & 7) * 8), s1 = __shfl(scale[1], (c & 7) * 8);
        s *= c < 8 ? s0 : s1;
      } else {
        put(j & 1, b.x[j][0][0], b.x[j][1][0]);
      }
      const i32x8 x = get(j & 1);
      const f32x4 p0 = mma128(w0, x), p1 = mma128(w1, x);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[0][j][i] = __builtin_fmaf(s, p0[i], acc[0][j][i]);
        acc[1][j][i] = __builtin_fmaf(s, p1[i], acc[1][j][i]);
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
      if (j < live) reinterpret_cast<f32x4*>(lds)[(wave * G + j) * kWave + lane] = acc[f][j];
    __syncthreads();
    if (wave < live) {
      f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kSmallWaves; ++w)
        v += reinterpret_cast<const f32x4*>(lds)[(w * G + wave) * kWave + lane];
      const int r = wave * 16 + c, n = t.n0 + f * 16 + 4 * q;
      if (r < t.rows && n < g.N) store4<kBlockDense>(g, t.row0 + r, n, v);
    }
  }
}

// ---- tiles of BM rows x BN weight rows, WM x WN waves, one K block per step.  The
// rows' codes and scales go from memory straight into LDS (NBUF buffers, NBUF - 1
// steps under way); rows are 128 bytes, chunk x of row r lies at
// x ^ ((r / 2) % 8), so that the 16 rows of an operand read fall on distinct
// banks.  The weights go straight into registers (WBUF operands per wave and
// group, WBUF - 1 steps under way): a weight is read by the WM waves of a column
// and no other, so LDS would only add a way, while a row serves all WN waves.
// Where weights come from memory once (decode) the bound is HBM: 64 tokens of
// uneven use read 92 experts, 0.92 GB, in 154 us of both products, 6.0 TB/s (a plain
// stream of reads reaches 7.1); where they are shared, no unit is busy for more than
// half the time (8192 x 8192 x 4096: 2.06 PFLOP/s, matrix units about 45 %), and what
// is left is the waves' own order of LDS reads, products and multiply-adds between
// barriers.
template <int MODE, int BM, int BN, int WM, int WN, int NBUF, int WBUF, bool ONCE>
__global__ __launch_bounds__(WM* WN * 64) void block_gemm_kernel(BlockArgs g) {
  constexpr int NW = WM * WN;
  constexpr int WTM = BM / WM, WTN = BN / WN;
  constexpr int MS = WTM / 16, NS = WTN / 16;  // 16 x 16 products of a wave
  constexpr bool kHalf = MODE == kBlockUp;     // exact products, in fp16
  constexpr int QA = BM / 8 / NW;              // loads of 8 rows per wave and step
  constexpr int kRowLoads = QA + 1;            // and one of 64 scales
  constexpr int kRowsAhead = (NBUF - 2) * kRowLoads;         // loads that may be under way: of rows,
  // Loads go between the products, weights first, so that the matrix unit starts
  // with the step and not after them (3712 x 2688, M = 4096 50.9 -> 46.6 us, M = 1024
  // 18.8 -> 16.9); all at once, rows first, where the step is short of time for
  // them: two buffers, or weights from memory (T = 4096 571 us, spread 583).
  constexpr bool kSpread = NBUF == 4 && !ONCE;
  // with the weights': those of steps from this one on that were issued after
  // the rows of this one
  constexpr int kAhead = kRowsAhead + (kSpread ? WBUF / 2 : WBUF - 1) * 2 * NS;
  constexpr int SOFF = BM * 128;
  constexpr int kParts = BM < 64 ? 1 : BM / 64;  // loads of 64 rows' scales
  constexpr int WOFF = SOFF + kParts * 256;
  constexpr int BUF = WOFF + 256;
  static_assert(QA * 8 * NW == BM && 128 % WTN == 0 && BN % WTN == 0, "tile");
  static_assert(BM % 64 == 0 || BM == 32, "scales come 64 at a time");
  static_assert(NS == 1 || NS == 2 || NS == 4, "columns of a wave");
  static_assert((NBUF == 2 || NBUF == 4) && (WBUF == 2 || WBUF == 4) && kAhead < 64, "buffers");
  __shared__ __attribute__((aligned(1024))) uint8_t lds0[BUF];
  __shared__ __attribute__((aligned(1024))) uint8_t lds1[BUF];
  __shared__ __attribute__((aligned(1024))) uint8_t lds2[NBUF == 4 ? BUF : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t lds3[NBUF == 4 ? BUF : 16];
  TileAt t;
  if (!find_tile<MODE>(g, BM, BN, t)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int c = lane & 15, q = lane >> 4;
  const int K = g.K, steps = (K + 127) / 128;

  // Rows: gathered ones are addressed from the first activation row (fewer than
  // 2^32 bytes, checked by the caller), others from the tile's first.
  const bool gather = MODE == kBlockUp;
  const size_t first = gather ? 0 : static_cast<size_t>(t.row0);
  const uint32_t a_bytes = static_cast<uint32_t>(static_cast<size_t>(gather ? g.a_rows : t.rows) * K);
  const uint8_t* const a = g.a + first * K;
  uint32_t ar[QA];
#pragma unroll
  for (int i = 0; i < QA; ++i) {
    const int r = (wave * QA + i) * 8 + (lane >> 3);
    const int ch = ((lane & 7) ^ swz(r)) * 16;
    const uint32_t row = static_cast<uint32_t>(source_row<MODE>(g, t.row0 + min(r, t.rows - 1)) - first);
    ar[i] = row * K + ch;
  }
  // Scales: wave p < kParts loads those of 64 rows, the others those of the
  // weights' 128-row blocks (all the same words to the same place), so that
  // every wave issues the same number of loads.
  const bool of_rows = wave < kParts;
  const int w_blk = t.n0 / 128, w_blks = (g.N + 127) / 128;
  const uint32_t s_at =
      4 * (of_rows ? static_cast<uint32_t>(source_row<MODE>(g, t.row0 + min(wave * 64 + lane, t.rows - 1)))
                   : static_cast<uint32_t>(min(lane, w_blks - 1 - w_blk) * steps));
  const float* const s_from = of_rows ? g.a_s : g.w_s + (t.w_blk + w_blk) * steps;
  const int s_step = of_rows ? g.a_rows : 1;
  const uint32_t s_bytes = 4u * (of_rows ? g.a_rows : (w_blks - w_blk) * steps);
  const int s_to = of_rows ? SOFF + wave * 256 : WOFF;
  // load i of kRowLoads
  const auto load_row = [&](int step, uint8_t* buf, int i) __attribute__((always_inline)) {
    const bool in = step < steps;
    if (i < QA) {
      const Buffer b = buffer_of(a, in ? a_bytes : 0u);
      const int chunks = min(K / 16 - step * 8, 8);  // a last block may be short
      const int ch = (lane & 7) ^ swz((wave * QA + i) * 8 + (lane >> 3));
      load16_to_lds(b, ch < chunks ? ar[i] : kPastEnd, in ? step * 128 : 0, buf + (wave * QA + i) * 1024);
    } else {
      const Buffer sb = buffer_of(s_from + static_cast<size_t>(in ? step : 0) * s_step, in ? s_bytes : 0u);
      load4_to_lds(sb, s_at, 0, buf + s_to);
    }
    __builtin_amdgcn_sched_barrier(0);  // the order of the loads is what the waits count on
  };
  const auto load_rows = [&](int step, uint8_t* buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kRowLoads; ++i) load_row(step, buf, i);
  };
  // weights: the wave's groups of 16 rows; the last one stands in for those past N
  const int m0 = wm * WTM, nw0 = wn * WTN;
  const int groups = (g.N - t.n0 - nw0 + 15) / 16;
  const uint8_t* const w_at = t.w + static_cast<size_t>(t.n0 + nw0) / 16 * steps * 2048;
  const uint32_t w_bytes = groups <= 0 ? 0u : static_cast<uint32_t>(groups < NS ? groups : NS) * steps * 2048;
  typedef u32x4 Weights[NS][2];
  const auto load_w1 = [&](Weights& w, int step, int i) __attribute__((always_inline)) {
    const Buffer b = buffer_of(w_at, step < steps ? w_bytes : 0u);
    load_weights<ONCE>(w[i], b, lane * 16, step < steps ? (max(min(i, groups - 1), 0) * steps + step) * 2048 : 0);
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
  f32x4 acc[NS][MS];
#pragma unroll
  for (int i = 0; i < NS; ++i)
#pragma unroll
    for (int j = 0; j < MS; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  // this lane's two chunks of row c of a 16-row group (groups are 2 KB apart,
  // and a group's first row is a multiple of 16, so its swizzle is c's)
  const int off0 = c * 128 + (((2 * q) ^ swz(c)) << 4), off1 = c * 128 + (((2 * q + 1) ^ swz(c)) << 4);
  const auto frag = [&](const uint8_t* group) __attribute__((always_inline)) {
    return join(*reinterpret_cast<const u32x4*>(group + off0), *reinterpret_cast<const u32x4*>(group + off1));
  };
  // Products run kDeep ahead of the multiply-adds that take their results, so
  // that a wave has other products to issue while one is in the matrix unit.
  const auto compute = [&](const uint8_t* buf, const Weights& w, auto live_c, auto issue)
                           __attribute__((always_inline)) {
    constexpr int ML = decltype(live_c)::value;
    constexpr int kDeep = 2;
    const uint8_t* const xrow = buf + m0 * 128;
    const float* const srow = reinterpret_cast<const float*>(buf + SOFF) + m0 + c;
    const float sw = reinterpret_cast<const float*>(buf + WOFF)[nw0 / 128];
    i32x8 x[2];
    x[0] = frag(xrow);
    float s[2];
    s[0] = srow[0];
    f32x4 p[kDeep + 1];
#pragma unroll
    for (int u = 0; u < ML * NS + kDeep; ++u) {
      if (u < ML * NS) {
        const int j = u / NS, i = u % NS;
        if (i == 0 && j + 1 < ML) x[(j + 1) & 1] = frag(xrow + (j + 1) * 2048);
        p[u % (kDeep + 1)] = mma128(join(w[i][0], w[i][1]), x[j & 1]);
        issue(u);
      }
      if (u >= kDeep) {
        const int v = u - kDeep, j = v / NS, i = v % NS;
        if (i == 0) s[j & 1] *= sw;
        if (i == 0 && j + 1 < ML) s[(j + 1) & 1] = srow[(j + 1) * 16];
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[i][j][r] = __builtin_fmaf(s[j & 1], p[v % (kDeep + 1)][r], acc[i][j][r]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // The same with codes turned into fp16, which is exact: four products of 32
  // values a block, chained in fp32, over the lane's 32 values of k in their order.
  const auto compute_half = [&](const uint8_t* buf, const Weights& w, auto live_c, auto issue)
                                __attribute__((always_inline)) {
    constexpr int ML = decltype(live_c)::value;
    const uint8_t* const xrow = buf + m0 * 128;
    const float* const srow = reinterpret_cast<const float*>(buf + SOFF) + m0 + c;
    const float sw = reinterpret_cast<const float*>(buf + WOFF)[nw0 / 128];
    const auto half = [&](uint32_t lo, uint32_t hi) __attribute__((always_inline)) {
      const f16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, false);
      const f16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(lo, 1.0f, true);
      const f16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, false);
      const f16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(hi, 1.0f, true);
      return f16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
    };
    u32x4 x[2][2];
    const auto read = [&](u32x4 (&to)[2], int j) __attribute__((always_inline)) {
      to[0] = *reinterpret_cast<const u32x4*>(xrow + j * 2048 + off0);
      to[1] = *reinterpret_cast<const u32x4*>(xrow + j * 2048 + off1);
    };
    read(x[0], 0);
    f16x8 wf[NS][4];
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        wf[i][h] = half(w[i][h >> 1][(h & 1) * 2], w[i][h >> 1][(h & 1) * 2 + 1]);
      }
    f32x4 p[2][NS];
    float s[2];
#pragma unroll
    for (int j = 0; j <= ML; ++j) {
      if (j < ML) {
        if (j + 1 < ML) read(x[(j + 1) & 1], j + 1);
        s[j & 1] = srow[j * 16] * sw;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const f16x8 xf = half(x[j & 1][h >> 1][(h & 1) * 2], x[j & 1][h >> 1][(h & 1) * 2 + 1]);
#pragma unroll
          for (int i = 0; i < NS; ++i) {
            const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
            p[j & 1][i] =
                __builtin_amdgcn_mfma_f32_16x16x32_f16(wf[i][h], xf, h == 0 ? zero : p[j & 1][i], 0, 0, 0);
          }
          if (h * NS % 4 == 0) issue(j * NS + h * NS / 4);
        }
      }
      if (j > 0) {
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[i][j - 1][r] = __builtin_fmaf(s[(j - 1) & 1], p[(j - 1) & 1][i][r], acc[i][j - 1][r]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // One step: its rows have arrived (this wave's, then at the barrier
  // everyone's), those of step + NBUF - 1 start into the buffer that everyone
  // has read, the weights of step + WBUF - 1 into the registers of step - 1,
  // then the products.  A load that nothing uses is not there to be counted, the
  // compiler drops it: a wave without products loads no weights and counts none,
  // and the last steps of all (TAIL, fewer than 4) wait for all that is under way.
  const auto body = [&](int step, const uint8_t* cur, uint8_t* ahead, const Weights& now, Weights& next,
                        auto live_c, auto tail_c) __attribute__((always_inline)) {
    constexpr bool TAIL = decltype(tail_c)::value, kAny = decltype(live_c)::value > 0;
    __builtin_amdgcn_s_waitcnt(vmcnt_imm(TAIL ? 0 : (kAny ? kAhead : kRowsAhead)));
    __asm__ volatile("s_barrier" ::: "memory");
    if constexpr (kAny && !TAIL && kSpread) {
      constexpr int kLoads = kRowLoads + NS, kProducts = decltype(live_c)::value * NS;
      const auto issue = [&](int u) __attribute__((always_inline)) {
#pragma unroll
        for (int l = 0; l < kLoads; ++l) {
          if (l * kProducts / kLoads != u) continue;
          if (l < NS) load_w1(next, step + WBUF - 1, l);
          else load_row(step + NBUF - 1, ahead, l - NS);
        }
      };
      if constexpr (kHalf) compute_half(cur, now, live_c, issue);
      else compute(cur, now, live_c, issue);
    } else {
      if (!TAIL || NBUF == 2) load_rows(step + NBUF - 1, ahead);
      if (kAny && (!TAIL || WBUF == 2)) load_w(next, step + WBUF - 1);
      if constexpr (kAny && kHalf) compute_half(cur, now, live_c, [](int) {});
      else if constexpr (kAny) compute(cur, now, live_c, [](int) {});
    }
  };
  const auto run = [&](auto live_c) __attribute__((always_inline)) {
    Weights w0, w1, w2, w3;
    load_rows(0, lds0);
    if (NBUF == 4) {
      load_rows(1, lds1);
      load_rows(2, lds2);
    }
    if (decltype(live_c)::value > 0) load_w(w0, 0);
    if (decltype(live_c)::value > 0 && WBUF == 4) {
      load_w(w1, 1);
      load_w(w2, 2);
    }
    // (the buffers' and operands' places are fixed in the code, so that the
    // compiler sees which loads each step has to wait for)
    int step = 0;
    const auto one = [&](auto k_c, auto tail_c) __attribute__((always_inline)) {
      constexpr int k = decltype(k_c)::value, n = k % NBUF, a = (k + NBUF - 1) % NBUF;
      constexpr int v = k % WBUF, y = (k + WBUF - 1) % WBUF;
      const uint8_t* const cur = n == 0 ? lds0 : (n == 1 ? lds1 : (n == 2 ? lds2 : lds3));
      uint8_t* const ahead = a == 0 ? lds0 : (a == 1 ? lds1 : (a == 2 ? lds2 : lds3));
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
  // a ragged expert's last rows: products of the groups that hold rows only
  if (live == 0) run(std::integral_constant<int, 0>{});
  else if (MODE != kBlockDense && live <= MS / 2) run(std::integral_constant<int, MS / 2>{});
  else run(std::integral_constant<int, MS>{});
  if constexpr (MODE == kBlockUp) {
    // bf16(relu(h)^2), then E4M3 with the scale of the row's block of 128
    // columns, as block_quant_kernel makes them: the tile holds whole blocks, a
    // block lies in 128 / WTN waves, which join their maxima through LDS.
    // Columns come in whole groups of 16 (N is a multiple of 16).
    static_assert(BN % 128 == 0, "whole blocks");
    __shared__ float part[WN][BM];
    // Half the work of this part is the rounding of the squares: the fast form
    // rounds the fp32 square, which is wrong only where that lies on a midpoint
    // (as one in 2^16 does); then the wave takes the exact form.
    u16x2 v[MS][NS][2];  // four bf16 values each
    u16x2 least = {0xffff, 0xffff};
#pragma unroll
    for (int j = 0; j < MS; ++j)
#pragma unroll
      for (int i = 0; i < NS; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float a = fmaxf(acc[i][j][2 * h], 0.f), b = fmaxf(acc[i][j][2 * h + 1], 0.f);
          const f32x2 sq = {a * a, b * b};
          v[j][i][h] = __builtin_bit_cast(u16x2, __builtin_convertvector(sq, bf16x2));
          const u16x2 low = __builtin_bit_cast(
              u16x2, __builtin_amdgcn_perm(__float_as_uint(sq[1]), __float_as_uint(sq[0]), 0x05040100u));
          least = __builtin_elementwise_min(least, low ^ 0x8000);
        }
    if (__ballot(least[0] == 0 || least[1] == 0)) {
#pragma unroll
      for (int j = 0; j < MS; ++j)
#pragma unroll
        for (int i = 0; i < NS; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            v[j][i][h] = u16x2{relu_sq_bf16(acc[i][j][2 * h]), relu_sq_bf16(acc[i][j][2 * h + 1])};
    }
#pragma unroll
    for (int j = 0; j < MS; ++j) {
      u16x2 m2 = {0, 0};  // bf16 values of one sign compare as integers
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (i < groups) m2 = __builtin_elementwise_max(m2, __builtin_elementwise_max(v[j][i][0], v[j][i][1]));
      int amax = m2[0] > m2[1] ? m2[0] : m2[1];
      amax = max(amax, __shfl_xor(amax, 16));
      amax = max(amax, __shfl_xor(amax, 32));
      if (q == 0) part[wn][m0 + j * 16 + c] = __uint_as_float(static_cast<uint32_t>(amax) << 16);
    }
    __syncthreads();
    constexpr int kSharers = 128 / WTN;
    uint8_t* const codes = static_cast<uint8_t*>(g.out);
    const int w0 = wn / kSharers * kSharers;
#pragma unroll
    for (int j = 0; j < MS; ++j) {
      const int r = m0 + j * 16 + c;
      if (j >= live || r >= t.rows) continue;
      float amax = 0.f;
#pragma unroll
      for (int w = 0; w < kSharers; ++w) amax = fmaxf(amax, part[w0 + w][r]);
      const bool any = amax >= kTinyAmax;
      const float inv = any ? __fdiv_rn(448.f, amax) : 0.f;
      const size_t row = static_cast<size_t>(t.row0 + r);
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (i < groups)
          *reinterpret_cast<uint32_t*>(codes + row * g.N + t.n0 + nw0 + i * 16 + 4 * q) =
              encode4(__builtin_bit_cast(uint32_t, v[j][i][0]), __builtin_bit_cast(uint32_t, v[j][i][1]), inv);
      if (wn == w0 && q == 0)
        g.out_s[static_cast<size_t>((t.n0 + nw0) / 128) * g.M + row] = any ? __fdiv_rn(amax, 448.f) : 0.f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < MS; ++j) {
      const int r = m0 + j * 16 + c;
      if (j >= live || r >= t.rows) continue;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const int n = t.n0 + nw0 + i * 16 + 4 * q;
        if (n < g.N) store4<MODE>(g, t.row0 + r, n, acc[i][j]);
      }
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

template <int G, bool QUANT, bool ONCE = true>
hipError_t launch_small(const BlockArgs& g, hipStream_t stream) {
  return dispatch(reinterpret_cast<const void*>(&block_small_kernel<G, QUANT, ONCE>),
                  tiles_of(g, kBlockDense, 16 * G, kSmallN), kSmallWaves * kWave, g, stream, KernelEvents{});
}


template <int MODE, int BM, int BN, int WM, int WN, int NBUF, int WBUF, bool ONCE = false>
hipError_t launch_large(const BlockArgs& g, hipStream_t stream, const KernelEvents& ev = KernelEvents{}) {
  return dispatch(reinterpret_cast<const void*>(&block_gemm_kernel<MODE, BM, BN, WM, WN, NBUF, WBUF, ONCE>),
                  tiles_of(g, MODE, BM, BN), WM * WN * 64, g, stream, ev);
}

}  // namespace

// Rows per tile of the experts' products.  Experts of a few rows take tiles of 32,
// which read each weight once or twice; from 16 rows per expert on, tiles of 128
// (full layer, T = 256, 12 rows per expert: 243 us with 32 rows, 275 with 128;
// T = 384: 287 and 285; T = 768: 364 and 319).  So do short batches of few
// experts, whose 128-row tiles are too few for the chip.
int block_tile_rows(int R, int E) { return R < (16 * E > 256 ? 16 * E : 256) ? 32 : 128; }

// Full layer (128 experts, 2688 -> 1856 -> 2688), whole forward, graph replay.
// Decode tiles 32 x 64 (32 x 128 where the tile makes the codes) with the weights
// 3 steps ahead, since nearly each is read once and from memory: T = 5 54 us, T = 64
// 157.  Prefill tiles 128 x 128 in 4 waves, two workgroups or more to a CU, were the
// best with E4M3 products in both projections (T = 4096 573 us; 128 x 256 in 8 waves
// 581, 128 x 128 in 8 607, 64 x 128 620, 256 x 256 631; column tiles dealt round the
// XCDs 605), and still are for the down projection.  With the up projection in fp16:
// 128 x 128 in 2 x 2 waves 669, in a row of 4 waves 684, 128 x 256 in 8 waves 677,
// 2 x 4 waves 709; tokens handed over in fp16 instead of codes, which is half the
// conversions and twice the LDS reads, 688.  Counters at T = 4096 say what is left:
// the up projection (331 us, 740 TFLOP/s) has the matrix unit busy for 33 % of the
// time and the vector unit, with the conversions of both operands in every wave,
// for 42, at 1.7 waves per SIMD, so the two hardly overlap; LDS is busy for 10 %, HBM
// reads 2.7 TB/s.  The down projection (255 us): matrix unit 23, vector unit 30, LDS
// 26 %, HBM 3.2 TB/s of reads and 264 MB of rows written.
hipError_t launch_block_experts(int stage, const BlockArgs& g, hipStream_t stream, const KernelEvents& ev) {
  if (block_tile_rows(g.M, g.E) == 32)
    return stage == 0 ? launch_large<kBlockUp, 32, 128, 1, 4, 4, 4, true>(g, stream, ev)
                      : launch_large<kBlockDown, 32, 64, 1, 4, 4, 4, true>(g, stream, ev);
  return stage == 0 ? launch_large<kBlockUp, 128, 128, 2, 2, 4, 2>(g, stream, ev)
                    : launch_large<kBlockDown, 128, 128, 1, 4, 2, 2>(g, stream, ev);
}

// One matrix.  Few rows (up to 128) split K over the waves of a workgroup, since
// there are too few tiles for the 256 CUs.  Past that the largest tile is taken
// that still has about a tile per CU (kFill); each halving of the tile costs
// 10-20 % of the rate and is worth it only to fill the chip.  3712 x 2688 weights:
// M = 256 9.2 us with 64 x 64, M = 512 12.0 with 64 x 128, M = 1024 16.9 with 128 x
// 128, M = 2048 27.6 with 128 x 256, M = 4096 46.4 with 256 x 256 (one size larger,
// loads not yet spread: 12.8, 17.8, 30.6, 33.6; one smaller: 15.4, 22.0, 31.1,
// 55.7); 1856 x 2688, M = 4096 29.5 with 128 x 256 (256 x 256, half the chip, 47.7).
constexpr int kFill = 200;
hipError_t launch_block_dense(const BlockArgs& g, hipStream_t stream) {
  if (g.M <= 16) return launch_small<1, false>(g, stream);
  if (g.M <= 32) return launch_small<2, false>(g, stream);
  if (g.M <= 64) return launch_small<4, false>(g, stream);
  if (g.M <= 128) return launch_small<4, false, false>(g, stream);  // two row tiles
  const auto fills = [&](int bm, int bn) { return tiles_of(g, kBlockDense, bm, bn) >= kFill; };
  if (fills(256, 256)) return launch_large<kBlockDense, 256, 256, 2, 4, 4, 2>(g, stream);
  if (fills(128, 256)) return launch_large<kBlockDense, 128, 256, 1, 8, 4, 2>(g, stream);
  if (fills(128, 128)) return launch_large<kBlockDense, 128, 128, 2, 4, 4, 2>(g, stream);
  if (fills(64, 128)) return launch_large<kBlockDense, 64, 128, 2, 4, 4, 2>(g, stream);
  return launch_large<kBlockDense, 64, 64, 2, 4, 4, 4>(g, stream);
}

// Quantised by every workgroup that multiplies them, which for one tile of rows
// costs less than a kernel of its own: 3712 x 2688, M = 1 5.8 us (two kernels
// 6.9, and 3.5 us more on the host), M = 16 7.3 (7.6), M = 24 9.5 (9.3); with more
// rows it loses: M = 77 18.9 us (11.3).
hipError_t launch_block_few_linear(const BlockArgs& g, hipStream_t stream) {
  return g.M <= 16 ? launch_small<1, true>(g, stream) : launch_small<2, true>(g, stream);
}

hipError_t launch_block_quant(const BlockQuantArgs& q, hipStream_t stream) {
  if (q.rows <= 0) return hipSuccess;
  hipLaunchKernelGGL(block_quant_kernel, dim3(quant_groups(q)), dim3(kQThreads), 0, stream, q);
  return hipGetLastError();
}

hipError_t launch_block_pack_codes(const uint8_t* q, int N, int K, uint8_t* codes, hipStream_t stream) {
  const int64_t n = static_cast<int64_t>((N + 15) / 16 * 16) * ((K + 127) / 128) * 8;
  int64_t blocks = (n + kQThreads - 1) / kQThreads;
  if (blocks > 8192) blocks = 8192;
  hipLaunchKernelGGL(block_pack_codes_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kQThreads), 0,
                     stream, q, N, K, codes);
  return hipGetLastError();
}

hipError_t launch_block_pack(const uint16_t* w, int E, int N, int K, uint8_t* codes, float* scales,
                             hipStream_t stream) {
  hipLaunchKernelGGL(block_pack_kernel, dim3((K + 127) / 128, (N + 127) / 128, E), dim3(kQThreads), 0,
                     stream, w, N, K, codes, scales);
  return hipGetLastError();
}

}  // namespace moe
