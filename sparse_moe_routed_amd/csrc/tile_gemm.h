// Tiles of the grouped and dense products whose operands both go through LDS, so
// that a tile's every byte is fetched once.
//
// A stage is KH instructions' depth along the sum, 64 bytes each (32 bf16, 64 integers).
// Operands come in three forms:
//   contiguous  rows with the sum along memory: 64 KH bytes of a row, chunks of 16 moved
//               by row_swz; a lane's operand is one chunk
//   packed      weights in operand order (moe.h): copied as they lie
//   turned      the sum runs over the rows of memory: 32 KH of them as they lie, pairs of
//               chunks moved by tr_swz; ds_read_b64_tr_b16 hands lane i of 16 column i
//               of four rows, so two of them are a lane's 8 values
//
// Products run with operands that are in registers already; among them go the reads
// of the next depth's operands.  At the last depth of a stage the next stage has
// arrived, the operands of this one have been read, and one barrier says so for
// everyone; then the reads are of the next stage, and the loads of the stage NBUF
// further on go into the buffer that has been read.  So the matrix unit waits for no
// LDS read, there is one barrier a stage, and NBUF - 1 stages are under way.
//
// What bounds it: on 8192^3, where a tile of 256 x 256 needs 64 KB of operands for each
// 8.4 million products, the matrix unit: 1150 to 1360 TFLOP/s in bf16 in the three
// forms (library products 1171 to 1458), and 2.10 POP/s in integers at 4096 x 3712 x 2688.
// Grouped by expert the weights bind, each read once: 4.1 to 4.4 TB/s with their rows and
// results at 192 rows an expert, 5.8 TB/s at 12.
#pragma once
#include "products.h"

namespace moe {

typedef short s16x4 __attribute__((ext_vector_type(4)));

enum TileForm { kContig = 0, kPackedForm = 1, kTurned = 2 };
// what a reduction row's 32-byte pairs of 16-byte chunks are moved by: the rows that
// the lanes of half a wave read at once (k % 32 in 0..3 and 8..11, then 16..19 and
// 24..27, each then 4 on) lie on distinct banks
__device__ __forceinline__ int tr_swz(int k) { return (k & 3) | ((k >> 3) & 1) << 2; }

struct ProductTile {
  int rows, cols;   // valid rows and columns of the tile
  int row0, n0;     // first row (of all rows) and column
  int length;       // of the sum, in values
  const uint8_t *a, *b;
  uint32_t a_stride, b_stride;  // bytes between rows of memory
  uint32_t a_bytes;             // of contiguous rows
  size_t out;                   // first value of the output tile
  int ldo;                      // values between rows of the output
  const float* w_s;
};

// values that all lanes share, in scalar registers (a division leaves them in vector ones)
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ uint32_t uniform(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(v)));
}
__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  return reinterpret_cast<const uint8_t*>(static_cast<uint64_t>(uniform(static_cast<uint32_t>(u >> 32))) << 32 |
                                          uniform(static_cast<uint32_t>(u)));
}

template <typename T, int MODE, int BM, int BN>
__device__ __forceinline__ bool tile_find(const NtArgs& g, ProductTile& t) {
  if constexpr (MODE == kGradWeights) {
    // a row of tiles of one expert is one XCD's, the rows of tiles go round: experts
    // of many rows are then shared by all
    const int n_rt = (g.N + BM - 1) / BM, n_ct = (g.K + BN - 1) / BN;
    const int b = blockIdx.x - g.warm, l = b >> 3, panel = l / n_ct * 8 + (b & 7), ct = l % n_ct;
    if (panel >= g.E * g.splits * n_rt) return false;
    const int es = panel / n_rt, rt = panel - es * n_rt, e = es / g.splits, split = es - e * g.splits;
    int lo = min(max(g.offsets[e], 0), g.M), hi = min(max(g.offsets[e + 1], 0), g.M);
    if (g.splits > 1) {  // a part of the expert's rows, whole stages of them
      const int part = (max(hi - lo, 0) + g.splits * 32 - 1) / (g.splits * 32) * 32;
      const int from = min(lo + split * part, hi);
      hi = min(from + part, hi);
      lo = from;
    }
    const int first = __builtin_amdgcn_readfirstlane(lo);
    t.length = __builtin_amdgcn_readfirstlane(max(hi - lo, 0));
    if (t.length == 0 && g.accumulate) return false;
    t.row0 = rt * BM;
    t.n0 = ct * BN;
    t.rows = min(BM, g.N - t.row0);
    t.cols = min(BN, g.K - t.n0);
    t.a_stride = g.N * 2u;
    t.b_stride = g.K * 2u;
    t.a = g.a + static_cast<size_t>(first) * t.a_stride + t.row0 * 2;
    t.b = g.w + static_cast<size_t>(first) * t.b_stride + t.n0 * 2;
    t.ldo = g.K;
    t.out = ((static_cast<size_t>(split) * g.E + e) * g.N + t.row0) * g.K + t.n0;
  } else {
    const int width = MODE == kGradRows ? g.K : g.N;  // of the output
    t.length = MODE == kGradRows ? g.N : g.K;
    const int n_nt = (width + BN - 1) / BN;
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
    t.cols = min(BN, width - t.n0);
    t.a_stride = t.length * T::kBytes;
    t.a = g.a + static_cast<size_t>(t.row0) * t.a_stride;
    t.a_bytes = static_cast<uint32_t>(t.rows) * t.a_stride;
    const uint8_t* const w = g.w + static_cast<size_t>(e) * nt_matrix_bytes<T>(g.N, g.K);
    if constexpr (MODE == kGradRows) {
      t.b_stride = g.K * 2u;
      t.b = w + t.n0 * 2;
    } else {
      t.b_stride = T::kPacked ? (g.K + 127) / 128 * 2048u : g.K * 2u;  // of 16 rows, of one
      t.b = w + static_cast<size_t>(T::kPacked ? t.n0 / 16 : t.n0) * t.b_stride;
    }
    t.ldo = width;
    t.out = static_cast<size_t>(t.row0) * width + t.n0;
    t.w_s = g.w_s;
  }
  t.a = uniform(t.a);
  t.b = uniform(t.b);
  t.rows = uniform(t.rows);
  t.cols = uniform(t.cols);
  t.length = uniform(t.length);
  t.a_bytes = uniform(t.a_bytes);
  t.a_stride = uniform(t.a_stride);
  t.b_stride = uniform(t.b_stride);
  t.row0 = uniform(t.row0);
  t.n0 = uniform(t.n0);
  return true;
}

// 16 bytes a lane from memory straight into LDS, 1 KB from `to` on.  In assembly because
// the compiler, which cannot tell the two buffers apart in every form of read, would
// wait for all of them before the next read; the waits are the step's own.  A load
// past the descriptor's end writes zeros.  m0, which holds `to`, is an operand, so that the
// compiler knows what is in it.  It does not look into the assembly for what the scalar
// operands need: five wait states between a vector instruction (a readfirstlane) that
// writes one and the load that reads it, one after m0.
__device__ __forceinline__ void dma16(i32x4 rsrc, uint32_t at, uint32_t step_at, Lds to) {
  __asm__ volatile("s_nop 4\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"{m0}"(
                       uniform(static_cast<uint32_t>(reinterpret_cast<uintptr_t>(to)))),
                   "v"(at), "s"(rsrc), "s"(uniform(step_at))
                   : "memory");
}

__device__ __forceinline__ i32x4 descriptor(const uint8_t* p, uint32_t bytes) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  return i32x4{uniform(static_cast<int>(u)), uniform(static_cast<int>(u >> 32) & 0xffff),
               uniform(static_cast<int>(bytes)), kRawBuffer};
}

// Reads all rows of dy and x once, expert after expert, g.warm workgroups side by side,
// and drops them: they are in the last-level cache then, where the tiles find them.
// A tile's own loads are a few stages ahead of its products, which is too little for
// memory that is busy with the writes of dw.
__device__ __forceinline__ void warm_rows(const NtArgs& g, Lds to, int waves) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t mine = (blockIdx.x * waves + wave) * 1024u + lane * 16u, all = g.warm * waves * 1024u;
  const Lds at = to + wave * 1024;
  const auto read = [&](const uint8_t* p, size_t bytes) __attribute__((always_inline)) {
    read_once(bytes, mine, all, [&](size_t base, uint32_t n, uint32_t o, uint32_t step_at) __attribute__((always_inline)) {
      dma16(descriptor(p + base, n), o, step_at, at);
      __asm__ volatile("s_waitcnt vmcnt(24)" ::: "memory");
    });
  };
  const int E = g.E;
  for (int e = 0; e < E; ++e) {
    const int lo = uniform(min(max(g.offsets[e], 0), g.M)), hi = uniform(min(max(g.offsets[e + 1], 0), g.M));
    if (hi <= lo) continue;
    read(g.w + static_cast<size_t>(lo) * g.K * 2, static_cast<size_t>(hi - lo) * g.K * 2);
    read(g.a + static_cast<size_t>(lo) * g.N * 2, static_cast<size_t>(hi - lo) * g.N * 2);
  }
  __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// chunk x of row r of a contiguous operand lies at x ^ row_swz(r).  16 lanes at a time read
// LDS: rows 0 to 3 and 12 to 15 of one chunk with rows 4 to 11 of its neighbour (x ^ 1), or
// the other way round; they fall on distinct banks.
template <int KH>
__device__ __forceinline__ int row_swz(int r) {
  return KH == 1 ? -(r >> 2) & 3 : swz(r);
}

template <typename T, int MODE, int BM, int BN, int WM, int WN, int KH, int NBUF>
__global__ __launch_bounds__(WM* WN * 64, 2) void tile_kernel(NtArgs g) {
  typedef typename T::Acc Acc;
  constexpr int AF = MODE == kGradWeights ? kTurned : kContig;
  constexpr int BF = MODE >= kGradRows ? kTurned : (T::kPacked ? kPackedForm : kContig);
  constexpr int NW = WM * WN, WTM = BM / WM, WTN = BN / WN, MS = WTM / 16, NS = WTN / 16;
  constexpr int kRow = 64 * KH;  // bytes of a row
  constexpr int ABYTES = BM * kRow, BBYTES = BN * kRow, BUF = ABYTES + BBYTES;
  constexpr int QA = ABYTES / 1024 / NW, QB = BBYTES / 1024 / NW;  // loads per wave and stage
  constexpr int kLoads = QA + QB;
  constexpr int kStep = kRow / T::kBytes;  // values of the sum
  static_assert(QA * NW * 1024 == ABYTES && QB * NW * 1024 == BBYTES, "tile");
  static_assert((AF != kTurned || BM >= 128) && (BF != kTurned || BN >= 128), "a turned row covers the banks");
  static_assert(MODE == kNtDense || MODE == kNtGroups || MODE >= kGradRows, "rows as they lie");
  static_assert(BF != kPackedForm || KH == 2, "whole steps of packed weights");
  static_assert((KH == 1 || KH == 2) && NBUF >= 2 && NBUF * BUF <= 160 * 1024 && (NBUF - 1) * kLoads < 64, "buffers");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[NBUF * BUF];
  if (MODE == kGradWeights && static_cast<int>(blockIdx.x) < g.warm) {
    warm_rows(g, (Lds)lds, NW);
    return;
  }
  ProductTile t;
  if (!tile_find<T, MODE, BM, BN>(g, t)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int c = lane & 15, q = lane >> 4;
  const int steps = (t.length + kStep - 1) / kStep;

  constexpr int kChunks = kRow / 16, kRows = 64 / kChunks;  // of a row, in a piece
  // Piece p = wave + NW i (1 KB) of an operand's stage: where this lane's 16 bytes come
  // from.  What the stage or the tile does not hold is past the end, as are the stages
  // past the last: rows by the descriptor, chunks of a row by their offset.
  const auto place = [&](auto form_c, int width, uint32_t stride, int valid, int i) __attribute__((always_inline)) {
    constexpr int kForm = decltype(form_c)::value;
    const int p = wave + NW * i;
    if constexpr (kForm == kTurned) {
      const int at = p * 1024 + lane * 16, k = at / (width * 2), ch = at % (width * 2) / 16;
      const int col = (((ch >> 1) ^ tr_swz(k)) << 4) + ((ch & 1) << 3);  // first of 8 columns
      return col < valid ? k * stride + col * 2u : kPastEnd;
    } else if constexpr (kForm == kPackedForm) {
      return (p >> 1) * stride + (p & 1) * 1024u + lane * 16u;
    } else {
      const int r = p * kRows + lane / kChunks;
      return r * stride + ((lane % kChunks) ^ row_swz<KH>(r)) * 16u;
    }
  };
  // pieces of a wave lie a fixed distance apart where chunks move alike in them
  constexpr bool kAlikeA = AF != kTurned || NW * 512 / BM % 16 == 0;
  constexpr bool kAlikeB = BF != kTurned || NW * 512 / BN % 16 == 0;
  static_assert(KH == 1 || NW % 2 == 0, "contiguous rows and packed groups move alike");
  const uint32_t apart_a = AF == kTurned ? NW * 512 / BM * t.a_stride : NW * kRows * t.a_stride;
  const uint32_t apart_b =
      BF == kTurned ? NW * 512 / BN * t.b_stride : (BF == kPackedForm ? NW / 2 : NW * kRows) * t.b_stride;
  const int chunk = (lane % kChunks) ^ row_swz<KH>(wave * kRows + lane / kChunks);  // of a contiguous row
  uint32_t aa[kAlikeA ? 1 : QA], ba[kAlikeB ? 1 : QB];
#pragma unroll
  for (int i = 0; i < (kAlikeA ? 1 : QA); ++i)
    aa[i] = place(std::integral_constant<int, AF>{}, BM, t.a_stride, t.rows, i);
#pragma unroll
  for (int i = 0; i < (kAlikeB ? 1 : QB); ++i)
    ba[i] = place(std::integral_constant<int, BF>{}, BN, t.b_stride, t.cols, i);
  const uint32_t b_bytes = (BF == kPackedForm ? (t.cols + 15) / 16 : t.cols) * t.b_stride;
  // load l of QA + QB of a stage (load_at.h)
  const auto load1 = [&](int step, Lds buf, auto l_c) __attribute__((always_inline)) {
    constexpr int l = decltype(l_c)::value;
    constexpr bool kIsA = l < QA;
    constexpr int i = kIsA ? l : l - QA, kForm = kIsA ? AF : BF;
    const int left = max(min(t.length - step * kStep, kStep), 0);  // of the sum's values
    const uint8_t* const base = kIsA ? t.a : t.b;
    const uint32_t stride = kIsA ? t.a_stride : t.b_stride;
    const Lds to = buf + (kIsA ? 0 : ABYTES) + (wave + NW * i) * 1024;
    uint32_t at;
    if constexpr (kIsA) at = kAlikeA ? aa[0] + i * apart_a : aa[kAlikeA ? 0 : i];
    else at = kAlikeB ? ba[0] + i * apart_b : ba[kAlikeB ? 0 : i];
    if constexpr (kForm == kTurned) {
      dma16(descriptor(base + static_cast<size_t>(step) * kStep * stride, left * stride), at, 0, to);
    } else if constexpr (kForm == kPackedForm) {
      const StageLoad g = load_packed(b_bytes, at, step, left);
      dma16(descriptor(base, g.records), g.at, g.step_at, to);
    } else {
      const StageLoad g = load_rows(kIsA ? t.a_bytes : b_bytes, at, step, kRow, left, chunk * (16 / T::kBytes));
      dma16(descriptor(base, g.records), g.at, g.step_at, to);
    }
  };
  const auto load_part = [&](int step, Lds buf, auto from_c, auto to_c) __attribute__((always_inline)) {
    constexpr int kFrom = decltype(from_c)::value, kTo = decltype(to_c)::value;
    const auto go = [&](auto self, auto l_c) __attribute__((always_inline)) {
      constexpr int l = decltype(l_c)::value;
      if constexpr (l < kTo) {
        load1(step, buf, l_c);
        self(self, std::integral_constant<int, l + 1>{});
      }
    };
    go(go, std::integral_constant<int, kFrom>{});
  };

  // operands of a stage: row group j of this wave is j WM + wm, so that a ragged
  // tile's rows are shared out; `live` of them hold rows
  const int live = __builtin_amdgcn_readfirstlane(min(MS, (((t.rows + 15) >> 4) - wm + WM - 1) / WM));
  const int tr_row = 8 * q + (c >> 2), tr_f = tr_swz(tr_row);
  const uint32_t contig_lane = c * kRow + ((q ^ row_swz<KH>(c)) << 4);
  typedef const __attribute__((address_space(3))) u32x4* Chunk;
  const auto operand = [&](Lds tile, auto form, int width, int group, int h) __attribute__((always_inline)) {
    constexpr int kForm = decltype(form)::value;
    if constexpr (kForm == kTurned) {
      typedef __attribute__((address_space(3))) s16x4* Quad;
      const Lds p = tile + (h * 32 + tr_row) * width * 2 + ((group ^ tr_f) << 5) + ((c & 3) << 3);
      const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Quad)p);
      const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((Quad)(p + 8 * width));
      return __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      return *(Chunk)(tile + group * KH * 1024 + (kForm == kPackedForm ? h * 1024u + lane * 16u : contig_lane ^ (h * 64u)));
    }
  };
  const auto row_operand = [&](Lds buf, int j, int h) __attribute__((always_inline)) {
    return operand(buf, std::integral_constant<int, AF>{}, BM, j * WM + wm, h);
  };
  const auto col_operand = [&](Lds buf, int i, int h) __attribute__((always_inline)) {
    return operand(buf + ABYTES, std::integral_constant<int, BF>{}, BN, wn * NS + i, h);
  };
  Acc acc[NS][MS];
#pragma unroll
  for (int i = 0; i < NS; ++i)
#pragma unroll
    for (int j = 0; j < MS; ++j) acc[i][j] = Acc{};
  typedef u32x4 Cols[NS];
  u32x4 x[MS];
  Cols w0, w1;
  // with products of the wave's first ML row groups
  const auto run = [&](auto live_c) __attribute__((always_inline)) {
    constexpr int ML = decltype(live_c)::value;
    constexpr int kPer = (NS + ML - 1) / ML;  // column operands read beside one row operand
    constexpr std::integral_constant<int, 0> kFirst{};
    // The products of one depth (x, w), the operands of depth h in `from` into `next` and x (a
    // row operand is read into the place of the one that has been multiplied), and with
    // `load` stage `step` into `to`.
    const auto depth = [&](const Cols& w, Cols& next, Lds from, int h, auto load_c, int step, Lds to)
                           __attribute__((always_inline)) {
      const auto part = [&](auto self, auto j_c) __attribute__((always_inline)) {
        constexpr int j = decltype(j_c)::value;
        if constexpr (j < ML) {
#pragma unroll
          for (int i = j * kPer; i < (j + 1) * kPer && i < NS; ++i) next[i] = col_operand(from, i, h);
          if constexpr (decltype(load_c)::value)
            load_part(step, to, std::integral_constant<int, j * kLoads / ML>{},
                      std::integral_constant<int, (j + 1) * kLoads / ML>{});
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int i = 0; i < NS; ++i) acc[i][j] = T::mma(w[i], x[j], acc[i][j]);
          x[j] = row_operand(from, j, h);
          __builtin_amdgcn_sched_barrier(0);
          self(self, std::integral_constant<int, j + 1>{});
        }
      };
      part(part, kFirst);
    };
    // the stage's last depth, w its column operands
    const auto last = [&](int step, uint32_t cur_at, uint32_t other_at, const Cols& w, Cols& next)
                          __attribute__((always_inline)) {
      __asm__ volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((NBUF - 2) * kLoads) : "memory");
      depth(w, next, (Lds)lds + other_at, 0, std::true_type{}, step + NBUF, (Lds)lds + cur_at);
    };
#pragma unroll
    for (int b = 0; b < NBUF; ++b)
      load_part(b, (Lds)lds + b * BUF, kFirst, std::integral_constant<int, kLoads>{});
    __asm__ volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((NBUF - 1) * kLoads) : "memory");
#pragma unroll
    for (int i = 0; i < NS; ++i) w0[i] = col_operand((Lds)lds, i, 0);
#pragma unroll
    for (int j = 0; j < ML; ++j) x[j] = row_operand((Lds)lds, j, 0);
    uint32_t cur = 0, other = BUF;
    const auto forward = [&]() __attribute__((always_inline)) {
      cur = other;
      other = other == (NBUF - 1) * BUF ? 0 : other + BUF;
    };
    for (int step = 0;;) {
      if constexpr (KH == 2) {
        depth(w0, w1, (Lds)lds + cur, 1, std::false_type{}, 0, (Lds)lds);
        last(step, cur, other, w1, w0);
      } else {
        last(step, cur, other, w0, w1);
        forward();
        if (++step >= steps) break;
        last(step, cur, other, w1, w0);
      }
      forward();
      if (++step >= steps) break;
    }
    __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");  // nothing is under way into LDS from here on
  };
  constexpr int kQuarter = MS < 4 ? 1 : MS / 4;
  if (steps > 0) {
    if (live <= kQuarter) run(std::integral_constant<int, kQuarter>{});
    else if (MS > 2 && live <= MS / 2) run(std::integral_constant<int, MS / 2>{});
    else if (MS > 2 && live <= MS / 2 + kQuarter) run(std::integral_constant<int, MS / 2 + kQuarter>{});
    else run(std::integral_constant<int, MS>{});
  }

  const auto buffers = [&](int) __attribute__((always_inline)) { return (Lds)lds; };
  store_tile<T, MODE, BM, BN, WM, WN, 1, NBUF * BUF>(g, {t.row0, t.rows, t.n0, t.cols, t.ldo, t.out, t.w_s}, buffers, acc);
}

template <typename T, int MODE, int BM, int BN, int WM, int WN, int KH, int NBUF>
hipError_t launch_tile(const NtArgs& g, hipStream_t stream) {
  const long long width = MODE >= kGradRows ? g.K : g.N, n_ct = (width + BN - 1) / BN;
  long long blocks;
  if (MODE == kGradWeights) blocks = (g.E * static_cast<long long>(g.splits) * ((g.N + BM - 1) / BM) + 7) / 8 * 8 * n_ct + g.warm;
  else if (MODE == kNtDense) blocks = (n_ct * ((g.M + BM - 1) / BM) + 7) / 8 * 8;
  else blocks = group_tiles(g.M, g.E, BM, n_ct);
  return launch_tiles(reinterpret_cast<const void*>(&tile_kernel<T, MODE, BM, BN, WM, WN, KH, NBUF>), blocks, WM * WN * 64, g,
                      stream);
}

}  // namespace moe
