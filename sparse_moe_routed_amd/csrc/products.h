// What the products of channel.hip and grouped.hip share: element types, operands, the
// tile a workgroup takes, and how results are stored.
//   out[m, n] = sum_k a[m, k] w[n, k]     (and grouped.hip's gradients)
// over one matrix or over groups of rows with a matrix each, in bf16 or in 8-bit
// integers.  Sums are fp32 of exact products, or exact int32.  An instruction's depth is
// 64 bytes of a row in both types, 32 bf16 or 64 integers, and its operands are one
// 16-byte chunk per lane: row lane % 16, chunk lane / 16 of four.
#pragma once
#include <hip/hip_runtime.h>
#include <type_traits>

#include "moe_common.h"
#include "moe_internal.h"
#include "tile.h"

namespace moe {

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) uint8_t* Lds;  // so that the compiler sees which buffer is read

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
  kNtDown = 3,    // experts: fp32 gate * h
  kGradRows = 4,     // dx: rows of dy, columns of w, the sum over w's rows
  kGradWeights = 5   // dw: columns of dy by columns of x, the sum over the expert's rows
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

// four results of a row: columns n .. n + 3 of `width`, at value `at` of the output, in
// fp32 or bf16; WHOLE: rows of whole quads, and quads aligned
template <typename T, int MODE, bool F32, bool WHOLE>
__device__ __forceinline__ void nt_store(const NtArgs& g, size_t at, int width, int n, typename T::Acc v, float rs,
                                         f32x4 cs, float gate) {
  f32x4 h;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = nt_value(v[i], rs, cs[i]);
    if constexpr (MODE == kNtDown) h[i] *= gate;
  }
  if constexpr (F32) {
    float* const o = static_cast<float*>(g.out) + at;
    if constexpr (WHOLE) {
      *reinterpret_cast<f32x4*>(o) = h;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < width) o[i] = h[i];
    }
  } else {
    uint16_t* const o = static_cast<uint16_t*>(g.out) + at;
    const auto pair = [&](int i) __attribute__((always_inline)) {
      return MODE == kNtUp ? relu_sq_bf16_pair(h[i], h[i + 1]) : bf16_pair(h[i], h[i + 1]);
    };
    const uint2 b = make_uint2(pair(0), pair(2));
    if constexpr (WHOLE) {
      *reinterpret_cast<uint2*>(o) = b;
    } else {
      if (n < width) o[0] = static_cast<uint16_t>(b.x);
      if (n + 1 < width) o[1] = static_cast<uint16_t>(b.x >> 16);
      if (n + 2 < width) o[2] = static_cast<uint16_t>(b.y);
      if (n + 3 < width) o[3] = static_cast<uint16_t>(b.y >> 16);
    }
  }
}

// store(fp32?, whole?) as the call's output asks for: experts' widths are multiples of
// 64, those of grouped products of 8
template <typename T, int MODE, typename Store>
__device__ __forceinline__ void nt_store_as(const NtArgs& g, int width, Store store) {
  constexpr std::true_type yes{};
  constexpr std::false_type no{};
  if constexpr (MODE == kNtUp) store(no, yes);
  else if constexpr (MODE == kNtDown) store(yes, yes);
  else if constexpr (MODE == kNtDense) {
    if (width % 4 == 0) {
      if (g.out_f32) store(yes, yes);
      else store(no, yes);
    } else {
      if (g.out_f32) store(yes, no);
      else store(no, no);
    }
  } else {
    if (g.out_f32) store(yes, yes);
    else store(no, yes);
  }
}

// ---- the results of a tile
struct StoreAt {
  int row0, rows, n0, cols;  // first row of all and column, valid rows and columns of the tile
  int ldo;                   // values between rows of the output
  size_t out;                // first value of the output tile
  const float* w_s;
};

// Stores a tile's results.  They go through LDS, so that a store instruction writes
// whole rows of the tile: a lane holds four columns of a row and its neighbours other
// rows, which would be a part of 16 lines.  buffer(0) to buffer(NB - 1) are parts of LDS of
// kBytes each, which take as many rows as fit at a time; chunk x of row r lies at x ^ (r % 16), on
// other banks than its neighbours.  Row group j of a wave is j WM + wm.  Stores are
// non-temporal: of y, dx and dw nothing is read again before it has left the caches (dw of
// 1500 rows 246 us, with ordinary stores 333; of 24576 rows in fp32 561 and 724).  What the
// experts write is read by the next kernel, but ordinary stores gain nothing there either
// (the layer of 640, 2048 and 4096 tokens 316, 402 and 551 us, with ordinary stores of the
// intermediate and of the rows 317, 405 and 555).
template <typename T, int MODE, int BM, int BN, int WM, int WN, int NB, int kBytes, typename Buffers>
__device__ __forceinline__ void store_tile(const NtArgs& g, const StoreAt& t, Buffers buffer,
                                           const typename T::Acc (&acc)[BN / WN / 16][BM / WM / 16]) {
  constexpr int MS = BM / WM / 16, NS = BN / WN / 16, NW = WM * WN;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN, c = lane & 15, q = lane >> 4;
  // scales of this lane's rows and columns, all loads at once
  float rs[MS], gate[MS];
  f32x4 cs[NS];
  if constexpr (T::kBytes == 1) {
    size_t source[MS];
#pragma unroll
    for (int j = 0; j < MS; ++j) {
      const int r = t.row0 + min((j * WM + wm) * 16 + c, t.rows - 1);
      source[j] = nt_source<MODE>(g, r);
      if constexpr (MODE == kNtDown) gate[j] = g.row_gate[r];
    }
#pragma unroll
    for (int j = 0; j < MS; ++j) rs[j] = g.a_s[source[j]];
#pragma unroll
    for (int i = 0; i < NS; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) cs[i][k] = t.w_s[min(t.n0 + (wn * NS + i) * 16 + 4 * q + k, g.N - 1)];
  }
  // this lane's four results of column group i, row group j
  const auto scaled = [&](int i, int j) __attribute__((always_inline)) {
    f32x4 h;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (T::kBytes == 1) h[k] = nt_value(acc[i][j][k], rs[j], cs[i][k]);
      else h[k] = acc[i][j][k];
      if constexpr (MODE == kNtDown) h[k] *= gate[j];
    }
    return h;
  };
  const auto rows = [&](auto f32_c) __attribute__((always_inline)) {
    constexpr bool kF32 = decltype(f32_c)::value;
    constexpr int kRowBytes = BN * (kF32 ? 4 : 2), kChunks = kRowBytes / 16;
    constexpr int kFit = kBytes / kRowBytes / (16 * WM) * (16 * WM);  // rows of a buffer
    constexpr int kGroups = kFit / (16 * WM);                         // row groups of a wave in it
    constexpr int kRounds = (MS + NB * kGroups - 1) / (NB * kGroups);
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    typedef __attribute__((address_space(3))) u32x4* Chunk16;
    typedef __attribute__((address_space(3))) u32x2* Chunk8;
    static_assert(kFit > 0 && kChunks >= 16, "rows of a buffer");
#pragma unroll
    for (int round = 0; round < kRounds; ++round) {
      __syncthreads();  // what was there has been read
#pragma unroll
      for (int i = 0; i < NS; ++i) {
#pragma unroll
        for (int jj = 0; jj < NB * kGroups; ++jj) {
          const int j = round * NB * kGroups + jj;
          if (j >= MS) continue;
          const f32x4 h = scaled(i, j);
          const int group = wn * NS + i;
          const Lds row = buffer(jj / kGroups) + ((jj % kGroups * WM + wm) * 16 + c) * kRowBytes;
          if constexpr (kF32) {
            *(Chunk16)(row + (((group * 4 + q) ^ c) << 4)) = __builtin_bit_cast(u32x4, h);
          } else {
            u32x2 v;
            if constexpr (MODE == kNtUp) {
              v = u32x2{relu_sq_bf16_pair(h[0], h[1]), relu_sq_bf16_pair(h[2], h[3])};
            } else {
              v = u32x2{bf16_pair(h[0], h[1]), bf16_pair(h[2], h[3])};
            }
            *(Chunk8)(row + (((group * 2 + (q >> 1)) ^ c) << 4) + ((q & 1) << 3)) = v;
          }
        }
      }
      __syncthreads();
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int first = (round * NB + b) * kFit;
        for (int at = wave * 64 + lane; at < kFit * kChunks; at += NW * 64) {
          const int lr = at / kChunks, ch = at % kChunks, r = first + lr, n = ch * (kF32 ? 4 : 8);
          if (r >= t.rows) break;
          if (n >= t.cols) continue;
          u32x4 v = *(Chunk16)(buffer(b) + lr * kRowBytes + ((ch ^ (lr & 15)) << 4));
          const size_t to = t.out + static_cast<size_t>(r) * t.ldo + n;
          if constexpr (kF32) {
            u32x4* const o = reinterpret_cast<u32x4*>(static_cast<float*>(g.out) + to);
            if (MODE == kGradWeights && g.accumulate)
              v = __builtin_bit_cast(u32x4, __builtin_bit_cast(f32x4, v) +
                                                __builtin_bit_cast(f32x4, __builtin_nontemporal_load(o)));
            __builtin_nontemporal_store(v, o);
          } else {
            __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(static_cast<uint16_t*>(g.out) + to));
          }
        }
      }
    }
  };
  // results one by one, where rows of the output are no multiple of 16 bytes
  const auto each = [&](auto f32_c) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int n = (wn * NS + i) * 16 + 4 * q;
#pragma unroll
      for (int j = 0; j < MS; ++j) {
        const int r = (j * WM + wm) * 16 + c;
        if (r >= t.rows) continue;
        const f32x4 h = scaled(i, j);
        const size_t to = t.out + static_cast<size_t>(r) * t.ldo + n;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (n + k >= t.cols) continue;
          if constexpr (decltype(f32_c)::value) static_cast<float*>(g.out)[to + k] = h[k];
          else static_cast<uint16_t*>(g.out)[to + k] = f32_to_bf16(h[k]);
        }
      }
    }
  };
  constexpr std::true_type kYes{};
  constexpr std::false_type kNo{};
  if constexpr (MODE == kNtUp) {
    rows(kNo);
  } else if constexpr (MODE == kNtDown) {
    rows(kYes);
  } else {
    if (MODE == kNtDense && t.ldo % (g.out_f32 ? 4 : 8)) {
      if (g.out_f32) each(kYes);
      else each(kNo);
    } else if (g.out_f32) {
      rows(kYes);
    } else {
      rows(kNo);
    }
  }
}

template <int MODE, int BM, int BN>
long long row_tiles(const NtArgs& g) {
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

}  // namespace moe
