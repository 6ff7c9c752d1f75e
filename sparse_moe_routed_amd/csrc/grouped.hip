// Products of bf16 rows grouped by expert, with both gradients:
//   y[r, n]      = sum_k x[r, k] w[e, n, k]         rows r of expert e
//   dx[r, k]     = sum_n dy[r, n] w[e, n, k]
//   dw[e, n, k] (+)= sum_{r of e} dy[r, n] x[r, k]
// Sums are fp32 of exact products; results are rounded once.
//
// All three are tile_gemm.h's kernel.  The first has both operands contiguous along the
// sum; in the others the sum runs over the rows of a matrix: of w for dx, of dy and x
// for dw.
#include "products.h"
#include "small.h"
#include "tile_gemm.h"

namespace moe {

namespace {

// rows of no expert, before offsets[0] and from offsets[E] on, set to zero: 16 bytes a
// thread.  For the few rows that pad a batch it is a launch's time (1 to 2 us); for those of
// other experts their fill (24576 rows of 2688 bf16, a quarter of the experts: 124 us, without
// 102)
__global__ __launch_bounds__(256) void zero_rest_kernel(const int32_t* __restrict__ offsets, int E, int R,
                                                        size_t row_bytes, uint8_t* __restrict__ out) {
  const size_t head = min(max(offsets[0], 0), R) * row_bytes, tail = min(max(offsets[E], 0), R) * row_bytes;
  const size_t end = R * row_bytes, step = static_cast<size_t>(gridDim.x) * 256 * 16;
  const size_t at = (static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x) * 16;
  const u32x4 zero = {0u, 0u, 0u, 0u};
  for (size_t i = at; i < head; i += step) *reinterpret_cast<u32x4*>(out + i) = zero;
  for (size_t i = tail + at; i < end; i += step) *reinterpret_cast<u32x4*>(out + i) = zero;
}

// dw of its parts [splits, n], added up in their order, eight loads at a time (64 parts of
// 64 x 64: 18 us with the product, 41 one by one)
__global__ __launch_bounds__(256) void join_kernel(const float* __restrict__ parts, int splits, size_t n,
                                                   void* __restrict__ out, int out_f32, int accumulate) {
  for (size_t i = (static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x) * 4; i < n;
       i += static_cast<size_t>(gridDim.x) * 1024) {
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int s = 0; s < splits; ++s) v += *reinterpret_cast<const f32x4*>(parts + s * n + i);
    if (out_f32) {
      f32x4* const o = reinterpret_cast<f32x4*>(static_cast<float*>(out) + i);
      *o = accumulate ? v + *o : v;
    } else {
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + i) =
          make_uint2(bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3]));
    }
  }
}

hipError_t launch_zero_rest(const GroupedArgs& g, int width, hipStream_t stream) {
  hipLaunchKernelGGL(zero_rest_kernel, dim3(256), dim3(256), 0, stream, g.offsets, g.E, g.R,
                     static_cast<size_t>(width) * (g.out_f32 ? 4 : 2), static_cast<uint8_t*>(g.out));
  return hipGetLastError();
}

NtArgs product_args(const GroupedArgs& g, const void* rows, const void* cols) {
  NtArgs a{};
  a.M = a.a_rows = g.R;
  a.N = g.N;
  a.K = g.K;
  a.a = static_cast<const uint8_t*>(rows);
  a.w = static_cast<const uint8_t*>(cols);
  a.out = g.out;
  a.out_f32 = g.out_f32;
  a.E = g.E;
  a.offsets = g.offsets;
  a.accumulate = g.accumulate;
  return a;
}

}  // namespace

// tiles of 256 x 256 that full rows would make
long long large_tiles(int R, int width) {
  return static_cast<long long>((R + 255) / 256) * ((width + 255) / 256);
}

// Tiles by size, measured at N = 1856 and K = 2688:
//   - few rows, whose tiles of 64 x 128 would leave many CUs without one: 32 columns a
//     workgroup and the sum dealt to its waves (1 row 8.6 us, in tiles 13.9; 16 rows of 4
//     experts 11.0 and 14.5; but of 8 experts 19.5 and 16.0);
//   - 256 x 256, which read least from the caches for each product, where the experts have
//     rows for them and the chip enough of them (192 rows an expert of 128: 315 us, 393 in
//     128 x 128; 8192 rows of one 68 and 81; but 128 rows an expert 289 and 279, and 4096
//     rows of one expert, 128 tiles, 56 and 41);
//   - 128 x 128 where there is more than one for each CU (2500 rows of one expert 36 us, 43
//     in 64 x 128; 4096 rows 41 and 58);
//   - 64 x 128 for the rest, two workgroups to a CU and two stages under way in each (1000
//     rows of one expert 19 us, 31 in 128 x 128; 1000 rows of 16 experts 26 and 30).  With
//     one stage under way in each of three workgroups 1000 rows of one expert take 26 us,
//     and 400 rows of 128 experts with weights in memory 216, now 196.
hipError_t launch_grouped_matmul(const GroupedArgs& g, hipStream_t stream) {
  const NtArgs a = product_args(g, g.x, g.w);
  const int experts = g.R < g.E ? g.R : g.E;  // at most, with rows
  const int row_tiles = (g.R + 127) / 128;
  const long long cols = (g.N + 127) / 128;
  hipError_t err;
  if (g.R <= 256 && ((g.R + 63) / 64 + experts) * cols < 128)
    err = g.R <= 64 ? launch_small<NtBf16, kNtGroups, 1, false>(a, stream)
                    : launch_small<NtBf16, kNtGroups, 4, false>(a, stream);
  else if (g.R >= 144 * g.E && large_tiles(g.R, g.N) >= 160)
    err = launch_tile<NtBf16, kNtGroups, 256, 256, 2, 4, 2, 2>(a, stream);
  else if (g.R >= 4 * g.E && (row_tiles > experts ? row_tiles : experts) * cols >= 280)
    err = launch_tile<NtBf16, kNtGroups, 128, 128, 2, 2, 2, 2>(a, stream);
  else err = launch_tile<NtBf16, kNtGroups, 64, 128, 1, 4, 2, 3>(a, stream);
  return err == hipSuccess && g.zero_rest ? launch_zero_rest(g, g.N, stream) : err;
}

// As above, but w's tile is read turned, a stage of 32 of its rows: four of them in LDS
// beat two of 64 until the matrix instructions bind (192 rows an expert of 128 317 us and
// 322, 512 rows 638 and 618; 8192 rows of 8 experts 97 and 89).  64 x 128 for few rows:
// 1500 rows of 128 experts 221 us, 228 in 256 x 256; 12288 rows 334 and 270; 1000 rows of
// one expert 23 us, 2048 rows 34, where 256 x 256 have too few tiles.  128 x 128 beat
// neither (12288 rows 267 us, 1500 rows 236).
hipError_t launch_grouped_input_grad(const GroupedArgs& g, hipStream_t stream) {
  const NtArgs a = product_args(g, g.dy, g.w);
  hipError_t err;
  if (g.R < 16 * g.E || large_tiles(g.R, g.K) < 128)
    err = launch_tile<NtBf16, kGradRows, 64, 128, 1, 4, 1, 4>(a, stream);
  else if (g.R < 320 * g.E) err = launch_tile<NtBf16, kGradRows, 256, 256, 2, 4, 1, 4>(a, stream);
  else err = launch_tile<NtBf16, kGradRows, 256, 256, 2, 4, 2, 2>(a, stream);
  return err == hipSuccess && g.zero_rest ? launch_zero_rest(g, g.K, stream) : err;
}

// dw in tiles of 128 x 256, whose four waves read two operands of rows for each of columns:
// at 128 experts of 1856 x 2688 and 24576 rows 472 us, in 256 x 256 522, in 128 x 128 542;
// at 1500 rows, where the fill of dw binds, 237, 287 and 298.
//
// Parts of an expert's rows side by side, 128 rows a part at least, each a sum of its own,
// joined in order, where the experts' tiles are too few for the chip and the experts' rows
// many enough to pay for the second kernel: 24576 rows of one expert, 64 x 64, 18 us, in one
// part 249; 1500 rows of each of 16, 256 x 256, 22 and 28; 1024 rows each 21 and 21; 512 rows
// each 18 and 14.
constexpr int kDwRows = 128, kDwCols = 256;
int weight_grad_splits(int R, int E, int N, int K) {
  if (R < 1024ll * E) return 1;
  const long long tiles = static_cast<long long>(E) * ((N + kDwRows - 1) / kDwRows) * ((K + kDwCols - 1) / kDwCols);
  const long long by_tiles = 256 / tiles, by_rows = R / (128ll * E);
  const long long s = by_tiles < by_rows ? by_tiles : by_rows;
  return s < 2 ? 1 : static_cast<int>(s < 64 ? s : 64);
}

hipError_t launch_grouped_weight_grad(const GroupedArgs& g, hipStream_t stream) {
  NtArgs a = product_args(g, g.dy, g.x);
  a.splits = weight_grad_splits(g.R, g.E, g.N, g.K);
  // Rows are read ahead where there are enough of them, the last-level cache (256 MB) holds
  // them and the writes of dw would keep memory from them: R = 24576, 1856 x 2688, bf16,
  // 128 experts (dw 5.7 times the rows' bytes) 472 us, 520 without; 64 experts (2.9 times)
  // 349 and 354; but 32 (1.4 times) 315 and 294.
  const size_t bytes = static_cast<size_t>(g.R) * (g.N + g.K) * 2;
  const size_t dw_bytes = static_cast<size_t>(g.E) * g.N * g.K * (g.out_f32 ? 4 : 2);
  a.warm = bytes >= (32u << 20) && bytes <= (240u << 20) && dw_bytes >= 2 * bytes ? 32 : 0;
  if (a.splits > 1) {
    a.out = g.partial;
    a.out_f32 = 1;
    a.accumulate = 0;
  }
  const hipError_t err = launch_tile<NtBf16, kGradWeights, kDwRows, kDwCols, 1, 4, 1, 3>(a, stream);
  if (err != hipSuccess || a.splits == 1) return err;
  const size_t n = static_cast<size_t>(g.E) * g.N * g.K;
  const size_t groups = (n / 4 + 255) / 256;
  hipLaunchKernelGGL(join_kernel, dim3(static_cast<unsigned>(groups < 4096 ? groups : 4096)), dim3(256), 0, stream,
                     g.partial, a.splits, n, g.out, g.out_f32, g.accumulate);
  return hipGetLastError();
}

}  // namespace moe
