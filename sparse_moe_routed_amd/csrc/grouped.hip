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
#include "tile_gemm.h"

namespace moe {

namespace {

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

// Tiles of 256 rows read each weight once where an expert has no more rows; tiles of 64
// are three or four to a CU and keep more bytes under way.
hipError_t launch_grouped_matmul(const GroupedArgs& g, hipStream_t stream) {
  const NtArgs a = product_args(g, g.x, g.w);
  const hipError_t err = g.R < 96 * g.E ? launch_tile<NtBf16, kNtGroups, 64, 128, 1, 4, 2, 2>(a, stream)
                                        : launch_tile<NtBf16, kNtGroups, 256, 256, 2, 4, 2, 2>(a, stream);
  return err == hipSuccess && g.zero_rest ? launch_zero_rest(g, g.N, stream) : err;
}

hipError_t launch_grouped_input_grad(const GroupedArgs& g, hipStream_t stream) {
  const NtArgs a = product_args(g, g.dy, g.w);
  hipError_t err;
  if (g.R < 16 * g.E) err = launch_tile<NtBf16, kGradRows, 64, 128, 1, 4, 1, 4>(a, stream);
  else if (g.R < 320 * g.E) err = launch_tile<NtBf16, kGradRows, 256, 256, 2, 4, 1, 4>(a, stream);
  else err = launch_tile<NtBf16, kGradRows, 256, 256, 2, 4, 2, 2>(a, stream);
  return err == hipSuccess && g.zero_rest ? launch_zero_rest(g, g.K, stream) : err;
}

hipError_t launch_grouped_weight_grad(const GroupedArgs& g, hipStream_t stream) {
  return launch_tile<NtBf16, kGradWeights, 128, 256, 1, 4, 1, 3>(product_args(g, g.dy, g.x), stream);
}

}  // namespace moe
