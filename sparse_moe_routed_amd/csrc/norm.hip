// The norms around a block, fused with the block's gate, the residual scale
// and the residual add:
//   n  = y / sqrt(mean(y^2) + eps) * w_post   (or n = y without the post-norm)
//   x' = bf16(x + scale * gate * n)
//   out = bf16(x' / sqrt(mean(x'^2) + eps) * w_pre)
// Everything between the loads and the two roundings is fp32; the pre-norm
// takes the rounded x', as the next reader of x does.
//
// HBM bound: 2 B (x) + 4 or 2 B (y) read and 2 + 2 B written per value.  A row
// belongs to W waves and stays in their registers from the first load to the
// last store, so both means cost no second pass over memory.  4096 rows of 2688
// with fp32 y move 110 MB in 22 us, 5.0 TB/s (a large copy: 4.9 to 5.0 TB/s).
#include "moe_common.h"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kNormThreads = 256;

// 8 values from p, which need not be aligned beyond its elements (rows of odd
// width); global loads of this target take any dword pieces
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  f32x4 a, b;
  __builtin_memcpy(&a, p, 16);
  __builtin_memcpy(&b, p + 4, 16);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = a[i];
    v[4 + i] = b[i];
  }
}

__device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
  u32x4 a;
  __builtin_memcpy(&a, p, 16);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(a[i] << 16);
    v[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_to_f32(*p); }

// chunk at p: 8 values, or the first n of them and zeros
template <class Tp>
__device__ __forceinline__ void load_chunk(const Tp* p, int n, float (&v)[8]) {
  if (n >= 8) {
    load8(p, v);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < n ? load1(p + i) : 0.f;
  }
}

__device__ __forceinline__ void store_chunk(uint16_t* p, int n, const uint16_t (&b)[8]) {
  if (n >= 8) {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = b[2 * i] | (static_cast<uint32_t>(b[2 * i + 1]) << 16);
    // streamed: the next reader is another kernel, mostly on another XCD's L2
    // (4096 x 2688, graph replay: 26.7 us, through the caches 30.8; loads gain
    // nothing by it)
    typedef u32x4 Out __attribute__((aligned(2)));
    __builtin_nontemporal_store(o, reinterpret_cast<Out*>(p));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = b[i];
  }
}

// sum over the W waves of a row, in every lane (fixed order)
template <int W>
__device__ __forceinline__ float row_sum(float v, float* part) {
  v = wave_sum(v);
  if constexpr (W > 1) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) v += part[w];
  }
  return v;
}

// W waves per row, C chunks of 8 values per lane; a workgroup takes one row, or
// with W = 1 four.
template <int W, int C, class Y>
__global__ __launch_bounds__(W > 1 ? W * kWave : kNormThreads) void residual_norm_kernel(
    int T, int H, const uint16_t* x, const Y* y, const float* gate, int gate_kind,
    const float* __restrict__ post_w, const float* __restrict__ pre_w, float scale, float eps,
    int post_norm, uint16_t* x_out, uint16_t* out) {
  __shared__ float part[2][W > 1 ? W : 1];
  constexpr int kRows = W > 1 ? 1 : kNormThreads / kWave;
  const int t = blockIdx.x * kRows + threadIdx.x / (W * kWave);
  if (t >= T) return;  // whole rows; with W > 1 the whole workgroup
  const int lane = threadIdx.x % (W * kWave);
  const size_t row = static_cast<size_t>(t) * H;
  const int chunks = (H + 7) / 8;
  const float* const gp = gate_kind == kGateChannel ? gate : (gate_kind == kGateElement ? gate + row : nullptr);
  const float* const post = post_norm ? post_w : nullptr;
  const auto load = [&](auto p, float (&v)[C][8]) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int c = lane + j * W * kWave;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = 0.f;
      if (c < chunks) load_chunk(p + 8 * c, H - 8 * c, v[j]);
    }
  };
  // chunk c times its factors from p
  const auto times = [&](float (&v)[8], const float* p, int c) __attribute__((always_inline)) {
    if (!p) return;
    float w[8];
    load_chunk(p + 8 * c, H - 8 * c, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= w[i];
  };

  float xv[C][8];
  load(x + row, xv);
  if (y) {
    float yv[C][8];
    float ss = 0.f;
    load(y + row, yv);
    float f = scale;
    if (gate_kind == kGateToken) f *= gate[t];
    if (post_norm) {
#pragma unroll
      for (int j = 0; j < C; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += yv[j][i] * yv[j][i];
      f *= 1.0f / sqrtf(row_sum<W>(ss, part[0]) / static_cast<float>(H) + eps);
    }
#pragma unroll
    for (int j = 0; j < C; ++j) {
      const int c = lane + j * W * kWave;
      if (c >= chunks) continue;
      const int n = H - 8 * c;
      float m[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) m[i] = f * yv[j][i];
      times(m, post, c);
      times(m, gp, c);
      uint16_t b[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        b[i] = f32_to_bf16(xv[j][i] + m[i]);
        xv[j][i] = i < n ? bf16_to_f32(b[i]) : 0.f;
      }
      store_chunk(x_out + row + 8 * c, n, b);
    }
  }
  if (!out) return;
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < C; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += xv[j][i] * xv[j][i];
  const float r = 1.0f / sqrtf(row_sum<W>(ss, part[1]) / static_cast<float>(H) + eps);
#pragma unroll
  for (int j = 0; j < C; ++j) {
    const int c = lane + j * W * kWave;
    if (c >= chunks) continue;
    const int n = H - 8 * c;
    float m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = r * xv[j][i];
    times(m, pre_w, c);
    uint16_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = f32_to_bf16(m[i]);
    store_chunk(out + row + 8 * c, n, b);
  }
}

template <int W, int C, class Y>
hipError_t launch_rows(const ResidualNormArgs& a, hipStream_t stream) {
  constexpr int kThreads = W > 1 ? W * kWave : kNormThreads;
  constexpr int kRows = kThreads / (W * kWave);
  hipLaunchKernelGGL((residual_norm_kernel<W, C, Y>), dim3((a.T + kRows - 1) / kRows), dim3(kThreads),
                     0, stream, a.T, a.H, a.x, static_cast<const Y*>(a.y), a.gate, a.gate_kind,
                     a.post_w, a.pre_w, a.scale, a.eps, a.post_norm, a.x_out, a.out);
  return hipGetLastError();
}

// Few rows are latency: as many lanes as a row has chunks, so that each lane
// waits for one load of a kind (H = 2688, T = 1 4.2 us, 3 waves of 2 chunks 5.3,
// one wave of 6 8.6; T = 333 7.4, 9.1, 14.4).  Many rows are bandwidth: fewer
// waves to a row and more rows in a CU (T = 2048 13.7 us, 6 waves 17.2; T = 4096
// 26.7 us by graph replay, 4.2 of them launch, 6 waves 30.3, one wave 39.2).  Wider rows alike:
// H = 8192, T = 64 6.3 us with 16 waves (8 waves 6.9, 4 9.6), T = 4096 74 us with
// 8 (16 waves 80.5, 4 76); H = 12288, T = 4096 106 us (6 chunks 129).
constexpr int kFewRows = 1536;
template <class Y>
hipError_t launch_type(const ResidualNormArgs& a, hipStream_t stream) {
  const bool few = a.T <= kFewRows;
  if (a.H <= 512) return launch_rows<1, 1, Y>(a, stream);
  if (a.H <= 6 * 512) return few ? launch_rows<6, 1, Y>(a, stream) : launch_rows<3, 2, Y>(a, stream);
  if (a.H <= 16 * 512) return few ? launch_rows<16, 1, Y>(a, stream) : launch_rows<8, 2, Y>(a, stream);
  if (a.H <= 32 * 512) return launch_rows<16, 2, Y>(a, stream);
  return launch_rows<16, 6, Y>(a, stream);
}

}  // namespace

int residual_norm_max_width() { return 16 * 6 * 512; }

hipError_t launch_residual_norm(const ResidualNormArgs& a, hipStream_t stream) {
  if (a.T <= 0) return hipSuccess;
  return a.y_bf16 ? launch_type<uint16_t>(a, stream) : launch_type<float>(a, stream);
}

}  // namespace moe
