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
// last store, so both means cost no second pass over memory.
#include "moe_common.h"
#include "moe_internal.h"

namespace moe {

namespace {

constexpr int kNormChunks = 6;  // 8-value chunks per lane
constexpr int kNormThreads = 256;
constexpr int kNormWave = kNormChunks * 8 * kWave;  // values one wave holds

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
    __builtin_memcpy(p, &o, 16);
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

// W waves per row; a workgroup of kNormThreads takes kNormThreads / (64 W)
// rows (one row of 16 waves for the widest).
template <int W, class Y>
__global__ __launch_bounds__(W > 4 ? W * kWave : kNormThreads) void residual_norm_kernel(
    int T, int H, const uint16_t* x, const Y* y, const float* gate, int gate_kind,
    const float* __restrict__ post_w, const float* __restrict__ pre_w, float scale, float eps,
    int post_norm, uint16_t* x_out, uint16_t* out) {
  __shared__ float part[2][W > 1 ? W : 1];
  constexpr int kRows = W > 4 ? 1 : kNormThreads / (W * kWave);
  static_assert(W == 1 || kRows == 1, "the waves of a row meet at workgroup barriers");
  const int t = blockIdx.x * kRows + threadIdx.x / (W * kWave);
  if (t >= T) return;  // whole rows; with W > 1 the whole workgroup
  const int lane = threadIdx.x % (W * kWave);
  const size_t row = static_cast<size_t>(t) * H;
  const int chunks = (H + 7) / 8;

  float xv[kNormChunks][8];
#pragma unroll
  for (int j = 0; j < kNormChunks; ++j) {
    const int c = lane + j * W * kWave;
#pragma unroll
    for (int i = 0; i < 8; ++i) xv[j][i] = 0.f;
    if (c < chunks) load_chunk(x + row + 8 * c, H - 8 * c, xv[j]);
  }
  if (y) {
    float yv[kNormChunks][8];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < kNormChunks; ++j) {
      const int c = lane + j * W * kWave;
#pragma unroll
      for (int i = 0; i < 8; ++i) yv[j][i] = 0.f;
      if (c < chunks) load_chunk(y + row + 8 * c, H - 8 * c, yv[j]);
    }
    float f = scale;
    if (post_norm) {
#pragma unroll
      for (int j = 0; j < kNormChunks; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss += yv[j][i] * yv[j][i];
      f *= 1.0f / sqrtf(row_sum<W>(ss, part[0]) / static_cast<float>(H) + eps);
    }
    if (gate_kind == kGateToken) f *= gate[t];
    const float* gp = gate_kind == kGateChannel ? gate : (gate_kind == kGateElement ? gate + row : nullptr);
#pragma unroll
    for (int j = 0; j < kNormChunks; ++j) {
      const int c = lane + j * W * kWave;
      if (c >= chunks) continue;
      const int n = H - 8 * c;
      float m[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) m[i] = f * yv[j][i];
      if (post_norm && post_w) {
        float w[8];
        load_chunk(post_w + 8 * c, n, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i] *= w[i];
      }
      if (gp) {
        float g[8];
        load_chunk(gp + 8 * c, n, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i] *= g[i];
      }
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
  for (int j = 0; j < kNormChunks; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += xv[j][i] * xv[j][i];
  const float r = 1.0f / sqrtf(row_sum<W>(ss, part[1]) / static_cast<float>(H) + eps);
#pragma unroll
  for (int j = 0; j < kNormChunks; ++j) {
    const int c = lane + j * W * kWave;
    if (c >= chunks) continue;
    const int n = H - 8 * c;
    float m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = r * xv[j][i];
    if (pre_w) {
      float w[8];
      load_chunk(pre_w + 8 * c, n, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) m[i] *= w[i];
    }
    uint16_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = f32_to_bf16(m[i]);
    store_chunk(out + row + 8 * c, n, b);
  }
}

template <int W, class Y>
hipError_t launch_rows(const ResidualNormArgs& a, hipStream_t stream) {
  constexpr int kThreads = W > 4 ? W * kWave : kNormThreads;
  constexpr int kRows = kThreads / (W * kWave);
  hipLaunchKernelGGL((residual_norm_kernel<W, Y>), dim3((a.T + kRows - 1) / kRows), dim3(kThreads),
                     0, stream, a.T, a.H, a.x, static_cast<const Y*>(a.y), a.gate, a.gate_kind,
                     a.post_w, a.pre_w, a.scale, a.eps, a.post_norm, a.x_out, a.out);
  return hipGetLastError();
}

template <class Y>
hipError_t launch_type(const ResidualNormArgs& a, hipStream_t stream) {
  if (a.H <= kNormWave) return launch_rows<1, Y>(a, stream);
  if (a.H <= 4 * kNormWave) return launch_rows<4, Y>(a, stream);
  return launch_rows<16, Y>(a, stream);
}

}  // namespace

int residual_norm_max_width() { return 16 * kNormWave; }

hipError_t launch_residual_norm(const ResidualNormArgs& a, hipStream_t stream) {
  if (a.T <= 0) return hipSuccess;
  return a.y_bf16 ? launch_type<uint16_t>(a, stream) : launch_type<float>(a, stream);
}

}  // namespace moe
