// The whole layer for a few tokens (T <= 16) in two kernels:
//   l = x W_r^T + b;  ids, gates = top-k and softmax of l
//   a_{t,j} = bf16(relu(W_up,e x~_t)^2),  e = ids[t, j]
//   y_t = sum_e g_{t,e} W_down,e a~_{t,e}
// with x~, a~ quantised per tensor as moe_forward does (FP8, NVFP4).
//
// Such a batch reads every selected expert's weights once (20 / 10 / 5.6 MB
// per expert at the full width) and computes next to nothing, so the bound is
// HBM, and below it the latency of the chain router -> selection -> up ->
// (tensor scale of a) -> down, which as separate launches costs more than the
// weights of one token.  Full layer, T = 1 and T = 4: BF16 36 and 81 us, FP8 28
// and 53, NVFP4 28 and 48 (as separate launches 54 and 81, 46 and 64, 42 and 53);
// from 4 tokens on BF16 has enough weights to read that the launches hardly count.
// Of NVFP4's 28 us the router's kernel takes 5, the start of 256 workgroups 3, the
// selection 4, the up projection 7, the wait for it 2, fetching a 2 and the down
// projection 2.5; with more tokens the products stream at 5 to 5.7 TB/s.
//
// few_router_kernel writes partial logits.  few_layer_kernel does the rest: its
// workgroups each redo the selection (a few KB of partial logits), then take
// work items from a ticket counter: first the up projection's rounds, then the
// down projection's column tiles.  A down item waits until every up round is
// done.  The wait ends: tickets are handed out in order, so all up rounds
// belong to workgroups that are running, and none of those waits before its
// round is done, however few workgroups the GPU runs at a time.  It is bounded
// all the same: if another call writes to the workspace meanwhile, which the header
// forbids, done words are lost, and the columns that waited for them become NaN.
//
// Weights go from HBM straight into registers in MFMA operand order.  The
// matrix instruction takes 16 weight rows x 16 tokens: with at most 16 tokens
// each weight is loaded once whatever the routing, and the columns of tokens
// that the expert does not serve are computed and dropped, which costs
// nothing at this ratio of bytes to products.
#include "moe_common.h"
#include "moe_internal.h"
#include "topk.h"

namespace moe {

namespace {

constexpr int kWaves = 16;
constexpr int kThreads = kWaves * kWave;
constexpr int kTok = kFewTokens;        // MFMA columns
constexpr int kMaxRows = kTok * 8;      // (token, slot) pairs
constexpr int kRouterThreads = 256;
constexpr int kMaxPolls = 1 << 22;      // some seconds; an up projection takes milliseconds at most

__device__ __forceinline__ bf16x8 fp8_frag(uint32_t w0, uint32_t w1) {
  const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, false);
  const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, true);
  const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, false);
  const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, true);
  return bf16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// ---- activation quantisers, 8 values of one lane (the recipes of quant.hip)
template <int FMT>
struct TensorScale {
  float s = 1.f;  // value = stored * s
  float a = 0.f;  // FP8: 448 / amax (0 where infinite); NVFP4: 6 s
  __device__ explicit TensorScale(float amax) {
    if constexpr (FMT == kFP8) {
      s = amax > 0.f ? __fdiv_rn(amax, 448.f) : 0.f;
      a = quotient_or_zero(448.f, amax);
    } else if constexpr (FMT == kNVFP4) {
      s = amax > 0.f ? __fdiv_rn(amax, 2688.f) : 0.f;
      a = 6.f * s;
    }
  }
};

__device__ __forceinline__ float amax8(u32x4 v) {
  float m = 0.f;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    m = fmaxf(m, fabsf(__uint_as_float(v[w] << 16)));
    m = fmaxf(m, fabsf(__uint_as_float(v[w] & 0xffff0000u)));
  }
  return m;
}

// 8 bf16 values as the GEMM operand: dec(code) in bf16 (FP8), dec(code) *
// dec(block scale) in fp16 (NVFP4; the other half of the 16-value block is on
// the neighbouring lane, which must be active).  The values are those of the
// encoders of moe_common.h; a code's sign may be that of -0, whose products
// add nothing.
// POSITIVE: values of 0 or more, so that v * ts.a is at most 448 and nothing is
// left to clamp (FP8).
template <int FMT, bool POSITIVE = false>
__device__ __forceinline__ u32x4 quantise8(u32x4 v, const TensorScale<FMT>& ts) {
  if constexpr (FMT == kBF16) {
    return v;
  } else {
    float f[8];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      f[2 * w] = __uint_as_float(v[w] << 16);
      f[2 * w + 1] = __uint_as_float(v[w] & 0xffff0000u);
    }
    if constexpr (FMT == kFP8 && POSITIVE) {
      uint32_t c[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h] * ts.a, f[4 * h + 1] * ts.a, 0, false);
        c[h] = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h + 2] * ts.a, f[4 * h + 3] * ts.a, lo, true);
      }
      return __builtin_bit_cast(u32x4, fp8_frag(c[0], c[1]));
    } else if constexpr (FMT == kFP8) {
      const uint32_t c0 = e4m3_encode4(f[0] * ts.a, f[1] * ts.a, f[2] * ts.a, f[3] * ts.a);
      const uint32_t c1 = e4m3_encode4(f[4] * ts.a, f[5] * ts.a, f[6] * ts.a, f[7] * ts.a);
      return __builtin_bit_cast(u32x4, fp8_frag(c0, c1));
    } else {
      float m = fabsf(f[0]);
#pragma unroll
      for (int j = 1; j < 8; ++j) m = fmaxf(m, fabsf(f[j]));
      // quad_perm [1, 0, 3, 2]: the value of the neighbouring lane
      const float mo = __builtin_bit_cast(
          float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, m), 0xb1, 0xf, 0xf, false));
      const uint32_t sb = ts.s > 0.f ? e4m3_encode(__fdiv_rn(fmaxf(m, mo), ts.a)) : 0u;
      const f16x2 s2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sb | (sb << 8), 1.0f, false);
      const float sbf = static_cast<float>(s2[0]);
      const float r = quotient_or_zero(1.f, sbf * ts.s);
      // |f r| is below 6 (1 + 2^-4) for a normal block scale and below 9 for a
      // subnormal one, which may be two thirds of what it rounds: the hardware
      // conversion saturates it to 6
      uint32_t q = 0u;
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[0] * r, f[1] * r, 1.0f, 0);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[2] * r, f[3] * r, 1.0f, 1);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[4] * r, f[5] * r, 1.0f, 2);
      q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, f[6] * r, f[7] * r, 1.0f, 3);
      const f16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, 1.0f, 0) * s2;
      const f16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, 1.0f, 1) * s2;
      const f16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, 1.0f, 2) * s2;
      const f16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, 1.0f, 3) * s2;
      return u32x4{__builtin_bit_cast(uint32_t, p0), __builtin_bit_cast(uint32_t, p1),
                   __builtin_bit_cast(uint32_t, p2), __builtin_bit_cast(uint32_t, p3)};
    }
  }
}

// ---- first kernel.  Workgroups [0, E / 16 * kFewSlices) write partial logits:
// 16 experts over one K slice each, its K steps dealt to the 4 waves in
// contiguous ranges, the waves' sums added in wave order.  The others (FP8,
// NVFP4) quantise a part of the tokens each, the tensor's amax taken by every
// one of them; BF16 copies them where y overlaps x, since the second kernel's
// first workgroups write y while its last ones may not have read their tokens.
// Workgroup 0 clears the counters of the second kernel.
constexpr int kQuantGroups = 16;

template <int FMT>
__global__ __launch_bounds__(kRouterThreads) void few_router_kernel(FewArgs g) {
  constexpr int U = 6;  // K steps of loads in flight
  __shared__ f32x4 red[4][kWave];
  const int T = g.T, H = g.H, E = g.E;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n_router = E / 16 * kFewSlices;
  if (blockIdx.x == 0)
    for (int j = threadIdx.x; j < kFewCounters; j += kRouterThreads) g.ctr[j] = 0u;
  if (static_cast<int>(blockIdx.x) >= n_router) {
    const u32x4* x = reinterpret_cast<const u32x4*>(g.x);
    const int n8 = T * H / 8;
    float amax = 0.f;
    if constexpr (FMT != kBF16) {
      float* part = reinterpret_cast<float*>(red);
#pragma unroll 8
      for (int i = threadIdx.x; i < n8; i += kRouterThreads) amax = fmaxf(amax, amax8(x[i]));
      amax = wave_max(amax);
      if (lane == 0) part[wave] = amax;
      __syncthreads();
      amax = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
    }
    const TensorScale<FMT> ts(amax);
    const int b = static_cast<int>(blockIdx.x) - n_router;
    if (b == 0 && threadIdx.x == 0) *g.x_scale = ts.s;
    // pairs of chunks (a block's halves) stay together: the stride is even
    for (int i = b * kRouterThreads + threadIdx.x; i < n8; i += kQuantGroups * kRouterThreads)
      reinterpret_cast<u32x4*>(g.x_q)[i] = quantise8<FMT>(x[i], ts);
    return;
  }
  const int eb = blockIdx.x / kFewSlices, s = blockIdx.x % kFewSlices;
  const int row = lane & 15;
  const int kq = (lane >> 4) * 8;
  const int steps = H / 32;
  const int i = s * 4 + wave;
  const int k0 = steps * i / (4 * kFewSlices), k1 = steps * (i + 1) / (4 * kFewSlices);
  const size_t n = static_cast<size_t>(E) * H;
  const uint16_t* xr = g.x + static_cast<size_t>(min(row, T - 1)) * H + kq;
  const uint16_t* hi = g.w_router + static_cast<size_t>(eb * 16 + row) * H + kq;
  const uint16_t* mid = hi + n;
  const uint16_t* lo = mid + n;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int kb = k0; kb < k1; kb += U) {
    bf16x8 a[U], bh[U], bm[U], bl[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (kb + u < k1) {
        const int kk = (kb + u) * 32;
        a[u] = *reinterpret_cast<const bf16x8*>(xr + kk);
        bh[u] = *reinterpret_cast<const bf16x8*>(hi + kk);
        bm[u] = *reinterpret_cast<const bf16x8*>(mid + kk);
        bl[u] = *reinterpret_cast<const bf16x8*>(lo + kk);
      }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kb + u >= k1) break;
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[u], bl[u], acc, 0, 0, 0);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[u], bm[u], acc, 0, 0, 0);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[u], bh[u], acc, 0, 0, 0);
    }
  }
  red[wave][lane] = acc;
  __syncthreads();
  if (wave == 0) {
    f32x4 v = red[0][lane];
#pragma unroll
    for (int w = 1; w < 4; ++w) v += red[w][lane];
    // lane holds column (expert) lane % 16, rows (tokens) 4 (lane / 16) + r
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = (lane >> 4) * 4 + r;
      if (t < T) g.part[(static_cast<size_t>(s) * T + t) * E + eb * 16 + row] = v[r];
    }
  }
}

// ---- weight units.  A unit is what a wave takes of 16 weight rows at a time:
//   BF16, FP8  one 128-byte line of each row (64 / 128 K values): two 16-byte
//              loads a lane, 8 lanes to a row, so that every load instruction
//              reads whole lines; the wave turns them into MFMA operand order
//              through 2 KB of LDS of its own.  (Loading in operand order
//              puts 16 rows on neighbouring lanes: every 16 lanes touch 16
//              lines, and four tokens BF16 ran at 2.5 TB/s that way.)
//   NVFP4      two 64-value steps of the panel layout (128 K values), which is
//              operand order as it stands: one 16-byte load of codes and one
//              2-byte load of block scales a lane
// Loads go through a buffer descriptor of one expert's matrix, so a unit past
// the end, or the part of a last unit past K, reads nothing and is zero.
template <int FMT>
struct Unit {
  u32x4 v[FMT == kNVFP4 ? 1 : 2];
  uint32_t sb;
};
template <int FMT>
constexpr int kUnitK = FMT == kBF16 ? 64 : 128;

template <int FMT>
__host__ __device__ constexpr int units_of(int K) {
  return (K + kUnitK<FMT> - 1) / kUnitK<FMT>;
}

constexpr uint32_t kPastEnd = 0xffffff00u;  // beyond every matrix: reads as zero
constexpr int kRawBuffer = 0x00027000;      // descriptor word 3: raw 32-bit data
constexpr int kStreamOnce = 2;              // cache policy: non-temporal

// One expert's matrix for the 16 rows of a tile: descriptors, and this lane's
// byte offsets in unit 0 (a unit further on adds a scalar).  DOWN selects the
// FP8 code layout: row-major (up) or panels (down).
template <int FMT, bool DOWN>
struct Tile {
  const uint8_t *codes, *scales;
  uint32_t bytes;          // of the codes; a block scale for every 8 of them (NVFP4)
  uint32_t at, at_last;    // codes; of the last unit (past K: kPastEnd)
  uint32_t step, row8;     // from unit to unit, from rows 0..7 to 8..15
  uint32_t row8_last;
  uint32_t sat, sat_last;  // scales
  int last;                // index of the last unit

  // e: expert (matrix index), n0: first row, uniform over the wave
  __device__ __forceinline__ void point(const void* w, const uint8_t* bs, int e, int n0, int N, int K) {
    const int lane = threadIdx.x & 63;
    const size_t n = static_cast<size_t>(N) * K;
    const size_t size = FMT == kBF16 ? 2 * n : (FMT == kFP8 ? n : n / 2);
    bytes = static_cast<uint32_t>(size);
    codes = static_cast<const uint8_t*>(w) + size * e;
    last = units_of<FMT>(K) - 1;
    if constexpr (FMT == kNVFP4) {
      scales = bs + n / 16 * e;
      const int q = lane >> 4, p = n0 / kNvPanel, rows = nv_panel_rows(N, p);
      const uint32_t pr = n0 + (lane & 15) - p * kNvPanel;
      at = static_cast<uint32_t>(p) * kNvPanel * (K / 2) + (q >> 1) * rows * 32 + pr * 32 + (q & 1) * 16;
      sat = static_cast<uint32_t>(p) * kNvPanel * (K / 16) + (q >> 1) * rows * 4 + pr * 4 + (q & 1) * 2;
      step = 2 * rows * 32;
      const bool in = (2 * last + (q >> 1)) * kNvStepK < K;
      at_last = in ? at : kPastEnd;
      sat_last = in ? sat : kPastEnd;
    } else {
      const int row = lane >> 3, ch = lane & 7;
      const uint32_t width = FMT == kBF16 ? 2 * K : K;  // row bytes
      const bool in = last * 128 + ch * 16 < static_cast<int>(width);
      if constexpr (FMT == kFP8 && DOWN) {
        const int p = n0 / kNvPanel, rows = nv_panel_rows(N, p), pr = n0 + row - p * kNvPanel;
        const int sb = min(kFp8StepK, K - last * kFp8StepK);  // row bytes of the last step
        const uint32_t base = static_cast<uint32_t>(p) * kNvPanel * K + ch * 16;
        at = base + pr * kFp8StepK;
        at_last = in ? base + pr * sb : kPastEnd;
        step = rows * kFp8StepK;
        row8 = 8 * kFp8StepK;
        row8_last = in ? 8 * sb : 0;
      } else {
        at = static_cast<uint32_t>(n0 + row) * width + ch * 16;
        at_last = in ? at : kPastEnd;
        step = 128;
        row8 = 8 * width;
        row8_last = in ? row8 : 0;
      }
    }
  }

  // loads of unit u; none (zeros) unless `in`.  The scheduling fence keeps the
  // loads of a stream in order, so that a wait for the oldest unit waits for no
  // later one.
  __device__ __forceinline__ Unit<FMT> load(int u, bool in) const {
    const __amdgpu_buffer_rsrc_t rc = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(codes), 0, in ? static_cast<int>(bytes) : 0, kRawBuffer);
    Unit<FMT> r{};
    const bool tail = u == last;
    // past the end by the lane's own offset (no records, scalar offset 0, or
    // kPastEnd), whether or not the range check counts the scalar offset
    const uint32_t so = in ? u * step : 0u;
    if constexpr (FMT == kNVFP4) {
      const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<uint8_t*>(scales), 0, in ? static_cast<int>(bytes / 8) : 0, kRawBuffer);
      r.sb = __builtin_amdgcn_raw_buffer_load_b16(rs, tail ? sat_last : sat, so / 8, kStreamOnce);
      r.v[0] = __builtin_amdgcn_raw_buffer_load_b128(rc, tail ? at_last : at, so, kStreamOnce);
    } else {
      const uint32_t o = tail ? at_last : at;
      r.v[0] = __builtin_amdgcn_raw_buffer_load_b128(rc, o, so, kStreamOnce);
      r.v[1] = __builtin_amdgcn_raw_buffer_load_b128(rc, o + (tail ? row8_last : row8), so, kStreamOnce);
    }
    __builtin_amdgcn_sched_barrier(0);
    return r;
  }
};

// acc += 16 weight rows of a unit times the tokens' values: lane l has weight
// row and token column l % 16 and, of each MFMA, the K values of one 16-byte
// chunk of the tokens.  x points at the unit's first chunk of this lane's
// column, chunks lie dx bytes apart.  `turn` is the wave's 2 KB of LDS: chunk c
// of a row lies at c ^ (row % 8), free of bank conflicts both ways.
template <int FMT>
__device__ __forceinline__ f32x4 mul_unit(const Unit<FMT>& w, const uint8_t* x, int dx,
                                          uint8_t* turn, f32x4 acc) {
  const int lane = threadIdx.x & 63, q = lane >> 4;
  if constexpr (FMT == kNVFP4) {
    // E2M1 codes times the block scale as fp16 (exact, at most 6 significant
    // bits)
    const f16x2 sc = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w.sb, 1.0f, false);
    x += q * 4 * dx;
    f16x8 b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = *reinterpret_cast<const f16x8*>(x + i * dx);
    f32x4 odd = {0.f, 0.f, 0.f, 0.f};  // two chains of products
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f16x2 s2 = {sc[i >> 1], sc[i >> 1]};
      const f16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w.v[0][i], 1.0f, 0) * s2;
      const f16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w.v[0][i], 1.0f, 1) * s2;
      const f16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w.v[0][i], 1.0f, 2) * s2;
      const f16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w.v[0][i], 1.0f, 3) * s2;
      const f16x8 a = {p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
      if (i & 1) odd = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b[i], odd, 0, 0, 0);
      else acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b[i], acc, 0, 0, 0);
    }
    acc += odd;
  } else {
    const int row = lane >> 3, r = lane & 15;
    u32x4* const put = reinterpret_cast<u32x4*>(turn + row * 128 + (((lane & 7) ^ row) << 4));
    wave_lds_order();  // the unit before this one has been read
    put[0] = w.v[0];
    put[64] = w.v[1];  // 8 rows on, the same row % 8
    wave_lds_order();
    const auto get = [&](int c) {
      return *reinterpret_cast<const u32x4*>(turn + r * 128 + ((c ^ (r & 7)) << 4));
    };
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (FMT == kBF16) {
        const bf16x8 b = *reinterpret_cast<const bf16x8*>(x + (i * 4 + q) * dx);
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, get(i * 4 + q)), b,
                                                      acc, 0, 0, 0);
      } else {
        // E4M3 codes as bf16 (exact), so the products are exact in fp32
        const u32x4 v = get(i * 4 + q);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bf16x8 b = *reinterpret_cast<const bf16x8*>(x + ((i * 4 + q) * 2 + h) * dx);
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp8_frag(v[2 * h], v[2 * h + 1]), b, acc, 0,
                                                        0, 0);
        }
      }
    }
  }
  return acc;
}

// n units through a ring of P in flight: load(i) starts the i-th (nothing past
// n), use(unit, i) consumes it.  prime() may run ahead of what use() needs.
template <int FMT, int P>
struct Stream {
  Unit<FMT> ring[P];
  template <class Load>
  __device__ __forceinline__ void prime(Load load) {
#pragma unroll
    for (int j = 0; j < P; ++j) ring[j] = load(j);
  }
  template <class Load, class Use>
  __device__ __forceinline__ void run(int n, Load load, Use use) {
    for (int i = 0; i < n; i += P) {
#pragma unroll
      for (int j = 0; j < P; ++j) {
        if (i + j < n) use(ring[j], i + j);
        ring[j] = load(i + j + P);
      }
    }
  }
};

// routing of the batch, the same in every workgroup
struct Routing {
  uint32_t mask[kMaxE];          // tokens of each expert, a bit each
  uint32_t used[kMaxE / 32];     // experts with tokens, a bit each
  __attribute__((aligned(16))) uint32_t key[kMaxRows / 2];  // 16 bits a row, ~0: none
  uint8_t slot[kMaxE][kTok];     // slot of a token at an expert it selected
  float gate[kTok][8];
  int16_t id[kTok][8];           // -1: none
  uint8_t expert[kMaxRows];      // distinct experts, ascending
  uint16_t off[kMaxRows + 1];    // first row of each: rows go by expert, then token
  uint8_t src[kMaxRows];         // (token * 8 + slot) of each row
  int n_experts;
};

struct Shared {
  Routing rt;
  // of each wave: its part of a sum, and where its weights are turned around
  __attribute__((aligned(16))) uint8_t turn[kWaves][2048];
  float wave_part[kWaves];
  int next;
};

__device__ __forceinline__ void clear_routing(Shared& sm) {
  for (int e = threadIdx.x; e < kMaxE; e += kThreads) sm.rt.mask[e] = 0u;
  if (threadIdx.x < kMaxE / 32) sm.rt.used[threadIdx.x] = 0u;
  if (threadIdx.x < kMaxRows / 2) sm.rt.key[threadIdx.x] = 0xffffffffu;
}

// top-k and gates of the tokens wave, wave + kWaves, ... of up to 64 N experts
template <int N>
__device__ __forceinline__ void select_experts(const FewArgs& g, Shared& sm) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  Routing& rt = sm.rt;
  for (int t = wave; t < g.T; t += kWaves) {
    float v[N];
    uint32_t key[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int e = lane + 64 * i;
      v[i] = -INFINITY;
      key[i] = 0u;
      if (e < g.E) {
        float l = 0.f;
#pragma unroll
        for (int s = 0; s < kFewSlices; ++s) l += g.part[(static_cast<size_t>(s) * g.T + t) * g.E + e];
        v[i] = l + (g.bias ? g.bias[e] : 0.f);
        key[i] = float_key(v[i]);
      }
    }
    float sel_v[8];
    int sel_i[8];
    wave_topk(v, key, g.k, sel_v, sel_i);
    float z[8], sum = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      z[j] = j < g.k ? expf(sel_v[j] - sel_v[0]) : 0.f;
      sum += z[j];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (lane != j || j >= g.k) continue;
      const int e = sel_i[j];
      rt.id[t][j] = static_cast<int16_t>(e);
      rt.gate[t][j] = z[j] / sum;
      if (e >= 0) {
        rt.slot[e][t] = static_cast<uint8_t>(j);
        atomicOr(&rt.mask[e], 1u << t);
        atomicOr(&rt.used[e >> 5], 1u << (e & 31));
        reinterpret_cast<uint16_t*>(rt.key)[t * g.k + j] = static_cast<uint16_t>(e * kTok + t);
      }
    }
  }
}

// The rows by expert, then token: a row's place is the number of smaller keys
// (expert * 16 + token), its expert's place the number of smaller experts used.
__device__ __forceinline__ void list_rows(const FewArgs& g, Shared& sm) {
  Routing& rt = sm.rt;
  const int n = g.T * g.k, p = threadIdx.x;
  if (p < n) {
    const uint32_t mine = reinterpret_cast<const uint16_t*>(rt.key)[p];
    if (mine != 0xffffu) {
      int at = 0;
      for (int i = 0; i < (n + 7) / 8; ++i) {
        const u32x4 v = reinterpret_cast<const u32x4*>(rt.key)[i];
#pragma unroll
        for (int w = 0; w < 4; ++w) at += ((v[w] & 0xffffu) < mine) + ((v[w] >> 16) < mine);
      }
      const int e = static_cast<int>(mine) / kTok, t = static_cast<int>(mine) % kTok;
      rt.src[at] = static_cast<uint8_t>(t * 8 + rt.slot[e][t]);
      if (!(rt.mask[e] & ((1u << t) - 1u))) {  // the expert's first row
        int d = __popc(rt.used[e >> 5] & ((1u << (e & 31)) - 1u));
        for (int w = 0; w < (e >> 5); ++w) d += __popc(rt.used[w]);
        rt.expert[d] = static_cast<uint8_t>(e);
        rt.off[d] = static_cast<uint16_t>(at);
      }
    }
  }
  if (p == kThreads - 1) {
    int d = 0, rows = 0;
    for (int w = 0; w < kMaxE / 32; ++w) d += __popc(rt.used[w]);
    for (int i = 0; i < n; ++i) rows += reinterpret_cast<const uint16_t*>(rt.key)[i] != 0xffffu;
    rt.off[d] = static_cast<uint16_t>(rows);
    rt.n_experts = d;
  }
}

// this lane's token column of expert e: whether it is served, and its row
// among the expert's (0 for a column that is dropped)
struct Column {
  bool live;
  int rank;
};
__device__ __forceinline__ Column column_of(const Routing& rt, int e) {
  const int c = threadIdx.x & 15;
  const uint32_t m = rt.mask[e];
  const bool live = (m >> c) & 1u;
  return Column{live, live ? static_cast<int>(__popc(m & ((1u << c) - 1u))) : 0};
}

constexpr int kBatch = 6;  // 16-byte loads a thread starts together when it stages

// stages rows x chunks of 8 values: get(row) is a row's first value, put(row,
// chunk) where its chunk goes, make(v) what goes there.  Thread pairs (2 i,
// 2 i + 1) hold neighbouring chunks (chunks is even).  The threads of the last
// waves go first: the first ones may still be routing.
template <class Get, class Put, class Make>
__device__ __forceinline__ void stage_rows(int rows, int chunks, Get get, Put put, Make make) {
  const int n = rows * chunks;
  const float inv = 1.0f / static_cast<float>(chunks);
  const int me = static_cast<int>(kThreads - 1 - threadIdx.x);
  for (int i0 = me; i0 < n; i0 += kBatch * kThreads) {
    u32x4 v[kBatch];
    int r[kBatch], c[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int i = i0 + j * kThreads;
      if (i >= n) break;
      // i / chunks: i < 2^14 here, so the quotient is off by less than the
      // distance of (i + 1/2) / chunks from a whole number
      r[j] = static_cast<int>((static_cast<float>(i) + 0.5f) * inv);
      c[j] = i - r[j] * chunks;
      v[j] = reinterpret_cast<const u32x4*>(get(r[j]))[c[j]];
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (i0 + j * kThreads >= n) break;  // both threads of a pair, or neither
      *reinterpret_cast<u32x4*>(put(r[j], c[j])) = make(v[j]);
    }
  }
}

// chunks of K values a unit's operand reads: whole units, zeros past K
template <int FMT>
__host__ __device__ constexpr int chunks_of(int K) {
  return units_of<FMT>(K) * kUnitK<FMT> / 8;
}

template <int FMT>
__global__ __launch_bounds__(kThreads) void few_layer_kernel(FewArgs g) {
  // units in flight per wave: 16 waves keep 32 KB to 64 KB of loads under way per
  // CU; 3 and 4 are 1 % slower, 5 and 6 up to 10 % (loads past a stream's end
  // touch no memory but are issued)
  constexpr int P = 2;
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  Shared& sm = *reinterpret_cast<Shared*>(dyn);
  uint8_t* const stage = dyn + (sizeof(Shared) + 15) / 16 * 16;  // tokens, later rows of a
  Routing& rt = sm.rt;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c = lane & 15, q = lane >> 4;
  const int H = g.H, F = g.F, T = g.T;
  uint8_t* const turn = sm.turn[wave];
  const auto part_of = [&](int w) { return reinterpret_cast<f32x4*>(sm.turn[w]) + lane; };

  if (tid == 0) sm.next = static_cast<int>(atomicAdd(&g.ctr[kFewTicket], 1u));
  clear_routing(sm);
  __syncthreads();
  if (g.E <= 128) select_experts<2>(g, sm);
  else select_experts<kMaxE / 64>(g, sm);
  // The tokens as the operand: chunk ch of token t at (ch * T + t) * 16, so the
  // lanes of one MFMA read consecutive addresses.
  const int T16 = T * 16;
  stage_rows(
      T, H / 8, [&](int t) { return g.tokens + static_cast<size_t>(t) * H; },
      [&](int t, int ch) { return stage + ch * T16 + t * 16; }, [](u32x4 v) { return v; });
  for (int i = H / 8 * T16 + tid * 16; i < chunks_of<FMT>(H) * T16; i += kThreads * 16)
    *reinterpret_cast<u32x4*>(stage + i) = u32x4{0u, 0u, 0u, 0u};
  __syncthreads();
  list_rows(g, sm);
  __syncthreads();
  int ticket = __builtin_amdgcn_readfirstlane(sm.next);
  if (ticket == 0)
    for (int i = tid; i < T * g.k; i += kThreads) {
      g.ids[i] = rt.id[i / g.k][i % g.k];
      g.gates[i] = rt.gate[i / g.k][i % g.k];
    }

  const int D = __builtin_amdgcn_readfirstlane(rt.n_experts);
  const int f16 = F / 16;
  const int up_tiles = D * f16;
  const int groups = static_cast<int>(gridDim.x);
  const int up_items = min(up_tiles, groups);  // an item: an even share of the tiles

  // ---- up.  An item's tiles go in rounds of n = 16, 8, 4, 2, 1 of them, a
  // tile's K split over 16 / n waves, so that nearly every wave streams to the
  // end of the item; a round's first loads start before the sums of the round
  // before it are joined.  A last round may hold fewer than n tiles, down to
  // 5/8: idle waves cost less there than one more round.
  const uint8_t* const col = stage + min(c, T - 1) * 16;
  while (static_cast<uint32_t>(ticket) < static_cast<uint32_t>(up_items)) {
    float local = 0.f;
    // (up_tiles * up_items < 2^31: at most 128 experts, 256 items, F < 2^16)
    const int t1 = static_cast<int>(static_cast<uint32_t>(up_tiles * (ticket + 1)) / static_cast<uint32_t>(up_items));
    int t0 = static_cast<int>(static_cast<uint32_t>(up_tiles * ticket) / static_cast<uint32_t>(up_items));
    const int U = units_of<FMT>(H);
    Tile<FMT, false> w;
    int ksl = 0, e = 0, n0 = 0, u0 = 0, n = 0;  // of the round that is streaming
    bool live = false;                          // this wave stores a tile of it
    const auto start = [&]() {
      const int left = t1 - t0;
      ksl = 0;
      while ((kWaves >> ksl) * 5 > left * 8) ++ksl;
      const bool mine = t0 + (wave >> ksl) < t1;
      const int tile = mine ? t0 + (wave >> ksl) : t0, d = tile / f16;
      const int part = wave & ((1 << ksl) - 1);
      n0 = __builtin_amdgcn_readfirstlane(tile - d * f16) * 16;
      e = __builtin_amdgcn_readfirstlane(rt.expert[d]);
      u0 = __builtin_amdgcn_readfirstlane((U * part) >> ksl);
      n = mine ? __builtin_amdgcn_readfirstlane((U * (part + 1)) >> ksl) - u0 : 0;
      live = mine && part == 0;
      w.point(g.up, g.up_bs, e, n0, F, H);
    };
    const auto load = [&](int i) { return w.load(u0 + i, i < n); };
    Stream<FMT, P> st;
    start();
    st.prime(load);
    int seen = 0;
    if (tid == 0)
      seen = static_cast<int>(__hip_atomic_load(&g.ctr[kFewTicket], __ATOMIC_RELAXED,
                                                __HIP_MEMORY_SCOPE_AGENT));
    while (true) {
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
      st.run(n, load, [&](const Unit<FMT>& v, int i) {
        acc = mul_unit<FMT>(v, col + (u0 + i) * (kUnitK<FMT> / 8) * T16, T16, turn, acc);
      });
      const int ks = 1 << ksl, ce = e, cn0 = n0;
      const bool first = live;
      t0 += kWaves >> ksl;
      const bool more = t0 < t1;
      if (more) {
        start();
        st.prime(load);
      }
      if (ks > 1) {
        *part_of(wave) = acc;
        __syncthreads();
        if (first)
          for (int v = 1; v < ks; ++v) acc += *part_of(wave + v);
      }
      if (first && ((rt.mask[ce] >> c) & 1u)) {
        float scale = 1.f;
        if constexpr (FMT != kBF16) scale = *g.x_scale * g.up_s[ce];
        uint16_t b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          b[i] = relu_sq_bf16(FMT == kBF16 ? acc[i] : acc[i] * scale);
          local = fmaxf(local, bf16_to_f32(b[i]));
        }
        const size_t row = static_cast<size_t>(c) * g.k + rt.slot[ce][c];
        const uint32_t lo = b[0] | (static_cast<uint32_t>(b[1]) << 16);
        const uint32_t hi = b[2] | (static_cast<uint32_t>(b[3]) << 16);
        __hip_atomic_store(reinterpret_cast<uint64_t*>(g.act + row * F + cn0 + 4 * q),
                           lo | (static_cast<uint64_t>(hi) << 32), __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
      }
      if (!more) break;
      if (ks > 1) __syncthreads();  // the parts are read before the next round
    }
    // The item's rows are in memory before it counts as done: agent-scope
    // stores write through every cache, and this waits for their answers.
    __builtin_amdgcn_s_waitcnt(0);
    local = wave_max(local);
    if (lane == 0) sm.wave_part[wave] = local;
    __syncthreads();
    if (tid == 0) {
#pragma unroll
      for (int v = 1; v < kWaves; ++v) local = fmaxf(local, sm.wave_part[v]);
      // done, with the item's largest a (its sign bit is free)
      __hip_atomic_store(&g.ctr[kFewDone + ticket], kFewDoneBit | __float_as_uint(local),
                         __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      // Items that no workgroup has taken yet are taken before anyone waits; the
      // count only grows, so what was seen earlier may already say that there
      // are none.
      if (seen < up_items) seen = static_cast<int>(atomicAdd(&g.ctr[kFewTicket], 1u));
      sm.next = seen;
    }
    __syncthreads();
    ticket = __builtin_amdgcn_readfirstlane(sm.next);
  }

  // ---- down: 16 output columns over all experts
  const int F8 = F / 8, cF = chunks_of<FMT>(F);
  const int stride = cF * 16 + 16;  // LDS row of a: padded against bank conflicts
  const int U = units_of<FMT>(F);
  bool ready = false;
  bool late = false;  // wave 0: the wait was given up
  TensorScale<FMT> ts(0.f);
  for (int item = blockIdx.x; item < H / 16; item += groups) {
    const int n0 = item * 16;
    f32x4 tot = {0.f, 0.f, 0.f, 0.f};
    for (int d0 = 0; d0 < D;) {
      // experts whose rows fit the stage (one expert's always do)
      int d1 = d0 + 1;
      while (d1 < D && rt.off[d1 + 1] - rt.off[d0] <= g.stage_rows) ++d1;
      d1 = __builtin_amdgcn_readfirstlane(d1);
      const int r0 = __builtin_amdgcn_readfirstlane(rt.off[d0]);
      const int rows = __builtin_amdgcn_readfirstlane(rt.off[d1]) - r0;
      const int all = (d1 - d0) * U;
      const int i0 = __builtin_amdgcn_readfirstlane(all * wave / kWaves);
      const int n = __builtin_amdgcn_readfirstlane(all * (wave + 1) / kWaves) - i0;
      int ld = d0 + i0 / U, lu = i0 % U;  // expert and unit of the next load
      int cd = ld, cu = lu;               // and of the next product
      const auto expert = [&](int d) { return __builtin_amdgcn_readfirstlane(rt.expert[d < D ? d : 0]); };
      Tile<FMT, true> w;
      w.point(g.down, g.down_bs, expert(ld), n0, H, F);
      const auto load = [&](int i) {
        const Unit<FMT> v = w.load(lu, i < n);
        if (++lu == U) {
          lu = 0;
          w.point(g.down, g.down_bs, expert(++ld), n0, H, F);
        }
        return v;
      };
      Stream<FMT, P> st;
      st.prime(load);  // the weights do not wait for a
      if (!ready) {
        // every up item is done; the largest a gives the tensor scale
        if (wave == 0) {
          float amax = 0.f;
          for (int i = lane; i < up_items && !late; i += kWave) {
            uint32_t v;
            int polls = 0;
            while (!((v = __hip_atomic_load(&g.ctr[kFewDone + i], __ATOMIC_RELAXED,
                                            __HIP_MEMORY_SCOPE_AGENT)) & kFewDoneBit) && ++polls < kMaxPolls)
              __builtin_amdgcn_s_sleep(4);
            late = polls == kMaxPolls;
            amax = fmaxf(amax, __uint_as_float(v & ~kFewDoneBit));
          }
          amax = wave_max(amax);
          late = __any(late);
          // what the other workgroups stored is read from memory from here on
          __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
          if (lane == 0) sm.wave_part[0] = amax;
        }
        __syncthreads();
        ts = TensorScale<FMT>(sm.wave_part[0]);
        ready = true;
      }
      __syncthreads();  // the stage is free
      stage_rows(
          rows, F8,
          [&](int r) {
            const int s = rt.src[r0 + r];
            return g.act + (static_cast<size_t>(s >> 3) * g.k + (s & 7)) * F;
          },
          [&](int r, int ch) { return stage + r * stride + ch * 16; },
          [&](u32x4 v) { return quantise8<FMT, true>(v, ts); });
      if (cF > F8)
        for (int i = tid; i < rows * (cF - F8); i += kThreads)
          *reinterpret_cast<u32x4*>(stage + i / (cF - F8) * stride + (F8 + i % (cF - F8)) * 16) =
              u32x4{0u, 0u, 0u, 0u};
      __syncthreads();
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
      int ce = expert(cd);
      Column col_c = column_of(rt, ce);
      const uint8_t* row = stage + (rt.off[cd < D ? cd : 0] - r0 + col_c.rank) * stride;
      const auto flush = [&]() {
        if (col_c.live) {
          float f = rt.gate[c][rt.slot[ce][c]];
          if constexpr (FMT != kBF16) f *= ts.s * g.down_s[ce];
#pragma unroll
          for (int i = 0; i < 4; ++i) tot[i] += f * acc[i];
        }
        acc = f32x4{0.f, 0.f, 0.f, 0.f};
      };
      st.run(n, load, [&](const Unit<FMT>& v, int) {
        acc = mul_unit<FMT>(v, row + cu * (kUnitK<FMT> * 2), 16, turn, acc);
        if (++cu == U) {
          flush();
          cu = 0;
          if (++cd < d1) {
            ce = expert(cd);
            col_c = column_of(rt, ce);
            row = stage + (rt.off[cd] - r0 + col_c.rank) * stride;
          }
        }
      });
      if (n > 0 && cu != 0) flush();
      d0 = d1;
    }
    *part_of(wave) = tot;
    __syncthreads();
    if (wave == 0 && c < T) {
#pragma unroll
      for (int w = 1; w < kWaves; ++w) tot += *part_of(w);
      if (late) tot = f32x4{NAN, NAN, NAN, NAN};
      const size_t at = static_cast<size_t>(c) * H + n0 + 4 * q;
      if (g.y_bf16) {
        const uint32_t lo = f32_to_bf16(tot[0]) | (static_cast<uint32_t>(f32_to_bf16(tot[1])) << 16);
        const uint32_t hi = f32_to_bf16(tot[2]) | (static_cast<uint32_t>(f32_to_bf16(tot[3])) << 16);
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(g.y) + at) = make_uint2(lo, hi);
      } else {
        *reinterpret_cast<f32x4*>(static_cast<float*>(g.y) + at) = tot;
      }
    }
    __syncthreads();  // the parts are read before they are written again
  }
}

constexpr size_t kLdsBytes = 160 * 1024;
constexpr size_t kFixedLds = (sizeof(Shared) + 15) / 16 * 16;
constexpr size_t kMaxStage = 120 * 1024;
static_assert(kFixedLds + kMaxStage <= kLdsBytes, "the stage fits");
constexpr int kGroups = kFewGroups;

// bytes of an LDS row of a, and of the stage for T tokens: the tokens, or rows
// of a for one expert that all of them select.  Whole units of 128 values
// cover the three formats.
size_t row_bytes(int F) { return (static_cast<size_t>(F) + 127) / 128 * 256 + 16; }
size_t stage_need(int T, int H, int F) {
  const size_t xs = (static_cast<size_t>(H) + 127) / 128 * 256;
  return static_cast<size_t>(T) * (xs > row_bytes(F) ? xs : row_bytes(F));
}

template <int FMT>
hipError_t launch_layer(const FewArgs& a, hipStream_t stream) {
  FewArgs g = a;
  g.tokens = FMT == kBF16 && !g.y_over_x ? g.x : g.x_q;
  const int blocks = g.E / 16 * kFewSlices + (g.tokens == g.x ? 0 : kQuantGroups);
  hipLaunchKernelGGL(few_router_kernel<FMT>, dim3(blocks), dim3(kRouterThreads), 0, stream, g);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const size_t need = stage_need(g.T, g.H, g.F);
  const size_t all = static_cast<size_t>(g.T) * g.k * row_bytes(g.F);
  const size_t stage = all > need ? (all < kMaxStage ? all : kMaxStage) : need;
  g.stage_rows = static_cast<int>(stage / row_bytes(g.F));
  const size_t lds = kFixedLds + stage;
  hipLaunchKernelGGL(few_layer_kernel<FMT>, dim3(kGroups), dim3(kThreads), lds, stream, g);
  return hipGetLastError();
}

}  // namespace

// The operands fit LDS, one expert's matrix is addressed by 32 bits, and the two
// kernels are not slower than moe_route and moe_forward.  What they save is
// launches, about 20 us; what they cost grows with the rows of a that every
// workgroup stages, and for NVFP4 quantises, T k F values.  Full layer (k F =
// 11136), us of these against the two calls: BF16 T = 1 36 (54), 4 81 (81), 8 104
// (110), 12 154 (159), 16 189 (182); NVFP4 T = 1 28 (42), 5 52 (56), 6 59 (57), 16
// 103 (84); FP8 T = 1 28 (46), 8 75 (86), 16 117 (130).  At 1024 -> 512, 64 experts,
// top-4, they are ahead at every T in every format (17 to 34 us against 28 to 35).
// At 2048 -> 768, 128 experts, top-8, NVFP4 T = 8 takes 41 (47), and BF16 12 74 (75)
// but 16 96 (90): there the border, drawn at the full layer, comes 7 % late.
bool few_pays(int fmt, int T, int H, int F, int k) {
  const size_t staged = static_cast<size_t>(T) * k * F;
  if (fmt == kFP8Block || (fmt == kBF16 && staged > 140000) || (fmt == kNVFP4 && staged > 60000)) return false;
  return stage_need(T, H, F) <= kMaxStage &&
         static_cast<size_t>(H) * F * 2 < (static_cast<size_t>(1) << 31);
}

hipError_t launch_few(int fmt, const FewArgs& g, hipStream_t stream) {
  switch (fmt) {
    case kBF16: return launch_layer<kBF16>(g, stream);
    case kFP8: return launch_layer<kFP8>(g, stream);
    case kNVFP4: return launch_layer<kNVFP4>(g, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace moe
