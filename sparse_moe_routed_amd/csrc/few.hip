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
// weights of one token.
//
// few_router_kernel writes partial logits.  few_layer_kernel does the rest: its
// workgroups each redo the selection (a few KB of partial logits), then take
// work items from a ticket counter: first the up projection's rounds, then the
// down projection's column tiles.  A down item waits until every up round is
// done.  The wait ends: tickets are handed out in order, so all up rounds
// belong to workgroups that are running, and none of those waits before its
// round is done, however few workgroups the GPU runs at a time.
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

constexpr int kWaves = 8;
constexpr int kThreads = kWaves * kWave;
constexpr int kTok = kFewTokens;        // MFMA columns
constexpr int kMaxRows = kTok * 8;      // (token, slot) pairs
constexpr int kRouterThreads = 256;

// ---- partial logits: grid (E / 16, kFewSlices), 4 waves; the K steps are
// dealt to slices and waves in contiguous ranges, the waves' sums added in
// wave order.  Also clears the counters of the second kernel.
__global__ __launch_bounds__(kRouterThreads) void few_router_kernel(
    const uint16_t* __restrict__ x, const uint16_t* __restrict__ wp, int T, int H, int E,
    float* __restrict__ part, uint32_t* __restrict__ ctr) {
  constexpr int U = 6;  // K steps of loads in flight
  __shared__ f32x4 red[4][kWave];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int eb = blockIdx.x, s = blockIdx.y;
  if (eb == 0 && s == 0 && threadIdx.x < kFewCounters) ctr[threadIdx.x] = 0u;
  const int row = lane & 15;
  const int kq = (lane >> 4) * 8;
  const int steps = H / 32;
  const int i = s * 4 + wave;
  const int k0 = steps * i / (4 * kFewSlices), k1 = steps * (i + 1) / (4 * kFewSlices);
  const size_t n = static_cast<size_t>(E) * H;
  const uint16_t* xr = x + static_cast<size_t>(min(row, T - 1)) * H + kq;
  const uint16_t* hi = wp + static_cast<size_t>(eb * 16 + row) * H + kq;
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
      if (t < T) part[(static_cast<size_t>(s) * T + t) * E + eb * 16 + row] = v[r];
    }
  }
}

// ---- weight units.  A unit is what one wave loads of 16 weight rows with one
// 16-byte load a lane (NVFP4: and one 2-byte load of block scales): lane l
// holds row l % 16 and, with q = l / 16, the K values
//   BF16   32 per unit:  8 at 32 u + 8 q                      (1 MFMA)
//   FP8    64 per unit: 16 at 64 u + 16 q                     (2 MFMAs)
//   NVFP4 128 per unit: 32 at 128 u + 32 q, two scale blocks  (4 MFMAs)
// MFMA i of a unit multiplies values 8 i .. 8 i + 7 of each lane; the tokens'
// operand is read at the same K values.  Loads go through a buffer descriptor
// of one expert's matrix, so a unit past the end reads nothing and is zero.
template <int FMT>
struct Unit {
  u32x4 v;
  uint32_t sb;
};
template <int FMT>
constexpr int kUnitK = FMT == kBF16 ? 32 : (FMT == kFP8 ? 64 : 128);

template <int FMT>
__host__ __device__ constexpr int units_of(int K) {
  return (K + kUnitK<FMT> - 1) / kUnitK<FMT>;
}

constexpr uint32_t kPastEnd = 0xffffff00u;  // beyond every matrix: reads as zero
constexpr int kRawBuffer = 0x00027000;      // descriptor word 3: raw 32-bit data
constexpr int kStreamOnce = 2;              // cache policy: non-temporal

struct Matrix {
  __amdgpu_buffer_rsrc_t codes, scales;
};

template <int FMT>
__device__ __forceinline__ Matrix matrix_of(const void* w, const uint8_t* bs, int e, int N, int K) {
  const size_t n = static_cast<size_t>(N) * K;
  const size_t bytes = FMT == kBF16 ? 2 * n : (FMT == kFP8 ? n : n / 2);
  Matrix m;
  m.codes = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint8_t*>(static_cast<const uint8_t*>(w) + bytes * e), 0, static_cast<int>(bytes),
      kRawBuffer);
  if constexpr (FMT == kNVFP4)
    m.scales = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(bs + n / 16 * e), 0,
                                                 static_cast<int>(n / 16), kRawBuffer);
  else
    m.scales = m.codes;
  return m;
}

// DOWN selects the FP8 code layout: row-major (up) or panels (down)
template <int FMT, bool DOWN>
__device__ __forceinline__ Unit<FMT> load_unit(const Matrix& m, int n0, int N, int K, int u, bool in) {
  const int lane = threadIdx.x & 63, q = lane >> 4;
  const int n = n0 + (lane & 15);
  uint32_t at;
  Unit<FMT> r{};
  if constexpr (FMT == kBF16) {
    at = static_cast<uint32_t>(n) * (2 * K) + u * 64 + q * 16;
  } else if constexpr (FMT == kFP8 && !DOWN) {
    at = static_cast<uint32_t>(n) * K + u * 64 + q * 16;
  } else if constexpr (FMT == kFP8) {
    const int p = n0 / kNvPanel, rows = nv_panel_rows(N, p);
    const int st = u >> 1, sb = min(kFp8StepK, K - st * kFp8StepK);
    at = static_cast<uint32_t>(p) * kNvPanel * K + static_cast<uint32_t>(st) * rows * kFp8StepK +
         (n - p * kNvPanel) * sb + (u & 1) * 64 + q * 16;
  } else {
    const int p = n0 / kNvPanel, rows = nv_panel_rows(N, p);
    const int st = 2 * u + (q >> 1);  // 64-value step of this lane
    in = in && st * kNvStepK < K;
    const uint32_t pr = n - p * kNvPanel;
    const uint32_t sat = static_cast<uint32_t>(p) * kNvPanel * (K / 16) +
                         static_cast<uint32_t>(st) * rows * 4 + pr * 4 + (q & 1) * 2;
    at = static_cast<uint32_t>(p) * kNvPanel * (K / 2) + static_cast<uint32_t>(st) * rows * 32 +
         pr * 32 + (q & 1) * 16;
    r.sb = __builtin_amdgcn_raw_buffer_load_b16(m.scales, in ? sat : kPastEnd, 0, kStreamOnce);
  }
  r.v = __builtin_amdgcn_raw_buffer_load_b128(m.codes, in ? at : kPastEnd, 0, kStreamOnce);
  return r;
}

__device__ __forceinline__ bf16x8 fp8_frag(uint32_t w0, uint32_t w1) {
  const bf16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, false);
  const bf16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w0, 1.0f, true);
  const bf16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, false);
  const bf16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w1, 1.0f, true);
  return bf16x8{p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
}

// acc += 16 weight rows of the unit times the tokens' values; tok(c) points at
// the 16-byte chunk (8 values) c of this lane's token column
template <int FMT, class Tok>
__device__ __forceinline__ f32x4 mul_unit(const Unit<FMT>& w, int u, int last_chunk, Tok tok,
                                          f32x4 acc) {
  const int q = (threadIdx.x & 63) >> 4;
  if constexpr (FMT == kBF16) {
    const bf16x8 b = *reinterpret_cast<const bf16x8*>(tok(u * 4 + q));
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, w.v), b, acc, 0, 0, 0);
  } else if constexpr (FMT == kFP8) {
    // E4M3 codes as bf16 (exact), so the products are exact in fp32
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bf16x8 b = *reinterpret_cast<const bf16x8*>(tok(u * 8 + q * 2 + i));
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fp8_frag(w.v[2 * i], w.v[2 * i + 1]), b, acc, 0,
                                                    0, 0);
    }
  } else {
    // E2M1 codes times the block scale as fp16 (exact, at most 6 significant
    // bits); a unit half past K holds zero codes and reads the last chunk
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f16x8 b = *reinterpret_cast<const f16x8*>(tok(min(u * 16 + q * 4 + i, last_chunk)));
      const _Float16 sh = static_cast<_Float16>(e4m3_decode((w.sb >> (i >> 1 ? 8 : 0)) & 0xffu));
      const f16x2 s2 = {sh, sh};
      const f16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w.v[i], 1.0f, 0) * s2;
      const f16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w.v[i], 1.0f, 1) * s2;
      const f16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w.v[i], 1.0f, 2) * s2;
      const f16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w.v[i], 1.0f, 3) * s2;
      const f16x8 a = {p0[0], p0[1], p1[0], p1[1], p2[0], p2[1], p3[0], p3[1]};
      acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, acc, 0, 0, 0);
    }
  }
  return acc;
}

// n units through a ring of P loads in flight: load(i) starts the i-th (none
// past n), use(unit, i) consumes it
template <int FMT, int P, class Load, class Use>
__device__ __forceinline__ void stream_units(int n, Load load, Use use) {
  Unit<FMT> ring[P];
#pragma unroll
  for (int j = 0; j < P; ++j) ring[j] = load(j);
  for (int i = 0; i < n; i += P) {
#pragma unroll
    for (int j = 0; j < P; ++j) {
      if (i + j < n) use(ring[j], i + j);
      ring[j] = load(i + j + P);
    }
  }
}

// ---- activation quantisers, 8 values of one lane (the recipes of quant.hip)
template <int FMT>
struct TensorScale {
  float s = 1.f;  // value = stored * s
  float a = 0.f;  // FP8: 448 / amax; NVFP4: 6 s
  __device__ explicit TensorScale(float amax) {
    if constexpr (FMT == kFP8) {
      s = amax > 0.f ? __fdiv_rn(amax, 448.f) : 0.f;
      a = amax > 0.f ? __fdiv_rn(448.f, amax) : 0.f;
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
// the neighbouring lane, which must be active)
template <int FMT>
__device__ __forceinline__ u32x4 quantise8(u32x4 v, const TensorScale<FMT>& ts) {
  if constexpr (FMT == kBF16) {
    return v;
  } else if constexpr (FMT == kFP8) {
    uint32_t c[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t a = v[2 * h], b = v[2 * h + 1];
      c[h] = e4m3_encode4(__uint_as_float(a << 16) * ts.a, __uint_as_float(a & 0xffff0000u) * ts.a,
                          __uint_as_float(b << 16) * ts.a, __uint_as_float(b & 0xffff0000u) * ts.a);
    }
    return __builtin_bit_cast(u32x4, fp8_frag(c[0], c[1]));
  } else {
    const float m = amax8(v);
    // quad_perm [1, 0, 3, 2]: the value of the neighbouring lane
    const float mo = __builtin_bit_cast(
        float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, m), 0xb1, 0xf, 0xf, false));
    float sbf = 0.f;
    if (ts.s > 0.f) sbf = e4m3_decode(e4m3_encode(__fdiv_rn(fmaxf(m, mo), ts.a)));
    const float r = sbf > 0.f ? __fdiv_rn(1.f, sbf * ts.s) : 0.f;
    float t[8];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      t[2 * w] = __uint_as_float(v[w] << 16) * r;
      t[2 * w + 1] = __uint_as_float(v[w] & 0xffff0000u) * r;
    }
    const uint32_t q = e2m1_encode8(t);
    const _Float16 sh = static_cast<_Float16>(sbf);
    const f16x2 s2 = {sh, sh};
    const f16x2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, 1.0f, 0) * s2;
    const f16x2 p1 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, 1.0f, 1) * s2;
    const f16x2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, 1.0f, 2) * s2;
    const f16x2 p3 = __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(q, 1.0f, 3) * s2;
    return u32x4{__builtin_bit_cast(uint32_t, p0), __builtin_bit_cast(uint32_t, p1),
                 __builtin_bit_cast(uint32_t, p2), __builtin_bit_cast(uint32_t, p3)};
  }
}

// routing of the batch, the same in every workgroup
struct Routing {
  uint32_t mask[kMaxE];          // tokens of each expert, a bit each
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
  f32x4 red[kWaves][kWave];
  float wave_part[kWaves];
  int next, ready;
};

// element r of the packed partial logits of token t; every wave takes the
// tokens wave, wave + kWaves, ...
__device__ void route_tokens(const FewArgs& g, Shared& sm) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  Routing& rt = sm.rt;
  for (int e = threadIdx.x; e < kMaxE; e += kThreads) rt.mask[e] = 0u;
  __syncthreads();
  for (int t = wave; t < g.T; t += kWaves) {
    float v[kMaxE / 64];
    uint32_t key[kMaxE / 64];
#pragma unroll
    for (int i = 0; i < kMaxE / 64; ++i) {
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
    if (lane == 0) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = j < g.k ? sel_i[j] : -1;
        rt.id[t][j] = static_cast<int16_t>(e);
        rt.gate[t][j] = z[j] / sum;
        if (e >= 0) {
          rt.slot[e][t] = static_cast<uint8_t>(j);
          atomicOr(&rt.mask[e], 1u << t);
        }
      }
    }
  }
  __syncthreads();
  if (wave == 0) {
    int base = 0, row = 0;
    for (int e0 = 0; e0 < g.E; e0 += 64) {
      const int e = e0 + lane;
      const uint32_t m = e < g.E ? rt.mask[e] : 0u;
      const uint64_t any = __ballot(m != 0u);
      const int cnt = __popc(m);
      int incl = cnt;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const int n = __shfl_up(incl, o);
        if (lane >= o) incl += n;
      }
      if (m) {
        const int d = base + __popcll(any & ((1ull << lane) - 1));
        int at = row + incl - cnt;
        rt.expert[d] = static_cast<uint8_t>(e);
        rt.off[d] = static_cast<uint16_t>(at);
        for (uint32_t b = m; b; b &= b - 1) {
          const int t = __ffs(static_cast<int>(b)) - 1;
          rt.src[at++] = static_cast<uint8_t>(t * 8 + rt.slot[e][t]);
        }
      }
      base += __popcll(any);
      row += __shfl(incl, 63);
    }
    if (lane == 0) {
      rt.off[base] = static_cast<uint16_t>(row);
      rt.n_experts = base;
    }
  }
  __syncthreads();
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

// one token row's values as operand chunks of 16 bytes, with the tensor scale
// over all T rows.  Chunk c of token t sits at (c * T + t) * 16, so the lanes
// of one MFMA operand read consecutive addresses.
template <int FMT>
__device__ float stage_tokens(const FewArgs& g, uint8_t* xs, Shared& sm) {
  const int h8 = g.H / 8;
  float m = 0.f;
  for (int t = 0; t < g.T; ++t)
    for (int c = threadIdx.x; c < h8; c += kThreads) {
      const u32x4 v = reinterpret_cast<const u32x4*>(g.x + static_cast<size_t>(t) * g.H)[c];
      if constexpr (FMT != kBF16) m = fmaxf(m, amax8(v));
      *reinterpret_cast<u32x4*>(xs + (static_cast<size_t>(c) * g.T + t) * 16) = v;
    }
  if constexpr (FMT == kBF16) return 1.f;
  m = wave_max(m);
  if ((threadIdx.x & 63) == 0) sm.wave_part[threadIdx.x >> 6] = m;
  __syncthreads();
  m = 0.f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) m = fmaxf(m, sm.wave_part[w]);
  const TensorScale<FMT> ts(m);
  // each thread quantises the chunks it stored (a block's halves are on
  // neighbouring lanes: h8 is even)
  for (int t = 0; t < g.T; ++t)
    for (int c = threadIdx.x; c < h8; c += kThreads) {
      u32x4* p = reinterpret_cast<u32x4*>(xs + (static_cast<size_t>(c) * g.T + t) * 16);
      *p = quantise8<FMT>(*p, ts);
    }
  return ts.s;
}

// waves that share one 16-row tile of the up projection: as many as leave at
// least one round for every workgroup, so that a few experts still spread over
// all of them
__device__ __forceinline__ int up_split(int tiles, int n_groups) {
  int ks = 1;
  while (ks < kWaves && tiles * ks < n_groups * kWaves) ks *= 2;
  return ks;
}

template <int FMT>
__global__ __launch_bounds__(kThreads) void few_layer_kernel(FewArgs g) {
  constexpr int P = 8;  // loads in flight per wave
  extern __shared__ __attribute__((aligned(16))) uint8_t dyn[];
  Shared& sm = *reinterpret_cast<Shared*>(dyn);
  uint8_t* const stage = dyn + (sizeof(Shared) + 15) / 16 * 16;  // tokens, later rows of a
  Routing& rt = sm.rt;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c = lane & 15, q = lane >> 4;
  const int H = g.H, F = g.F, T = g.T;

  int ticket = 0;
  if (tid == 0) ticket = static_cast<int>(atomicAdd(&g.ctr[0], 1u));
  route_tokens(g, sm);
  const float s_x = stage_tokens<FMT>(g, stage, sm);
  if (tid == 0) {
    sm.next = ticket;
    sm.ready = 0;
  }
  __syncthreads();
  ticket = __builtin_amdgcn_readfirstlane(sm.next);
  if (ticket == 0)
    for (int i = tid; i < T * g.k; i += kThreads) {
      g.ids[i] = rt.id[i / g.k][i % g.k];
      g.gates[i] = rt.gate[i / g.k][i % g.k];
    }

  const int D = __builtin_amdgcn_readfirstlane(rt.n_experts);
  const int f16 = F / 16;
  const int up_tiles = D * f16;
  const int ks = up_split(up_tiles, static_cast<int>(gridDim.x));
  const int per_round = kWaves / ks;
  const int up_rounds = (up_tiles + per_round - 1) / per_round;
  const int down_tiles = H / 16;
  const int stride = F * 2 + 16;  // LDS row of a: padded against bank conflicts

  while (ticket < up_rounds + down_tiles) {
    int nxt = 0;
    if (tid == 0) nxt = static_cast<int>(atomicAdd(&g.ctr[0], 1u));
    if (ticket < up_rounds) {
      // ---- up: a tile of 16 expert rows per ks waves, K split over them
      const int tile = ticket * per_round + wave / ks;
      const bool have = tile < up_tiles;
      const int d = __builtin_amdgcn_readfirstlane(have ? tile / f16 : 0);
      const int n0 = __builtin_amdgcn_readfirstlane(have ? tile % f16 : 0) * 16;
      const int e = __builtin_amdgcn_readfirstlane(rt.expert[d]);
      const int U = units_of<FMT>(H);
      const int part = wave % ks;
      const int u0 = U * part / ks;
      const int n = have ? U * (part + 1) / ks - u0 : 0;
      const Matrix m = matrix_of<FMT>(g.up, g.up_bs, e, F, H);
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
      const uint8_t* col = stage + min(c, T - 1) * 16;
      stream_units<FMT, P>(
          n, [&](int i) { return load_unit<FMT, false>(m, n0, F, H, u0 + i, i < n); },
          [&](const Unit<FMT>& w, int i) {
            acc = mul_unit<FMT>(
                w, u0 + i, H / 8 - 1, [&](int ch) { return col + static_cast<size_t>(ch) * T * 16; },
                acc);
          });
      if (ks > 1) {
        sm.red[wave][lane] = acc;
        __syncthreads();
        if (part == 0)
          for (int w = 1; w < ks; ++w) acc += sm.red[wave + w][lane];
      }
      float local = 0.f;
      if (have && part == 0) {
        float scale = 1.f;
        if constexpr (FMT != kBF16) scale = s_x * g.up_s[e];
        if ((rt.mask[e] >> c) & 1u) {
          uint16_t b[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            b[i] = relu_sq_bf16(FMT == kBF16 ? acc[i] : acc[i] * scale);
            local = fmaxf(local, bf16_to_f32(b[i]));
          }
          const size_t row = static_cast<size_t>(c) * g.k + rt.slot[e][c];
          *reinterpret_cast<uint2*>(g.act + row * F + n0 + 4 * q) =
              make_uint2(b[0] | (static_cast<uint32_t>(b[1]) << 16),
                         b[2] | (static_cast<uint32_t>(b[3]) << 16));
        }
        if constexpr (FMT != kBF16) {
          local = wave_max(local);
          if (lane == 0) atomic_max_nonneg(&g.ctr[kFewAmax + (tile % kAmaxSlots)], local);
        }
        __threadfence();  // the tile is in memory before the round counts as done
      }
      __syncthreads();
      if (tid == 0) {
        __threadfence();
        atomicAdd(&g.ctr[1], 1u);
      }
    } else {
      // ---- down: 16 output columns over all experts
      if (!sm.ready) {
        if (tid == 0) {
          while (__hip_atomic_load(&g.ctr[1], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) <
                 static_cast<uint32_t>(up_rounds))
            __builtin_amdgcn_s_sleep(2);
        }
        __syncthreads();
        __threadfence();  // what the other workgroups wrote is read from memory
        if (tid == 0) sm.ready = 1;
      }
      float amax = 0.f;
      if constexpr (FMT != kBF16)
        amax = wave_max(__uint_as_float(__hip_atomic_load(&g.ctr[kFewAmax + lane], __ATOMIC_RELAXED,
                                                          __HIP_MEMORY_SCOPE_AGENT)));
      const TensorScale<FMT> ts(amax);
      const int n0 = (ticket - up_rounds) * 16;
      const int U = units_of<FMT>(F);
      const int f8 = F / 8;
      f32x4 tot = {0.f, 0.f, 0.f, 0.f};
      for (int d0 = 0; d0 < D;) {
        // experts whose rows fit the stage (one expert's always do)
        int d1 = d0 + 1;
        while (d1 < D && rt.off[d1 + 1] - rt.off[d0] <= g.stage_rows) ++d1;
        const int r0 = rt.off[d0];
        __syncthreads();  // the stage is free
        for (int r = r0 + wave; r < rt.off[d1]; r += kWaves) {
          const int s = rt.src[r];
          const u32x4* src = reinterpret_cast<const u32x4*>(
              g.act + (static_cast<size_t>(s >> 3) * g.k + (s & 7)) * F);
          u32x4* dst = reinterpret_cast<u32x4*>(stage + static_cast<size_t>(r - r0) * stride);
          for (int ch = lane; ch < f8; ch += kWave) dst[ch] = quantise8<FMT>(src[ch], ts);
        }
        __syncthreads();
        const int all = (d1 - d0) * U;
        const int i0 = __builtin_amdgcn_readfirstlane(all * wave / kWaves);
        const int n = __builtin_amdgcn_readfirstlane(all * (wave + 1) / kWaves) - i0;
        int ld = d0 + i0 / U, lu = i0 % U;  // expert and unit of the next load
        int cd = ld, cu = lu;               // and of the next product
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
        int ce = __builtin_amdgcn_readfirstlane(rt.expert[cd < D ? cd : 0]);
        Column col = column_of(rt, ce);
        const uint8_t* row = stage + static_cast<size_t>(rt.off[cd < D ? cd : 0] - r0 + col.rank) * stride;
        auto flush = [&]() {
          if (col.live) {
            float f = rt.gate[c][rt.slot[ce][c]];
            if constexpr (FMT != kBF16) f *= ts.s * g.down_s[ce];
#pragma unroll
            for (int i = 0; i < 4; ++i) tot[i] += f * acc[i];
          }
          acc = f32x4{0.f, 0.f, 0.f, 0.f};
        };
        stream_units<FMT, P>(
            n,
            [&](int i) {
              const int e = __builtin_amdgcn_readfirstlane(rt.expert[ld < D ? ld : 0]);
              const Matrix m = matrix_of<FMT>(g.down, g.down_bs, e, H, F);
              const Unit<FMT> w = load_unit<FMT, true>(m, n0, H, F, lu, i < n);
              if (++lu == U) {
                lu = 0;
                ++ld;
              }
              return w;
            },
            [&](const Unit<FMT>& w, int i) {
              acc = mul_unit<FMT>(w, cu, f8 - 1, [&](int ch) { return row + ch * 16; }, acc);
              if (++cu == U) {
                flush();
                cu = 0;
                if (++cd < d1) {
                  ce = __builtin_amdgcn_readfirstlane(rt.expert[cd]);
                  col = column_of(rt, ce);
                  row = stage + static_cast<size_t>(rt.off[cd] - r0 + col.rank) * stride;
                }
              }
            });
        if (n > 0 && cu != 0) flush();
        d0 = d1;
      }
      sm.red[wave][lane] = tot;
      __syncthreads();
      if (wave == 0 && c < T) {
#pragma unroll
        for (int w = 1; w < kWaves; ++w) tot += sm.red[w][lane];
        const size_t at = static_cast<size_t>(c) * H + n0 + 4 * q;
        if (g.y_bf16) {
          const uint32_t lo = f32_to_bf16(tot[0]) | (static_cast<uint32_t>(f32_to_bf16(tot[1])) << 16);
          const uint32_t hi = f32_to_bf16(tot[2]) | (static_cast<uint32_t>(f32_to_bf16(tot[3])) << 16);
          *reinterpret_cast<uint2*>(static_cast<uint16_t*>(g.y) + at) = make_uint2(lo, hi);
        } else {
          *reinterpret_cast<f32x4*>(static_cast<float*>(g.y) + at) = tot;
        }
      }
    }
    if (tid == 0) sm.next = nxt;
    __syncthreads();
    ticket = __builtin_amdgcn_readfirstlane(sm.next);
    __syncthreads();
  }
}

constexpr size_t kLdsBytes = 160 * 1024;
constexpr size_t kFixedLds = (sizeof(Shared) + 15) / 16 * 16;
constexpr size_t kMaxStage = 144 * 1024;
static_assert(kFixedLds + kMaxStage <= kLdsBytes, "the stage fits");
// two workgroups per CU where the tokens' operand allows it
constexpr size_t kHalfLds = kLdsBytes / 2;
constexpr int kGroups = 512;

// bytes of the stage for T tokens: the tokens, and rows of a for at least one
// expert that all of them select
size_t stage_need(int T, int H, int F) {
  const size_t xs = static_cast<size_t>(T) * H * 2;
  const size_t as = static_cast<size_t>(T) * (static_cast<size_t>(F) * 2 + 16);
  return xs > as ? xs : as;
}

template <int FMT>
hipError_t launch_layer(const FewArgs& a, hipStream_t stream) {
  FewArgs g = a;
  const size_t need = stage_need(g.T, g.H, g.F);
  const size_t all = static_cast<size_t>(g.T) * g.k * (static_cast<size_t>(g.F) * 2 + 16);
  const bool two = kFixedLds + need <= kHalfLds;
  const size_t room = two ? kHalfLds - kFixedLds : kMaxStage;
  const size_t stage = all > need ? (all < room ? all : room) : need;
  g.stage_rows = static_cast<int>(stage / (static_cast<size_t>(g.F) * 2 + 16));
  const size_t lds = kFixedLds + stage;
  const int grid = two ? kGroups : kGroups / 2;
  hipLaunchKernelGGL(few_layer_kernel<FMT>, dim3(grid), dim3(kThreads), lds, stream, g);
  return hipGetLastError();
}

}  // namespace

// the operands fit LDS and one expert's matrix is addressed by 32 bits
bool few_fits(int T, int H, int F) {
  return stage_need(T, H, F) <= kMaxStage &&
         static_cast<size_t>(H) * F * 2 < (static_cast<size_t>(1) << 31);
}

hipError_t launch_few(int fmt, const FewArgs& g, hipStream_t stream) {
  hipLaunchKernelGGL(few_router_kernel, dim3(g.E / 16, kFewSlices), dim3(kRouterThreads), 0, stream,
                     g.x, g.w_router, g.T, g.H, g.E, g.part, g.ctr);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  switch (fmt) {
    case kBF16: return launch_layer<kBF16>(g, stream);
    case kFP8: return launch_layer<kFP8>(g, stream);
    case kNVFP4: return launch_layer<kNVFP4>(g, stream);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace moe
