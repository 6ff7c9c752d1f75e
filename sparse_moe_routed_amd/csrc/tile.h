// Device code shared by the tiled products: buffer descriptors, loads straight
// into LDS, and the owner of a tile among ragged groups of rows.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <type_traits>

#include "load_at.h"
#include "moe_common.h"
#include "moe_internal.h"

namespace moe {

// Buffer descriptors: raw 32-bit data; a load past num_records reads zero and
// touches no memory, so loads past the last K block are issued all the same, and
// every wave has the same number of loads under way.  What lies past the end is
// past it by the lane's own offset (kPastEnd, or a descriptor of no records with
// a scalar offset of 0), whether or not the range check counts the scalar offset.
constexpr int kRawBuffer = 0x00027000;
static_assert(kPastEnd == kBlockMaxBytes, "beyond every buffer");
typedef __amdgpu_buffer_rsrc_t Buffer;

__device__ __forceinline__ Buffer buffer_of(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, static_cast<int>(bytes), kRawBuffer);
}

__device__ __forceinline__ void load16_to_lds(Buffer b, uint32_t at, uint32_t step_at, uint8_t* to) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (__attribute__((address_space(3))) void*)to, 16, at, step_at, 0, 0);
}
__device__ __forceinline__ void load4_to_lds(Buffer b, uint32_t at, uint32_t step_at, uint8_t* to) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (__attribute__((address_space(3))) void*)to, 4, at, step_at, 0, 0);
}

// chunk x of a 128-byte row r lies at x ^ swz(r), so that the 16 rows of an
// operand read fall on distinct banks
__device__ __forceinline__ int swz(int r) { return (r >> 1) & 7; }

// s_waitcnt immediate: at most n vector memory operations outstanding
constexpr int vmcnt_imm(int n) { return (n & 15) | (7 << 4) | (15 << 8) | ((n >> 4) << 14); }

// ---- groups of rows: rows offsets[e] to offsets[e + 1] belong to group e.  The
// offsets are device data: bounds outside [0, R] are taken as the nearest of them and
// a group that ends before it starts is empty, so that what a kernel reads and writes
// stays inside its buffers whatever they hold.
struct GroupTile {
  int e, row0, rows;  // rows: valid rows of the tile
  int nt;             // column tile
};

// inclusive sum over the lanes
__device__ __forceinline__ int wave_scan(int v) {
  const auto add = [&](auto how, auto rows) {
    v += __builtin_amdgcn_update_dpp(0, v, decltype(how)::value, decltype(rows)::value, 0xf, false);
  };
  add(std::integral_constant<int, 0x111>{}, std::integral_constant<int, 0xf>{});  // lane - 1 of the row of 16
  add(std::integral_constant<int, 0x112>{}, std::integral_constant<int, 0xf>{});  // - 2
  add(std::integral_constant<int, 0x114>{}, std::integral_constant<int, 0xf>{});  // - 4
  add(std::integral_constant<int, 0x118>{}, std::integral_constant<int, 0xf>{});  // - 8
  add(std::integral_constant<int, 0x142>{}, std::integral_constant<int, 0xa>{});  // last lane of row 0 to row 1, 2 to 3
  add(std::integral_constant<int, 0x143>{}, std::integral_constant<int, 0xc>{});  // lane 31 to rows 2 and 3
  return v;
}

// The tile of this workgroup among those of E <= 256 groups, BM rows by one of n_nt
// column tiles, false for a surplus one.  Workgroups go round robin to the 8 XCDs;
// each XCD takes a contiguous eighth of the tiles (group, column tile, row tile), so
// that sharers of a weight panel share an L2.  Every wave works it out for itself: a
// kernel that did it once would cost a launch, this costs two loads and a scan.
template <int BM>
__device__ __forceinline__ bool find_group_tile(const int32_t* __restrict__ offsets, int E, int R, int n_nt,
                                                GroupTile& t) {
  const int lane = threadIdx.x & 63;
  int first[4], count[4], upto[4], total = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    first[q] = count[q] = upto[q] = 0;
    if (64 * q >= E) continue;
    const int e = 64 * q + lane;
    const int lo = min(max(offsets[min(e, E)], 0), R), hi = min(max(offsets[min(e + 1, E)], 0), R);
    first[q] = lo;
    count[q] = max(hi - lo, 0);
    upto[q] = wave_scan((count[q] + BM - 1) / BM) + total;
    total = __builtin_amdgcn_readlane(upto[q], 63);
  }
  // (groups that overlap may have more tiles than the launch: those past its bound are left)
  const int tiles = min(total, (R + BM - 1) / BM + min(R, E)) * n_nt, per_xcd = (tiles + 7) >> 3;
  const int local = blockIdx.x >> 3;
  const int logical = (blockIdx.x & 7) * per_xcd + local;
  if (local >= per_xcd || logical >= tiles) return false;
  const int panel = logical / n_nt;
  int e = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (64 * q < E) e += __popcll(__ballot(64 * q + lane < E && upto[q] <= panel));
  e = __builtin_amdgcn_readfirstlane(e);
  int lo = 0, n = 0, last = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q)
    if (e >> 6 == q) {
      lo = __builtin_amdgcn_readlane(first[q], e & 63);
      n = __builtin_amdgcn_readlane(count[q], e & 63);
      last = __builtin_amdgcn_readlane(upto[q], e & 63);
    }
  const int te = (n + BM - 1) / BM;
  const int loc = logical - (last - te) * n_nt;
  t.e = e;
  t.nt = loc / te;
  const int mt = loc - t.nt * te;
  t.row0 = lo + mt * BM;
  t.rows = min(BM, n - mt * BM);
  return true;
}

// upper bound of the workgroups that find_group_tile<BM> needs
inline long long group_tiles(int R, int E, int bm, long long n_nt) {
  return (((R + bm - 1) / bm + (R < E ? R : E)) * n_nt + 7) / 8 * 8;
}

}  // namespace moe
