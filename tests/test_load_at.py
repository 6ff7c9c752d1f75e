"""Where the loads of the tiled products go (csrc/load_at.h), on the host: whichever way a
buffer's range check takes the scalar offset, what is not dropped is inside the buffer."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_moe_routed_amd", "csrc")

CHECK = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "load_at.h"
using namespace moe;

// `valid`: bytes of the buffer from the descriptor's first on.  The check may take the
// lane's offset alone, the sum, or what the scalar offset leaves of the records (in 32 bits).
static bool dropped[3];
static void look(size_t valid, uint32_t records, uint32_t at, uint32_t step_at) {
  dropped[0] = at >= records;
  dropped[1] = static_cast<uint64_t>(at) + step_at >= records;
  dropped[2] = at >= static_cast<uint32_t>(records - step_at);
  for (int r = 0; r < 3; ++r)
    if (!dropped[r] && static_cast<uint64_t>(at) + step_at + 16 > valid) {
      std::printf("reading %d: valid %zu records %u at %u scalar %u\n", r, valid, records, at, step_at);
      std::exit(1);
    }
}
"""


def _run(tmp_path, body):
    src, exe = tmp_path / "check.cc", tmp_path / "check"
    src.write_text(CHECK + body)
    # the header's attributes mean nothing to the host's compiler
    subprocess.run([shutil.which("g++"), "-O2", "-std=c++17", "-D__host__=", "-D__device__=", "-D__forceinline__=inline",
                    "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout


needs_compiler = pytest.mark.skipif(shutil.which("g++") is None, reason="no g++")


@needs_compiler
def test_rows_read_ahead(tmp_path):
    """Every byte is read, none behind the last."""
    _run(tmp_path, r"""
int main() {
  const uint32_t all = 32 * 4 * 1024;
  for (size_t bytes : {size_t(16), size_t(1024), size_t(all - 16), size_t(all), size_t(all + 16), size_t(5 * all - 2032),
                       (size_t(1) << 30) + 48}) {
    size_t read[3] = {0, 0, 0};
    for (uint32_t mine = 0; mine < all; mine += 16)
      read_once(bytes, mine, all, [&](size_t base, uint32_t n, uint32_t at, uint32_t step_at) {
        if (base + n > bytes) std::exit(2);
        look(bytes - base, n, at, step_at);
        for (int r = 0; r < 3; ++r) read[r] += dropped[r] ? 0 : 16;
      });
    for (int r = 0; r < 3; ++r)
      if (read[r] != bytes) {
        std::printf("reading %d: %zu of %zu bytes\n", r, read[r], bytes);
        return 3;
      }
  }
}
""")


@needs_compiler
def test_stages_of_rows_and_of_packed_weights(tmp_path):
    """Loads of all stages of a tile and of those past the last one: contiguous rows and
    packed groups of 16 rows.  A chunk that holds values is read, no other is, and none behind the buffer."""
    _run(tmp_path, r"""
static void see(bool holds) {
  for (int r = 0; r < 3; ++r)
    if (dropped[r] == holds) {
      std::printf("reading %d: a chunk is %s\n", r, holds ? "left out" : "read");
      std::exit(2);
    }
}
int main() {
  for (int row_bytes : {16, 64, 80, 128, 144, 2688, 131072})
    for (int rows : {1, 3, 16, 17})
      for (int stage : {64, 128})
        for (int step = 0; step < (row_bytes + stage - 1) / stage + 5; ++step) {
          const int left = row_bytes - step * stage < stage ? row_bytes - step * stage : stage;  // bytes
          const uint32_t bytes = rows * row_bytes;
          for (int r = 0; r < 32; ++r)
            for (int chunk = 0; chunk < stage / 16; ++chunk) {
              const StageLoad l = load_rows(bytes, r * row_bytes + chunk * 16, step, stage, left, chunk * 16);
              look(bytes, l.records, l.at, l.step_at);
              see(r < rows && chunk * 16 < left);
            }
        }
  for (int steps : {1, 2, 21})
    for (int groups : {1, 2, 5})
      for (int step = 0; step < steps + 5; ++step) {
        const uint32_t bytes = groups * steps * 2048;
        for (int g = 0; g < 8; ++g)
          for (int at = 0; at < 2048; at += 16) {
            const StageLoad l = load_packed(bytes, g * steps * 2048 + at, step, step < steps ? 128 : 0);
            look(bytes, l.records, l.at, l.step_at);
            see(g < groups && step < steps);
          }
      }
}
""")


DMA = r"""
#include "tile_gemm.h"
namespace moe {
__global__ void loads(const uint8_t* p, uint8_t* out) {
  __shared__ __attribute__((aligned(1024))) uint8_t a[1024], b[1024];
  const Buffer d = buffer_of(p, 4096);
  load16_to_lds(d, threadIdx.x * 16, 0, a);
  dma16(descriptor(p, 4096), threadIdx.x * 16, 0, (Lds)b);
  load16_to_lds(d, threadIdx.x * 16 + 1024, 0, a);
  __asm__ volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  out[threadIdx.x] = a[threadIdx.x] + b[threadIdx.x];
}
}  // namespace moe
"""


def test_load_into_lds_and_the_compilers_own(tmp_path):
    """dma16 between two of the compiler's loads into another buffer of LDS: m0, the
    buffer's place, is written anew for each of the three."""
    from sparse_moe_routed_amd import build

    src, out = tmp_path / "loads.hip", tmp_path / "loads.s"
    src.write_text(DMA)
    subprocess.run([build.hipcc(), *build.HIPCC_FLAGS, "-I", CSRC, "--cuda-device-only", "-S", str(src), "-o", str(out)],
                   check=True, capture_output=True)
    places = []
    for line in out.read_text().splitlines():
        op = line.split()
        if len(op) > 1 and op[1] == "m0,":
            m0 = op[2]
        elif op and op[0].startswith("buffer_load") and op[-1] == "lds":
            places.append(m0)
    assert len(places) == 3 and places[0] == places[2] != places[1]
