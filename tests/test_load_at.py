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
