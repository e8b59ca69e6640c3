"""Which bytes the tiles of the 8-bit product read, lane by lane on the host: the
arithmetic of csrc/fp8_stage.hpp, compiled for the CPU."""
import subprocess
from pathlib import Path

import pytest

CSRC = Path(__file__).resolve().parent.parent / "adapter_lora_bgmv_amd" / "csrc"
PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "fp8_stage.hpp"
using namespace lora;
// An n-row matrix of k codes a row by tiles of T rows, whose resource ends with
// the last row's k codes: transfers outside every row's codes, taken that the
// scalar offset is not checked, and codes of the matrix that no lane brings.
int main(int argc, char **argv) {
  const long long n = atoll(argv[1]), k = atoll(argv[2]), stride = atoll(argv[3]), T = atoll(argv[4]);
  const bool step_back = atoi(argv[5]);
  long long outside = 0, missing = 0;
  for (long long r0 = 0; r0 < n; r0 += T) {
    const long long records = (n - r0 - 1) * stride + k;
    for (long long k0 = 0; k0 < k; k0 += kFp8Block) {
      for (long long r = 0; r < T; ++r) {
        long long brought = 0;
        for (int slot = 0; slot < 8; ++slot) {
          const uint32_t chunk = stage_chunk(r, slot), c = step_back ? stage_column(chunk, k0, k) : chunk;
          const long long checked = r * stride + c, row = r0 + r, column = k0 + c;
          if (checked >= records) continue;  // not read
          if (row >= n || column + 16 > k) ++outside;
          else if (c == chunk) ++brought;
        }
        const long long due = (k - k0 < kFp8Block ? k - k0 : kFp8Block) / 16;
        if (r0 + r < n && brought != due) ++missing;
      }
    }
  }
  printf("%lld %lld\n", outside, missing);
}
"""
SIZES = [(n, k, pad, tile) for n in (1, 65, 257) for k in (16, 128, 144, 240, 272, 4096, 4208) for pad in (0, 16) for tile in (64, 128, 256)]


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    d = tmp_path_factory.mktemp("stage")
    (d / "stage.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", "-I", str(CSRC), str(d / "stage.cpp"), "-o", str(d / "stage")], check=True)

    def run(n, k, pad, tile, step_back=1):
        out = subprocess.run([str(d / "stage"), *map(str, (n, k, k + pad, tile, step_back))], check=True, capture_output=True, text=True)
        return tuple(map(int, out.stdout.split()))
    return run


def test_a_tile_reads_codes_of_its_rows_and_all_of_them(program):
    for size in SIZES:
        assert program(*size) == (0, 0), size


def test_lanes_past_a_cut_row_would_leave_it(program):
    """The mistake, planted here: without the step back a cut last block reads past the rows' ends."""
    for n, k, pad, tile in SIZES:
        outside, _ = program(n, k, pad, tile, 0)
        assert (outside > 0) == (k % 128 != 0 and (k > 128 or n > 1)), (n, k, pad, tile)
