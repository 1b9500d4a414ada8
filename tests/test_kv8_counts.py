"""The 8-bit cache's counts of work at sizes that no test attends over: the
kernels' own host/device functions, compiled for the host, against whole
numbers (no GPU)."""
import subprocess

import pytest

from compressed_sparse_attention_topk_b200 import build as csa2_build

PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include "kv8_steps.cuh"
using namespace csa2::kv8;

template <int SLOTS>
int ring(long long n) {  // use n of a ring against its 64-bit count
  return ring_slot<SLOTS>((uint32_t)n) == n % SLOTS &&
         ring_parity<SLOTS>((uint32_t)n) == (uint32_t)(n / SLOTS & 1);
}

int main(int argc, char **argv) {
  if (argc == 2) {  // uses of a ring of any size, in tiles of so many
    const int used = atoi(argv[1]);
    long long n = 0;
    for (int slots = 2; slots <= 6; ++slots) {
      int base = 0;
      for (n = 0; n < (5ll << 31); n += used, base = ring_after(base, used, slots))
        if (base < 0 || base >= 2 * slots || base % slots != n % slots ||
            (base / slots & 1) != (n / slots & 1))
          return 1;
    }
    for (n = -3; n <= 3; ++n)
      for (long long at : {4ll, 1ll << 31, 1ll << 32, 3ll << 32})
        if (!ring<4>(at + n) || !ring<8>(at + n)) return 1;
    return 0;
  }
  // T pos0 G reach: a sequence's steps (the sum over a warp's lanes), the last tile's
  const long long T = atoll(argv[1]), pos0 = atoll(argv[2]), G = atoll(argv[3]);
  ChunkSeq s{};
  s.T = (int)T;
  s.pos0 = (int)pos0;
  s.tiles = (int)((T * G + kChunkRows - 1) / kChunkRows);
  s.reach = (int)atoll(argv[4]);
  auto sum = chunk_steps_of(s, (int)G, 0, 32);
  for (int lane = 1; lane < 32; ++lane) sum += chunk_steps_of(s, (int)G, lane, 32);
  printf("%lld %lld\n", (long long)sum, (long long)chunk_steps(s, (int)G, s.tiles - 1));
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    at = tmp_path_factory.mktemp("kv8_counts")
    src, exe = at / "counts.cu", at / "counts"
    src.write_text(PROGRAM)
    subprocess.run([csa2_build.NVCC, "-O2", "-std=c++17", "-I", csa2_build.CSRC, "-I",
                    csa2_build.INCLUDE, "-o", str(exe), str(src)], check=True)

    def run(*args):
        out = subprocess.run([str(exe), *map(str, args)], check=True, capture_output=True,
                             text=True, timeout=120).stdout
        return [int(x) for x in out.split()]

    return run


def steps(T, pos0, G, reach):
    """Per tile of 256 rows (row = token * G + head), the 64-key steps up to its
    last row's position; their sum and the last tile's."""
    total = last = 0
    for end in range(256, T * G + 256, 256):
        at = min(pos0 + (min(end, T * G) - 1) // G, reach - 1)
        last = 1 if at < 0 else at // 64 + 1
        total += last
    return [total, last]


@pytest.mark.parametrize("T,pos0,G,reach", [
    (1, 0, 1, 64), (300, -20, 4, 1 << 14), (2048, 14336, 4, 1 << 14), (77, 166758, 8, 1 << 18),
    (1 << 20, 0, 64, 1 << 20), (1 << 20, 0, 128, 1 << 20), (1 << 21, 0, 16, 1 << 21),
    (1 << 17, (1 << 30) - (1 << 17), 32, 1 << 30), (1 << 20, 0, 128, 1 << 16)])
def test_steps_of_a_sequence(program, T, pos0, G, reach):
    assert program(T, pos0, G, reach) == steps(T, pos0, G, reach)


def test_rows_that_end_at_the_limit_of_32_bits(program):
    """n * H just below 2^31: the last tile's end is row 2^31."""
    T = (1 << 24) - 1
    total, last = program(T, 0, 128, 1 << 24)
    assert last == (T - 1) // 64 + 1
    # two tokens to a tile, 32 tiles to a step count (the last tile: one token)
    assert total == sum(32 * k for k in range(1, last + 1))


@pytest.mark.parametrize("used", [1 << 25, (1 << 25) - 1, 1000003])
def test_rings_used_more_than_2_to_the_32_times(program, used):
    """Slot and phase of every use follow the 64-bit count."""
    assert program(used) == []
