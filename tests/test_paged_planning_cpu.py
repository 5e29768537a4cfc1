"""The closed form of the attention's planning step, compiled for the host, against a plain sum."""
import os
import random
import subprocess

from gated_deltanet_02_gb300 import build as B

SRC = """
#include <stdio.h>
#include "paged_sched.cuh"
int main() {
  unsigned n, a, b;
  while (scanf("%u %u %u", &n, &a, &b) == 3) printf("%lld\\n", glinattn::paged::tiles_sum(n, a, b));
  return 0;
}
"""


def test_sum_of_cache_tiles(tmp_path):
    src, exe = tmp_path / "sum.cu", tmp_path / "sum"
    src.write_text(SRC)
    subprocess.run([B.nvcc(), *B.ARCH, "-std=c++17", "-I", B.INCLUDE, "-I", B.CSRC, str(src), "-o", str(exe)], check=True)
    rng = random.Random(1)
    cases = [(n, a, b) for n in (1, 2, 3, 4, 5, 31, 127, 128, 129, 255) for a in range(1, 257) for b in (0, 1, 127, 128, 300)]
    cases += [(rng.randrange(1, 5000), rng.randrange(1, 257), rng.randrange(1 << 31)) for _ in range(500)]
    cases += [((1 << 24) - 1, a, (1 << 31) - 1) for a in (1, 85, 127, 128, 255, 256)]
    got = subprocess.run([str(exe)], input="\n".join("%d %d %d" % c for c in cases), capture_output=True, text=True, check=True)

    def plain(n, a, b):      # 128 terms a further 128 a on add a whole number to each
        head = [(a * i + b) // 128 for i in range(min(n, 128))]
        rounds, rest = divmod(n, 128)
        total = rounds * sum(head) + 128 * a * (rounds * (rounds - 1) // 2) if rounds else 0
        return total + sum(head[:rest]) + rest * a * rounds

    want = [plain(*c) if c[0] > 5000 else sum((c[1] * i + c[2]) // 128 for i in range(c[0])) for c in cases]
    assert [int(x) for x in got.stdout.split()] == want
