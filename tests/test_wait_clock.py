"""The bound of the kernels' waits, compiled for the host: a timer that steps back
between two readings does not end a wait."""
import os
import subprocess

import pytest

from key_retention_scoring_b200 import build as tria_build

PROGRAM = r"""
#include <cstdio>
#include "tria_internal.h"
int main() {
  unsigned long long t0, now, limit;
  while (std::scanf("%llu %llu %llu", &t0, &now, &limit) == 3)
    std::printf("%d\n", tria::time_over(t0, now, limit) ? 1 : 0);
}
"""

CASES = [  # first reading, second, limit, over
    (1000, 1000, 1, False), (1000, 1001, 1, False), (1000, 1002, 1, True),
    (1000, 999, 1, False), (1000, 968, 2_000_000_000, False), (1000, 968, 0, False),
    (10 ** 18, 10 ** 18 + 2_000_000_000, 2_000_000_000, False), (10 ** 18, 10 ** 18 + 2_000_000_001, 2_000_000_000, True),
    (10 ** 18, 10 ** 18 - 1, 2 ** 63 - 1, False), (10 ** 18, 3 * 10 ** 18, 2 ** 63 - 1, False),
]


@pytest.fixture(scope="module")
def answers(tmp_path_factory):
    d = tmp_path_factory.mktemp("clock")
    src, exe = d / "clock.cu", d / "clock"
    src.write_text(PROGRAM)
    subprocess.run([tria_build.nvcc(), *tria_build.ARCH, "-std=c++17", "-I", tria_build.INCLUDE, "-I", tria_build.CSRC,
                    "-o", str(exe), str(src)], check=True, capture_output=True)
    text = "".join(f"{a} {b} {n}\n" for a, b, n, _ in CASES)
    return subprocess.run([str(exe)], input=text, check=True, capture_output=True, text=True).stdout.split()


def test_time_over(answers):
    assert answers == ["1" if over else "0" for *_, over in CASES]


def test_every_wait_on_the_global_timer_uses_it():
    for name in os.listdir(tria_build.CSRC):
        text = open(os.path.join(tria_build.CSRC, name)).read()
        assert "global_timer() -" not in text, name
