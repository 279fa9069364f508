"""How many workgroups a launch takes, and how many share the passes of a 4-bit product over a group's rows (host arithmetic,
built by itself)."""

import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

DRIVER = r"""
#include <cstdio>
#include <cstdlib>
#include "launch_size.h"
int main(int argc, char** argv) {
  if (argc == 2) std::printf("%lld\n", (long long)mgs::most_workgroups(std::atoi(argv[1])));
  for (int i = 1; i + 2 < argc; i += 3)
    std::printf("%lld\n", (long long)mgs::shared_passes(std::atoll(argv[i]), std::atoll(argv[i + 1]), std::atoi(argv[i + 2])));
}
"""

# (passes of the fullest group, workgroups of one pass, threads, shared by)
CASES = [
    (1, 1, 512, 1), (7, 100, 256, 7), (16, 100, 256, 16), (1000, 100, 256, 16),
    (16, 131072, 256, 16),                       # 128 experts x 16384 pairs, or 256 x 8192: 2^21 workgroups
    (16, (1 << 20) - 1, 256, 16), (16, 1 << 20, 256, 15), (17, 1 << 20, 256, 15),  # 2^32 threads and just below
    (16, 1 << 21, 256, 7), (3, 1 << 21, 256, 3), (16, 1 << 22, 256, 3), (16, 1 << 22, 128, 7),
    (1, 1 << 23, 256, 1), (16, 1 << 23, 256, 1),  # one pass where the launch takes no more
]


@pytest.fixture(scope="module")
def shared(tmp_path_factory):
    d = tmp_path_factory.mktemp("launch")
    (d / "driver.cpp").write_text(DRIVER)
    exe = str(d / "driver")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", os.path.join(ROOT, "moe_grouped_scaled_amd", "csrc"),
                    str(d / "driver.cpp"), "-o", exe], check=True, timeout=120)

    def run(cases):
        out = subprocess.run([exe] + [str(v) for c in cases for v in c[:3]], check=True, stdout=subprocess.PIPE, text=True, timeout=60)
        return [int(v) for v in out.stdout.split()]

    run.exe = exe
    return run


@pytest.mark.parametrize("threads", [64, 128, 256, 512])
def test_most_workgroups(shared, threads):
    most = int(subprocess.run([shared.exe, str(threads)], check=True, stdout=subprocess.PIPE, text=True, timeout=60).stdout)
    assert most * threads < 1 << 32 <= (most + 1) * threads


def test_shared_passes(shared):
    assert shared(CASES) == [c[3] for c in CASES]


def test_a_launch_stays_below_its_threads(shared):
    cases = [(want, base, threads) for want in (1, 5, 16, 99) for threads in (128, 256, 512)
             for base in (1, 1000, 4097, (1 << 19) + 1, 1 << 20, (1 << 22) - 1, 1 << 22, 1 << 23) if base * threads < 1 << 32]
    for (want, base, threads), got in zip(cases, shared(cases)):
        assert 1 <= got <= min(want, 16) and got * base * threads < 1 << 32
        assert got == min(want, 16) or (got + 1) * base * threads >= 1 << 32
