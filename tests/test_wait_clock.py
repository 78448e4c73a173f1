"""The clock of the tensor-core kernels' bounded waits, on the host (not gpu)."""

import os
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "zero_sharded_mixed_flatparameter_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "zero_wait.h"
using namespace zfs;
// polls `step` ns apart, from a time near the counter's end, until the wait is spent: polls, -1 if it never is
static long long polls(unsigned long long step, long long most) {
  unsigned long long now = ~0ull - 5 * kWaitNs;
  Patience p(now);
  for (long long i = 1; i <= most; ++i)
    if (p.spent(now += step)) return i;
  return -1;
}
int main() {
  std::printf("%lld %lld\n", polls(1000, 10000000), polls(5000000, 10000));   // running: a second of polls
  // off the GPU for two seconds once, then running: the two seconds do not count
  Patience p(0);
  unsigned long long now = 1000;
  int early = p.spent(now);
  early |= p.spent(now += 2000000000ull);
  long long i = 0;
  while (!p.spent(now += 1000)) ++i;
  std::printf("%d %lld\n", early, i);
  std::printf("%lld\n", polls(20000000, 100000));                             // every poll late: it ends all the same
}
"""


@pytest.fixture(scope="module")
def figures(tmp_path_factory):
    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    where = tmp_path_factory.mktemp("wait")
    (where / "main.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-I" + CSRC, str(where / "main.cpp"), "-o", str(where / "main")], check=True)
    return [int(x) for x in subprocess.run([str(where / "main")], capture_output=True, text=True, check=True,
                                           timeout=60).stdout.split()]


def test_a_running_wait_ends_after_a_second(figures):
    assert figures[0] == 1_000_001 and figures[1] == 201


def test_time_off_the_gpu_does_not_count(figures):
    assert figures[2] == 0 and 990_000 <= figures[3] <= 1_000_001


def test_every_wait_ends(figures):
    assert 1000 < figures[4] <= 1100
