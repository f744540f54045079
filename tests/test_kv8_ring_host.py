"""The 8-bit attention's ring of stages, host side: which units a producer
waits for before its CTA ends.  A copy that is still in flight then would land
in another CTA's shared memory, so every stage's last copy has to be among
them wherever the producer stopped, at the end of its units or after a wait
that gave up halfway."""
import os
import shutil
import subprocess

import pytest

from sparse_long_context_02_b200 import build as dsa_build

SOURCE = """
#include <cstdio>
#include "kv8.cuh"
template <int S, int P> void show() {
    for (int issued = -1; issued < 40; ++issued) {
        std::printf("%d %d %d:", S, P, issued);
        dsa::kv8::drain<S, P>(issued, [](int j) { std::printf(" %d", j); });
        std::printf("\\n");
    }
}
int main() {
    show<6, 3>();
    show<8, 4>();
    show<16, 4>();
    show<4, 1>();
}
"""


@pytest.fixture(scope="module")
def lines(tmp_path_factory):
    if shutil.which(dsa_build.nvcc()) is None:
        pytest.skip("no nvcc")
    at = tmp_path_factory.mktemp("ring")
    src, exe = at / "ring.cu", at / "ring"
    src.write_text(SOURCE)
    subprocess.check_call([dsa_build.nvcc(), "-gencode", "arch=compute_100a,code=sm_100a",
                           "-std=c++17", "-O0", "-I", dsa_build.CSRC, "-o", str(exe), str(src)])
    return subprocess.check_output([str(exe)], text=True).splitlines()


def test_a_producer_waits_for_every_copy_in_flight(lines):
    assert len(lines) == 4 * 41
    for line in lines:
        head, _, tail = line.partition(":")
        stages, producers, issued = map(int, head.split())
        last = {}  # stage -> the producer's newest unit there
        for j in range(issued % producers if issued >= 0 else 0, issued + 1, producers):
            last[j % stages] = j
        assert sorted(map(int, tail.split())) == sorted(last.values()), line


def test_the_kernel_leaves_through_it():
    code = open(os.path.join(dsa_build.CSRC, "kv8.cuh")).read()
    assert code.count("drain<C::STAGES, C::PRODUCERS>(issued,") == 1
