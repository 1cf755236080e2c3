"""How the few-rows MXFP4 product is laid out and split: the header that the kernel
is built from, compiled for the host."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "decode_gemm_exl3_amd", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <initializer_list>
#include "mxfp4_plan.hpp"
using namespace exl3::mx;
static_assert(spans_of(2147483616) == 4194304 && held_rows(2147483616, 64) == 0, "no sum past 32 bits");
int main() {
    for (int held : {0, HELD_SPANS, MORE_HELD_SPANS})
        for (int whole : {0, 1}) printf("lds %d %d %d %d\n", held, whole, small_slots(held, whole) * 16, small_per_cu(held, whole));
    const int inputs[] = {32, 96, 512, 1056, 2048, 2080, 4096, 4128, 8192, 8224, 14336, 16384};
    const int outputs[] = {1, 16, 40, 1001, 2816, 4096, 4097, 8192, 14336, 28672, 100000};
    const int tiles[] = {1, 2, 7, 64, 300};
    for (int n_in : inputs) for (int n_out : outputs) for (int t : tiles) for (int held : {0, HELD_SPANS, MORE_HELD_SPANS})
        printf("split %d %d %d %d %d %d\n", n_in, n_out, t, held, small_split(n_out, t, n_in, held), held ? held_rows(n_in, held) : 16);
}
"""


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    compiler = shutil.which("g++") or shutil.which("clang++")
    if compiler is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(PROGRAM)
    subprocess.run([compiler, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(d / "plan.cpp"), "-o", str(d / "plan")], check=True)
    lines = subprocess.run([str(d / "plan")], capture_output=True, text=True, check=True).stdout.split("\n")
    rows = [line.split() for line in lines if line]
    return [tuple(map(int, r[1:])) for r in rows if r[0] == "lds"], [tuple(map(int, r[1:])) for r in rows if r[0] == "split"]


def test_workgroups_of_a_cu(plan):
    per_cu = {(held, whole): n for held, whole, _, n in plan[0]}
    for held, whole, nbytes, n in plan[0]:
        assert 1 <= n and n * nbytes <= 160 * 1024
    # whatever the input's length
    assert per_cu[32, 0] == per_cu[32, 1] == 2


def test_a_split_fits_one_round(plan):
    per_cu = {(held, whole): n for held, whole, _, n in plan[0]}
    for n_in, n_out, tiles, held, split, _ in plan[1]:
        assert split in (1, 2, 4, 8)
        runs, places = -(-n_out // 16), 256 * per_cu[held, int(n_in % 128 == 0)]
        # the runs' waves, counted as waves: workgroups of the last outputs may be partly empty
        assert split == 1 or runs * tiles * split <= 8 * places, (n_in, n_out, tiles, held, split)
        assert split == 1 or split // 2 < -(-n_in // 512)


def test_held_rows_fit(plan):
    for n_in, _, _, held, _, rows in plan[1]:
        assert rows <= 16 and (held == 0 or rows * -(-n_in // 512) <= held)
