"""Which kernel makes a product of 8-bit rows: the header that the launches are chosen by, compiled for the host."""
import os
import shutil
import subprocess

import pytest

import _int8_cases as C

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "decode_gemm_exl3_amd", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "int8_plan.hpp"
using namespace exl3::i8;
static_assert(choose_product(ProductShape{false, 1 << 23, 1, 16, 1 << 12}).kernel == LARGE_256, "no sum past 32 bits");
const char* name(ProductKernel k) {
    switch (k) {
        case SMALL_STAGED: return "SMALL_STAGED";
        case SMALL_STREAMED: return "SMALL_STREAMED";
        case STRIP_16: return "STRIP_16";
        case STRIP_32: return "STRIP_32";
        case STRIP_64: return "STRIP_64";
        case MEDIUM_LONG: return "MEDIUM_LONG";
        case MEDIUM_SHORT: return "MEDIUM_SHORT";
        case MIDDLE: return "MIDDLE";
        case LARGE_128: return "LARGE_128";
        case LARGE_256: return "LARGE_256";
        case LARGE_BOTH: return "LARGE_BOTH";
    }
    return "";
}
int main() {
    int grouped, rows, groups, n_in, n_out;
    while (std::scanf("%d %d %d %d %d", &grouped, &rows, &groups, &n_in, &n_out) == 5) {
        const ProductChoice c = choose_product(ProductShape{grouped != 0, rows, groups, n_in, n_out});
        std::printf("%s %d\n", name(c.kernel), c.cols);
    }
}
"""


@pytest.fixture(scope="module")
def choose(tmp_path_factory):
    compiler = shutil.which("g++") or shutil.which("clang++")
    if compiler is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("plan")
    (d / "plan.cpp").write_text(PROGRAM)
    subprocess.run([compiler, "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(d / "plan.cpp"), "-o", str(d / "plan")], check=True)

    def run(shapes):
        text = "\n".join(" ".join(map(str, s)) for s in shapes)
        out = subprocess.run([str(d / "plan")], input=text, capture_output=True, text=True, check=True).stdout.split("\n")
        return [(line.split()[0], int(line.split()[1])) for line in out if line]
    return run


def test_the_grouped_cases_of_the_gpu_tests_reach_their_kernels(choose):
    cases = [(kernel, c) for kernel, cs in C.GROUPED.items() for c in cs]
    got = choose([(1, rows, groups, n_in, n_out) for _, (groups, rows, _, n_in, n_out, _) in cases])
    assert [(k, c) for (k, _), (_, c) in zip(got, cases)] == cases


def test_the_long_cases_of_the_gpu_tests_reach_their_kernels(choose):
    got = choose([(0, m, 1, C.LONGEST, n_out) for m, n_out in C.LONG.values()])
    assert [k for k, _ in got] == list(C.LONG)
    cols = got[list(C.LONG).index("LARGE_BOTH")][1]
    assert 0 < cols < C.LONG["LARGE_BOTH"][1] and cols % 256 == 0


def test_every_number_of_kept_groups_is_covered(choose):
    """Both sides of 64 and 128 groups, and of 256 offsets, in each tile that looks for groups in that way."""
    for kernel in ("MEDIUM_SHORT", "MIDDLE", "LARGE_128", "LARGE_256"):
        groups = {c[0] for c in C.GROUPED[kernel]}
        assert {64, 127, 128, 300} <= groups and any(g < 128 and c[2] for c in C.GROUPED[kernel] for g in [c[0]])
    for cs in C.GROUPED.values():
        for groups, rows, behind, *_ in cs:
            counts = C.uneven(groups, rows - behind, 0)
            assert sum(counts) == rows - behind and counts[0] and counts[-1] and (groups < 8 or 0 in counts)
