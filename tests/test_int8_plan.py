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


# Sizes at which both sides were timed: few rows of long inputs against tiles for rows that are not there, and where those are as fast
@pytest.mark.parametrize("shape, kernel", [
    ((0, 16, 1, 4096, 128256), "STRIP_32"), ((0, 16, 1, 4096, 40000), "STRIP_32"), ((0, 2, 1, 20480, 20480), "STRIP_32"),
    ((0, 5, 1, 8192, 28672), "STRIP_32"), ((1, 12, 8, 14336, 4096), "STRIP_32"), ((1, 16, 8, 14336, 4096), "STRIP_32"),
    ((1, 32, 8, 14336, 4096), "STRIP_32"), ((1, 64, 8, 14336, 4096), "STRIP_32"),
    ((1, 200, 16, 8192, 4096), "MEDIUM_SHORT"), ((1, 128, 8, 4096, 14336), "MEDIUM_SHORT"),
    ((1, 256, 8, 4096, 14336), "MEDIUM_SHORT"), ((1, 384, 64, 2816, 2048), "MEDIUM_SHORT"), ((1, 1024, 128, 1024, 1024), "SMALL_STAGED"),
    ((0, 16, 1, 2048, 28672), "MEDIUM_SHORT"), ((0, 13, 1, 14336, 4096), "SMALL_STREAMED"), ((1, 6, 8, 14336, 4096), "STRIP_64"),
    ((0, 32, 1, 8192, 28672), "MEDIUM_SHORT"), ((0, 13, 1, 4096, 6144), "STRIP_32")])
def test_few_rows(choose, shape, kernel):
    assert choose([shape])[0][0] == kernel


def test_few_rows_of_the_gpu_tests_reach_their_kernels(choose):
    cases = [(k, c) for k, cs in C.FEW.items() for c in cs]
    assert [(k, c) for (k, _), (_, c) in zip(choose([(0, m, 1, n_in, n_out) for _, (m, n_in, n_out, _) in cases]), cases)] == cases
    cases = [(k, c) for k, cs in C.FEW_GROUPED.items() for c in cs]
    assert [(k, c) for (k, _), (_, c) in zip(choose([(1, m, g, n_in, n_out) for _, (g, m, _, n_in, n_out, _) in cases]), cases)] == cases


def test_strips_of_few_rows_fit_a_launch(choose):
    """2^24 workgroups of 256 threads are a launch's end: the largest sizes that the entry points take."""
    for shape in ((0, 16, 1, 4096, 1 << 24), (1, 4096, 4096, 4096, 1 << 17), (1, 16 * 4096, 4096, 4096, 1 << 17)):
        kernel, _ = choose([shape])[0]
        _, rows, groups, _, n_out = shape
        assert kernel != "STRIP_32" or (rows // 32 + groups + 1) * -(-n_out // 32) + 127 < 1 << 24, shape
