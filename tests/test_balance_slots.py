"""Which of a token's slots each lane reads: the header that the balance kernels are built
from, compiled for the host."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "decode_gemm_exl3_amd", "csrc")

# Walks a lane's slots; the end of the program with 1 at a slot that the token does not have.
PROGRAM = r"""
#include <cstdio>
#include <cstdlib>
#include <initializer_list>
#include "slots.hpp"
template <int LANES> void lane_of(int top_k, int lane) {
    int64_t next = lane, reads = 0, taken = 0;
    exl3::lane_slots<LANES>(top_k, lane, lane < top_k ? lane : -1, [&](int64_t j) {
        next += LANES;
        if (j != next || j >= top_k) {
            printf("top_k %d, lane %d of %d: slot %lld after %lld reads\n", top_k, lane, LANES, (long long)j, (long long)reads);
            exit(1);
        }
        ++reads;
        return j;
    }, [&](int64_t id) { taken += id >= 0; });
    const int64_t want = lane < top_k ? ((int64_t)top_k - lane + LANES - 1) / LANES : 0;
    if (taken != want || reads != (want > 0 ? want - 1 : 0)) {
        printf("top_k %d, lane %d of %d: %lld slots, not %lld\n", top_k, lane, LANES, (long long)taken, (long long)want);
        exit(1);
    }
}
template <int LANES> void all(int top_k) {
    for (int lane = 0; lane < LANES; ++lane) lane_of<LANES>(top_k, lane);
}
int main() {
    for (int k = 0; k < 200; ++k) {
        all<1>(k); all<2>(k); all<4>(k); all<8>(k); all<16>(k); all<32>(k); all<64>(k);
    }
    // the last numbers of slots that 32 bits hold: a lane's next slot would pass them
    for (int back : {0, 1, 31, 62, 63, 64}) {
        for (int lane : {0, 1, 62, 63}) lane_of<64>(0x7FFFFFFF - back, lane);
        lane_of<32>(0x7FFFFFFF - back, 31);
    }
}
"""


def test_every_slot_once_and_none_behind_the_last(tmp_path):
    compiler = shutil.which("g++") or shutil.which("clang++")
    if compiler is None:
        pytest.skip("no host compiler")
    (tmp_path / "slots.cpp").write_text(PROGRAM)
    # -fwrapv: a sum past 32 bits wraps, as it does on the GPU
    subprocess.run([compiler, "-std=c++17", "-O1", "-fwrapv", "-Wall", "-Werror", "-I", CSRC, str(tmp_path / "slots.cpp"), "-o", str(tmp_path / "slots")],
                   check=True)
    run = subprocess.run([str(tmp_path / "slots")], capture_output=True, text=True, timeout=100)
    assert run.returncode == 0, run.stdout
