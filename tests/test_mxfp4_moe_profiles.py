"""The counters committed for the large MXFP4 products: derived figures follow from the raw ones."""
import csv
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def table():
    lines = [line for line in open(os.path.join(ROOT, "profiles", "mxfp4_moe_counters.txt")) if not line.startswith("#")]
    end = next(i for i, line in enumerate(lines) if line.startswith("instruction,"))
    return list(csv.DictReader(lines[:end])), list(csv.DictReader(lines[end:]))


def test_derived_figures():
    products, _ = table()
    assert {r["case"] for r in products} == {"dense", "zeros", "square", "experts"}
    for r in products:
        v = {k: float(x) for k, x in r.items() if k not in ("case", "kernel")}
        cycles = v["sq_busy_cycles"] / 32
        assert v["clock_ghz"] == pytest.approx(cycles / v["run_ns"], abs=6e-4)
        assert v["mfma_busy"] == pytest.approx(v["sq_valu_mfma_busy_cycles"] / 1024 / cycles, abs=6e-4)
        assert v["wait_any"] == pytest.approx(v["sq_wait_any"] / v["sq_wave_cycles"], abs=6e-4)
        assert v["wait_inst"] == pytest.approx(v["sq_wait_inst_any"] / v["sq_wave_cycles"], abs=6e-4)
        # a 32 x 32 x 64 instruction keeps its matrix core busy 32 cycles
        assert v["sq_valu_mfma_busy_cycles"] == pytest.approx(32 * v["sq_insts_mfma"], rel=1e-3)


def test_work_of_the_counted_products():
    products, _ = table()
    by = {}
    for r in products:
        by[r["case"]] = by.get(r["case"], 0) + int(r["sq_insts_mfma"])
    each = 32 * 32 * 64
    assert by["dense"] == by["zeros"] == 2048 * 28672 * 8192 // each and by["square"] == 8192 ** 3 // each
    assert by["experts"] >= 0.98 * 16384 * 2816 * 2048 / each  # and the padding of ragged groups


def test_issue_rates():
    _, issue = table()
    assert [r["workgroups"] for r in issue] == ["256", "256"]  # one wave a SIMD
    for r in issue:
        flops = {"16x16x128": 2 * 16 * 16 * 128, "32x32x64": 2 * 32 * 32 * 64}[r["instruction"]]
        # a SIMD each, so at most flops a SIMD over its cycles at the card's 2.4 GHz
        assert float(r["pflops"]) <= 1.001 * 1024 * flops / float(r["cycles_each"]) * 2.4e9 / 1e15
