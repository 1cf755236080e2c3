"""The figures committed for the 8-bit products and the balance loss: derived ones follow from the raw ones."""
import csv
import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def lines(name):
    return [line for line in open(os.path.join(ROOT, "profiles", name)) if not line.startswith("#")]


def table():
    rows = lines("int8_balance_counters.txt")
    end = next(i for i, line in enumerate(rows) if line.startswith("instruction,"))
    return list(csv.DictReader(rows[:end])), list(csv.DictReader(rows[end:]))


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
        # a 16 x 16 x 64 instruction keeps its matrix core busy 16 cycles
        assert v["sq_valu_mfma_busy_cycles"] == pytest.approx(16 * v["sq_insts_mfma"], rel=1e-3)


def test_work_of_the_counted_products():
    products, _ = table()
    by = {}
    for r in products:
        by[r["case"]] = by.get(r["case"], 0) + int(r["sq_insts_mfma"])
    each = 16 * 16 * 64
    assert by["dense"] == by["zeros"] == 2048 * 28672 * 8192 // each and by["square"] == 8192 ** 3 // each
    assert by["experts"] >= 16384 * 2816 * 2048 / each  # and the padding of ragged groups


def test_issue_rates():
    _, issue = table()
    assert [(r["instruction"], r["waves_a_cu"]) for r in issue] == [
        ("16x16x64", "4"), ("16x16x64", "8"), ("32x32x32", "4"), ("32x32x32", "8")]
    for r in issue:  # both make 2048 operations a cycle and SIMD, at the card's 2.4 GHz at most
        assert 3.0 < float(r["pops"]) <= 1024 * 2048 * 2.4e9 / 1e15


def test_every_measured_case_has_its_kernels():
    spec = importlib.util.spec_from_file_location("more_operators", os.path.join(ROOT, "perf", "more_operators.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    rows = list(csv.DictReader(lines("int8_balance_kernel_stats.txt")))
    cases = list(dict.fromkeys(r["case"] for r in rows))
    assert cases == [c["name"] for c in module.listed()]
    sources = "".join(open(os.path.join(ROOT, "decode_gemm_exl3_amd", "csrc", f)).read() for f in ("int8.hip", "int8_rows.hip", "balance.hip"))
    for r in rows:
        assert f"void {r['kernel'].split('<')[0]}(" in sources
        assert int(r["calls"]) == 33 and int(r["min_ns"]) <= int(r["median_ns"]) <= int(r["max_ns"])
