"""The committed times of the 8-bit products' kernels say which of them the launch takes, and it is what it takes; derived counters."""
import csv
import os

from test_int8_plan import choose  # noqa: F401  (a fixture)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NAMES = {"SMALL_STAGED": "small staged", "SMALL_STREAMED": "small streamed", "STRIP_16": "strip 32x16", "STRIP_32": "strip 32x32", "STRIP_64": "strip 32x64",
         "MEDIUM_LONG": "64x64 long", "MEDIUM_SHORT": "64x64 short", "MIDDLE": "128x128", "LARGE_128": "128x256", "LARGE_256": "256x256",
         "LARGE_BOTH": "256x256 and 128x256"}


def test_the_chosen_kernels(choose):  # noqa: F811
    lines = [line for line in open(os.path.join(ROOT, "profiles", "int8_product_rules.txt")) if not line.startswith("#")]
    by = {}
    for r in csv.DictReader(lines):
        shape = tuple(int(r[k]) for k in ("groups", "rows", "n_in", "n_out"))
        by.setdefault(shape, {})[r["kernel"]] = (float(r["us"]), r["chosen"] == "1")
    shapes = list(by)
    got = choose([(int(g > 0), m, max(g, 1), n_in, n_out) for g, m, n_in, n_out in shapes])
    for shape, (kernel, _) in zip(shapes, got):
        assert [k for k, (_, chosen) in by[shape].items() if chosen] == [NAMES[kernel]], shape
        assert len(by[shape]) > 1 and all(us > 0 for us, _ in by[shape].values())


def test_the_balance_counters():
    rows = list(csv.DictReader(line for line in open(os.path.join(ROOT, "profiles", "balance_counters.txt")) if not line.startswith("#")))
    assert [r["kernel"].split("<")[0] for r in rows] == ["sum_kernel", "loss_kernel", "backward_kernel"]
    for r in rows:
        v = {k: float(x) for k, x in r.items() if k != "kernel"}
        cycles = v["sq_busy_cycles"] / 32
        assert abs(v["clock_ghz"] - cycles / v["run_ns"]) < 6e-4 and abs(v["wait_any"] - v["sq_wait_any"] / v["sq_wave_cycles"]) < 6e-4
        assert abs(v["valu_busy"] - 4 * v["sq_active_inst_valu"] / 1024 / cycles) < 6e-4 and v["sq_active_inst_valu"] >= v["sq_insts_valu"]
