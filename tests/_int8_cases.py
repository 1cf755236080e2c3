"""Sizes of 8-bit products by the kernel that choose_product (csrc/int8_plan.hpp) takes for them: the CPU tests
check the choice, the GPU tests the products."""
import numpy as np

# groups, rows (those behind the last group among them), rows behind, n_in, n_out, dtype.  The tiles' search keeps 128
# groups in two registers (the rows behind the last are one more), or reads 256 offsets at a time.
GROUPED = {
    "STRIP_16": [(3, 140, 2, 144, 500, "fp32")],
    "STRIP_32": [(70, 2000, 0, 80, 50, "bf16")],
    "STRIP_64": [(20, 400, 5, 144, 520, "fp16")],
    "MEDIUM_LONG": [(63, 63 * 20, 4, 144, 300, "bf16")],
    "MEDIUM_SHORT": [(64, 64 * 20, 9, 144, 1101, "bf16"), (100, 100 * 25, 0, 272, 603, "fp32"), (127, 127 * 18, 1, 112, 700, "fp16"),
                     (128, 128 * 31, 40, 128, 517, "bf16"), (255, 255 * 17, 3, 64, 300, "fp16"), (256, 256 * 17, 0, 48, 301, "bf16"),
                     (300, 300 * 20, 70, 144, 330, "fp16"), (1030, 1030 * 18, 2, 32, 130, "bf16")],
    "MIDDLE": [(63, 63 * 100, 20, 144, 299, "bf16"), (64, 64 * 100, 130, 272, 1100, "fp16"), (100, 100 * 40, 0, 80, 1101, "fp32"),
               (127, 127 * 70, 1, 128, 300, "bf16"), (128, 128 * 70, 5, 144, 301, "fp16"), (300, 300 * 70, 200, 48, 300, "bf16"),
               (1030, 1030 * 36, 9, 16, 150, "fp16")],
    "LARGE_128": [(63, 63 * 40, 3, 144, 2500, "bf16"), (64, 64 * 40, 90, 400, 6001, "fp16"), (100, 100 * 70, 0, 144, 2500, "fp32"),
                  (127, 127 * 40, 200, 272, 2500, "bf16"), (128, 128 * 40, 1, 128, 2499, "fp16"), (300, 300 * 40, 500, 80, 1101, "bf16"),
                  (1030, 1030 * 34, 4, 16, 700, "bf16")],
    "LARGE_256": [(63, 63 * 70, 100, 144, 2500, "fp16"), (64, 64 * 70, 0, 272, 1100, "bf16"), (100, 100 * 100, 7, 80, 1101, "fp32"),
                  (127, 127 * 70, 300, 144, 1100, "bf16"), (128, 128 * 70, 1, 400, 1099, "fp16"), (300, 300 * 100, 50, 32, 2500, "bf16")],
}

# rows, outputs of one weight; with the longest inputs there are
LONG = {"SMALL_STREAMED": (20, 200), "STRIP_16": (100, 600), "STRIP_32": (100, 1500), "STRIP_64": (100, 3001), "MEDIUM_LONG": (250, 4090),
        "MEDIUM_SHORT": (450, 4090), "MIDDLE": (770, 4090), "LARGE_128": (2040, 4090), "LARGE_256": (1000, 28672), "LARGE_BOTH": (2048, 28672)}
LONGEST = (1 << 17) - 16


def uneven(groups, rows, seed):
    """Counts of `groups` groups, a quarter of them empty, some an order of magnitude larger than others; `rows` in all, and
    some of them in the first and the last group."""
    rng = np.random.default_rng([31, groups, rows, seed])
    weight = np.exp2(rng.uniform(-2, 2, groups)) * (rng.random(groups) > 0.25)
    weight[[0, -1]] = 1.0
    counts = rng.multinomial(rows - 2, weight / weight.sum())
    counts[0] += 1
    counts[-1] += 1
    return [int(c) for c in counts]


# Few rows whose outputs are too many for one strip a CU: rows, n_in, n_out, dtype of one weight; and of groups as above
FEW = {"STRIP_32": [(5, 4112, 20001, "bf16"), (16, 4096, 34001, "fp16"), (11, 4096, 16500, "fp32")],
       "MEDIUM_SHORT": [(9, 2064, 28673, "bf16"), (30, 4096, 20001, "fp16")]}
FEW_GROUPED = {"STRIP_32": [(8, 13, 2, 8208, 4100, "bf16"), (8, 60, 0, 8192, 6001, "fp16"), (40, 300, 30, 8208, 1050, "fp32")],
               "MEDIUM_SHORT": [(8, 100, 3, 8192, 4100, "bf16"), (20, 150, 1, 8176, 1500, "fp16")]}
