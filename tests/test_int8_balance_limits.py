"""Limits of the 8-bit operators whose products of sizes pass 64 bits, at the C ABI.  No kernel is launched here."""
import pytest

import decode_gemm_exl3_amd as ex

A = 1 << 24  # stand-ins for device addresses: no call below reaches the device
F16, F32, EINVAL, EUNSUPPORTED = 0, 2, -1, -2


@pytest.fixture(scope="module")
def lib():
    from decode_gemm_exl3_amd import int8
    for f in (int8._quantize, int8._dequantize, int8._norm):
        f.load()
    return ex.load()


# rows times values: 2^64, 2^64 - 2^44 (negative in 64 bits), 2^63, 2^57
@pytest.mark.parametrize("rows, n", [(1 << 40, 1 << 24), (1 << 40, (1 << 24) - 16), (1 << 40, 1 << 23), (1 << 34, 1 << 23)])
def test_sizes_whose_product_passes_what_there_is(lib, rows, n):
    for dtype in (F16, F32):
        assert lib.exl3_int8_quantize(A, dtype, rows, n, n, 2 * A, 3 * A, None) == EUNSUPPORTED
        assert lib.exl3_int8_dequantize(A, 2 * A, rows, n, 3 * A, dtype, None) == EUNSUPPORTED
        assert lib.exl3_int8_rms_norm(A, dtype, rows, n, n, 2 * A, n, 3 * A, F32, 0.0, 4 * A, 5 * A, 6 * A, None) == EUNSUPPORTED


def test_errors_of_the_arguments_come_first(lib):
    assert lib.exl3_int8_quantize(A, F16, 1 << 40, 1 << 24, 1 << 24, 2 * A + 8, 3 * A, None) == EINVAL
    assert lib.exl3_int8_dequantize(A, 2 * A, 1 << 40, 1 << 24, 3 * A, 7, None) == EINVAL
