"""MXFP4 and expert operators on the GPU: calls at the edge of what they allow."""
import numpy as np
import pytest
import torch

import _mxfp4_ref as R

pytestmark = pytest.mark.gpu
DTYPES = R.DTYPES


@pytest.fixture(scope="module")
def ex():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import decode_gemm_exl3_amd as ex
    ex.load()
    return ex


def dev(a):
    return (torch.from_numpy(a) if isinstance(a, np.ndarray) else a).cuda()


@pytest.mark.parametrize("dtype", DTYPES)
def test_results_between_the_rows_of_an_input(ex, dtype):
    """Rows of a wider buffer whose rest holds the results: no byte is shared."""
    rng = np.random.default_rng(1)
    m, n_in, n_out, dt = 3, 64, 48, DTYPES[dtype]
    x = R.rows(rng, m, n_in, dt)
    codes, scales = R.weight(rng, n_out, n_in)
    buf = torch.full((m, n_in + 160), 7.0, dtype=dt, device="cuda")
    buf[:, :n_in] = x.cuda()
    y = buf.view(-1)[n_in:n_in + m * n_out].view(m, n_out)
    ex.mxfp4_linear(buf[:, :n_in], dev(codes), dev(scales), y=y)
    R.assert_product(y, R.dequantize(*R.quantize(x)), R.dequantize(codes, scales), dt)
    assert torch.equal(buf[:, :n_in].cpu(), x) and (buf[1:, n_in:] == 7).all() and (buf[0, n_in + m * n_out:] == 7).all()
