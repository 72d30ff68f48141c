"""GPU: the norm of rows whose squares leave the fp32 range below, with no eps (or next to none) to
hide it.  Bounds as in test_fp8_gpu.check_norm; a product r * weight below 2^-126 is off by 2^-150 at
most, which the statistic scales like the row."""
import numpy as np
import pytest

from tests import fp8_ref as R
from tests.test_fp8_gpu import bytes_of, host, norm_case

torch = pytest.importorskip("torch")
import ternary_quantized_moe_b200 as tq  # noqa: E402

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def run(x, r, w, eps):
    T, d = x.shape
    y = torch.empty((T, d), dtype=BF16, device="cuda")
    codes = torch.empty((T, d), dtype=torch.uint8, device="cuda")
    scales = torch.empty((T, -(-d // 128)), dtype=torch.uint8, device="cuda")
    tq.scion_rmsnorm_forward(x.to("cuda"), T, w.to("cuda"), eps, resid=None if r is None else r.to("cuda"), y=y,
                             y_codes=codes, y_scales=scales)
    return y, codes, scales


@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-40, 1e-30, 1e-20])
@pytest.mark.parametrize("d", [272, 2048, 8192, 16400])
@pytest.mark.parametrize("size", [1e-8, 1e-10, 1e-18, 1e-20, 1e-22, 1e-24, 1e-30, 1e-37, 1e-40])
def test_rows_whose_squares_underflow(d, size, eps):
    x, _, w = norm_case(3, d, F32, None)
    x = (x.double() * size).float()
    x[1, ::3] = 0
    x[2, 1:] = 0  # one element alone
    eps = float(np.float32(eps))  # (what the argument, an fp32, holds: 1e-45 is 1.4e-45)
    _, ry = R.rmsnorm(host(x), None, host(w), eps)
    rms = np.sqrt((host(x) ** 2).mean(1, keepdims=True) + eps)
    y, codes, scales = run(x, None, w, eps)
    err = np.abs(ry) * ((d + 4) / 2 + 9) * 2.0 ** -24 + 2.0 ** -150 * (1 + 1.01 / rms)
    err[host(x) == 0] = 0  # (0 w rms is 0 exactly, and a block of zeros has byte 127)
    # (a bf16 below 2^-126 is off by 2^-134 at most)
    assert (np.abs(host(y) - ry) <= np.abs(ry) * 2.0 ** -8 + 2.0 ** -134 + 2 * err).all()
    R.check_codes(bytes_of(codes), bytes_of(scales), ry, err)


@pytest.mark.parametrize("d", [272, 2048])
def test_zero_rows_without_eps_are_nan(d):
    """0 / 0, all of the row alike, and no effect on the rows beside it; with any eps they are zero."""
    x, _, w = norm_case(3, d, F32, None)
    x[1] = 0
    y, codes, scales = run(x, -x, w, 0.0)  # r = 0 everywhere
    assert torch.isnan(y).all() and (scales == 255).all() and (codes & 0x7F == 0x7F).all()
    y, codes, scales = run(x, None, w, 0.0)
    assert torch.isnan(y[1]).all() and (scales[1] == 255).all() and torch.isfinite(y[[0, 2]]).all()
    for eps in (1e-45, 1e-38, 1e-6):
        y, codes, scales = run(x, None, w, eps)
        assert (y[1] == 0).all() and (codes[1] & 0x7F == 0).all() and (scales[1] == 127).all()
