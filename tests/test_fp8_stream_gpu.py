"""GPU: shapes of the streaming product that the layers of test_fp8_gpu.py do not reach (bounds as there)."""
import numpy as np
import pytest

from tests import fp8_ref as R
from tests.test_fp8_gpu import Case, bytes_of, dev_codes, dev_scales, gated_reference, host

torch = pytest.importorskip("torch")
import ternary_quantized_moe_b200 as tq  # noqa: E402

pytestmark = pytest.mark.gpu


def repeated(T, K, N):
    """A case of 128 outputs, its layer's rows repeated to N, and the result of all of them."""
    c = Case(T, K, 128)
    codes = dev_codes(c.w[0][0]).view(torch.uint8).repeat(N // 128, 1)
    scales = dev_scales(c.w[0][1]).view(torch.uint8).repeat(N // 128, 1)
    layer = tq.scion_fp8_create(codes, scales)
    out = torch.full((T + 1, N), 7.0, device="cuda")
    tq.scion_fp8_forward(c.dx, c.dsx, T, layer, out[:T])
    assert tq.scion_fp8_check(layer) == 0 and (out[T] == 7).all()
    return c, out[:T].view(T, N // 128, 128)


@pytest.mark.parametrize("T", [70, 96, 112, 128])
def test_more_tiles_of_many_tokens_than_sms(T):
    """160 and 256 tiles of weights with tiles of 80 to 128 tokens: a ring that is used many times over, with
    two CTAs per SM where two fit and one where they would have one stage each."""
    for K, N in ((8192, 20480), (8208, 32768)):
        c, out = repeated(T, K, N)
        c.check(out[:, 0])
        assert (out == out[:, :1]).all()


@pytest.mark.parametrize("T", [1, 7, 8, 9, 16])
@pytest.mark.parametrize("K,N", [(528, 20480), (144, 37888), (1024, 32768)])
def test_few_tokens_and_many_short_rows(T, K, N):
    """Layers of more rows than two rounds of the mma.sync kernel's CTAs hold."""
    c, out = repeated(T, K, N)
    c.check(out[:, 0])
    assert (out == out[:, :1]).all()


@pytest.mark.parametrize("T,K,F", [(1, 528, 8192), (8, 256, 4352), (3, 2576, 9600), (16, 1040, 4864)])
def test_gated_few_tokens_and_many_short_rows(T, K, F):
    c = Case(T, K, 128, gated=True)
    ref, err = gated_reference(c)
    args = []
    for codes, scales in c.w:
        args += [dev_codes(codes).view(torch.uint8).repeat(F // 128, 1), dev_scales(scales).view(torch.uint8).repeat(F // 128, 1)]
    layer = tq.scion_fp8_create(*args)
    codes = torch.empty((T, F // 128, 128), dtype=torch.uint8, device="cuda")
    scales = torch.empty((T, F // 128), dtype=torch.uint8, device="cuda")
    h = torch.empty((T, F // 128, 128), dtype=torch.bfloat16, device="cuda")
    tq.scion_fp8_gated_forward(c.dx, c.dsx, T, layer, h_codes=codes, h_scales=scales)
    tq.scion_fp8_gated_forward(c.dx, c.dsx, T, layer, h=h)
    assert tq.scion_fp8_check(layer) == 0
    R.check_codes(bytes_of(codes[:, 0].contiguous()), bytes_of(scales[:, :1].contiguous()), ref, err)
    assert (np.abs(host(h[:, 0]) - ref) <= np.abs(ref) * 2.0 ** -8 + 2 * err).all()
    assert (codes == codes[:, :1]).all() and (scales == scales[:, :1]).all() and (h == h[:, :1]).all()
