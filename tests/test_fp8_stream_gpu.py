"""GPU: shapes of the streaming product that the layers of test_fp8_gpu.py do not reach (bounds as there)."""
import pytest

from tests.test_fp8_gpu import Case, dev_codes, dev_scales

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
