"""GPU: the few-token products where their clusters, loops and tiles are least regular, against 64 bits
(bounds as in test_fp8_gpu.py)."""
import pytest

from tests import fp8_ref as R
from tests.test_fp8_gpu import Case, bytes_of, gated_reference

torch = pytest.importorskip("torch")
import ternary_quantized_moe_b200 as tq  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("F", [16, 32, 144, 272, 400, 1040])
@pytest.mark.parametrize("T", [1, 8])
def test_gated_clusters_with_ctas_without_rows(T, F):
    """Widths that leave the last cluster of eight CTAs (16 features each) partly without rows: those
    CTAs have nothing to multiply and meet the others at the exchange of magnitudes at once."""
    c = Case(T, 2064, F, gated=True)
    ref, err = gated_reference(c)
    codes = torch.empty((64, T, F), dtype=torch.uint8, device="cuda")
    scales = torch.empty((64, T, -(-F // 128)), dtype=torch.uint8, device="cuda")
    for i in range(64):
        tq.scion_fp8_gated_forward(c.dx, c.dsx, T, c.layer, h_codes=codes[i], h_scales=scales[i])
    assert tq.scion_fp8_check(c.layer) == 0
    R.check_codes(bytes_of(codes[0]), bytes_of(scales[0]), ref, err)
    assert (codes == codes[0]).all() and (scales == scales[0]).all()
