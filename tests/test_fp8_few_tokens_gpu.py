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


@pytest.mark.parametrize("T", [2, 40, 600])
def test_captured_fork_and_join(T):
    """Two streams captured into one graph: the products of one layer's input on both, joined by a third
    that reads both results; replayed on new inputs, and two such graphs of one handle at once."""
    K, N = 1040, 640
    c = Case(T, K, N)
    d = Case(T, N, 272)
    x = torch.empty((T, K), device="cuda")
    w = torch.ones(K, dtype=torch.bfloat16, device="cuda")

    def make():
        b = {"codes": torch.empty((T, K), dtype=torch.uint8, device="cuda"),
             "scales": torch.empty((T, -(-K // 128)), dtype=torch.uint8, device="cuda"),
             "ncodes": torch.empty((T, K), dtype=torch.uint8, device="cuda"),
             "nscales": torch.empty((T, -(-K // 128)), dtype=torch.uint8, device="cuda"),
             "a": torch.empty((T, N), device="cuda"), "b": torch.empty((T, N), device="cuda"),
             "hc": torch.empty((T, N), dtype=torch.uint8, device="cuda"),
             "hs": torch.empty((T, -(-N // 128)), dtype=torch.uint8, device="cuda"),
             "out": torch.empty((T, 272), device="cuda")}
        return b

    def step(b, side):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            tq.scion_rmsnorm_forward(x, T, w, 1e-6, y_codes=b["ncodes"], y_scales=b["nscales"])
            tq.scion_fp8_forward(b["ncodes"], b["nscales"], T, c.layer, b["a"])
        tq.scion_fp8_quantize_device(x, b["codes"], b["scales"])
        tq.scion_fp8_forward(b["codes"], b["scales"], T, c.layer, b["b"])
        main.wait_stream(side)
        tq.scion_fp8_forward(b["codes"], b["scales"], T, c.layer, b["a"], base=b["a"])
        tq.scion_fp8_quantize_device(b["a"], b["hc"], b["hs"])
        tq.scion_fp8_forward(b["hc"], b["hs"], T, d.layer, b["out"])

    x.normal_()
    sides = [torch.cuda.Stream() for _ in range(2)]
    bufs, graphs, want = [make(), make()], [torch.cuda.CUDAGraph() for _ in range(2)], make()
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        step(want, sides[0])
    torch.cuda.current_stream().wait_stream(warm)
    for b, g, s in zip(bufs, graphs, sides):
        with torch.cuda.graph(g):
            step(b, s)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        x.normal_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        step(want, sides[0])
        torch.cuda.synchronize()
        for b in bufs:
            assert all(torch.equal(b[k], want[k]) for k in want)
    assert torch.isfinite(want["out"]).all() and tq.scion_fp8_check(c.layer) == 0
