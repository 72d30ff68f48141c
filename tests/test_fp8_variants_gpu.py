"""GPU: every variant of the product kernels, at a shape that its rule sends there (the launched kernel's
name is read from the profiler), against 64 bits and to the precision of fp32 sums.

Precision.  Each K step of 32 rounds a partial sum once, by at most half a unit of it (2^-24), and no
partial sum is larger in the mean than the whole; roundings of unrelated signs add in squares, so that the
relative error of all outputs together is at most 2^-24 sqrt(K / 32) times the roundings' own spread
(1 / sqrt 3 of the largest), below 2^-24 sqrt(K / 64), and one more rounding for the sums of parts."""
import re

import numpy as np
import pytest

from tests import fp8_ref as R
from tests.test_fp8_gpu import Case, bytes_of, dev_codes, dev_scales, gated_reference, host

torch = pytest.importorskip("torch")
import ternary_quantized_moe_b200 as tq  # noqa: E402

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


def launched(call):
    """Names of the library's product kernels that a call launches, or None where nothing is recorded."""
    from torch.profiler import ProfilerActivity, profile

    call()
    torch.cuda.synchronize()
    with profile(activities=[ProfilerActivity.CUDA], acc_events=True) as p:
        call()
        torch.cuda.synchronize()
    names = [m.group(0) for e in p.events() for m in [re.search(r"fp8_\w+_kernel<[^>]*>", e.name)] if m]
    return names or None


def check_launched(call, kernel):
    names = launched(call)
    if names is None:
        pytest.skip("no kernel activity is recorded on this machine")
    assert names == [kernel]


def check_precision(out, ref, K):
    off = np.linalg.norm(host(out) - ref) / np.linalg.norm(ref)
    assert off <= 2.0 ** -24 * (1 + np.sqrt(K / 64)), "%.2e" % off


ROWS = [("fp8_rows_kernel<1, 1, 4, false, 1>", 1, 2064, 2360), ("fp8_rows_kernel<1, 1, 4, false, 1>", 8, 8192, 40),
        ("fp8_rows_kernel<1, 1, 2, false, 2>", 3, 2048, 2000), ("fp8_rows_kernel<1, 1, 2, false, 2>", 8, 4112, 4001),
        ("fp8_rows_kernel<1, 1, 2, false, 4>", 1, 1040, 4801), ("fp8_rows_kernel<1, 1, 2, false, 4>", 7, 2064, 9472),
        ("fp8_rows_kernel<1, 2, 2, false, 1>", 9, 4112, 1000), ("fp8_rows_kernel<1, 2, 2, false, 1>", 16, 144, 2368),
        ("fp8_rows_kernel<1, 2, 1, false, 2>", 12, 2064, 2401), ("fp8_rows_kernel<1, 2, 1, false, 2>", 16, 1040, 9000),
        ("fp8_rows_kernel<1, 4, 1, false, 1>", 17, 2048, 1111), ("fp8_rows_kernel<1, 4, 1, false, 1>", 32, 1040, 2368),
        ("fp8_rows_kernel<1, 4, 1, false, 2>", 24, 1040, 2500), ("fp8_rows_kernel<1, 4, 1, false, 2>", 32, 528, 4736)]


@pytest.mark.parametrize("kernel,T,K,N", ROWS)
def test_rows_kernel(kernel, T, K, N):
    c = Case(T, K, N)
    base = torch.from_numpy(c.base).to("cuda")
    for out_type in (F32, BF16):
        c.check(c.run(out_type))
        c.check(c.run(out_type, base), c.base)
    out = torch.empty((T, N), dtype=F32, device="cuda")
    check_launched(lambda: tq.scion_fp8_forward(c.dx, c.dsx, T, c.layer, out), kernel)
    check_precision(out, c.products()[0][0], K)


ROWS_GATED = [("fp8_rows_kernel<2, 1, 1, %s, 2>", 1, 2064, 2400), ("fp8_rows_kernel<2, 1, 1, %s, 2>", 8, 4096, 1008),
              ("fp8_rows_kernel<2, 2, 1, %s, 1>", 9, 2064, 912), ("fp8_rows_kernel<2, 2, 1, %s, 1>", 16, 2064, 912),
              ("fp8_rows_kernel<2, 2, 1, %s, 1>", 12, 1168, 1792), ("fp8_rows_kernel<2, 2, 1, %s, 1>", 16, 144, 400)]


def check_gated(kernel, T, K, F, forms):
    c = Case(T, K, F, gated=True)
    ref, err = gated_reference(c)
    codes = torch.empty((T, F), dtype=torch.uint8, device="cuda")
    scales = torch.empty((T, -(-F // 128)), dtype=torch.uint8, device="cuda")
    h = torch.empty((T, F), dtype=BF16, device="cuda")
    runs = {"true": lambda: tq.scion_fp8_gated_forward(c.dx, c.dsx, T, c.layer, h_codes=codes, h_scales=scales),
            "false": lambda: tq.scion_fp8_gated_forward(c.dx, c.dsx, T, c.layer, h=h)}
    for form in forms:
        runs[form]()
    if "true" in forms:
        R.check_codes(bytes_of(codes), bytes_of(scales), ref, err)
    if "false" in forms:
        assert (np.abs(host(h) - ref) <= np.abs(ref) * 2.0 ** -8 + 2 * err).all()
    assert tq.scion_fp8_check(c.layer) == 0
    for form in forms:
        check_launched(runs[form], kernel % form if "%" in kernel else kernel)


@pytest.mark.parametrize("kernel,T,K,F", ROWS_GATED)
def test_rows_kernel_gated(kernel, T, K, F):
    check_gated(kernel, T, K, F, ("true", "false"))


@pytest.mark.parametrize("T,K,F", [(9, 528, 2352), (12, 768, 2368), (16, 656, 2320)])
def test_rows_kernel_gated_more_clusters_than_run_at_once(T, K, F):
    """19 clusters of eight CTAs: 148 SMs hold 18 at most."""
    check_gated("fp8_rows_kernel<2, 2, 1, true, 2>", T, K, F, ("true",))


# (kernel, T, K, N, base): scale rows and outputs of any alignment in the "true" of the third place
PLAIN = [("fp8_stream_kernel<1, true, false>", 64, 4096, 2048, False), ("fp8_stream_kernel<1, true, false>", 64, 8192, 512, True),
         ("fp8_stream_kernel<1, true, true>", 64, 4112, 2052, False), ("fp8_stream_kernel<1, true, true>", 64, 2048, 2049, True),
         ("fp8_stream_kernel<1, false, false>", 500, 1024, 2048, False),
         ("fp8_stream_kernel<1, false, false>", 600, 512, 2048, True),
         ("fp8_stream_kernel<1, false, true>", 500, 1040, 2047, True), ("fp8_stream_kernel<1, false, true>", 500, 1040, 2048, False),
         ("fp8_pair_kernel<0>", 2600, 1040, 2304, False), ("fp8_pair_kernel<1>", 2600, 1040, 2304, False),
         ("fp8_pair_kernel<2>", 2600, 1040, 2304, True), ("fp8_pair_kernel<5>", 2600, 1040, 2303, False),
         ("fp8_pair_kernel<5>", 2600, 1040, 2303, True)]


@pytest.mark.parametrize("kernel,T,K,N,with_base", PLAIN)
def test_stream_and_pair_kernels(kernel, T, K, N, with_base):
    c = Case(T, K, N)
    base = torch.from_numpy(c.base).to("cuda") if with_base else None
    for out_type in (F32, BF16):
        c.check(c.run(out_type, base), c.base if with_base else None)
    out = torch.empty((T, N), dtype=BF16 if kernel.endswith("<0>") else F32, device="cuda")
    check_launched(lambda: tq.scion_fp8_forward(c.dx, c.dsx, T, c.layer, out, base=base), kernel)
    check_precision(c.run(F32), c.products()[0][0], K)


@pytest.mark.parametrize("kernel,T,K,F,forms", [
    ("fp8_stream_kernel<2, true, false>", 50, 2048, 5456, ("true", "false")),
    ("fp8_stream_kernel<2, true, true>", 50, 2064, 5456, ("true", "false")),
    ("fp8_stream_kernel<2, false, false>", 33, 512, 16384, ("true", "false")),
    ("fp8_stream_kernel<2, false, true>", 33, 528, 16384, ("true", "false")),
    ("fp8_pair_kernel<3>", 2600, 1040, 1040, ("false",)), ("fp8_pair_kernel<4>", 2600, 1040, 1040, ("true",))])
def test_stream_and_pair_kernels_gated(kernel, T, K, F, forms):
    check_gated(kernel, T, K, F, forms)
