"""The 64-bit reference of the 8-bit operators against torch's own e4m3 conversion and hand-worked
values, and the refusals of the library's entry points (no GPU needed: they precede any CUDA call)."""
import ctypes as C

import numpy as np
import pytest

import ternary_quantized_moe_b200 as tq
from tests import fp8_ref as R

torch = pytest.importorskip("torch")


def test_table_is_torchs():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(R.TABLE, t)


def test_rounding_is_torchs():
    rng = np.random.default_rng(5)
    v = np.concatenate([rng.uniform(-448, 448, 20000), rng.normal(0, 0.01, 20000), R.TABLE[np.isfinite(R.TABLE)]])
    mid = (R.POSITIVE[1:] + R.POSITIVE[:-1]) / 2  # ties
    v = np.concatenate([v, mid, -mid]).astype(np.float32)
    ref = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    got = R.round_e4m3(v.astype(np.float64))
    np.testing.assert_array_equal(R.TABLE[got], R.TABLE[ref])


def test_scale_bytes_by_hand():
    a = np.array([448.0, 448.0000001, 449.0, 1.75, 1.7500001, 1.0, 0.0, np.inf, np.nan, 2.0 ** -140, 3.4e38])
    assert R.scale_bytes(a).tolist() == [127, 128, 128, 119, 120, 119, 127, 255, 255, 0, 247]


def test_values_by_hand():
    codes = np.array([[0x38, 0xB8, 0x7E, 0x01]], np.uint8)  # 1, -1, 448, 2^-9
    np.testing.assert_array_equal(R.values(codes, np.array([[128]], np.uint8), 1), [[2.0, -2.0, 896.0, 2.0 ** -8]])


# ------------------------------------------------------------------ refusals
P = 0x100000  # a 16-byte aligned address that is never read: the checks fail first


def quant(**kw):
    a = dict(t=0, src=P, rows=4, cols=256, br=1, codes=P, scales=P) | kw
    return tq._load().scion_fp8_quantize_device(a["t"], a["src"], a["rows"], a["cols"], a["br"], a["codes"], a["scales"], None)


@pytest.mark.parametrize("bad", [dict(t=2), dict(t=-1), dict(src=None), dict(rows=-1), dict(cols=0), dict(cols=24),
                                 dict(cols=1 << 21), dict(br=0), dict(br=64), dict(codes=None), dict(scales=None),
                                 dict(src=P + 8), dict(codes=P + 4), dict(rows=1 << 41),
                                 dict(rows=1 << 40, cols=1 << 20, br=128)])
def test_quantize_refusals(bad):
    assert quant(**bad) == tq.SCION_EINVAL


def norm(**kw):
    a = dict(x=P, xt=0, r=P, rt=0, w=P, eps=1e-6, T=4, d=256, ro=P, y=P, c=P, s=P) | kw
    return tq._load().scion_rmsnorm_forward(a["x"], a["xt"], a["r"], a["rt"], a["w"], a["eps"], a["T"], a["d"], a["ro"],
                                            a["y"], a["c"], a["s"], None)


@pytest.mark.parametrize("bad", [dict(x=None), dict(xt=2), dict(rt=5), dict(w=None), dict(eps=-1.0), dict(eps=float("nan")),
                                 dict(eps=float("inf")), dict(T=-1), dict(d=0), dict(d=8), dict(d=100), dict(d=32784),
                                 dict(ro=None, y=None, c=None, s=None), dict(c=None), dict(s=None), dict(x=P + 8),
                                 dict(r=P + 4), dict(w=P + 2), dict(ro=P + 8), dict(y=P + 8), dict(c=P + 1),
                                 dict(xt=1, ro=P, rt=0)])
def test_norm_refusals(bad):
    assert norm(**bad) == tq.SCION_EINVAL


def create(**kw):
    D = tq._Fp8Desc()
    a = dict(n=256, k=256, w_codes=P, w_scales=P, up_codes=None, up_scales=None) | kw
    for name, v in a.items():
        setattr(D, name, v)
    h = C.c_void_p()
    st = tq._load().scion_fp8_create(C.byref(D), None, C.byref(h))
    assert not h.value
    return st


@pytest.mark.parametrize("bad", [dict(n=0), dict(n=(1 << 20) + 1), dict(k=0), dict(k=8), dict(k=72), dict(k=65552),
                                 dict(w_codes=None), dict(w_scales=None), dict(w_codes=P + 8), dict(up_codes=P),
                                 dict(up_scales=P), dict(up_codes=P + 8, up_scales=P), dict(n=200, up_codes=P, up_scales=P)])
def test_create_refusals(bad):
    assert create(**bad) == tq.SCION_EINVAL


def test_null_handles():
    lib = tq._load()
    assert lib.scion_fp8_create(None, None, None) == tq.SCION_EINVAL
    assert lib.scion_fp8_forward(P, P, 1, None, None, P, 0, None) == tq.SCION_EINVAL
    assert lib.scion_fp8_gated_forward(P, P, 1, None, P, None, None, None) == tq.SCION_EINVAL
    assert lib.scion_fp8_check(None, None) == tq.SCION_EINVAL
    assert lib.scion_fp8_device_bytes(None) == 0
    lib.scion_fp8_destroy(None)


def test_empty_batches_launch_nothing():
    assert quant(rows=0, src=None, codes=None, scales=None) == tq.SCION_OK
    assert norm(T=0, x=None, r=None) == tq.SCION_OK
    assert norm(T=0, x=None, r=None, ro=None, y=None, c=None, s=None) == tq.SCION_OK
