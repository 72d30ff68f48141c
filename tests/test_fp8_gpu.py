"""GPU parity of the 8-bit dense operators against their definitions in 64 bits.

Tolerances.  A sum of n fp32 products carries at most n 2^-23 of the sum of their magnitudes (each
addition is off by at most one unit of its partial sum, truncation included); the products of two e4m3
codes and the scalings by powers of two are exact.  A rounding to bf16 is off by at most 2^-8 of the
value.  8-bit results are held to half a step of their code (fp8_ref.check_codes)."""
import numpy as np
import pytest

from tests import fp8_ref as R

torch = pytest.importorskip("torch")
import ternary_quantized_moe_b200 as tq  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def host(t):
    return t.double().cpu().numpy()


def bytes_of(t):
    return t.view(torch.uint8).cpu().numpy()


def dev_codes(c):
    return torch.from_numpy(c).to(DEV).view(torch.float8_e4m3fn)


def dev_scales(b):
    return torch.from_numpy(b).to(DEV).view(torch.float8_e8m0fnu)


def activations(rng, T, K):
    v = rng.standard_normal((T, K)) * np.exp(rng.standard_normal((T, 1)))
    v[:, rng.integers(0, K, max(1, K // 100))] *= 30
    return v


# ------------------------------------------------------------------ quantizer
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 128), (3, 144), (128, 128), (129, 2048), (300, 1936), (1000, 48)])
def test_quantize(dtype, block_rows, rows, cols):
    rng = np.random.default_rng(rows * 7 + cols)
    v = torch.from_numpy(activations(rng, rows, cols)).to(dtype)
    if rows > 2:
        v[1] = 0  # a group of zeros (block_rows 1)
        v[2, :16] = torch.tensor([448.0, 224, 1.75, -448, 0, 1, -0.0, 3] * 2)
    codes, scales = tq.scion_fp8_quantize_device(v.to(DEV), block_rows=block_rows)
    rc, rb = R.quantize(host(v), block_rows)
    np.testing.assert_array_equal(bytes_of(scales), rb)
    np.testing.assert_array_equal(bytes_of(codes), rc)


def test_quantize_extremes():
    """Infinities and NaN mark their block alone; the largest and smallest magnitudes keep their scales."""
    v = torch.zeros((6, 256), dtype=F32)
    v[0, 3], v[1, 130], v[1, 0] = float("inf"), float("nan"), 1.0
    v[2, :128], v[2, 128:] = 3.4e38, 1.2e-38
    v[3, 0], v[3, 128] = 1e-45, 2.0 ** -126
    v[4, 0], v[4, 128] = 1.75, 1.7500001
    v[5, :8] = torch.tensor([1.0, -1, 2.0 ** -18, 2.0 ** -19, 2.0 ** -17 * 1.5, 0.4375, 1.0625, 1.1875])
    codes, scales = tq.scion_fp8_quantize_device(v.to(DEV))
    b, c = bytes_of(scales), bytes_of(codes)
    rc, rb = R.quantize(host(v), 1)
    np.testing.assert_array_equal(b, rb)
    bad = R.spread(rb, v.shape, 1) == 255
    assert bad.sum() == 256 and (c[bad] & 0x7F == 0x7F).all()
    np.testing.assert_array_equal(c[~bad], rc[~bad])


# ------------------------------------------------------------------ norm
def norm_case(T, d, xt, rt, seed=0):
    rng = np.random.default_rng(seed + T * 31 + d)
    x = torch.from_numpy(rng.standard_normal((T, d))).to(xt)
    r = None if rt is None else torch.from_numpy(activations(rng, T, d)).to(rt)
    w = torch.from_numpy(1 + 0.2 * rng.standard_normal(d)).to(BF16)
    return x, r, w


def check_norm(x, r, w, eps, resid_out, y, codes, scales):
    rr, ry = R.rmsnorm(host(x), None if r is None else host(r), host(w), eps)
    d = x.shape[1]
    # fp32: r 2^-24; the mean at most (d + 4) 2^-24 by the additions' bound; rsqrt, two products
    err = np.abs(ry) * ((d + 4) / 2 + 8) * 2.0 ** -24
    err += 2.0 ** -24 * np.abs(rr) / np.maximum(np.abs(rr), 1e-30) * np.abs(ry)
    if resid_out is not None:
        got = host(resid_out)
        if resid_out.dtype == F32:
            np.testing.assert_array_equal(got, rr.astype(np.float32).astype(np.float64))
        else:
            assert (np.abs(got - rr) <= np.abs(rr) * (2.0 ** -8 + 2.0 ** -23)).all()
    if y is not None:
        assert (np.abs(host(y) - ry) <= np.abs(ry) * 2.0 ** -8 + 2 * err).all()
    if codes is not None:
        R.check_codes(bytes_of(codes), bytes_of(scales), ry, err)


@pytest.mark.parametrize("xt,rt", [(F32, F32), (BF16, F32), (F32, BF16), (BF16, BF16), (F32, None), (BF16, None)])
@pytest.mark.parametrize("T,d", [(1, 16), (1, 2048), (5, 144), (33, 1936), (64, 2048), (3, 8192), (2, 16400), (2, 32768)])
def test_norm(T, d, xt, rt):
    x, r, w = norm_case(T, d, xt, rt)
    ro = None if r is None else torch.full((T + 1, d), 7.0, dtype=rt, device=DEV)
    y = torch.full((T + 1, d), 7.0, dtype=BF16, device=DEV)
    codes = torch.full((T + 1, d), 9, dtype=torch.uint8, device=DEV)
    scales = torch.full((T + 1, -(-d // 128)), 9, dtype=torch.uint8, device=DEV)
    rd = None if r is None else r.to(DEV)
    tq.scion_rmsnorm_forward(x.to(DEV), T, w.to(DEV), 1e-6, resid=rd, resid_out=None if ro is None else ro[:T], y=y[:T],
                             y_codes=codes[:T], y_scales=scales[:T])
    check_norm(x, r, w, 1e-6, None if ro is None else ro[:T], y[:T], codes[:T], scales[:T])
    # rows behind the last token stay as they were; the residual is only read
    assert (y[T] == 7).all() and (codes[T] == 9).all() and (scales[T] == 9).all() and (ro is None or (ro[T] == 7).all())
    assert r is None or torch.equal(rd.cpu(), r)


@pytest.mark.parametrize("rt", [F32, BF16])
def test_norm_in_place_and_single_outputs(rt):
    T, d = 9, 2064
    x, r, w = norm_case(T, d, rt, rt)
    want = torch.empty((T, d), dtype=BF16, device=DEV)
    ro = torch.empty((T, d), dtype=rt, device=DEV)
    tq.scion_rmsnorm_forward(x.to(DEV), T, w.to(DEV), 1e-5, resid=r.to(DEV), resid_out=ro, y=want)
    for target in ("resid", "x"):
        xd, rd = x.to(DEV), r.to(DEV)
        buf = rd if target == "resid" else xd
        y = torch.empty_like(want)
        tq.scion_rmsnorm_forward(xd, T, w.to(DEV), 1e-5, resid=rd, resid_out=buf, y=y)
        assert torch.equal(buf, ro) and torch.equal(y, want)
    # the sum alone, and resid_out without a residual (a copy in another type)
    only = torch.empty_like(ro)
    tq.scion_rmsnorm_forward(x.to(DEV), T, w.to(DEV), 1e-5, resid=r.to(DEV), resid_out=only)
    assert torch.equal(only, ro)
    cast = torch.empty((T, d), dtype=BF16 if rt == F32 else F32, device=DEV)
    tq.scion_rmsnorm_forward(x.to(DEV), T, w.to(DEV), 1e-5, resid_out=cast)
    assert torch.equal(cast.cpu(), x.to(cast.dtype))


def test_norm_special_rows():
    """Zero rows, rows with infinities or NaN (NaN in all of their outputs, no effect on their neighbours)
    and rows of large and small magnitude."""
    T, d = 7, 272
    x, _, w = norm_case(T, d, F32, None)
    x[0] = 0
    x[1, 5] = float("inf")
    x[2, 200] = float("nan")
    x[3] *= 1e15
    x[4] *= 1e-15
    x[5] = 0
    x[5, 3] = 2.0
    y = torch.empty((T, d), dtype=BF16, device=DEV)
    codes = torch.empty((T, d), dtype=torch.uint8, device=DEV)
    scales = torch.empty((T, 3), dtype=torch.uint8, device=DEV)
    tq.scion_rmsnorm_forward(x.to(DEV), T, w.to(DEV), 1e-6, y=y, y_codes=codes, y_scales=scales)
    assert torch.isnan(y[1]).all() and torch.isnan(y[2]).all()
    assert (scales[1:3] == 255).all() and (codes[1:3] & 0x7F == 0x7F).all()
    assert (y[0] == 0).all() and (codes[0] & 0x7F == 0).all() and (scales[0] == 127).all()
    keep = [0, 3, 4, 5, 6]
    check_norm(x[keep], None, w, 1e-6, None, y[keep], codes[keep], scales[keep])
    assert torch.isfinite(y[keep]).all()


@pytest.mark.parametrize("d", [272, 2048])
@pytest.mark.parametrize("size", [1e-34, 1e-36, 3e-38, 1e-40])
def test_norm_of_rows_near_the_smallest_numbers(d, size):
    """The statistic is eps alone and the scale's inverse near the end of the fp32 range."""
    T = 3
    x, _, w = norm_case(T, d, F32, None)
    x = (x.double() * size).float()
    x[1, ::3] = 0
    y = torch.empty((T, d), dtype=BF16, device=DEV)
    codes = torch.empty((T, d), dtype=torch.uint8, device=DEV)
    scales = torch.empty((T, -(-d // 128)), dtype=torch.uint8, device=DEV)
    tq.scion_rmsnorm_forward(x.to(DEV), T, w.to(DEV), 1e-6, y=y, y_codes=codes, y_scales=scales)
    _, ry = R.rmsnorm(host(x), None, host(w), 1e-6)
    # as in check_norm, and below the smallest normal number 2^-150 per fp32 product: r w (then times
    # 10^3 = 1 / sqrt(eps)) and y
    err = np.abs(ry) * ((d + 4) / 2 + 9) * 2.0 ** -24 + 2.0 ** -150 * 1001
    # (a bf16 below 2^-126 is off by 2^-134 at most)
    assert (np.abs(host(y) - ry) <= np.abs(ry) * 2.0 ** -8 + 2.0 ** -134 + 2 * err).all()
    R.check_codes(bytes_of(codes), bytes_of(scales), ry, err)


# ------------------------------------------------------------------ products
def quantized(rng, rows, cols, block_rows, std=1.0):
    v = activations(rng, rows, cols) * std
    return R.quantize(v, block_rows)


class Case:
    """A layer and its input, both sides."""

    def __init__(self, T, K, N, gated=False, seed=0):
        rng = np.random.default_rng(seed + 1000003 * T + 1009 * K + N)
        self.T, self.K, self.N = T, K, N
        self.x, self.sx = quantized(rng, T, K, 1)
        self.w = [quantized(rng, N, K, 128, 0.7 * K ** -0.5) for _ in range(2 if gated else 1)]
        args = [f(a) for p in self.w for f, a in ((dev_codes, p[0]), (dev_scales, p[1]))]
        self.layer = tq.scion_fp8_create(*args)
        self.dx, self.dsx = dev_codes(self.x), dev_scales(self.sx)
        self.base = rng.standard_normal((T, N)).astype(np.float32)

    def products(self):
        """Per matrix: the exact product and a bound of the fp32 sums' error."""
        xv = R.values(self.x, self.sx, 1)
        out = []
        for c, s in self.w:
            wv = R.values(c, s, 128)
            out.append((xv @ wv.T, self.K * 2.0 ** -23 * (np.abs(xv) @ np.abs(wv).T)))
        return out

    def run(self, out_type, base=None):
        out = torch.full((self.T + 1, self.N), 7.0, dtype=out_type, device=DEV)
        tq.scion_fp8_forward(self.dx, self.dsx, self.T, self.layer, out[:self.T], base=base)
        assert tq.scion_fp8_check(self.layer) == 0
        assert (out[self.T] == 7).all()
        return out[:self.T]

    def check(self, out, base=None):
        ref, err = self.products()[0]
        if base is not None:
            ref, err = ref + base, err + 2.0 ** -23 * (np.abs(ref) + np.abs(base))
        tol = err + (np.abs(ref) * 2.0 ** -8 if out.dtype == BF16 else np.abs(ref) * 2.0 ** -23)
        worst = np.abs(host(out) - ref) - tol
        assert worst.max() <= 0, "off by %.3e more than the bound" % worst.max()


LINEAR = [(1, 16, 1), (1, 2048, 512), (1, 4096, 2048), (2, 128, 128), (7, 144, 100), (16, 512, 129), (17, 528, 300),
          (33, 2048, 257), (64, 4112, 384), (65, 256, 1000), (100, 2064, 256), (128, 640, 640), (129, 1024, 255),
          (200, 2048, 1111), (257, 512, 513), (300, 4096, 512), (513, 272, 2048), (1025, 1024, 768),
          (300, 640, 264), (400, 144, 260), (700, 16, 136), (2600, 640, 2304)]


@pytest.mark.parametrize("T,K,N", LINEAR)
def test_linear(T, K, N):
    c = Case(T, K, N)
    for out_type in (F32, BF16):
        c.check(c.run(out_type))
        c.check(c.run(out_type, torch.from_numpy(c.base).to(DEV)), c.base)
    inplace = torch.from_numpy(c.base).to(DEV)
    tq.scion_fp8_forward(c.dx, c.dsx, T, c.layer, inplace, base=inplace)
    c.check(inplace, c.base)


@pytest.mark.parametrize("T,K,N", [(1, 4112, 1000), (8, 4112, 2390), (3, 2064, 4800), (5, 272, 5000), (12, 2064, 2000),
                                   (16, 4112, 2390), (17, 144, 100), (24, 2064, 2000), (25, 2048, 2391), (31, 4096, 1000),
                                   (32, 4096, 2048), (32, 4112, 264)])
def test_linear_few_tokens(T, K, N):
    """Batches of up to 32 tokens: few and many weight rows, K of one round of blocks and more."""
    c = Case(T, K, N)
    for out_type in (F32, BF16):
        c.check(c.run(out_type, torch.from_numpy(c.base).to(DEV)), c.base)


@pytest.mark.parametrize("T,K,F", [(2, 4112, 2400), (8, 2064, 2400), (12, 4112, 1008), (16, 2064, 2000), (24, 2064, 400)])
def test_gated_few_tokens(T, K, F):
    c = Case(T, K, F, gated=True)
    ref, err = gated_reference(c)
    codes = torch.empty((T, F), dtype=torch.uint8, device=DEV)
    scales = torch.empty((T, -(-F // 128)), dtype=torch.uint8, device=DEV)
    tq.scion_fp8_gated_forward(c.dx, c.dsx, T, c.layer, h_codes=codes, h_scales=scales)
    R.check_codes(bytes_of(codes), bytes_of(scales), ref, err)
    h = torch.empty((T, F), dtype=BF16, device=DEV)
    tq.scion_fp8_gated_forward(c.dx, c.dsx, T, c.layer, h=h)
    assert (np.abs(host(h) - ref) <= np.abs(ref) * 2.0 ** -8 + 2 * err).all()


@pytest.mark.parametrize("T", [3, 70, 400])
def test_linear_is_reproducible_and_rows_are_independent(T):
    c = Case(T, 2048, 640)
    a, b = c.run(F32), c.run(F32)
    assert torch.equal(a, b)
    x, s = c.dx.clone(), c.dsx.clone()
    x.view(torch.uint8)[1:] = 0x7F  # every other row becomes NaN
    other = torch.empty_like(a)
    tq.scion_fp8_forward(x, s, T, c.layer, other)
    assert torch.equal(other[0], a[0]) and torch.isnan(other[1:]).all()


@pytest.mark.parametrize("T", [5, 300])
def test_linear_scale_range(T):
    """Scales far from 1 on both sides, a NaN scale in one row and one weight block, zero rows."""
    c = Case(T, 384, 256)
    c.sx[:, 0] = (c.sx[:, 0].astype(int) - 60).astype(np.uint8)
    c.sx[:, 1] = (c.sx[:, 1].astype(int) + 40).astype(np.uint8)
    c.w[0][1][:, 1] = (c.w[0][1][:, 1].astype(int) - 40).astype(np.uint8)
    c.w[0][1][:, 2] = (c.w[0][1][:, 2].astype(int) + 50).astype(np.uint8)
    c.x[1] = 0
    c.dx, c.dsx = dev_codes(c.x), dev_scales(c.sx)
    c.layer = tq.scion_fp8_create(dev_codes(c.w[0][0]), dev_scales(c.w[0][1]))
    out = c.run(F32)
    c.check(out)
    assert (out[1] == 0).all()
    c.sx[2, 1] = 255
    c.dsx = dev_scales(c.sx)
    out2 = c.run(F32)
    assert torch.isnan(out2[2]).all() and torch.equal(out2[3:], out[3:]) and torch.equal(out2[:2], out[:2])
    c.w[0][1][1, 0] = 255  # outputs 128 .. 255
    c.layer = tq.scion_fp8_create(dev_codes(c.w[0][0]), dev_scales(c.w[0][1]))
    out3 = c.run(F32)
    assert torch.isnan(out3[3:, 128:]).all() and torch.equal(out3[3:, :128], out[3:, :128])


@pytest.mark.parametrize("T,K,N", [(3, 272, 132), (20, 2048, 264), (70, 528, 512), (300, 2048, 512), (300, 48, 260)])
def test_linear_unaligned(T, K, N):
    """Outputs, bases and scales that start at addresses aligned to one element only."""
    c = Case(T, K, N)
    sx = torch.empty(c.dsx.numel() + 1, dtype=torch.uint8, device=DEV)
    sx[1:] = c.dsx.view(torch.uint8).flatten()
    sw = torch.empty(c.w[0][1].size + 1, dtype=torch.uint8, device=DEV)
    sw[1:] = dev_scales(c.w[0][1]).view(torch.uint8).flatten()
    c.layer = tq.scion_fp8_create(dev_codes(c.w[0][0]), sw[1:])
    base = torch.empty(T * N + 1, dtype=F32, device=DEV)
    base[1:] = torch.from_numpy(c.base).to(DEV).flatten()
    for out_type in (F32, BF16):
        buf = torch.full((T * N + 2,), 7.0, dtype=out_type, device=DEV)
        out = buf[1:-1].view(T, N)
        tq.scion_fp8_forward(c.dx, sx[1:], T, c.layer, out)
        c.check(out)
        tq.scion_fp8_forward(c.dx, sx[1:], T, c.layer, out, base=base[1:].view(T, N))
        c.check(out, c.base)
        assert buf[0] == 7 and buf[-1] == 7


@pytest.mark.parametrize("T,K,N", [(700, 2064, 2303), (1100, 640, 4100), (2600, 640, 1041), (2049, 272, 2306), (3000, 2048, 300)])
def test_linear_many_tokens_unaligned_rows(T, K, N):
    """Rows of outputs and bases at every alignment, in many tiles; in place; nothing beside them written."""
    c = Case(T, K, N)
    for out_type in (F32, BF16):
        buf = torch.full((T * N + 2,), 7.0, dtype=out_type, device=DEV)
        out = buf[1:-1].view(T, N)
        tq.scion_fp8_forward(c.dx, c.dsx, T, c.layer, out)
        c.check(out)
        tq.scion_fp8_forward(c.dx, c.dsx, T, c.layer, out, base=torch.from_numpy(c.base).to(DEV))
        c.check(out, c.base)
        assert buf[0] == 7 and buf[-1] == 7
    buf = torch.full((T * N + 2,), 7.0, dtype=F32, device=DEV)
    out = buf[1:-1].view(T, N)
    out.copy_(torch.from_numpy(c.base))
    tq.scion_fp8_forward(c.dx, c.dsx, T, c.layer, out, base=out)
    c.check(out, c.base)
    assert buf[0] == 7 and buf[-1] == 7 and tq.scion_fp8_check(c.layer) == 0


GATED = [(1, 16, 16), (1, 2048, 512), (2, 128, 128), (7, 144, 112), (16, 512, 144), (33, 2048, 272), (50, 2048, 528),
         (64, 4112, 384), (65, 256, 1008), (100, 2064, 256), (129, 1024, 240), (257, 512, 528), (300, 2048, 512),
         (1025, 1024, 768), (600, 16, 16), (2600, 640, 1040)]


def gated_value(g, u, eg, eu):
    """h = silu(g) u and the bound of its error: |silu'| <= 1.1; the exponential (ex2 of a rounded
    argument), quotient and product in fp32."""
    h = R.silu(g) * u
    return h, 1.1 * eg * np.abs(u) + (np.abs(R.silu(g)) + 1.1 * eg) * eu + np.abs(h) * (16 + 2 * np.abs(g)) * 2.0 ** -23


def gated_reference(c):
    (g, eg), (u, eu) = c.products()
    return gated_value(g, u, eg, eu)


@pytest.mark.parametrize("T,K,F", GATED)
def test_gated(T, K, F):
    c = Case(T, K, F, gated=True)
    ref, err = gated_reference(c)
    h = torch.full((T + 1, F), 7.0, dtype=BF16, device=DEV)
    tq.scion_fp8_gated_forward(c.dx, c.dsx, T, c.layer, h=h[:T])
    assert (np.abs(host(h[:T]) - ref) <= np.abs(ref) * 2.0 ** -8 + 2 * err).all()
    codes = torch.full((T + 1, F), 9, dtype=torch.uint8, device=DEV)
    scales = torch.full((T + 1, -(-F // 128)), 9, dtype=torch.uint8, device=DEV)
    tq.scion_fp8_gated_forward(c.dx, c.dsx, T, c.layer, h_codes=codes[:T], h_scales=scales[:T])
    assert tq.scion_fp8_check(c.layer) == 0
    R.check_codes(bytes_of(codes[:T]), bytes_of(scales[:T]), ref, err)
    assert (h[T] == 7).all() and (codes[T] == 9).all() and (scales[T] == 9).all()


@pytest.mark.parametrize("T", [4, 300])
def test_gated_special_rows(T):
    """A zero row gives zeros (scale byte 127), a NaN row NaN in all of its groups; gates far below and
    above zero saturate."""
    c = Case(T, 256, 272, gated=True)
    c.x[0], c.x[1, 7] = 0, 0x7F
    c.sx[2] = 134  # |gate| into the hundreds and beyond
    c.dx, c.dsx = dev_codes(c.x), dev_scales(c.sx)
    codes = torch.empty((T, 272), dtype=torch.uint8, device=DEV)
    scales = torch.empty((T, 3), dtype=torch.uint8, device=DEV)
    tq.scion_fp8_gated_forward(c.dx, c.dsx, T, c.layer, h_codes=codes, h_scales=scales)
    assert (codes[0] & 0x7F == 0).all() and (scales[0] == 127).all()
    assert (codes[1] & 0x7F == 0x7F).all() and (scales[1] == 255).all()
    keep = np.arange(T) != 1
    c.x[1] = 0
    ref, err = gated_reference(c)
    R.check_codes(bytes_of(codes)[keep], bytes_of(scales)[keep], ref[keep], err[keep])


# ------------------------------------------------------------------ far offsets
@pytest.mark.parametrize("N", [4096, 4097])
def test_linear_rows_past_32_bits(N):
    """An output of more than 2^31 elements: its first and last rows."""
    T, K = 540000, 16
    c = Case(256, K, N)
    x, sx = (t.view(torch.uint8).repeat(-(-T // 256), 1)[:T].contiguous() for t in (c.dx, c.dsx))
    out = torch.empty((T, N), dtype=BF16, device=DEV)
    tq.scion_fp8_forward(x, sx, T, c.layer, out)
    last = (T - 1) // 256 * 256  # a whole copy of the rows, and the part of one at the end
    c.check(out[:256])
    assert torch.equal(out[last - 256:last], out[:256]) and torch.equal(out[last:], out[:T - last])


def test_gated_rows_past_32_bits():
    T, K, F = 540000, 16, 4112
    c = Case(256, K, F, gated=True)
    x, sx = (t.view(torch.uint8).repeat(-(-T // 256), 1)[:T].contiguous() for t in (c.dx, c.dsx))
    codes, scales = torch.empty((T, F), dtype=torch.uint8, device=DEV), torch.empty((T, 33), dtype=torch.uint8, device=DEV)
    tq.scion_fp8_gated_forward(x, sx, T, c.layer, h_codes=codes, h_scales=scales)
    ref, err = gated_reference(c)
    R.check_codes(bytes_of(codes[:256]), bytes_of(scales[:256]), ref, err)
    last = (T - 1) // 256 * 256
    for t in (codes, scales):
        assert torch.equal(t[last - 256:last], t[:256]) and torch.equal(t[last:], t[:T - last])


@pytest.mark.parametrize("T", [1, 20])
def test_weights_past_32_bits(T):
    N, K = 1 << 20, 2064
    c = Case(T, K, 128)
    w = c.w[0][0]
    wd, sd = dev_codes(w).view(torch.uint8).repeat(N // 128, 1), dev_scales(c.w[0][1]).view(torch.uint8).repeat(N // 128, 1)
    want = c.run(F32)
    c.layer = tq.scion_fp8_create(wd, sd)
    out = torch.empty((T, N), dtype=F32, device=DEV)
    tq.scion_fp8_forward(c.dx, c.dsx, T, c.layer, out)
    c.check(out[:, :128].contiguous())
    c.check(out[:, -128:].contiguous())
    assert torch.equal(out[:, -128:], out[:, :128]) and want.shape == (T, 128)


def test_norm_and_quantize_past_32_bits():
    T, d = 270000, 8192
    x, _, w = norm_case(64, d, BF16, None)
    big = x.to(DEV).repeat(-(-T // 64), 1)[:T].contiguous()
    y = torch.empty_like(big)
    codes, scales = torch.empty((T, d), dtype=torch.uint8, device=DEV), torch.empty((T, 64), dtype=torch.uint8, device=DEV)
    tq.scion_rmsnorm_forward(big, T, w.to(DEV), 1e-6, y=y, y_codes=codes, y_scales=scales)
    last = (T - 1) // 64 * 64
    check_norm(x, None, w, 1e-6, None, y[:64], codes[:64], scales[:64])
    for t in (y, codes, scales):
        assert torch.equal(t[last - 64:last], t[:64]) and torch.equal(t[last:], t[:T - last])
    for block_rows in (1, 128):
        q, s = tq.scion_fp8_quantize_device(big, block_rows=block_rows)
        tail = T % 128  # (with block_rows 128 the last, shorter block of rows)
        rq, rs = R.quantize(host(big[T - tail:]), block_rows)
        np.testing.assert_array_equal(bytes_of(q[T - tail:]), rq)
        np.testing.assert_array_equal(bytes_of(s[-rs.shape[0]:]), rs)
        del q, s


# ------------------------------------------------------------------ use
@pytest.mark.parametrize("T", [2, 300])
def test_captured_and_replayed(T):
    """Norm, gated product and down projection captured into a CUDA graph and replayed on new inputs."""
    d, F = 512, 384
    rng = np.random.default_rng(T)
    gate, up, down = (quantized(rng, a, b, 128, b ** -0.5) for a, b in ((F, d), (F, d), (d, F)))
    ffn = tq.scion_fp8_create(dev_codes(gate[0]), dev_scales(gate[1]), dev_codes(up[0]), dev_scales(up[1]))
    proj = tq.scion_fp8_create(dev_codes(down[0]), dev_scales(down[1]))
    w = torch.ones(d, dtype=BF16, device=DEV)
    x, r = (torch.empty((T, d), dtype=F32, device=DEV) for _ in range(2))
    codes, scales = torch.empty((T, d), dtype=torch.uint8, device=DEV), torch.empty((T, 4), dtype=torch.uint8, device=DEV)
    hc, hs = torch.empty((T, F), dtype=torch.uint8, device=DEV), torch.empty((T, 3), dtype=torch.uint8, device=DEV)

    def step(x, r, out):
        tq.scion_rmsnorm_forward(x, T, w, 1e-6, resid=r, resid_out=out, y_codes=codes, y_scales=scales)
        tq.scion_fp8_gated_forward(codes, scales, T, ffn, h_codes=hc, h_scales=hs)
        tq.scion_fp8_forward(hc, hs, T, proj, out, base=out)

    out, want = torch.empty_like(x), torch.empty_like(x)
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    x.normal_(), r.normal_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, r, out)
    torch.cuda.current_stream().wait_stream(side)
    with torch.cuda.graph(g):
        step(x, r, out)
    for _ in range(3):
        x.normal_(), r.normal_()
        g.replay()
        step(x, r, want)
        assert torch.equal(out, want)


def test_calls_on_two_streams_overlap_safely():
    """One handle used on two streams at once: it holds no workspace."""
    a, b = Case(40, 2048, 1024), Case(300, 2048, 1024, seed=9)
    b.layer, b.w = a.layer, a.w
    want = a.run(F32).clone(), b.run(F32).clone()
    outs = [[torch.empty_like(w) for _ in range(8)] for w in want]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for i in range(8):
        for c, o, s in zip((a, b), outs, streams):
            tq.scion_fp8_forward(c.dx, c.dsx, c.T, a.layer, o[i], stream=s)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w, t) for t in o)


def test_python_refusals():
    c, g = Case(4, 256, 128), Case(4, 256, 128, gated=True)
    out = torch.empty((4, 128), dtype=F32, device=DEV)
    bad = [lambda: tq.scion_fp8_forward(c.dx.cpu(), c.dsx, 4, c.layer, out),
           lambda: tq.scion_fp8_forward(c.dx, c.dsx, 5, c.layer, out),
           lambda: tq.scion_fp8_forward(c.dx.t(), c.dsx, 4, c.layer, out),
           lambda: tq.scion_fp8_forward(c.dx, c.dsx, 4, c.layer, out.half()),
           lambda: tq.scion_fp8_forward(c.dx, c.dsx, 4, c.layer, out, base=out.bfloat16()),
           lambda: tq.scion_fp8_quantize_device(out.half()),
           lambda: tq.scion_fp8_create(c.dx, c.dsx[:, :1].contiguous()),
           lambda: tq.scion_rmsnorm_forward(out, 4, out[0], 1e-6, y=out.bfloat16())]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    hc, hs = torch.empty((4, 128), dtype=torch.uint8, device=DEV), torch.empty((4, 1), dtype=torch.uint8, device=DEV)
    einval = [lambda: tq.scion_fp8_forward(g.dx, g.dsx, 4, g.layer, out),
              lambda: tq.scion_fp8_gated_forward(c.dx, c.dsx, 4, c.layer, h=out.bfloat16()),
              lambda: tq.scion_fp8_gated_forward(g.dx, g.dsx, 4, g.layer),
              lambda: tq.scion_fp8_gated_forward(g.dx, g.dsx, 4, g.layer, h_codes=hc),
              lambda: tq.scion_fp8_gated_forward(g.dx, g.dsx, 4, g.layer, h=out.bfloat16(), h_codes=hc, h_scales=hs),
              lambda: tq.scion_fp8_quantize_device(out[:, :24].contiguous()),
              lambda: tq._check(tq._load().scion_fp8_forward(c.dx.data_ptr(), c.dsx.data_ptr(), (1 << 21) + 1, c.layer.handle,
                                                             None, out.data_ptr(), 0, None), "scion_fp8_forward")]
    for f in einval:
        with pytest.raises(tq.ScionError) as e:
            f()
        assert e.value.status == tq.SCION_EINVAL


def test_launches_are_counted():
    c = Case(3, 256, 128)
    before = tq.scion_kernel_launches()
    c.run(F32)
    tq.scion_rmsnorm_forward(torch.ones((2, 256), device=DEV), 2, torch.ones(256, dtype=BF16, device=DEV), 1e-6,
                             y=torch.empty((2, 256), dtype=BF16, device=DEV))
    assert tq.scion_kernel_launches() == before + 2


def test_empty_batches():
    c, g = Case(4, 256, 128), Case(4, 256, 128, gated=True)
    none = lambda n, t: torch.empty((0, n), dtype=t, device=DEV)  # noqa: E731
    x, s = none(256, torch.uint8), none(2, torch.uint8)
    tq.scion_fp8_forward(x, s, 0, c.layer, none(128, F32))
    tq.scion_fp8_gated_forward(x, s, 0, g.layer, h=none(128, BF16))
    tq.scion_fp8_gated_forward(x, s, 0, g.layer, h_codes=none(128, torch.uint8), h_scales=none(1, torch.uint8))
    tq.scion_rmsnorm_forward(none(256, F32), 0, torch.ones(256, dtype=BF16, device=DEV), 1e-6, y=none(256, BF16))
    codes, scales = tq.scion_fp8_quantize_device(none(256, F32))
    assert codes.shape == (0, 256) and scales.shape == (0, 2)


@pytest.mark.parametrize("T", [3, 200])
def test_block_with_an_8_bit_shared_expert(T):
    """The operators beside the ternary block as a model layer runs them: the residual add and norm feed
    the block (bf16) and an 8-bit shared expert, both added to the residual stream."""
    import oracle
    from tests.helpers import bf16, device_layer, oracle_layer_packed, packed_banks, with_margin
    from workloads import synth

    cfg = synth.Config("fp8 shared", 61, 256, 16, 4, 128, 0, synth.PQ2_0, 16, True, [8], 1)
    L = synth.layer_host(cfg)
    banks = packed_banks(cfg, L)
    ol = oracle_layer_packed(cfg, L, banks)
    y16 = with_margin(cfg, ol, synth.x_host(cfg, T))
    layer = device_layer(cfg, L, banks, max(T, 16))
    rng = np.random.default_rng(3)
    d, F = cfg.d, 144
    gate, up, down = (quantized(rng, a, b, 128, b ** -0.5) for a, b in ((F, d), (F, d), (d, F)))
    ffn = tq.scion_fp8_create(dev_codes(gate[0]), dev_scales(gate[1]), dev_codes(up[0]), dev_scales(up[1]))
    proj = tq.scion_fp8_create(dev_codes(down[0]), dev_scales(down[1]))
    # a residual stream whose norm with eps = 0 is close to the margin-filtered tokens; the block then runs
    # on the norm's own bf16 output, and tokens whose margin that rounding used up are left out below
    yv = bf16(y16).astype(np.float32)
    resid = torch.from_numpy(rng.standard_normal((T, d)).astype(np.float32)).to(DEV)
    x = torch.from_numpy(yv).to(DEV) - resid
    stream = torch.empty((T, d), dtype=F32, device=DEV)
    y = torch.empty((T, d), dtype=BF16, device=DEV)
    codes, scales = torch.empty((T, d), dtype=torch.uint8, device=DEV), torch.empty((T, 2), dtype=torch.uint8, device=DEV)
    hc, hs = torch.empty((T, F), dtype=torch.uint8, device=DEV), torch.empty((T, 2), dtype=torch.uint8, device=DEV)
    one = torch.ones(d, dtype=BF16, device=DEV)
    out = torch.empty((T, d), dtype=F32, device=DEV)
    tq.scion_rmsnorm_forward(x, T, one, 0.0, resid=resid, resid_out=stream, y=y, y_codes=codes, y_scales=scales)
    tq.scion_moe_forward_residual(y, T, layer, stream, out)
    tq.scion_fp8_gated_forward(codes, scales, T, ffn, h_codes=hc, h_scales=hs)
    tq.scion_fp8_forward(hc, hs, T, proj, out, base=out)
    # each step against its definition on the inputs it got
    check_norm(x.cpu(), resid.cpu(), one.cpu(), 0.0, stream, y, codes, scales)
    yb = y.view(torch.int16).cpu().numpy().view(np.uint16)
    logits, _, _ = oracle.route(ol, yb)
    top = -np.sort(-logits, axis=1)
    ok = top[:, cfg.top_k - 1] - top[:, cfg.top_k] >= 1e-4
    assert ok.sum() >= T * 0.9
    block, _, _ = oracle.forward(ol, yb)
    h = R.values(bytes_of(hc), bytes_of(hs), 1)
    xv = R.values(bytes_of(codes), bytes_of(scales), 1)
    gv, uv = R.values(*gate, 128), R.values(*up, 128)
    R.check_codes(bytes_of(hc), bytes_of(hs),
                  *gated_value(xv @ gv.T, xv @ uv.T, *(d * 2.0 ** -23 * (np.abs(xv) @ np.abs(m).T) for m in (gv, uv))))
    dv = R.values(*down, 128)
    ref = host(stream) + block + h @ dv.T
    err = np.linalg.norm(host(out) - ref, axis=1)
    # the block's own tolerance on its share, the sums' bound on the rest
    tol = 1e-3 * np.linalg.norm(block, axis=1) + np.linalg.norm(F * 2.0 ** -23 * (np.abs(h) @ np.abs(dv).T), axis=1)
    tol += 2.0 ** -22 * (np.linalg.norm(ref, axis=1) + np.linalg.norm(host(stream), axis=1))
    assert (err[ok] <= tol[ok]).all()
