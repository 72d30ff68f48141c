"""What is measured of the 8-bit operators: the block-scaled quantizer, the residual add with root-mean-square norm, the
block-scaled matrix product and the gated product, at the sizes a model around one MoE block runs them.

`run` calls the library where `own` is true and plain torch operations where it is false.  Values in 8 bits are e4m3 codes
(torch.float8_e4m3fn) with one power-of-two scale (torch.float8_e8m0fnu) per 128 columns of a row, or per 128 x 128 block of a
weight matrix: s is the smallest power of two with max|v| / s <= 448, and a block of zeros has s = 1.
"""
import math

import torch

own = False  # set from outside: True runs the library's kernels, False the plain forms

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2, "none": 0}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a decode batch's attention output quantised per token before its output projection
        {"name": "quant_rows_64x2048", "op": "quant", "rows": 64, "cols": 2048, "src": "bf16", "block_rows": 1},
        # a projection's weights quantised in 128 x 128 blocks when a model is loaded
        {"name": "quant_blocks_4096x2048", "op": "quant", "rows": 4096, "cols": 2048, "src": "f32", "block_rows": 128},
        # one token of decode: the previous block's fp32 output joins the fp32 residual stream; bf16 for the MoE
        # block and its router, 8 bits for the dense products
        {"name": "norm_t1_d2048", "op": "norm", "T": 1, "d": 2048, "x": "f32", "resid": "f32", "y": "both"},
        # a small ragged prompt of an odd width, bf16 residual stream, bf16 norm only
        {"name": "norm_t333_d1936", "op": "norm", "T": 333, "d": 1936, "x": "bf16", "resid": "bf16", "y": "bf16"},
        # a long prompt: bf16 sublayer output, fp32 residual stream, 8-bit output
        {"name": "norm_t16384_d4096", "op": "norm", "T": 16384, "d": 4096, "x": "bf16", "resid": "f32", "y": "fp8"},
        # one token through a projection (attention queries of a d = 2048 model)
        {"name": "linear_t1_2048x4096", "op": "linear", "T": 1, "K": 2048, "N": 4096, "out": "bf16", "base": False},
        # the largest decode batch through a projection back into the fp32 residual stream
        {"name": "linear_t64_4096x2048_base", "op": "linear", "T": 64, "K": 4096, "N": 2048, "out": "f32", "base": True},
        # a ragged prompt, K that ends inside a block of 128, an odd number of outputs
        {"name": "linear_t1000_2064x1111", "op": "linear", "T": 1000, "K": 2064, "N": 1111, "out": "bf16", "base": False},
        # a long prompt through a wide projection
        {"name": "linear_t16384_4096x4096", "op": "linear", "T": 16384, "K": 4096, "N": 4096, "out": "bf16", "base": False},
        # the shared expert of a 256-expert layer, one token
        {"name": "gated_t1_2048x512", "op": "gated", "T": 1, "K": 2048, "F": 512, "out": "fp8"},
        # a dense feed-forward layer at a ragged decode batch, a hidden width that ends inside a block
        {"name": "gated_t50_2048x5456", "op": "gated", "T": 50, "K": 2048, "F": 5456, "out": "fp8"},
        # the same layer's prefill
        {"name": "gated_t4096_2048x5504", "op": "gated", "T": 4096, "K": 2048, "F": 5504, "out": "fp8"},
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of `step` in [lo, hi], its logarithm uniform."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(["quant", "norm", "linear", "linear", "gated", "gated"])
    if op == "quant":
        rows = _spread(rng, 1, 16384)
        return {"op": op, "rows": rows, "cols": _spread(rng, 128, min(8192, 67108864 // rows), 16),
                "src": rng.choice(["f32", "bf16"]), "block_rows": rng.choice([1, 128])}
    T = _spread(rng, 1, 16384)
    if op == "norm":
        return {"op": op, "T": T, "d": _spread(rng, 128, min(8192, 67108864 // T), 16), "x": rng.choice(["f32", "bf16"]),
                "resid": rng.choice(["f32", "bf16", "none"]), "y": rng.choice(["bf16", "fp8", "both"])}
    K = _spread(rng, 128, 8192, 16)
    most = min(8192, (16384 * 4096 * 4096) // (T * K), 67108864 // T)
    if op == "linear":
        out = rng.choice(["f32", "bf16"])
        return {"op": op, "T": T, "K": K, "N": _spread(rng, 64, most), "out": out, "base": rng.choice([True, False])}
    return {"op": op, "T": T, "K": K, "F": _spread(rng, 64, max(64, most // 2), 16), "out": rng.choice(["bf16", "fp8"])}


# ------------------------------------------------------------------ inputs
def _blocks(v, block_rows):
    """v [R, C] fp32 -> [ceil(R/br), br, ceil(C/128), 128], zeros past the edges."""
    R, C = v.shape
    v = torch.nn.functional.pad(v, (0, -C % 128, 0, -R % block_rows))
    return v.reshape(v.shape[0] // block_rows, block_rows, -1, 128)


def _quantize(v, block_rows):
    """v [R, C] fp32 -> e4m3 codes [R, C], power-of-two scales [ceil(R/br), ceil(C/128)]."""
    R, C = v.shape
    b = _blocks(v, block_rows)
    amax = b.abs().amax(dim=(1, 3))
    m, e = torch.frexp(amax)  # amax = m 2^e, m in [1/2, 1);  448 = 7/8 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax == 0, torch.zeros_like(e), e)
    s = torch.ldexp(torch.ones_like(amax), e)
    q = (b / s[:, None, :, None]).reshape(b.shape[0] * block_rows, -1)[:R, :C]
    return q.to(torch.float8_e4m3fn).contiguous(), s.to(torch.float8_e8m0fnu)


def _values(codes, scales, block_rows):
    """The fp32 values that codes and scales stand for."""
    R, C = codes.shape
    s = scales.float().repeat_interleave(128, 1)[:, :C]
    if block_rows > 1:
        s = s.repeat_interleave(block_rows, 0)[:R]
    return codes.float() * s


def _activations(g, T, d):
    """Rows of different size with a few channels far above the rest, as a residual stream has them."""
    v = torch.randn(T, d, generator=g, device=DEV)
    v *= torch.exp(0.5 * torch.randn(T, 1, generator=g, device=DEV))
    far = torch.rand(d, generator=g, device=DEV) < 0.004
    return torch.where(far, 20 * v, v)


def _weights(g, N, K):
    w = torch.randn(N, K, generator=g, device=DEV) * K ** -0.5
    return _quantize(w * torch.exp(0.3 * torch.randn(N, 1, generator=g, device=DEV)), 128)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    op, st = case["op"], {"case": case}
    empty = lambda shape, t: torch.empty(shape, dtype=t, device=DEV)  # noqa: E731
    e4, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    groups = lambda n: (n + 127) // 128  # noqa: E731
    if op == "quant":
        R, C, br = case["rows"], case["cols"], case["block_rows"]
        v = _activations(g, R, C) if br == 1 else 0.02 * torch.randn(R, C, generator=g, device=DEV)
        st |= {"v": v.to(TYPES[case["src"]]), "codes": empty((R, C), e4), "scales": empty(((R + br - 1) // br, groups(C)), e8)}
    elif op == "norm":
        T, d = case["T"], case["d"]
        st["x"] = torch.randn(T, d, generator=g, device=DEV).to(TYPES[case["x"]])
        st["w"] = (1 + 0.1 * torch.randn(d, generator=g, device=DEV)).to(torch.bfloat16)
        st["resid"] = st["resid_out"] = st["y"] = st["codes"] = st["scales"] = None
        if case["resid"] != "none":
            st["resid"] = _activations(g, T, d).to(TYPES[case["resid"]])
            st["resid_out"] = torch.empty_like(st["resid"])
        if case["y"] in ("bf16", "both"):
            st["y"] = empty((T, d), torch.bfloat16)
        if case["y"] in ("fp8", "both"):
            st |= {"codes": empty((T, d), e4), "scales": empty((T, groups(d)), e8)}
    else:
        T, K = case["T"], case["K"]
        st["x"], st["sx"] = _quantize(_activations(g, T, K), 1)
        if op == "linear":
            N = case["N"]
            st["w"], st["sw"] = _weights(g, N, K)
            st["out"] = empty((T, N), TYPES[case["out"]])
            st["base"] = _activations(g, T, N) if case["base"] else None
        else:
            F = case["F"]
            st["w"], st["sw"] = _weights(g, F, K)
            st["up"], st["su"] = _weights(g, F, K)
            st["h"] = st["codes"] = st["scales"] = None
            if case["out"] == "bf16":
                st["h"] = empty((T, F), torch.bfloat16)
            else:
                st |= {"codes": empty((T, F), e4), "scales": empty((T, groups(F)), e8)}
        if own:
            import ternary_quantized_moe_b200 as tq

            st["layer"] = tq.scion_fp8_create(st["w"], st["sw"], st.get("up"), st.get("su"))
    return st


# ------------------------------------------------------------------ one pass
def _run_own(st):
    import ternary_quantized_moe_b200 as tq

    case = st["case"]
    op = case["op"]
    if op == "quant":
        tq.scion_fp8_quantize_device(st["v"], st["codes"], st["scales"], block_rows=case["block_rows"])
        return {"codes": st["codes"], "scales": st["scales"]}
    if op == "norm":
        tq.scion_rmsnorm_forward(st["x"], case["T"], st["w"], 1e-6, resid=st["resid"], resid_out=st["resid_out"], y=st["y"],
                                 y_codes=st["codes"], y_scales=st["scales"])
        return {k: st[k] for k in ("resid_out", "y", "codes", "scales")}
    if op == "linear":
        tq.scion_fp8_forward(st["x"], st["sx"], case["T"], st["layer"], st["out"], base=st["base"])
        return {"out": st["out"]}
    tq.scion_fp8_gated_forward(st["x"], st["sx"], case["T"], st["layer"], h=st["h"], h_codes=st["codes"], h_scales=st["scales"])
    return {k: st[k] for k in ("h", "codes", "scales")}


def run(st):
    if own:
        return _run_own(st)
    case = st["case"]
    op = case["op"]
    if op == "quant":
        codes, scales = _quantize(st["v"].float(), case["block_rows"])
        return {"codes": codes, "scales": scales}
    if op == "norm":
        r, out = st["x"].float(), {}
        if st["resid"] is not None:
            r = r + st["resid"].float()
            out["resid_out"] = r.to(st["resid"].dtype)
        y = r * torch.rsqrt(r.square().mean(1, keepdim=True) + 1e-6) * st["w"].float()
        if case["y"] in ("bf16", "both"):
            out["y"] = y.to(torch.bfloat16)
        if case["y"] in ("fp8", "both"):
            out["codes"], out["scales"] = _quantize(y, 1)
        return out
    x = _values(st["x"], st["sx"], 1)
    p = x @ _values(st["w"], st["sw"], 128).T
    if op == "linear":
        if st["base"] is not None:
            p = st["base"] + p
        return {"out": p.to(TYPES[case["out"]])}
    h = p * torch.sigmoid(p) * (x @ _values(st["up"], st["su"], 128).T)
    if case["out"] == "bf16":
        return {"h": h.to(torch.bfloat16)}
    codes, scales = _quantize(h, 1)
    return {"codes": codes, "scales": scales}


def work(case):
    op = case["op"]
    if op == "quant":
        R, C, br = case["rows"], case["cols"], case["block_rows"]
        return {"bytes": R * C * (BYTES[case["src"]] + 1) + ((R + br - 1) // br) * ((C + 127) // 128), "flops": 0}
    if op == "norm":
        T, d = case["T"], case["d"]
        per = BYTES[case["x"]] + 2 * BYTES[case["resid"]] + (2 if case["y"] != "fp8" else 0) + (1 if case["y"] != "bf16" else 0)
        return {"bytes": T * d * per + 2 * d + (T * ((d + 127) // 128) if case["y"] != "bf16" else 0), "flops": 0}
    T, K = case["T"], case["K"]
    kb = (K + 127) // 128
    if op == "linear":
        N = case["N"]
        moved = T * (K + kb) + N * K + (N + 127) // 128 * kb + T * N * (BYTES[case["out"]] + (4 if case["base"] else 0))
        return {"bytes": moved, "flops": 2 * T * N * K}
    F = case["F"]
    wide = F * 2 if case["out"] == "bf16" else F + (F + 127) // 128
    return {"bytes": T * (K + kb) + 2 * (F * K + (F + 127) // 128 * kb) + T * wide, "flops": 4 * T * F * K}


# ------------------------------------------------------------------ the definition in 64 bits
def _e4m3_table():
    """The 256 codes: sign, 4 exponent bits of bias 7, 3 mantissa bits; exponent and mantissa all ones is no number."""
    t = []
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        a = math.nan if (e, m) == (15, 7) else (m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10))
        t.append(-a if c & 128 else a)
    return torch.tensor(t, dtype=torch.float64, device=DEV)


def _exact_values(codes, scales, rows_per_scale):
    v = _e4m3_table()[codes.view(torch.uint8).int()]
    s = torch.exp2(scales.view(torch.uint8).double() - 127)
    rows = torch.arange(v.shape[0], device=DEV) // rows_per_scale
    cols = torch.arange(v.shape[1], device=DEV) // 128
    return v * s[rows][:, cols]


def _exact_codes(v, block_rows):
    """v / s before it is rounded to a code, s decided in 64 bits."""
    R, C = v.shape
    nr, nc = (R + block_rows - 1) // block_rows, (C + 127) // 128
    full = torch.zeros(nr * block_rows, nc * 128, dtype=torch.float64, device=DEV)
    full[:R, :C] = v
    amax = full.abs().view(nr, block_rows, nc, 128).amax(3).amax(1)
    e = torch.ceil(torch.log2(amax.clamp_min(1e-300) / 448)).clamp_min(-127)
    e = torch.where(amax * torch.exp2(-e) > 448, e + 1, e)
    e = torch.where(amax * torch.exp2(1 - e) <= 448, e - 1, e)
    s = torch.where(amax == 0, torch.ones_like(amax), torch.exp2(e))
    rows = torch.arange(R, device=DEV) // block_rows
    cols = torch.arange(C, device=DEV) // 128
    return v / s[rows][:, cols]


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "quant":
        # (a scale has no value before its rounding that it could be held to: the codes' values carry it)
        return {"codes": _exact_codes(st["v"].double(), case["block_rows"]), "scales": None}
    if op == "norm":
        r = st["x"].double() + (0 if st["resid"] is None else st["resid"].double())
        y = st["w"].double() * r / torch.sqrt((r * r).sum(1, keepdim=True) / case["d"] + 1e-6)
        return {"resid_out": None if st["resid"] is None else r, "y": None if st["y"] is None else y,
                "codes": None if st["codes"] is None else _exact_codes(y, 1), "scales": None}
    x = _exact_values(st["x"], st["sx"], 1)
    g = torch.matmul(x, _exact_values(st["w"], st["sw"], 128).t())
    if op == "linear":
        return {"out": g if st["base"] is None else g.add_(st["base"].double())}
    h = g / (1 + torch.exp(-g)) * torch.matmul(x, _exact_values(st["up"], st["su"], 128).t())
    return {"h": h} if case["out"] == "bf16" else {"codes": _exact_codes(h, 1), "scales": None}
