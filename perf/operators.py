"""Measured cases of the 4-bit layer and of the norms and gated residuals around it.

Four operators, each in its plain form (elementary torch operations in fp32)
and, with ``own``, as the calls a user makes of this package:

* quant     rows to 4-bit floating point (e2m1) codes with one power-of-two
            scale per 32 elements, returned as the values they stand for;
* linear    the 4-bit layer: such rows against 4-bit weights, from 16-bit
            activations (``codes`` false) or from codes in hand;
* norm      the norm before a block with its modulation, as 16-bit values
            or as int8 / e4m3 codes with a scale per row;
* residual  the gate, residual scale and norm after a block, with the next
            block's norm in the same call.
"""
import torch

own = False

DTYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}
BLOCK = 32
EPS = 1e-6


# ---- the cases ------------------------------------------------------------

def quant_case(m, k, dtype, **more):
    return {"op": "quant", "m": m, "k": k, "dtype": dtype, **more}


def linear_case(m, k, n, dtype, bias, codes, **more):
    return {"op": "linear", "m": m, "k": k, "n": n, "dtype": dtype, "bias": bias, "codes": codes, **more}


def norm_case(batch, tokens, k, dtype, kind, affine, modulated, vectors, out, **more):
    return {"op": "norm", "batch": batch, "tokens": tokens, "k": k, "dtype": dtype, "kind": kind,
            "affine": affine, "modulated": modulated, "vectors": vectors, "out": out, **more}


def residual_case(batch, tokens, k, dtype, stream, post, gate, kind, vectors, out, **more):
    return {"op": "residual", "batch": batch, "tokens": tokens, "k": k, "dtype": dtype,
            "stream": stream, "post": post, "gate": gate, "kind": kind, "vectors": vectors, "out": out, **more}


def listed():
    return [
        # One decoded token's activations on their way into a 4-bit layer.
        quant_case(1, 4096, "bfloat16", name="quant_token"),
        # The hidden rows of a feed-forward block in a large image batch.
        quant_case(8192, 12288, "bfloat16", name="quant_ffn_rows"),
        # One token through a fused-QKV layer: the 4-bit weight is what moves.
        linear_case(1, 4096, 12288, "bfloat16", False, False, name="linear_token"),
        # A ragged text prompt against an odd projection, fp16 with a bias.
        linear_case(77, 4128, 1111, "float16", True, False, name="linear_prompt_odd"),
        # The fused-QKV layer of a short image sequence.
        linear_case(512, 4096, 12288, "bfloat16", False, False, name="linear_fused_qkv"),
        # A down-projection over many rows whose codes are already there.
        linear_case(8192, 12288, 4096, "bfloat16", True, True, name="linear_ffn_down"),
        # A decoded token's norm in front of an int8 layer.
        norm_case(1, 1, 4096, "bfloat16", "rms", True, False, "bfloat16", "int8", name="norm_token_int8"),
        # The modulated norm of a diffusion block, two images with a vector each.
        norm_case(2, 4096, 4096, "bfloat16", "layer", False, True, "float32", "same", name="norm_modulated"),
        # Long rows in front of an e4m3 layer.
        norm_case(1, 8192, 12288, "bfloat16", "rms", True, False, "bfloat16", "fp8", name="norm_rows_fp8"),
        # A few decoded tokens back into the residual stream.
        residual_case(4, 1, 4096, "bfloat16", "bfloat16", "none", False, "rms", "bfloat16", "int8",
                      name="residual_tokens"),
        # An odd width in fp16 with an fp32 stream and nothing after it.
        residual_case(3, 333, 5001, "float16", "float32", "rms", True, "none", "float32", "same",
                      name="residual_odd_fp32"),
        # The end of a diffusion block and the start of the next.
        residual_case(2, 4096, 4096, "bfloat16", "bfloat16", "rms", True, "layer", "bfloat16", "same",
                      name="residual_block"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["quant", "linear", "linear", "norm", "residual"])
    half = rng.choice(["bfloat16", "float16"])
    if op == "quant":
        return quant_case(_log(rng, 1, 8192), BLOCK * _log(rng, 2, 384),
                          rng.choice(["bfloat16", "float16", "float32"]))
    if op == "linear":
        return linear_case(_log(rng, 1, 8192), BLOCK * _log(rng, 4, 384), _log(rng, 16, 4096), half,
                           rng.random() < 0.5, rng.random() < 0.4)
    batch = rng.choice([1, 2, 3, 4])
    tokens, k = _log(rng, 1, 2048), _log(rng, 48, 12288)
    vectors = rng.choice([half, "float32"])
    out = rng.choice(["same", "int8", "fp8"])
    if op == "norm":
        return norm_case(batch, tokens, k, half, rng.choice(["rms", "layer"]), rng.random() < 0.6,
                         rng.random() < 0.6, vectors, out)
    kind = rng.choice(["rms", "layer", "none"])
    return residual_case(batch, tokens, k, half, rng.choice([half, "float32"]),
                         rng.choice(["none", "rms", "layer"]), rng.random() < 0.7, kind, vectors,
                         "same" if kind == "none" else out)


def work(case):
    k = case["k"]
    if case["op"] == "quant":
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": case["m"] * k * (size + size), "flops": 4 * case["m"] * k}
    if case["op"] == "linear":
        m, n = case["m"], case["n"]
        packed = 17 / 32
        return {"bytes": m * k * (packed if case["codes"] else 2) + n * k * packed + 2 * m * n +
                (2 * n if case["bias"] else 0), "flops": 2 * m * n * k}
    m, g = case["batch"] * case["tokens"], case["batch"]
    vec = 4 if case["vectors"] == "float32" else 2
    made = 2 if case["out"] == "same" else 1
    if case["op"] == "norm":
        vectors = (1 if case["kind"] == "rms" else 2) * case["affine"] + 2 * g * case["modulated"]
        return {"bytes": m * k * (2 + made) + vectors * k * vec, "flops": 8 * m * k}
    stream = 4 if case["stream"] == "float32" else 2
    vectors = (case["post"] != "none") + g * case["gate"] + 2 * g * (case["kind"] != "none")
    return {"bytes": m * k * (2 + 2 * stream + (made if case["kind"] != "none" else 0)) + vectors * k * vec,
            "flops": 16 * m * k}


# ---- inputs ---------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows(g, m, k, dtype, outliers=True):
    """Activations: normal values, one column in a hundred 12 times as large,
    row magnitudes log-uniform over a factor of ten."""
    x = torch.randn(m, k, device="cuda", generator=g)
    if outliers:
        x *= torch.where(torch.rand(k, device="cuda", generator=g) < 0.01, 12.0, 1.0)
        x *= 10.0 ** (torch.rand(m, 1, device="cuda", generator=g) - 0.5)
    return x.to(dtype)


def _blocks(x):
    """Exponent of each block of 32 (fp32 [.., K/32, 1]) and the elements over
    2^exponent, rounded to the e2m1 grid (fp32 [.., K/32, 32])."""
    b = x.float().reshape(x.shape[0], -1, BLOCK)
    a = b.abs().amax(-1, keepdim=True)
    e = torch.where(a > 0, torch.frexp(a).exponent - 3, -127).clamp(-127, 127).float()
    v = b * torch.exp2(-e)
    step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0))
    return e, (torch.round(v / step) * step).clamp(-6, 6)


def _pack(x):
    """uint8 codes [M, K/2] (even k in the low nibble) and scale bytes [M, K/32]."""
    e, v = _blocks(x)
    a = v.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (code | (torch.signbit(v).to(torch.uint8) << 3)).reshape(x.shape[0], -1)
    return code[:, 0::2] | (code[:, 1::2] << 4), (e.squeeze(-1) + 127).to(torch.uint8)


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _values(codes, scales, dtype):
    """The values that packed codes and scales stand for, in fp32 or fp64."""
    table = torch.tensor(_E2M1, dtype=dtype, device=codes.device)
    nibbles = torch.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1, BLOCK)
    v = table[nibbles.int()] * torch.exp2(scales.to(dtype) - 127).unsqueeze(-1)
    return v.reshape(codes.shape[0], -1)


def prepare(case, seed):
    g = _generator(seed)
    dtype, k = DTYPES[case["dtype"]], case["k"]
    s = {"case": case}
    if case["op"] == "quant":
        s["x"] = _rows(g, case["m"], k, dtype)
        return s
    if case["op"] == "linear":
        n = case["n"]
        x = _rows(g, case["m"], k, dtype)
        w = torch.randn(n, k, device="cuda", generator=g) * 0.02
        s["wq"], s["ws"] = _pack(w)
        s["bias"] = (0.1 * torch.randn(n, device="cuda", generator=g)).to(dtype) if case["bias"] else None
        if case["codes"]:
            s["xq"], s["xs"] = _pack(x)
        else:
            s["x"] = x
        if own:
            from w8a8_int8_dynamic_amd import W8A8Linear, ops
            if case["codes"]:
                s["packed"], s["packed_scale"] = ops.fp4_prepack_weight(s["wq"], s["ws"])
            else:
                s["layer"] = W8A8Linear.from_quantized(s["wq"], s["ws"], s["bias"], scheme="fp4")
        return s
    batch, m = case["batch"], case["batch"] * case["tokens"]
    vec = DTYPES[case["vectors"]]

    def vectors(rows, mean, spread):
        shape = (k,) if rows is None else (rows, k)
        return (mean + spread * torch.randn(shape, device="cuda", generator=g)).to(vec)

    if case["op"] == "norm":
        s["x"] = _rows(g, m, k, dtype)
        s["weight"] = vectors(None, 1.0, 0.2) if case["affine"] else None
        s["bias"] = vectors(None, 0.0, 0.2) if case["affine"] and case["kind"] == "layer" else None
        # A model's modulation vectors are columns of one projection of its conditioning.
        if case["modulated"]:
            both = vectors(batch, 0.0, 0.3).repeat(1, 2)
            both[:, k:] = vectors(batch, 0.0, 0.3)
        s["scale"], s["shift"] = (both[:, :k], both[:, k:]) if case["modulated"] else (None, None)
        return s
    s["x"] = _rows(g, m, k, DTYPES[case["stream"]])
    s["y"] = _rows(g, m, k, dtype)
    s["post_weight"] = vectors(None, 1.0, 0.2) if case["post"] != "none" else None
    s["gate"] = vectors(batch, 0.0, 0.5) if case["gate"] else None
    s["scale"], s["shift"] = (vectors(batch, 0.0, 0.3), vectors(batch, 0.0, 0.3)) \
        if case["kind"] != "none" else (None, None)
    return s


# ---- the plain forms --------------------------------------------------------

def _normed(t, kind, weight, bias):
    if kind == "layer":
        t = t - t.mean(-1, keepdim=True)
    t = t * torch.rsqrt((t * t).mean(-1, keepdim=True) + EPS)
    if weight is not None:
        t = t * weight.to(t.dtype)
    return t if bias is None else t + bias.to(t.dtype)


def _modulated(t, scale, shift):
    if scale is None:
        return t
    t = t.reshape(scale.shape[0], -1, t.shape[-1])
    t = t * (1 + scale.to(t.dtype).unsqueeze(1)) + shift.to(t.dtype).unsqueeze(1)
    return t.reshape(-1, t.shape[-1])


def _gated(t, gate):
    if gate is None:
        return t
    return (t.reshape(gate.shape[0], -1, t.shape[-1]) * gate.to(t.dtype).unsqueeze(1)).reshape(t.shape)


def _out(h, out, dtype):
    """h as 16-bit values, or as (codes as the values they stand for, row scales)."""
    if out == "same":
        return h.to(dtype)
    top = 127.0 if out == "int8" else 448.0
    a = h.abs().amax(-1, keepdim=True)
    v = (h * (top / a)).clamp(-top, top)
    v = torch.round(v).to(torch.bfloat16) if out == "int8" else v.to(torch.float8_e4m3fn)
    return v, (a / top).squeeze(-1)


RESIDUAL_SCALE, BRANCH_SCALE = 0.9, 1.1


def _residual(s):
    """The updated residual stream and, where the case has one, the next norm of it (both before rounding)."""
    case = s["case"]
    y = s["y"].float()
    if case["post"] != "none":
        y = _normed(y, case["post"], s["post_weight"], None)
    r = RESIDUAL_SCALE * s["x"].float() + BRANCH_SCALE * _gated(y, s["gate"])
    if case["kind"] == "none":
        return r, None
    return r, _modulated(_normed(r, case["kind"], None, None), s["scale"], s["shift"])


def _plain(s):
    case = s["case"]
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "quant":
        e, v = _blocks(s["x"])
        return (v * torch.exp2(e)).reshape(s["x"].shape).to(dtype)
    if case["op"] == "linear":
        if case["codes"]:
            x = _values(s["xq"], s["xs"], torch.float32)
        else:
            e, v = _blocks(s["x"])
            x = (v * torch.exp2(e)).reshape(s["x"].shape)
        t = x @ _values(s["wq"], s["ws"], torch.float32).t()
        return (t if s["bias"] is None else t + s["bias"].float()).to(dtype)
    if case["op"] == "norm":
        h = _modulated(_normed(s["x"].float(), case["kind"], s["weight"], s["bias"]), s["scale"], s["shift"])
        return _out(h, case["out"], dtype)
    r, h = _residual(s)
    r = r.to(DTYPES[case["stream"]])
    return r if h is None else (r, _out(h, case["out"], dtype))


# ---- the framework's calls ----------------------------------------------------

def _codes(xq, xs, out):
    return (xq.to(torch.bfloat16) if out == "int8" else xq.view(torch.float8_e4m3fn)), xs


def _own(s):
    from w8a8_int8_dynamic_amd import ops
    case = s["case"]
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "quant":
        return ops.fp4_dequant(*ops.fp4_quant_per_block(s["x"]), dtype=dtype)
    if case["op"] == "linear":
        if not case["codes"]:
            return s["layer"](s["x"])
        return ops.fp4_scaled_mm(s["xq"], s["xs"], s["packed"], s["packed_scale"], case["n"], s["bias"],
                                   out_dtype=dtype)
    out = case["out"]
    if case["op"] == "norm":
        norm = ops.Norm(case["kind"], weight=s["weight"], bias=s["bias"], scale=s["scale"], shift=s["shift"],
                        eps=EPS)
        if out == "same":
            return ops.norm(s["x"], norm)
        quant = ops.norm_quant_per_token if out == "int8" else ops.fp8_norm_quant_per_token
        return _codes(*quant(s["x"], norm), out)
    post = None if case["post"] == "none" else ops.Norm(case["post"], weight=s["post_weight"], eps=EPS)
    more = {"gate": s["gate"], "post": post, "residual_scale": RESIDUAL_SCALE, "branch_scale": BRANCH_SCALE}
    if case["kind"] == "none":
        return ops.gated_residual(s["x"], s["y"], **more)
    norm = ops.Norm(case["kind"], scale=s["scale"], shift=s["shift"], eps=EPS)
    if out == "same":
        return ops.gated_residual_norm(s["x"], s["y"], norm, **more)
    quant = ops.gated_residual_norm_quant if out == "int8" else ops.fp8_gated_residual_norm_quant
    r, xq, xs = quant(s["x"], s["y"], norm, **more)
    return r, _codes(xq, xs, out)


def run(state):
    return _own(state) if own else _plain(state)


# ---- the definition in 64 bits ------------------------------------------------

def _grid64(x):
    """The values that x's 4-bit codes stand for, by distance to every grid value."""
    b = x.double().reshape(x.shape[0], -1, BLOCK)
    a = b.abs().amax(-1, keepdim=True)
    e = torch.where(a > 0, torch.floor(torch.log2(a)) - 2, -127.0).clamp(-127, 127)
    # floor(log2) of an exact power of two, whatever the logarithm's last bit
    e = torch.where(a >= torch.exp2(e + 3), e + 1, e)
    e = torch.where((a < torch.exp2(e + 2)) & (e > -127), e - 1, e)
    v = (b / torch.exp2(e)).abs()
    # steps of the grid 0, .5, 1, 1.5, 2, 3, 4, 6 past each halfway point: a tie goes to the even code
    q = 0.5 * (v > 0.25).double() + 0.5 * (v >= 0.75) + 0.5 * (v > 1.25) + 0.5 * (v >= 1.75) + \
        1.0 * (v > 2.5) + 1.0 * (v >= 3.5) + 2.0 * (v > 5.0)
    return (torch.copysign(q, b) * torch.exp2(e)).reshape(x.shape)


def _stats64(t, kind):
    mean = t.mean(-1, keepdim=True) if kind == "layer" else 0.0
    return (t - mean) / torch.sqrt(((t - mean) ** 2).mean(-1, keepdim=True) + EPS)


def _per_row(v, m):
    return v.double().repeat_interleave(m // v.shape[0], 0)


def _out64(h, out):
    if out == "same":
        return h
    top = 127.0 if out == "int8" else 448.0
    a = h.abs().amax(-1, keepdim=True)
    v = h * top / a
    if out == "int8":
        return torch.round(v), (a / top).squeeze(-1)
    # e4m3: 3 mantissa bits, smallest exponent -6
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))).clamp(-6, 8)
    return torch.round(v * torch.exp2(3 - e)) * torch.exp2(e - 3), (a / top).squeeze(-1)


def exact(case, seed):
    s = prepare(case, seed)
    m = s["x"].shape[0] if "x" in s else s["xq"].shape[0]
    if case["op"] == "quant":
        return _grid64(s["x"])
    if case["op"] == "linear":
        x = _values(s["xq"], s["xs"], torch.float64) if case["codes"] else _grid64(s["x"])
        t = torch.mm(x, _values(s["wq"], s["ws"], torch.float64).t())
        return t if s["bias"] is None else t + s["bias"].double()
    if case["op"] == "norm":
        h = _stats64(s["x"].double(), case["kind"])
        h = h if s["weight"] is None else h * s["weight"].double()
        h = h if s["bias"] is None else h + s["bias"].double()
        if s["scale"] is not None:
            h = h * (1 + _per_row(s["scale"], m)) + _per_row(s["shift"], m)
        return _out64(h, case["out"])
    y = s["y"].double()
    if case["post"] != "none":
        y = _stats64(y, case["post"]) * s["post_weight"].double()
    if s["gate"] is not None:
        y = y * _per_row(s["gate"], m)
    r = RESIDUAL_SCALE * s["x"].double() + BRANCH_SCALE * y
    if case["kind"] == "none":
        return r
    return r, _out64(_stats64(r, case["kind"]) * (1 + _per_row(s["scale"], m)) + _per_row(s["shift"], m), case["out"])
