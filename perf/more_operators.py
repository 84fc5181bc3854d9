"""Measured cases of the block-scaled 8-bit layer and of the mixture of experts built on it.

Four operators, each in its plain form (elementary torch operations in fp32,
in fp64 where a choice hangs on the last bits) and, with ``own``, as the calls
a user makes of this package:

* quant     rows to 8-bit floating point (e4m3) codes with one fp32 scale per
            128 elements, returned as the values they stand for;
* linear    such rows against e4m3 weights with one scale per 128 x 128
            block, from 16-bit activations (``codes`` false) or codes in hand;
* route     a router's logits to the experts of each token and their weights;
* experts   the chosen experts' gate, up and down products for each token and
            their weighted sum.
"""
import torch

own = False

DTYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}
BLOCK = 128
TOP = 448.0
LEAST = 2.0 ** -100


# ---- the cases ------------------------------------------------------------

def quant_case(m, k, dtype, **more):
    return {"op": "quant", "m": m, "k": k, "dtype": dtype, **more}


def linear_case(m, k, n, dtype, bias, codes, **more):
    return {"op": "linear", "m": m, "k": k, "n": n, "dtype": dtype, "bias": bias, "codes": codes, **more}


def route_case(tokens, experts, top_k, dtype, score, bias, groups, top_groups, renormalize, **more):
    return {"op": "route", "tokens": tokens, "experts": experts, "top_k": top_k, "dtype": dtype, "score": score,
            "bias": bias, "groups": groups, "top_groups": top_groups, "renormalize": renormalize, **more}


def experts_case(tokens, experts, top_k, k, inner, dtype, **more):
    return {"op": "experts", "tokens": tokens, "experts": experts, "top_k": top_k, "k": k, "inner": inner,
            "dtype": dtype, **more}


def listed():
    return [
        # One decoded token's activations on their way into a block-scaled layer.
        quant_case(1, 4096, "bfloat16", name="quant_token"),
        # The hidden rows of a feed-forward block over a long batch.
        quant_case(8192, 12288, "bfloat16", name="quant_ffn_rows"),
        # One token through a fused-QKV layer: the weight is what moves.
        linear_case(1, 4096, 12288, "bfloat16", False, False, name="linear_token"),
        # A ragged prompt against an odd projection, the last block of K part full, fp16 with a bias.
        linear_case(77, 4112, 1111, "float16", True, False, name="linear_prompt_odd"),
        # The fused-QKV layer of a short sequence.
        linear_case(512, 4096, 12288, "bfloat16", False, False, name="linear_fused_qkv"),
        # A down-projection over many rows whose codes are already there.
        linear_case(8192, 12288, 4096, "bfloat16", True, True, name="linear_ffn_down"),
        # A decoded token at a router that balances by a bias and picks groups first.
        route_case(1, 256, 8, "float32", "sigmoid", True, 8, 4, True, name="route_token"),
        # The same router over a long prompt.
        route_case(8192, 256, 8, "float32", "sigmoid", True, 8, 4, True, name="route_prompt"),
        # One decoded token: its experts' weights are what moves.
        experts_case(1, 64, 8, 4096, 1024, "bfloat16", name="experts_token"),
        # A decode batch that touches nearly every expert with a few rows each.
        experts_case(48, 64, 8, 4096, 1024, "bfloat16", name="experts_decode"),
        # A ragged prompt over fewer, narrower experts, whose last blocks are part full.
        experts_case(333, 24, 3, 2064, 720, "bfloat16", name="experts_prompt_odd"),
        # A long prompt: every expert has hundreds of rows.
        experts_case(4096, 64, 8, 4096, 1024, "bfloat16", name="experts_prompt"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    op = rng.choice(["quant", "linear", "linear", "route", "experts", "experts"])
    half = rng.choice(["bfloat16", "float16"])
    if op == "quant":
        return quant_case(_log(rng, 1, 8192), 16 * _log(rng, 2, 768),
                          rng.choice(["bfloat16", "float16", "float32"]))
    if op == "linear":
        return linear_case(_log(rng, 1, 8192), 16 * _log(rng, 4, 768), _log(rng, 16, 4096), half,
                           rng.random() < 0.5, rng.random() < 0.4)
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        experts = groups * _log(rng, 8, 512 // groups)
        top_groups = rng.randint(1, groups)
        top_k = min(_log(rng, 1, 16), experts // groups * top_groups)
        return route_case(_log(rng, 1, 8192), experts, top_k, rng.choice(["bfloat16", "float16", "float32"]),
                          rng.choice(["softmax", "sigmoid"]), rng.random() < 0.5, groups, top_groups,
                          rng.random() < 0.6)
    experts = _log(rng, 4, 64)
    return experts_case(_log(rng, 1, 2048), experts, min(_log(rng, 1, 8), experts), 16 * _log(rng, 8, 256),
                        16 * _log(rng, 4, 64), "bfloat16")


def _blocks_of(n):
    return -(-n // BLOCK)


def work(case):
    if case["op"] == "route":
        t, e = case["tokens"], case["experts"]
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": t * (e * size + 8 * case["top_k"]) + (4 * e if case["bias"] else 0), "flops": 8 * t * e}
    k = case["k"]
    if case["op"] == "quant":
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": case["m"] * k * (size + size), "flops": 4 * case["m"] * k}
    if case["op"] == "linear":
        m, n = case["m"], case["n"]
        rows = m * (k + 4 * _blocks_of(k)) if case["codes"] else 2 * m * k
        return {"bytes": rows + n * k + 4 * _blocks_of(n) * _blocks_of(k) + 2 * m * n +
                (2 * n if case["bias"] else 0), "flops": 2 * m * n * k}
    t, e, inner = case["tokens"], case["experts"], case["inner"]
    # How many experts t tokens with top_k different ones each touch, were all equally likely.
    touched = e * (1 - (1 - case["top_k"] / e) ** t)
    return {"bytes": int(touched * 3 * inner * k) + 4 * t * k + 8 * t * case["top_k"],
            "flops": 6 * t * case["top_k"] * inner * k}


# ---- inputs ---------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows(g, m, k, dtype):
    """Activations: normal values, one column in a hundred 12 times as large,
    row magnitudes log-uniform over a factor of ten."""
    x = torch.randn(m, k, device="cuda", generator=g)
    x *= torch.where(torch.rand(k, device="cuda", generator=g) < 0.01, 12.0, 1.0)
    x *= 10.0 ** (torch.rand(m, 1, device="cuda", generator=g) - 0.5)
    return x.to(dtype)


def _scales(a):
    """Scale and its reciprocal of blocks whose largest magnitude is a (fp32)."""
    live = a >= LEAST
    return torch.where(live, a / TOP, 0.0), torch.where(live, TOP / a, 0.0)


def _quant(x):
    """e4m3 codes (float8) [M, K] and scales [M, blocks] of rows, a scale per 128 elements."""
    m, k = x.shape
    b = torch.nn.functional.pad(x.float(), (0, -k % BLOCK)).reshape(m, -1, BLOCK)
    s, inv = _scales(b.abs().amax(-1, keepdim=True))
    q = (b * inv).clamp(-TOP, TOP).to(torch.float8_e4m3fn)
    return q.reshape(m, -1)[:, :k], s.squeeze(-1)


def _spread(s, k):
    """Scales per block to scales per element of K."""
    return s.repeat_interleave(BLOCK, -1)[..., :k]


def _weights(g, *shape):
    """A weight [.., N, K] as e4m3 codes (float8) and scales of its 128 x 128 blocks."""
    *lead, n, k = shape
    w = torch.randn(shape, device="cuda", generator=g) * 0.02
    p = torch.nn.functional.pad(w, (0, -k % BLOCK, 0, -n % BLOCK))
    del w
    p = p.reshape(*lead, _blocks_of(n), BLOCK, _blocks_of(k), BLOCK)
    s, inv = _scales(p.abs().amax((-3, -1), keepdim=True))
    q = (p * inv).clamp(-TOP, TOP).to(torch.float8_e4m3fn)
    del p
    q = q.reshape(*lead, _blocks_of(n) * BLOCK, _blocks_of(k) * BLOCK)[..., :n, :k]
    return q.contiguous(), s.squeeze(-1).squeeze(-2)


def _logits(g, tokens, experts, dtype):
    """A router's logits: some experts are more popular than others."""
    popular = 0.5 * torch.randn(experts, device="cuda", generator=g)
    return (torch.randn(tokens, experts, device="cuda", generator=g) + popular).to(dtype)


def prepare(case, seed):
    g = _generator(seed)
    dtype = DTYPES[case["dtype"]]
    s = {"case": case}
    if case["op"] == "route":
        s["logits"] = _logits(g, case["tokens"], case["experts"], dtype)
        s["bias"] = 0.1 * torch.randn(case["experts"], device="cuda", generator=g) if case["bias"] else None
        if own:
            from w8a8_int8_dynamic_amd import ops
            s["routing"] = ops.Routing(case["top_k"], case["score"], bias=s["bias"], groups=case["groups"],
                                       top_groups=case["top_groups"], renormalize=case["renormalize"],
                                       scale=ROUTE_SCALE)
        return s
    k = case["k"]
    if case["op"] == "quant":
        s["x"] = _rows(g, case["m"], k, dtype)
        return s
    if case["op"] == "linear":
        n = case["n"]
        x = _rows(g, case["m"], k, dtype)
        s["wq"], s["ws"] = _weights(g, n, k)
        s["bias"] = (0.1 * torch.randn(n, device="cuda", generator=g)).to(dtype) if case["bias"] else None
        if case["codes"]:
            s["xq"], s["xs"] = _quant(x)
        else:
            s["x"] = x
        if own:
            from w8a8_int8_dynamic_amd import W8A8Linear, ops
            if case["codes"]:
                s["packed"] = ops.fp8_block_prepack_weight(s["wq"].view(torch.uint8))
            else:
                s["layer"] = W8A8Linear.from_quantized(s["wq"].view(torch.uint8), s["ws"], s["bias"],
                                                       scheme="fp8_block")
        return s
    t, e, inner = case["tokens"], case["experts"], case["inner"]
    s["x"] = _rows(g, t, k, dtype)
    s["gate_up"], s["gate_up_scale"] = _gate_up(g, e, inner, k)
    s["down"], s["down_scale"] = _weights(g, e, k, inner)
    order = _logits(g, t, e, torch.float32).sort(dim=-1, descending=True, stable=True)
    s["ids"] = order.indices[:, :case["top_k"]].to(torch.int32).contiguous()
    s["weights"] = torch.softmax(order.values[:, :case["top_k"]], -1).contiguous()
    # The plain form's plan: rows set aside for each expert.
    s["room"] = int(torch.bincount(s["ids"].flatten(), minlength=e).max())
    if own:
        from w8a8_int8_dynamic_amd import W8A8Experts
        s["layer"] = W8A8Experts.from_quantized(s["gate_up"].view(torch.uint8), s["gate_up_scale"],
                                                s["down"].view(torch.uint8), s["down_scale"])
    return s


def _gate_up(g, e, inner, k):
    """Gate rows above up rows [E, 2 * inner, K], each half with block scales of its own."""
    gate, gs = _weights(g, e, inner, k)
    up, us = _weights(g, e, inner, k)
    both = torch.cat((gate.view(torch.uint8), up.view(torch.uint8)), 1).view(torch.float8_e4m3fn)
    return both, torch.cat((gs, us), 1)


ROUTE_SCALE = 2.5


# ---- the plain forms --------------------------------------------------------

def _values(q, s):
    """The values [.., N, K] in fp32 that a weight's codes and block scales stand for."""
    n, k = q.shape[-2:]
    return q.float() * s.repeat_interleave(BLOCK, -2)[..., :n, :].repeat_interleave(BLOCK, -1)[..., :k]


def _both_values(q, s):
    """The same of gate rows above up rows, each half with block scales of its own."""
    e, n, k = q.shape
    return _values(q.reshape(2 * e, n // 2, k), s.reshape(2 * e, s.shape[1] // 2, -1)).reshape(e, n, k)


def _through_codes(x):
    """Rows as the values of their codes, in fp32."""
    q, s = _quant(x)
    return q.float() * _spread(s, x.shape[1])


def _route(s):
    case, x = s["case"], s["logits"].double()
    t, e = x.shape
    score = torch.softmax(x, -1) if case["score"] == "softmax" else torch.sigmoid(x)
    choice = score if s["bias"] is None else score + s["bias"].double()
    if case["groups"] > 1:
        groups = choice.reshape(t, case["groups"], -1)
        two = groups.sort(-1, descending=True).values[..., :2].sum(-1)
        best = two.sort(dim=-1, descending=True, stable=True).indices[:, :case["top_groups"]]
        kept = torch.zeros_like(two, dtype=torch.bool).scatter_(1, best, True)
        choice = torch.where(kept.unsqueeze(-1), groups, -torch.inf).reshape(t, e)
    ids = choice.sort(dim=-1, descending=True, stable=True).indices[:, :case["top_k"]]
    w = score.gather(1, ids)
    if case["renormalize"]:
        w = w / w.sum(-1, keepdim=True)
    return ids.to(torch.int32), (w * ROUTE_SCALE).float()


def _gated(g, u):
    return g / (1 + torch.exp(-g)) * u


def _experts_few(s, x):
    """Each token's experts' weights gathered: for few slots."""
    t, top_k = s["ids"].shape
    ids = s["ids"].flatten().long()
    up = torch.bmm(_both_values(s["gate_up"].view(torch.uint8)[ids].view(torch.float8_e4m3fn),
                                s["gate_up_scale"][ids]), x.repeat_interleave(top_k, 0).unsqueeze(-1)).squeeze(-1)
    h = _through_codes(_gated(*up.chunk(2, -1)))
    y = torch.bmm(_values(s["down"].view(torch.uint8)[ids].view(torch.float8_e4m3fn), s["down_scale"][ids]),
                  h.unsqueeze(-1))
    return y.reshape(t, top_k, -1)


def _experts_many(s, x):
    """Rows set out by expert, each expert's in room for the busiest one's."""
    t, top_k = s["ids"].shape
    e, room = s["gate_up"].shape[0], s["room"]
    flat = s["ids"].flatten().long()
    order = flat.sort(stable=True).indices
    counts = torch.zeros(e, dtype=torch.long, device=flat.device).scatter_add_(0, flat, torch.ones_like(flat))
    first = counts.cumsum(0) - counts
    place = torch.empty_like(flat)
    place[order] = torch.arange(flat.numel(), device=flat.device) - first[flat[order]]
    at = flat * room + place
    rows = x.new_zeros(e * room, x.shape[1])
    rows[at] = x.repeat_interleave(top_k, 0)
    up = torch.bmm(rows.view(e, room, -1), _both_values(s["gate_up"], s["gate_up_scale"]).transpose(1, 2).contiguous())
    h = _through_codes(_gated(*up.chunk(2, -1)).reshape(e * room, -1)).view(e, room, -1)
    y = torch.bmm(h, _values(s["down"], s["down_scale"]).transpose(1, 2).contiguous())
    return y.reshape(e * room, -1)[at].reshape(t, top_k, -1)


def _plain(s):
    case = s["case"]
    if case["op"] == "route":
        return _route(s)
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "quant":
        return _through_codes(s["x"]).to(dtype)
    if case["op"] == "linear":
        x = s["xq"].float() * _spread(s["xs"], case["k"]) if case["codes"] else _through_codes(s["x"])
        t = x @ _values(s["wq"], s["ws"]).t()
        return (t if s["bias"] is None else t + s["bias"].float()).to(dtype)
    x = _through_codes(s["x"])
    y = (_experts_few if s["ids"].numel() < case["experts"] else _experts_many)(s, x)
    return (s["weights"].unsqueeze(-1) * y).sum(1).to(dtype)


# ---- the framework's calls ----------------------------------------------------

def _own(s):
    from w8a8_int8_dynamic_amd import ops
    case = s["case"]
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "quant":
        return ops.fp8_block_dequant(*ops.fp8_quant_per_block(s["x"]), dtype=dtype)
    if case["op"] == "linear":
        if not case["codes"]:
            return s["layer"](s["x"])
        return ops.fp8_block_scaled_mm(s["xq"].view(torch.uint8), s["xs"], s["packed"], s["ws"], case["n"],
                                       s["bias"], out_dtype=dtype)
    if case["op"] == "route":
        return ops.route_experts(s["logits"], s["routing"])
    return s["layer"](s["x"], s["ids"], s["weights"])


def run(state):
    return _own(state) if own else _plain(state)


# ---- the definition in 64 bits ------------------------------------------------

def _codes64(h):
    """The values of h's e4m3 codes times their scales: rounded by the exponent of each value. The
    factor of a block and its product with an element are fp32 numbers by the rule's definition, so that
    an element halfway between two codes is the same one to every reader."""
    m, k = h.shape
    b = torch.nn.functional.pad(h, (0, -k % BLOCK)).reshape(m, -1, BLOCK)
    a = b.abs().amax(-1, keepdim=True)
    v = torch.where(a >= LEAST, (b * (TOP / a.float()).double()).float().double(), 0.0)
    # 3 mantissa bits, smallest exponent -6
    e = (torch.frexp(v).exponent - 1).clamp(-6, 8).double()
    q = torch.round(v * torch.exp2(3 - e)) * torch.exp2(e - 3)
    return (q * (a / TOP)).reshape(m, -1)[:, :k]


def _weight64(q, s):
    n, k = q.shape[-2:]
    r = torch.arange(n, device=q.device) // BLOCK
    c = torch.arange(k, device=q.device) // BLOCK
    return q.double() * s.double()[r][:, c]


def _route64(case, s):
    x = s["logits"].double()
    if case["score"] == "softmax":
        score = torch.exp(x - x.amax(-1, keepdim=True))
        score = score / score.sum(-1, keepdim=True)
    else:
        score = 1 / (1 + torch.exp(-x))
    choice = score + (0 if s["bias"] is None else s["bias"].double())
    if case["groups"] > 1:
        size = x.shape[1] // case["groups"]
        first = choice.reshape(-1, case["groups"], size)
        top = first.topk(min(2, size), -1).values.sum(-1)
        # a group is kept where fewer than top_groups come before it
        before = (top.unsqueeze(1) > top.unsqueeze(2)).sum(-1)
        before += ((top.unsqueeze(1) == top.unsqueeze(2)).tril(-1)).sum(-1)
        choice = torch.where((before < case["top_groups"]).repeat_interleave(size, 1), choice, -torch.inf)
    ids = []
    for _ in range(case["top_k"]):
        best = choice.amax(-1, keepdim=True)
        ids.append((choice == best).to(torch.uint8).argmax(-1, keepdim=True))
        choice = choice.scatter(1, ids[-1], -torch.inf)
    ids = torch.cat(ids, 1)
    w = score.gather(1, ids)
    return ids.to(torch.int32), ROUTE_SCALE * (w / w.sum(-1, keepdim=True) if case["renormalize"] else w)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _route64(case, s)
    if case["op"] == "quant":
        return _codes64(s["x"].double())
    if case["op"] == "linear":
        x = s["xq"].double() * _spread(s["xs"].double(), case["k"]) if case["codes"] else _codes64(s["x"].double())
        t = torch.mm(x, _weight64(s["wq"], s["ws"]).t())
        return t if s["bias"] is None else t + s["bias"].double()
    x = _codes64(s["x"].double())
    out = torch.zeros_like(x)
    inner = case["inner"]
    for e in range(case["experts"]):
        token, slot = torch.nonzero(s["ids"] == e, as_tuple=True)
        if not token.numel():
            continue
        half = _blocks_of(inner)
        gate = torch.mm(x[token], _weight64(s["gate_up"][e, :inner], s["gate_up_scale"][e, :half]).t())
        up = torch.mm(x[token], _weight64(s["gate_up"][e, inner:], s["gate_up_scale"][e, half:]).t())
        h = _codes64(gate * torch.sigmoid(gate) * up)
        y = torch.mm(h, _weight64(s["down"][e], s["down_scale"][e]).t())
        out.index_add_(0, token, y * s["weights"][token, slot].double().unsqueeze(-1))
    return out
