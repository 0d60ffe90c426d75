"""Feed-forward operators of decoding with 8-bit weights and with experts, as cases to measure.

    quantize      s = max|x| / 127 of a row, q = x / s rounded to the nearest whole number
    linear_int8   y = act((q_x q_w^T) s_x s_w + b) + r, whole-number sums
    gated_int8    h = act(g) u, both projections as above
    route         the top_k of x router^T for each token, with the weights of their softmax or sigmoid
    moe           y = sum over a token's experts of weight * (act(x wg^T) (x wu^T)) wd^T + r

A case: op, dtype (of the activations), m tokens, k inputs, n outputs (the inner
width for the gated forms and the experts), act, the epilogue's parts, `pad`
(elements between the rows of x beyond k: a slice of a wider buffer).  `quantized`:
linear_int8 and gated_int8 get x as whole numbers with scales, else they quantise
it themselves.  route and moe: `experts` held here, top_k of `all_experts` chosen
by each token (the others live on other ranks: their numbers are given as -1), and
for moe `int8` weights.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"fp32": 4, "fp16": 2, "bf16": 2}


def _quantize(name, dtype, m, k, pad=0):
    return {"name": name, "op": "quantize", "dtype": dtype, "m": m, "k": k, "pad": pad}


def _product(name, op, dtype, m, k, n, act, bias=False, residual=False, quantized=False, pad=0):
    return {"name": name, "op": op, "dtype": dtype, "m": m, "k": k, "n": n, "act": act, "bias": bias,
            "residual": residual, "quantized": quantized, "pad": pad}


def _route(name, dtype, m, k, experts, top_k, scoring="softmax", normalize=True):
    return {"name": name, "op": "route", "dtype": dtype, "m": m, "k": k, "experts": experts, "top_k": top_k,
            "scoring": scoring, "normalize": normalize}


def _moe(name, dtype, m, k, n, experts, top_k, act="silu", int8=False, residual=False, all_experts=None):
    return {"name": name, "op": "moe", "dtype": dtype, "m": m, "k": k, "n": n, "experts": experts, "top_k": top_k,
            "act": act, "int8": int8, "residual": residual, "all_experts": all_experts or experts}


def listed():
    return [
        # a prompt's tokens before an 8-bit product
        _quantize("quantize_prompt_bf16", "bf16", 4096, 8192),
        # an odd small batch, rows of a wider buffer
        _quantize("quantize_odd_fp32", "fp32", 33, 1537, pad=13),
        # one decoded token through a narrow layer with its bias: the smallest call, all latency
        _product("linear_int8_1tok_small_fp16", "linear_int8", "fp16", 1, 512, 512, "gelu", bias=True),
        # one decoded token: a rank's row-parallel product at hidden 8192, an eighth of the inner width, with the residual
        _product("linear_int8_1tok_bf16", "linear_int8", "bf16", 1, 3584, 8192, "none", residual=True),
        # a ragged micro-batch through odd widths
        _product("linear_int8_odd_bf16", "linear_int8", "bf16", 333, 1537, 2047, "relu", bias=True, residual=True, pad=13),
        # a prompt's row-parallel product, its tokens quantised already
        _product("linear_int8_prompt_bf16", "linear_int8", "bf16", 8192, 3584, 8192, "none", quantized=True),
        # a decoding batch of 16: a rank's column-parallel gated projections
        _product("gated_int8_batch16_bf16", "gated_int8", "bf16", 16, 8192, 3584, "silu"),
        # a prompt's gated projections
        _product("gated_int8_prompt_fp16", "gated_int8", "fp16", 2048, 8192, 3584, "silu"),
        # one decoded token chooses among 64 experts
        _route("route_1tok_bf16", "bf16", 1, 4096, 64, 8),
        # a decoding batch, many experts
        _route("route_batch64_bf16", "bf16", 64, 8192, 256, 8, scoring="sigmoid"),
        # one decoded token through eight small experts of 64
        _moe("moe_1tok_bf16", "bf16", 1, 4096, 1024, 64, 8),
        # a decoding batch of 48 over eight large experts, a rank's share of their width, 8-bit weights
        _moe("moe_batch48_int8", "bf16", 48, 8192, 3584, 8, 2, int8=True, residual=True),
    ]


MOST_FLOPS = 2 * 8192 * 8192 * 3584
MOST_BYTES = 3 * 8 * 8192 * 3584


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """Most widths are multiples of 64."""
    v = _log(rng, lo, hi)
    return -(-v // 64) * 64 if rng.random() < 0.7 else v


def draw(rng):
    while True:
        op = rng.choice(["quantize", "linear_int8", "linear_int8", "gated_int8", "route", "moe", "moe"])
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        pad = rng.choice([0, 0, 8, 13])
        if op == "quantize":
            c = _quantize("", dtype, _log(rng, 1, 8192), _width(rng, 256, 16384), pad)
        elif op in ("linear_int8", "gated_int8"):
            plain = op == "linear_int8"
            act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"] if plain else ["silu", "silu", "gelu", "gelu_tanh"])
            c = _product("", op, dtype, _log(rng, 1, 8192), _width(rng, 256, 8192), _width(rng, 256, 8192), act,
                         plain and rng.random() < 0.5, plain and rng.random() < 0.5, rng.random() < 0.4, pad)
        else:
            experts, k = _log(rng, 4, 256), _width(rng, 256, 8192)
            top_k = rng.randint(1, min(8, experts))
            if op == "route":
                c = _route("", dtype, _log(rng, 1, 64), k, experts, top_k, rng.choice(["softmax", "softmax", "sigmoid"]),
                           rng.random() < 0.7)
            else:
                c = _moe("", dtype, _log(rng, 1, 64), k, _width(rng, 128, 4096), experts, top_k,
                         rng.choice(["silu", "silu", "gelu", "relu"]), rng.random() < 0.4, rng.random() < 0.3,
                         experts * rng.choice([1, 1, 4]))
                held = experts * 3 * k * c["n"] * (1 if c["int8"] else SIZE[dtype])
                if held > 2 * MOST_BYTES or work(c)["bytes"] > MOST_BYTES:
                    continue
        del c["name"]
        if work(c)["flops"] <= MOST_FLOPS:
            return c


def work(case):
    m, k, e, op = case["m"], case["k"], SIZE[case["dtype"]], case["op"]
    if op == "quantize":
        return {"bytes": m * k * (e + 1) + 4 * m, "flops": 3 * m * k}
    if op == "route":
        return {"bytes": (m + case["experts"]) * k * e + 8 * m * case["top_k"], "flops": 2 * m * case["experts"] * k}
    n = case["n"]
    if op == "moe":
        share = case["top_k"] / case["all_experts"]
        used = case["experts"] * (1 - (1 - share) ** m)  # expected number of experts that any token chose
        values = 3 * used * n * k * (1 if case["int8"] else e) + (4 * used * (2 * n + k) if case["int8"] else 0)
        return {"bytes": int(values) + m * k * e * (3 if case["residual"] else 2) + 8 * m * case["top_k"],
                "flops": int(6 * m * share * case["experts"] * n * k)}
    w = 2 if op == "gated_int8" else 1
    tokens = m * k + 4 * m if case["quantized"] else m * k * e
    return {"bytes": tokens + w * (n * k + 4 * n) + m * n * e * (2 if case["residual"] else 1)
            + (n * e if case["bias"] else 0), "flops": 2 * w * m * n * k}


# ---- inputs ------------------------------------------------------------------------

def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt, m, k, op = DTYPES[case["dtype"]], case["m"], case["k"], case["op"]

    def normal(rows, cols, scale, dtype=dt):
        return torch.empty(rows, cols, dtype=dtype, device="cuda").normal_(0.0, scale, generator=gen)

    def whole(*shape):
        """Rows of a quantised matrix: their largest values are about four standard deviations."""
        t = torch.empty(*shape, dtype=torch.int8, device="cuda")
        for part in t if len(shape) == 3 else [t]:
            part.copy_(torch.empty(part.shape, dtype=torch.float16, device="cuda").normal_(0.0, 32.0, generator=gen)
                       .round_().clamp_(-127, 127))
        return t

    def scales(*shape, width):
        return torch.empty(*shape, device="cuda").uniform_(0.8, 1.25, generator=gen) * (width ** -0.5 / 32)

    # some channels of the activations are larger than others
    gain = torch.exp(normal(1, k, 0.5, torch.float32))
    pad = case.get("pad", 0)
    wide = torch.zeros(m, k + pad, dtype=dt, device="cuda")
    wide[:, :k] = normal(m, k, 1.0, torch.float32) * gain
    s = {"x": wide[:, :k]}
    if op == "quantize":
        return s
    if op == "route":
        s["router"] = normal(case["experts"], k, k ** -0.5)
        return s
    n = case["n"]
    if op == "moe":
        count = case["experts"]
        chosen = torch.rand(m, case["all_experts"], device="cuda", generator=gen).argsort(dim=1)[:, :case["top_k"]]
        s["experts"] = torch.where(chosen < count, chosen, torch.full_like(chosen, -1)).int()
        s["weights"] = torch.softmax(normal(m, case["top_k"], 1.0, torch.float32), dim=1)
        for name, rows, cols in (("wg", n, k), ("wu", n, k), ("wd", k, n)):
            if case["int8"]:
                s[name], s[name + "_scale"] = whole(count, rows, cols), scales(count, rows, width=cols)
            else:
                t = torch.empty(count, rows, cols, dtype=dt, device="cuda")
                s[name], s[name + "_scale"] = t.normal_(0.0, cols ** -0.5, generator=gen), None
        s["r"] = normal(m, k, 1.0) if case["residual"] else None
        return s
    if case["quantized"]:
        wide = torch.zeros(m, k + pad, dtype=torch.int8, device="cuda")
        wide[:, :k] = whole(m, k)
        s["x"], s["x_scale"] = wide[:, :k], torch.empty(m, device="cuda").uniform_(0.02, 0.05, generator=gen)
    else:
        s["x_scale"] = None
    for name in ("w",) if op == "linear_int8" else ("wg", "wu"):
        s[name], s[name + "_scale"] = whole(n, k), scales(n, width=k)
    s["b"] = normal(1, n, 0.1)[0] if case["bias"] else None
    s["r"] = normal(m, n, 1.0) if case["residual"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = dict(case)
    return s


# ---- the plain form: 32 bits (64 next to a border), rounded once at the end ---------

def _act(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z / (1 + torch.exp(-z))


def _rows_quantized(x):
    """(q, scale) of the rows of a 32-bit matrix, q as 32-bit whole numbers."""
    scale = (x.abs().amax(dim=-1, keepdim=True).double() / 127).float()  # 64 bits: the nearest, where halves are common
    q = torch.round(x.double() / scale.double())
    q = torch.where(scale > 0, q, torch.zeros_like(q)).clamp(-127, 127)
    return q.float(), scale


def _plain_moe(s):
    c = s["case"]
    x, ids, count, int8 = s["x"].float(), s["experts"].long(), c["experts"], c["int8"]
    here = ids >= 0
    a = torch.where(here, s["weights"], torch.zeros_like(s["weights"]))
    ids = torch.where(here, ids, torch.zeros_like(ids))

    def product(t, scale, w, w_scale):
        y = torch.matmul(t, w.float().transpose(-1, -2).contiguous())
        return y * scale * w_scale.unsqueeze(-2) if int8 else y

    def block(t, scale, part):
        """The experts' blocks for rows t: part takes their weights, and scales, from the whole."""
        w = {name: part(s[name]) for name in ("wg", "wu", "wd")}
        ws = {name: part(s[name + "_scale"]) if int8 else None for name in w}
        h = _act(product(t, scale, w["wg"], ws["wg"]), c["act"]) * product(t, scale, w["wu"], ws["wu"])
        hq, h_scale = _rows_quantized(h) if int8 else (h, None)
        return product(hq, h_scale, w["wd"], ws["wd"])

    xq, x_scale = _rows_quantized(x) if int8 else (x, None)
    pairs = ids.numel()
    if pairs <= count:  # few choices: each one's expert, gathered
        rows = torch.arange(pairs, device=x.device) // c["top_k"]
        y = block(xq[rows].unsqueeze(1), x_scale[rows].unsqueeze(1) if int8 else None,
                  lambda t: t.index_select(0, ids.reshape(-1)))
        y = (y.squeeze(1) * a.reshape(-1, 1)).view(c["m"], c["top_k"], -1).sum(1)
    else:  # every expert for all tokens, weighted by zero where it was not chosen
        y = torch.zeros(c["m"], c["k"], device=x.device)
        for e in range(count):
            weight = torch.where(ids == e, a, torch.zeros_like(a)).sum(1, keepdim=True)
            y = y + weight * block(xq, x_scale, lambda t: t[e])
    return y if s["r"] is None else y + s["r"].float()


def _plain(s):
    c = s["case"]
    dt, op = DTYPES[c["dtype"]], c["op"]
    if op == "quantize":
        q, scale = _rows_quantized(s["x"].float())
        return {"values": q * scale, "scale": scale.squeeze(1)}
    if op == "route":
        logits = torch.matmul(s["x"].double(), s["router"].double().t())
        order = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :c["top_k"]]
        score = torch.softmax(logits, dim=1) if c["scoring"] == "softmax" else 1 / (1 + torch.exp(-logits))
        score = torch.gather(score, 1, order)
        if c["normalize"]:
            score = score / score.sum(1, keepdim=True)
        return {"weights": score.float(), "experts": order.int()}
    if op == "moe":
        return _plain_moe(s).to(dt)
    x, x_scale = s["x"].float(), None
    if c["quantized"]:
        x_scale = s["x_scale"].unsqueeze(1)
    else:
        x, x_scale = _rows_quantized(x)
    if op == "linear_int8":
        y = (x @ s["w"].float().t()) * x_scale * s["w_scale"]
        if s["b"] is not None:
            y = y + s["b"].float()
        y = _act(y, c["act"])
        return (y if s["r"] is None else y + s["r"].float()).to(dt)
    g = (x @ s["wg"].float().t()) * x_scale * s["wg_scale"]
    u = (x @ s["wu"].float().t()) * x_scale * s["wu_scale"]
    return (_act(g, c["act"]) * u).to(dt)


def _own(s):
    import message_allreduce_amd as llar
    c = s["case"]
    op = c["op"]
    if op == "quantize":
        q, scale = llar.quantize_rows(s["x"])
        return {"values": q * scale.unsqueeze(1), "scale": scale}
    if op == "route":
        weights, experts = llar.moe_route(s["x"], s["router"], c["top_k"], scoring=c["scoring"], normalize=c["normalize"])
        return {"weights": weights, "experts": experts}
    if op == "moe":
        return llar.moe_ffn(s["x"], s["experts"], s["weights"], s["wg"], s["wu"], s["wd"], activation=c["act"],
                            residual=s["r"], gate_scale=s["wg_scale"], up_scale=s["wu_scale"], down_scale=s["wd_scale"])
    if op == "linear_int8":
        return llar.linear_int8(s["x"], s["w"], s["w_scale"], x_scale=s["x_scale"], bias=s["b"], residual=s["r"],
                                activation=c["act"], dtype=DTYPES[c["dtype"]])
    return llar.gated_ffn_int8(s["x"], s["wg"], s["wu"], s["wg_scale"], s["wu_scale"], x_scale=s["x_scale"],
                               activation=c["act"], dtype=DTYPES[c["dtype"]])


def run(state):
    return _own(state) if own else _plain(state)


# ---- the definition in 64 bits ------------------------------------------------------

def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]

    def value(t):
        if case["act"] == "gelu":
            return t * 0.5 * torch.special.erfc(-t / 2 ** 0.5)
        if case["act"] == "gelu_tanh":
            return t * torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (t + 0.044715 * t ** 3))
        return {"none": lambda z: z, "relu": lambda z: z.clamp(min=0), "silu": lambda z: z * torch.sigmoid(z)}[case["act"]](t)

    def quantized(t):
        """Whole numbers and the row's scale, which is held in 32 bits."""
        top = t.abs().max(dim=-1).values
        scale = (top / 127).float().double()
        q = torch.round(t / scale.clamp(min=2.0 ** -1000)[..., None])
        return torch.clamp(q, -127, 127) * (scale > 0)[..., None], scale

    x = s["x"].double()
    if op == "quantize":
        q, scale = quantized(x)
        return {"values": q * scale[:, None], "scale": x.abs().max(dim=1).values / 127}
    if op == "route":
        logits = torch.mm(x, s["router"].double().T)
        # the count of better ones, with a lower number first among equals, is a choice's place
        less = torch.arange(case["experts"], device=x.device)
        top = []
        left = logits.clone()
        for _ in range(case["top_k"]):
            best = left.max(dim=1, keepdim=True).values
            pick = torch.where(left == best, less, case["experts"]).min(dim=1, keepdim=True).values
            top.append(pick)
            left.scatter_(1, pick, -math.inf)
        top = torch.cat(top, dim=1)
        if case["scoring"] == "softmax":
            shifted = torch.exp(logits - logits.max(dim=1, keepdim=True).values)
            score = shifted / shifted.sum(dim=1, keepdim=True)
        else:
            score = torch.sigmoid(logits)
        w = score.gather(1, top)
        return {"weights": w / w.sum(dim=1, keepdim=True) if case["normalize"] else w, "experts": top.int()}
    if op == "moe":
        xq, x_scale = quantized(x) if case["int8"] else (x, None)

        def product(t, scale, name, e):
            y = torch.mm(t, s[name][e].double().T)
            return y * scale[:, None] * s[name + "_scale"][e].double() if case["int8"] else y

        y = torch.zeros(case["m"], case["k"], dtype=torch.float64, device=x.device)
        for e in range(case["experts"]):
            token, place = (s["experts"] == e).nonzero(as_tuple=True)
            if token.numel() == 0:
                continue
            rows, scale = xq[token], x_scale[token] if case["int8"] else None
            h = value(product(rows, scale, "wg", e)) * product(rows, scale, "wu", e)
            hq, h_scale = quantized(h) if case["int8"] else (h, None)
            y.index_add_(0, token, product(hq, h_scale, "wd", e) * s["weights"][token, place].double()[:, None])
        return y if s["r"] is None else y + s["r"].double()
    xq, x_scale = (x, s["x_scale"].double()) if case["quantized"] else quantized(x)

    def scaled(name):
        return torch.mm(xq, s[name].double().T) * x_scale[:, None] * s[name + "_scale"].double()[None, :]

    if op == "linear_int8":
        z = scaled("w")
        y = value(z if s["b"] is None else z + s["b"].double())
        return y if s["r"] is None else y + s["r"].double()
    return value(scaled("wg")) * scaled("wu")
