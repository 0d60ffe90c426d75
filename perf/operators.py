"""The feed-forward operators of a tensor-parallel layer, as cases to measure.

What a rank computes around an AllReduce of partial outputs: the gated
feed-forward block (both column-parallel projections, the activation and the
product), the row-parallel matrix product with bias, activation and residual
in its epilogue, and both backward passes.

    linear        y = act(x w^T + b) + r
    linear_bwd    dz = dy act'(z);  dx = dz w,  dw = dz^T x,  db = sum of dz over the rows
    gated         g = x wg^T, u = x wu^T, h = act(g) u
    gated_bwd     dg = dh u act'(g), du = dh act(g);  dx = dg wg + du wu,  dwg = dg^T x,  dwu = du^T x

A case: op, dtype, m tokens, k inputs, n outputs (the block's inner width for
the gated forms), act, the epilogue's parts, `kn` (the weight lies k x n in
memory and is passed as its transposed view) and `pad` (elements between the
rows of x beyond k: a slice of a wider buffer).
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}
SIZE = {"fp32": 4, "fp16": 2, "bf16": 2}


def _case(name, op, dtype, m, k, n, act, bias=False, residual=False, save=False, kn=False, pad=0):
    return {"name": name, "op": op, "dtype": dtype, "m": m, "k": k, "n": n, "act": act, "bias": bias,
            "residual": residual, "save": save, "kn": kn, "pad": pad}


def listed():
    return [
        # one decoded token through a narrow layer with its bias: the smallest call, all latency
        _case("linear_1tok_small_fp16", "linear", "fp16", 1, 512, 512, "gelu", bias=True),
        # one decoded token: a rank's row-parallel product at hidden 8192, an eighth of the inner width, rank 0 adds the residual
        _case("linear_1tok_bf16", "linear", "bf16", 1, 3584, 8192, "none", residual=True),
        # a prompt of odd length through odd widths, the weight k x n as some checkpoints hold it
        _case("linear_odd_bf16", "linear", "bf16", 1001, 1537, 2047, "relu", bias=True, residual=True, kn=True),
        # a prompt's row-parallel product at the same widths as the decoded token's
        _case("linear_prompt_bf16", "linear", "bf16", 8192, 3584, 8192, "none", residual=True),
        # 32-bit training of a small model's ungated block
        _case("linear_fp32", "linear", "fp32", 512, 2048, 2048, "gelu_tanh", bias=True),
        # a training step's backward pass through the first product of an ungated block
        _case("linear_bwd_bf16", "linear_bwd", "bf16", 4096, 2048, 8192, "gelu", bias=True),
        # a ragged micro-batch's backward pass, rows taken from a wider buffer
        _case("linear_bwd_ragged_fp16", "linear_bwd", "fp16", 333, 1000, 1480, "none", bias=True, pad=24),
        # one decoded token: a rank's column-parallel gated projections, hidden 8192, an eighth of the inner width
        _case("gated_1tok_bf16", "gated", "bf16", 1, 8192, 3584, "silu"),
        # a decoding batch of 64 at the same widths
        _case("gated_batch64_fp16", "gated", "fp16", 64, 8192, 3584, "silu"),
        # a training step's forward pass, which keeps both projections for its backward pass
        _case("gated_train_bf16", "gated", "bf16", 4096, 8192, 3584, "silu", save=True),
        # the same step's backward pass
        _case("gated_bwd_bf16", "gated_bwd", "bf16", 4096, 8192, 3584, "silu"),
        # a small 32-bit model's backward pass at a ragged length
        _case("gated_bwd_fp32", "gated_bwd", "fp32", 777, 1024, 1408, "gelu_tanh"),
    ]


MOST_FLOPS = 8 * 4096 * 8192 * 3584


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["linear", "linear_bwd", "gated", "gated_bwd"])
        c = _case("", op, rng.choice(["bf16", "bf16", "fp16", "fp32"]), _log(rng, 1, 8192), _log(rng, 256, 8192),
                  _log(rng, 256, 8192), "silu")
        del c["name"]
        if rng.random() < 0.7:  # most widths are multiples of 64, and half the lengths of 16
            c["k"], c["n"] = -(-c["k"] // 64) * 64, -(-c["n"] // 64) * 64
        if c["m"] > 16 and rng.random() < 0.5:
            c["m"] = c["m"] // 16 * 16
        if op.startswith("linear"):
            c["act"] = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
            c["bias"] = rng.random() < 0.5
            c["residual"] = op == "linear" and rng.random() < 0.5
        else:
            c["act"] = rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"])
            c["save"] = op == "gated" and rng.random() < 0.4
        c["kn"] = rng.random() < 0.25
        c["pad"] = rng.choice([0, 0, 8, 13])
        if work(c)["flops"] <= MOST_FLOPS:
            return c


def work(case):
    m, k, n, e = case["m"], case["k"], case["n"], SIZE[case["dtype"]]
    op = case["op"]
    if op == "linear":
        values = m * k + n * k + m * n * (2 if case["residual"] else 1) + (n if case["bias"] else 0)
        flops = 2 * m * n * k
    elif op == "linear_bwd":
        values = m * n * (1 if case["act"] == "none" else 2) + 2 * m * k + 2 * n * k + (n if case["bias"] else 0)
        flops = 4 * m * n * k
    elif op == "gated":
        values = m * k + 2 * n * k + m * n * (3 if case["save"] else 1)
        flops = 4 * m * n * k
    else:
        values = 3 * m * n + 2 * m * k + 4 * n * k
        flops = 8 * m * n * k
    return {"bytes": values * e, "flops": flops}


def _inputs(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt, m, k, n = DTYPES[case["dtype"]], case["m"], case["k"], case["n"]

    def normal(rows, cols, scale, pad=0):
        t = torch.empty(rows, cols + pad, dtype=dt, device="cuda").normal_(0.0, scale, generator=gen)
        return t[:, :cols]

    def weight():
        t = normal(k, n, k ** -0.5).t() if case["kn"] else normal(n, k, k ** -0.5)
        return t

    s = {"x": normal(m, k, 1.0, case["pad"])}
    if case["op"].startswith("linear"):
        s["w"] = weight()
        if case["op"] == "linear":
            s["b"] = normal(1, n, 0.1)[0] if case["bias"] else None
            s["r"] = normal(m, n, 1.0) if case["residual"] else None
        else:
            s["dy"] = normal(m, n, 0.1)
            s["z"] = None if case["act"] == "none" else normal(m, n, 1.0)
    else:
        s["wg"], s["wu"] = weight(), weight()
        if case["op"] == "gated_bwd":
            s["dh"], s["g"], s["u"] = normal(m, n, 0.1), normal(m, n, 1.0), normal(m, n, 1.0)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = dict(case)
    return s


# ---- the plain form: 32 bits throughout, rounded once at the end -------------------

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


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (0.5 / math.pi) ** 0.5
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    sig = 1 / (1 + torch.exp(-z))
    return sig * (1 + z * (1 - sig))


def _plain(s):
    c = s["case"]
    dt, act, op = DTYPES[c["dtype"]], c["act"], c["op"]
    x = s["x"].float()
    if op == "linear":
        z = x @ s["w"].float().t()
        if s["b"] is not None:
            z = z + s["b"].float()
        y = _act(z, act)
        if s["r"] is not None:
            y = y + s["r"].float()
        return y.to(dt)
    if op == "linear_bwd":
        dz = s["dy"].float()
        if act != "none":
            dz = dz * _act_grad(s["z"].float(), act)
        out = {"dx": (dz @ s["w"].float()).to(dt), "dw": (dz.t() @ x).to(dt)}
        if c["bias"]:
            out["db"] = dz.sum(0).to(dt)
        return out
    wg, wu = s["wg"].float(), s["wu"].float()
    if op == "gated":
        g, u = x @ wg.t(), x @ wu.t()
        h = (_act(g, act) * u).to(dt)
        return {"h": h, "gate": g.to(dt), "up": u.to(dt)} if c["save"] else h
    dh, g, u = s["dh"].float(), s["g"].float(), s["u"].float()
    dg, du = dh * u * _act_grad(g, act), dh * _act(g, act)
    return {"dx": (dg @ wg + du @ wu).to(dt), "dw_gate": (dg.t() @ x).to(dt), "dw_up": (du.t() @ x).to(dt)}


def _own(s):
    import message_allreduce_amd as llar
    c = s["case"]
    act, op = c["act"], c["op"]
    if op == "linear":
        return llar.linear(s["x"], s["w"], s["b"], s["r"], activation=act)
    if op == "linear_bwd":
        dx, dw, db = llar.linear_backward(s["dy"], s["x"], s["w"], s["z"], activation=act, bias_grad=c["bias"])
        out = {"dx": dx, "dw": dw}
        if c["bias"]:
            out["db"] = db
        return out
    if op == "gated":
        if c["save"]:
            h, g, u = llar.gated_ffn(s["x"], s["wg"], s["wu"], activation=act, save=True)
            return {"h": h, "gate": g, "up": u}
        return llar.gated_ffn(s["x"], s["wg"], s["wu"], activation=act)
    dx, dwg, dwu = llar.gated_ffn_backward(s["dh"], s["x"], s["wg"], s["wu"], s["g"], s["u"], activation=act)
    return {"dx": dx, "dw_gate": dwg, "dw_up": dwu}


def run(state):
    return _own(state) if own else _plain(state)


# ---- the definition in 64 bits ------------------------------------------------------

def exact(case, seed):
    s = {k: None if v is None else v.double() for k, v in _inputs(case, seed).items()}
    act = case["act"]

    def phi(t):  # the normal distribution's function
        return 0.5 * torch.special.erfc(-t / 2 ** 0.5)

    def inner(t):
        return (2 / math.pi) ** 0.5 * (t + 0.044715 * t ** 3)

    value = {"none": lambda t: t, "relu": lambda t: t.clamp(min=0), "gelu": lambda t: t * phi(t),
             "gelu_tanh": lambda t: t * torch.sigmoid(2 * inner(t)), "silu": lambda t: t * torch.sigmoid(t)}[act]

    def slope(t):
        t = t.clone().requires_grad_(True)
        return torch.autograd.grad(value(t).sum(), t)[0]

    if case["op"] == "linear":
        z = torch.mm(s["x"], s["w"].T)
        y = value(z if s["b"] is None else z + s["b"])
        return y if s["r"] is None else y + s["r"]
    if case["op"] == "linear_bwd":
        dz = s["dy"] if act == "none" else s["dy"] * slope(s["z"])
        out = {"dx": torch.mm(dz, s["w"]), "dw": torch.mm(dz.T, s["x"])}
        if case["bias"]:
            out["db"] = dz.sum(dim=0)
        return out
    if case["op"] == "gated":
        g, u = torch.mm(s["x"], s["wg"].T), torch.mm(s["x"], s["wu"].T)
        h = value(g) * u
        return {"h": h, "gate": g, "up": u} if case["save"] else h
    dg, du = s["dh"] * s["u"] * slope(s["g"]), s["dh"] * value(s["g"])
    return {"dx": torch.mm(dg, s["wg"]) + torch.mm(du, s["wu"]), "dw_gate": torch.mm(dg.T, s["x"]),
            "dw_up": torch.mm(du.T, s["x"])}
