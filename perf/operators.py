"""Cases of the token operators: embedding lookup with scaling and its
gradient, RMS norm with the residual's addition and an int8 output, and the
int8 product with a scale for each token and channel.

A case is one call of one operator ("op").  `run` computes it in elementary
torch operations, or, where `own` is true, through this package's entry
points.  `exact` gives the same outputs from the definitions in 64 bits.

The int8 codes of the norm are returned as they are, whole numbers: a code is
decided from values in 64 bits on every side, so the codes have to be equal.
"""
import math

import numpy as np
import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
_BYTES = {"f32": 4, "bf16": 2, "fp8": 1}
_FP8_SCALE = 2.0 ** -8          # what the fp8 tables' codes stand for, per unit
_EPS = 1e-6


def listed():
    return [
        # one small request: 32 tokens of a small table, latency alone
        {"name": "lookup-short", "op": "lookup", "tokens": 32, "rows": 4096, "dim": 64,
         "table": "f32", "out": "f32", "dist": "uniform", "masked": 0.0},
        # a batch of long sequences into the first layer, a tenth of it padding
        {"name": "lookup-long", "op": "lookup", "tokens": 262144, "rows": 100000, "dim": 1024,
         "table": "bf16", "out": "bf16", "dist": "zipf", "masked": 0.1},
        # the gradient of a tiny table from a tiny batch
        {"name": "grad-short", "op": "grad", "tokens": 160, "rows": 1000, "dim": 16,
         "grad": "f32", "out": "f32", "dist": "uniform", "masked": 0.0, "accumulate": False},
        # 2048 histories of 20 items, the step added to a table of a million rows in place
        {"name": "grad-history", "op": "grad", "tokens": 40960, "rows": 1000000, "dim": 64,
         "grad": "f32", "out": "f32", "dist": "zipf", "masked": 0.05, "accumulate": True},
        # a training batch of long sequences, the whole gradient written
        {"name": "grad-long", "op": "grad", "tokens": 65536, "rows": 100000, "dim": 1024,
         "grad": "bf16", "out": "f32", "dist": "zipf", "masked": 0.0, "accumulate": False},
        # one token being decoded
        {"name": "norm-one", "op": "norm", "m": 1, "dim": 4096, "type": "bf16",
         "residual": True, "weight": True},
        # the interaction's odd row width
        {"name": "norm-odd", "op": "norm", "m": 2048, "dim": 415, "type": "f32",
         "residual": True, "weight": True},
        # a prompt's rows, wide
        {"name": "norm-long", "op": "norm", "m": 16384, "dim": 8192, "type": "bf16",
         "residual": True, "weight": True},
        # one token through one layer: the weights' bytes
        {"name": "product-one", "op": "product", "m": 1, "n": 4096, "k": 4096, "out": "bf16",
         "bias": False, "act": "none"},
        # a batch of single tokens
        {"name": "product-few", "op": "product", "m": 32, "n": 8192, "k": 8192, "out": "bf16",
         "bias": True, "act": "none"},
        # the top MLP's first layer, whose rows are of odd length
        {"name": "product-odd", "op": "product", "m": 2048, "n": 512, "k": 415, "out": "f32",
         "bias": True, "act": "relu"},
        # a prompt's rows through a wide layer: the matrix units' rate
        {"name": "product-long", "op": "product", "m": 8192, "n": 8192, "k": 8192, "out": "bf16",
         "bias": False, "act": "none"},
    ]


def _size(rng, low, high):
    """A whole number spread over the logarithm of [low, high]."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _width(rng, low, high):
    """A size that is odd, a multiple of 16, or anything."""
    v = _size(rng, low, high)
    kind = rng.randrange(3)
    return max(low, v // 16 * 16) if kind == 0 else v | 1 if kind == 1 and v < high else v


def draw(rng):
    op = rng.choice(("lookup", "grad", "norm", "product"))
    if op == "lookup":
        dim = _width(rng, 8, 4096)
        return {"op": op, "tokens": _size(rng, 1, (1 << 28) // dim // 2), "dim": dim,
                "rows": _size(rng, 100, (1 << 29) // dim),
                "table": rng.choice(("f32", "bf16", "fp8")), "out": rng.choice(("f32", "bf16")),
                "dist": rng.choice(("uniform", "zipf")), "masked": rng.choice((0.0, 0.05, 0.5))}
    if op == "grad":
        dim = _width(rng, 8, 4096)
        return {"op": op, "tokens": _size(rng, 1, min(1 << 19, (1 << 26) // dim)), "dim": dim,
                "rows": _size(rng, 100, 100_000_000 // dim),
                "grad": rng.choice(("f32", "bf16")), "out": rng.choice(("f32", "bf16")),
                "dist": rng.choice(("uniform", "zipf")), "masked": rng.choice((0.0, 0.05, 0.5)),
                "accumulate": False}
    if op == "norm":
        dim = _width(rng, 16, 8192)
        return {"op": op, "m": _size(rng, 1, (1 << 26) // dim), "dim": dim,
                "type": rng.choice(("f32", "bf16")), "residual": rng.random() < 0.7,
                "weight": rng.random() < 0.8}
    n, k = _width(rng, 16, 8192), _width(rng, 16, 8192)
    return {"op": op, "m": _size(rng, 1, 8192), "n": n, "k": k, "out": rng.choice(("f32", "bf16")),
            "bias": rng.random() < 0.5, "act": rng.choice(("none", "relu", "sigmoid"))}


# ----------------------------------------------------------------- inputs --
def _tokens(case, g):
    n, rows = case["tokens"], case["rows"]
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    if case["dist"] == "zipf":     # bounded power law of exponent 1.05, ranks scattered over rows
        e = -0.05
        rank = torch.floor(((float(rows + 1) ** e - 1.0) * u + 1.0) ** (1.0 / e)).long() - 1
        t = rank.clamp_(0, rows - 1) * 999983 % rows
    else:
        t = (u * rows).long().clamp_(0, rows - 1)
    if case["masked"]:
        gone = torch.rand(n, generator=g, device="cuda") < case["masked"]
        t = torch.where(gone, torch.full_like(t, -1), t)
    return t.to(torch.int32)


def _codes(x):
    """Rows of int8 codes and their scales, as a quantised model holds them."""
    s = x.abs().amax(1).clamp_(min=1e-12) / 127.0
    return torch.round(x / s[:, None]).clamp_(-127, 127).to(torch.int8), s


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1_000_003 + 17)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    st = {"case": case}
    if case["op"] in ("lookup", "grad"):
        st["tokens"] = _tokens(case, g)
        st["scale"] = math.sqrt(case["dim"])
    if case["op"] == "lookup":
        t = normal(case["rows"], case["dim"]).mul_(0.01)
        if case["table"] == "fp8":
            t.div_(_FP8_SCALE)
            st["scale"] *= _FP8_SCALE
        st["table"] = t.to(_DT[case["table"]])
    elif case["op"] == "grad":
        st["grad"] = normal(case["tokens"], case["dim"]).mul_(1e-3).to(_DT[case["grad"]])
        if case["accumulate"]:     # a step of plain gradient descent on the table itself
            st["scale"] *= -0.01
            st["table"] = normal(case["rows"], case["dim"]).mul_(0.01).to(_DT[case["out"]])
    elif case["op"] == "norm":
        dt = _DT[case["type"]]
        st["x"] = normal(case["m"], case["dim"]).to(dt)
        st["residual"] = normal(case["m"], case["dim"]).mul_(2.0).to(dt) if case["residual"] else None
        st["weight"] = normal(case["dim"]).mul_(0.1).add_(1.0) if case["weight"] else None
    else:
        st["a"], st["a_scale"] = _codes(normal(case["m"], case["k"]))
        st["w"], st["w_scale"] = _codes(normal(case["n"], case["k"]).mul_(case["k"] ** -0.5))
        st["bias"] = normal(case["n"]).mul_(0.1) if case["bias"] else None
    return st


# -------------------------------------------------------------------- run --
def _plain_lookup(case, st):
    t = st["tokens"].long()
    there = (t >= 0) & (t < case["rows"])
    rows = st["table"][t.clamp(0, case["rows"] - 1)].float() * st["scale"]
    return torch.where(there[:, None], rows, torch.zeros_like(rows)).to(_DT[case["out"]])


def _plain_grad(case, st):
    t = st["tokens"].long()
    there = (t >= 0) & (t < case["rows"])
    g = st["grad"].float() * st["scale"]
    g = torch.where(there[:, None], g, torch.zeros_like(g))
    t = t.clamp(0, case["rows"] - 1)
    if case["accumulate"]:
        return st["table"].index_add_(0, t, g)
    out = torch.zeros(case["rows"], case["dim"], dtype=torch.float32, device=g.device)
    return out.index_add_(0, t, g).to(_DT[case["out"]])


def _plain_norm(case, st):
    h = st["x"]
    if st["residual"] is not None:
        h = (h.float() + st["residual"].float()).to(h.dtype)
    d = h.double()                 # codes next to a border: in 64 bits
    y = d * torch.rsqrt(d.square().mean(1, keepdim=True) + _EPS)
    if st["weight"] is not None:
        y = y * st["weight"].double()
    s = (y.abs().amax(1) / 127.0).float()
    q = torch.where(s[:, None] > 0, torch.round(y / s.double()[:, None]), torch.zeros_like(y))
    return h, q.to(torch.int8), s


def _plain_product(case, st):
    c = st["a"].float() @ st["w"].float().t()
    c = c * (st["a_scale"][:, None] * st["w_scale"][None, :])
    if st["bias"] is not None:
        c = c + st["bias"]
    if case["act"] == "relu":
        c = torch.clamp(c, min=0.0)
    elif case["act"] == "sigmoid":
        c = 1.0 / (1.0 + torch.exp(-c))
    return c.to(_DT[case["out"]])


def _own(case, st):
    import dlrm_embedding_bag_amd as fw
    if case["op"] == "lookup":
        return {"rows": fw.emb_lookup_scaled(st["table"], st["tokens"], st["scale"],
                                             out_dtype=_DT[case["out"]])}
    if case["op"] == "grad":
        if case["accumulate"]:
            return {"table": fw.emb_lookup_grad(st["grad"], st["tokens"], scale=st["scale"],
                                                out=st["table"], accumulate=True)}
        return {"table": fw.emb_lookup_grad(st["grad"], st["tokens"], case["rows"],
                                            scale=st["scale"], out_dtype=_DT[case["out"]])}
    if case["op"] == "norm":
        h, q, s = fw.rms_norm_residual_i8(st["x"], st["weight"], st["residual"], eps=_EPS)
        return {"h": h, "codes": q, "scale": s}
    return {"out": fw.linear_i8_bias_act(st["a"], st["a_scale"], st["w"], st["w_scale"],
                                         st["bias"], case["act"], out_dtype=_DT[case["out"]])}


def run(state):
    case = state["case"]
    if own:
        return _own(case, state)
    if case["op"] == "lookup":
        return {"rows": _plain_lookup(case, state)}
    if case["op"] == "grad":
        return {"table": _plain_grad(case, state)}
    if case["op"] == "norm":
        h, q, s = _plain_norm(case, state)
        return {"h": h, "codes": q, "scale": s}
    return {"out": _plain_product(case, state)}


# ------------------------------------------------------------------- work --
def _distinct(case):
    """How many rows the case's tokens name, on the average."""
    n = case["tokens"] * (1.0 - case["masked"])
    if case["dist"] == "uniform":
        return case["rows"] * -math.expm1(-n / case["rows"])
    edge = np.arange(1, case["rows"] + 2, dtype=np.float64) ** -0.05
    p = (edge[:-1] - edge[1:]) / (edge[0] - edge[-1])
    return float(-np.expm1(-n * p).sum())


def work(case):
    if case["op"] == "lookup":
        n, d = case["tokens"], case["dim"]
        there = n * (1.0 - case["masked"])
        read = _distinct(case) * d * _BYTES[case["table"]]     # each row read once
        return {"bytes": 4 * n + read + n * d * _BYTES[case["out"]], "flops": there * d}
    if case["op"] == "grad":
        n, d = case["tokens"], case["dim"]
        there = n * (1.0 - case["masked"])
        wrote = case["rows"] * d * _BYTES[case["out"]]
        if case["accumulate"]:     # the rows that occur, read and written
            wrote = 2 * _distinct(case) * d * _BYTES[case["out"]]
        return {"bytes": 4 * n + there * d * _BYTES[case["grad"]] + wrote, "flops": 2 * there * d}
    if case["op"] == "norm":
        e = case["m"] * case["dim"]
        b = _BYTES[case["type"]]
        moved = e * (3 * b if case["residual"] else b) + e + 4 * case["m"]
        return {"bytes": moved + (4 * case["dim"] if case["weight"] else 0), "flops": 6 * e}
    m, n, k = case["m"], case["n"], case["k"]
    return {"bytes": m * k + n * k + 4 * m + (8 if case["bias"] else 4) * n
            + m * n * _BYTES[case["out"]], "flops": 2.0 * m * n * k}


# ------------------------------------------------------------------ exact --
def exact(case, seed):
    st = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "lookup":
        out = torch.zeros(case["tokens"], case["dim"], dtype=f64, device="cuda")
        at = torch.nonzero(st["tokens"] >= 0).squeeze(1)
        out[at] = st["table"].index_select(0, st["tokens"][at].long()).to(f64) * st["scale"]
        return {"rows": out}
    if case["op"] == "grad":
        # the rows that occur, numbered; their sums by number
        at = torch.nonzero(st["tokens"] >= 0).squeeze(1)
        names, back = torch.unique(st["tokens"][at].long(), return_inverse=True)
        sums = torch.zeros(names.numel(), case["dim"], dtype=f64, device="cuda")
        sums.scatter_add_(0, back[:, None].expand(-1, case["dim"]), st["grad"][at].to(f64))
        out = (st["table"].to(f64) if case["accumulate"] else
               torch.zeros(case["rows"], case["dim"], dtype=f64, device="cuda"))
        out[names] += sums * st["scale"]
        return {"table": out}
    if case["op"] == "norm":
        h = st["x"].to(f64)
        if st["residual"] is not None:
            h = (h + st["residual"].to(f64)).to(torch.float32).to(st["x"].dtype).to(f64)
        r = (h.pow(2).sum(1) / case["dim"] + _EPS).sqrt().reciprocal()
        y = torch.einsum("md,m->md", h, r)
        if st["weight"] is not None:
            y = torch.einsum("md,d->md", y, st["weight"].to(f64))
        s = y.abs().max(1).values / 127.0
        s32 = s.to(torch.float32).to(f64)
        return {"h": h, "codes": (y / s32[:, None]).round().to(torch.int8), "scale": s}
    a = st["a"].to(f64) * st["a_scale"].to(f64)[:, None]
    w = st["w"].to(f64) * st["w_scale"].to(f64)[:, None]
    c = torch.mm(a, w.t())
    if st["bias"] is not None:
        c += st["bias"].to(f64)
    if case["act"] == "relu":
        c = torch.where(c > 0, c, torch.zeros_like(c))
    elif case["act"] == "sigmoid":
        c = torch.reciprocal(1.0 + torch.exp(-c))
    return {"out": c}
