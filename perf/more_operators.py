"""Cases of the attention operators: norm and rotation of queries and keys with
their gradient, attention over packed sequences with its gradient, a paged
cache in 8 or 4 bits, and attention of single tokens over that cache.

A case is one call of one operator ("op"; "cache" writes and reads back).
`run` computes it in elementary torch operations, or, where `own` is true,
through this package's entry points.  `exact` gives the same outputs from the
definitions in 64 bits.

The cache holds groups of 32 values as codes (E4M3 in 8 bits, E2M1 in 4, the
lower half byte first) with a power of two for each group, the smallest that
clips nothing and at least 2^-117, kept as its exponent plus 127.  Codes lie as
(pages, heads, page, bytes), scales as (pages, heads, page, groups).
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "bf16": 2}
_EPS = 1e-6
_GROUP = 32
_TOP = {8: 448.0, 4: 6.0}
_CELLS = 1 << 28                # scores that the plain forms hold at once


def listed():
    return [
        # one token being decoded, far into its sequence
        {"name": "rope-one", "op": "rope", "tokens": 1, "heads": 32, "kv_heads": 8, "dim": 128,
         "pairs": 64, "type": "bf16", "interleaved": False, "weight": True, "first": 1000000},
        # a prompt's tokens
        {"name": "rope-long", "op": "rope", "tokens": 16384, "heads": 32, "kv_heads": 8,
         "dim": 128, "pairs": 64, "type": "bf16", "interleaved": False, "weight": True, "first": 0},
        # a training batch in 32 bits, two thirds of each head rotated
        {"name": "rope-grad", "op": "rope_grad", "tokens": 8191, "heads": 16, "kv_heads": 4,
         "dim": 96, "pairs": 32, "type": "f32", "interleaved": True, "weight": True, "first": 0},
        # 2048 histories of up to 20 items, embedding rows of 64 as heads
        {"name": "attention-history", "op": "attention", "batch": 2048, "longest": 20,
         "spread": 1.0, "past": 0, "heads": 4, "kv_heads": 4, "dim": 64, "type": "f32",
         "causal": True},
        # four prompts of different lengths in one batch
        {"name": "attention-prompt", "op": "attention", "batch": 4, "longest": 6500,
         "spread": 0.7, "past": 0, "heads": 32, "kv_heads": 8, "dim": 128, "type": "bf16",
         "causal": True},
        # pieces of prompts whose earlier keys are there already, a width that is no power of two
        {"name": "attention-piece", "op": "attention", "batch": 7, "longest": 1001,
         "spread": 0.9, "past": 777, "heads": 12, "kv_heads": 4, "dim": 80, "type": "bf16",
         "causal": True},
        # the gradient of the histories' attention, in 32 bits
        {"name": "attention-grad-history", "op": "attention_grad", "batch": 2048, "longest": 20,
         "spread": 1.0, "past": 0, "heads": 4, "kv_heads": 4, "dim": 64, "type": "f32",
         "causal": True},
        # a training batch of long sequences
        {"name": "attention-grad-long", "op": "attention_grad", "batch": 3, "longest": 5000,
         "spread": 0.6, "past": 0, "heads": 32, "kv_heads": 8, "dim": 128, "type": "bf16",
         "causal": True},
        # one step of 64 requests
        {"name": "cache-step", "op": "cache", "tokens": 64, "kv_heads": 8, "dim": 128, "bits": 4,
         "pages": 512, "page": 64, "type": "bf16"},
        # a prompt's keys and values
        {"name": "cache-prompt", "op": "cache", "tokens": 16384, "kv_heads": 8, "dim": 128,
         "bits": 8, "pages": 2048, "page": 16, "type": "bf16"},
        # one request with a long past
        {"name": "cached-long", "op": "cached", "batch": 1, "longest": 131001, "spread": 0.0,
         "heads": 32, "kv_heads": 8, "dim": 128, "bits": 4, "page": 64, "type": "bf16"},
        # a full server: requests of different lengths
        {"name": "cached-batch", "op": "cached", "batch": 64, "longest": 8000, "spread": 0.9,
         "heads": 32, "kv_heads": 8, "dim": 128, "bits": 8, "page": 16, "type": "bf16"},
    ]


def _size(rng, low, high):
    """A whole number spread over the logarithm of [low, high]."""
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _heads(rng):
    """Heads and key heads: groups of one to sixteen."""
    kv = rng.choice((1, 2, 3, 4, 8))
    return kv * rng.choice((1, 2, 3, 4, 8, 16) if kv < 8 else (1, 2, 4)), kv


def draw(rng):
    op = rng.choice(("rope", "rope_grad", "attention", "attention_grad", "cache", "cached"))
    kind = rng.choice(("f32", "bf16"))
    heads, kv = _heads(rng)
    if op in ("rope", "rope_grad"):
        dim = 8 * rng.randint(1, 32)
        row = (heads + kv) * dim
        return {"op": op, "tokens": _size(rng, 1, max(1, (1 << 25) // row)), "heads": heads,
                "kv_heads": kv, "dim": dim, "pairs": 4 * rng.randint(1, dim // 8), "type": kind,
                "interleaved": rng.random() < 0.5, "weight": rng.random() < 0.8,
                "first": rng.choice((0, 0, 5000, 1000000))}
    if op in ("attention", "attention_grad"):
        dim = rng.choice((64, 128, 8 * rng.randint(1, 16)))
        batch = _size(rng, 1, 1024)
        # at most about 2^38 operations, and 2^24 elements of queries
        most = math.sqrt((1 << 34) / (heads * max(dim, 64) * batch))
        longest = _size(rng, 1, max(1, int(min(most, (1 << 24) / (batch * heads * dim)))))
        return {"op": op, "batch": batch, "longest": longest, "spread": rng.choice((0.0, 0.5, 1.0)),
                "past": rng.choice((0, 0, _size(rng, 1, max(1, longest)))), "heads": heads,
                "kv_heads": kv, "dim": dim, "type": kind, "causal": rng.random() < 0.7}
    dim = rng.choice((32, 64, 128))
    page = rng.choice((16, 32, 64, 128, 256))
    if op == "cache":
        tokens = _size(rng, 1, (1 << 24) // (kv * dim))
        return {"op": op, "tokens": tokens, "kv_heads": kv, "dim": dim, "bits": rng.choice((4, 8)),
                "pages": tokens // page + rng.randint(1, 64), "page": page, "type": kind}
    batch = _size(rng, 1, 256)
    return {"op": op, "batch": batch, "longest": _size(rng, 1, (1 << 26) // (batch * kv * dim)),
            "spread": rng.choice((0.0, 0.5, 1.0)), "heads": heads, "kv_heads": kv, "dim": dim,
            "bits": rng.choice((4, 8)), "page": page, "type": kind}


def _lengths(case):
    """Sequence lengths of a case, spread below the longest."""
    return [int(round(case["longest"] * (1.0 - case["spread"] * ((i + 1) * 0.6180339887498949 % 1))))
            if i else case["longest"] for i in range(case["batch"])]


def _sums(lengths):
    out = [0]
    for n in lengths:
        out.append(out[-1] + n)
    return out


# ------------------------------------------------------------------ cache --
def _to_codes(x, bits):
    """Codes and scales of (..., dim) values, laid out as the cache holds them."""
    g = x.float().unflatten(-1, (-1, _GROUP))
    top = g.abs().amax(-1)
    mantissa, exponent = torch.frexp(top / _TOP[bits])      # the division may round up to
    e = torch.where(mantissa > 0.5, exponent, exponent - 1)  # a power of two, or down to one
    e = torch.where(torch.ldexp(torch.full_like(top, _TOP[bits]), e) < top, e + 1, e)
    e = torch.where(top > 0, e, -117).clamp(min=-117)
    y = torch.ldexp(g, -e[..., None])
    if bits == 8:
        codes = y.to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2)
    else:
        a = y.abs()
        c = (a > 0.25).to(torch.uint8)
        for border, even_above in ((0.75, True), (1.25, False), (1.75, True), (2.5, False),
                                   (3.5, True), (5.0, False)):
            c += (a >= border) if even_above else (a > border)
        c = (c + 8 * torch.signbit(y).to(torch.uint8)).flatten(-2)
        codes = c[..., 0::2] | c[..., 1::2] << 4
    return codes, (e + 127).to(torch.uint8)


def _from_codes(codes, scales, bits):
    """The float32 values that codes and scales stand for."""
    if bits == 8:
        v = codes.view(torch.float8_e4m3fn).float()
    else:
        c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).long()
        table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6],
                             device=codes.device)
        v = table[c]
    g = v.unflatten(-1, (-1, _GROUP))
    return torch.ldexp(g, scales.int()[..., None] - 127).flatten(-2)


# ----------------------------------------------------------------- inputs --
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1_000_003 + 17)
    dt = _DT[case["type"]]

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(scale)

    st = {"case": case}
    if case["op"] in ("rope", "rope_grad"):
        n, d = case["tokens"], case["dim"]
        st["q"] = normal(n, case["heads"], d, scale=2.0).to(dt)
        st["k"] = normal(n, case["kv_heads"], d, scale=2.0).to(dt)
        st["positions"] = torch.arange(n, device="cuda", dtype=torch.int32) + case["first"]
        i = torch.arange(case["pairs"], device="cuda", dtype=torch.float64)
        st["freqs"] = (500000.0 ** (-i / case["pairs"])).float()
        st["q_weight"] = normal(d, scale=0.1).add_(1.0) if case["weight"] else None
        st["k_weight"] = normal(d, scale=0.1).add_(1.0) if case["weight"] else None
        if case["op"] == "rope_grad":
            st["grad_q"] = normal(n, case["heads"], d, scale=1e-2).to(dt)
            st["grad_k"] = normal(n, case["kv_heads"], d, scale=1e-2).to(dt)
    elif case["op"] in ("attention", "attention_grad"):
        lengths = _lengths(case)
        st["sums"] = _sums(lengths)
        st["kv_sums"] = _sums([m + case["past"] for m in lengths])
        st["offsets"] = torch.tensor(st["sums"], dtype=torch.int32, device="cuda")
        st["kv_offsets"] = (torch.tensor(st["kv_sums"], dtype=torch.int32, device="cuda")
                            if case["past"] else None)
        n, m, d = st["sums"][-1], st["kv_sums"][-1], case["dim"]
        st["q"] = normal(n, case["heads"], d).to(dt)
        st["k"] = normal(m, case["kv_heads"], d).to(dt)
        st["v"] = normal(m, case["kv_heads"], d).to(dt)
        if case["op"] == "attention_grad":     # what the forward pass left
            done = _plain_attention(case, st)
            st["out"], st["lse"] = done["out"], done["lse"]
            st["grad"] = normal(n, case["heads"], d, scale=1e-2).to(dt)
    elif case["op"] == "cache":
        n, h, d = case["tokens"], case["kv_heads"], case["dim"]
        st["k"], st["v"] = normal(n, h, d).to(dt), normal(n, h, d).to(dt)
        slots = torch.randperm(case["pages"] * case["page"], generator=g, device="cuda")[:n]
        st["slots"] = slots.to(torch.int32)
        shape = (case["pages"], h, case["page"])
        for name in ("k", "v"):
            st[name + "_codes"] = torch.zeros(*shape, d * case["bits"] // 8, dtype=torch.uint8,
                                              device="cuda")
            st[name + "_scales"] = torch.zeros(*shape, d // _GROUP, dtype=torch.uint8,
                                               device="cuda")
    else:
        lengths = _lengths(case)
        h, d, page = case["kv_heads"], case["dim"], case["page"]
        st["lengths"] = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        most = max(1, -(-max(lengths) // page))
        used = [-(-n // page) for n in lengths]
        pages = max(1, sum(used))
        # pages lie in no order; entries behind a sequence's last page name none
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((case["batch"], most), -1, dtype=torch.int32)
        at = 0
        names = order.cpu()
        for b, c in enumerate(used):
            table[b, :c] = names[at:at + c]
            at += c
        st["table"] = table.cuda()
        st["q"] = normal(case["batch"], case["heads"], d).to(dt)
        for name in ("k", "v"):
            codes, scales = [], []
            for i in range(0, pages, 4096):
                some = _to_codes(normal(min(4096, pages - i), h, page, d), case["bits"])
                codes.append(some[0])
                scales.append(some[1])
            st[name + "_codes"], st[name + "_scales"] = torch.cat(codes), torch.cat(scales)
    return st


# -------------------------------------------------------------------- run --
def _rotation(case, st):
    a = st["positions"].double()[:, None] * st["freqs"].double()
    return torch.cos(a).float()[:, None, :], torch.sin(a).float()[:, None, :]


def _halves(case, x):
    """The two members of each pair, as views of (..., pairs)."""
    p = case["pairs"]
    if case["interleaved"]:
        return x[..., 0:2 * p:2], x[..., 1:2 * p:2]
    return x[..., :p], x[..., p:2 * p]


def _turn(case, x, cos, sin):
    out = x.clone()
    a, b = _halves(case, x)
    oa, ob = _halves(case, out)
    oa.copy_(a * cos - b * sin)
    ob.copy_(a * sin + b * cos)
    return out


def _plain_rope(case, st):
    cos, sin = _rotation(case, st)
    out = {}
    for name in ("q", "k"):
        x = st[name].float()
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS)
        if st[name + "_weight"] is not None:
            y = y * st[name + "_weight"]
        out[name] = _turn(case, y, cos, sin).to(st[name].dtype)
    return out


def _plain_rope_grad(case, st):
    cos, sin = _rotation(case, st)
    out = {}
    for name in ("q", "k"):
        x = st[name].float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS)
        dy = _turn(case, st["grad_" + name].float(), cos, -sin)
        if st[name + "_weight"] is not None:
            out[name + "_weight"] = (dy * x * r).sum((0, 1), dtype=torch.float64).float()
            dy = dy * st[name + "_weight"]
        dx = r * dy - x * (r * r * r) * (x * dy).mean(-1, keepdim=True)
        out[name] = dx.to(st[name].dtype)
    return out


def _blocks(case, st):
    """Sequences in blocks of padded rows: index and mask of queries and keys,
    and ranges of key heads, so that no block holds more than _CELLS scores."""
    lengths = _lengths(case)
    group = case["heads"] // case["kv_heads"]
    first = 0
    while first < len(lengths):
        last, lq = first + 1, lengths[first]
        while last < len(lengths):
            longer = max(lq, lengths[last])
            cells = (last + 1 - first) * longer * (longer + case["past"]) * case["heads"]
            if cells > _CELLS:
                break
            last, lq = last + 1, longer
        lk = lq + case["past"]
        if lk:
            at = torch.arange(first, last, device="cuda")
            q0, q1 = st["offsets"][at].long(), st["offsets"][at + 1].long()
            keys = st["offsets"] if st["kv_offsets"] is None else st["kv_offsets"]
            k0, k1 = keys[at].long(), keys[at + 1].long()
            iq = q0[:, None] + torch.arange(lq, device="cuda")
            ik = k0[:, None] + torch.arange(lk, device="cuda")
            there_q, there_k = iq < q1[:, None], ik < k1[:, None]
            seen = there_q[:, :, None] & there_k[:, None, :]
            if case["causal"]:     # the last query sees the last key
                pq = iq - q1[:, None]
                pk = ik - k1[:, None]
                seen = seen & (pk[:, None, :] <= pq[:, :, None])
            step = max(1, min(case["kv_heads"], _CELLS // max(1, (last - first) * lq * lk * group)))
            for h in range(0, case["kv_heads"], step):
                yield (torch.where(there_q, iq, 0), there_q, torch.where(there_k, ik, 0), there_k,
                       seen[:, None, None], h, min(h + step, case["kv_heads"]))
        first = last


def _rows(x, index, there, h0, h1, group):
    """(block, key heads, group, rows, dim) of float32, zeros where no row is."""
    y = x[index][:, :, h0 * group:h1 * group].float()
    y = torch.where(there[:, :, None, None], y, torch.zeros_like(y))
    return y.unflatten(2, (h1 - h0, group)).permute(0, 2, 3, 1, 4)


def _put(out, y, index, there, h0, h1, group):
    """Rows of a block back to where they belong."""
    rows = y.permute(0, 3, 1, 2, *range(4, y.dim())).flatten(2, 3)
    out[:, h0 * group:h1 * group].index_put_((index[there],), rows[there].to(out.dtype))


def _plain_attention(case, st):
    group, scale = case["heads"] // case["kv_heads"], case["dim"] ** -0.5
    out = torch.zeros_like(st["q"])
    lse = torch.full(st["q"].shape[:2], -math.inf, device="cuda")
    for iq, tq, ik, tk, seen, h0, h1 in _blocks(case, st):
        q = _rows(st["q"], iq, tq, h0, h1, group)
        k = _rows(st["k"], ik, tk, h0, h1, 1)
        v = _rows(st["v"], ik, tk, h0, h1, 1)
        s = torch.where(seen, q @ k.transpose(-1, -2) * scale, -math.inf)
        top = s.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, torch.zeros_like(top), top)
        p = torch.exp(s - top)
        total = p.sum(-1, keepdim=True)
        o = p @ v / torch.where(total > 0, total, torch.ones_like(total))
        _put(out, o, iq, tq, h0, h1, group)
        _put(lse, (torch.log(total) + top)[..., 0], iq, tq, h0, h1, group)
    return {"out": out, "lse": lse}


def _plain_attention_grad(case, st):
    group, scale = case["heads"] // case["kv_heads"], case["dim"] ** -0.5
    dq, dk, dv = (torch.zeros_like(st[name]) for name in ("q", "k", "v"))
    for iq, tq, ik, tk, seen, h0, h1 in _blocks(case, st):
        q = _rows(st["q"], iq, tq, h0, h1, group)
        k = _rows(st["k"], ik, tk, h0, h1, 1)
        v = _rows(st["v"], ik, tk, h0, h1, 1)
        do = _rows(st["grad"], iq, tq, h0, h1, group)
        delta = (do * _rows(st["out"], iq, tq, h0, h1, group)).sum(-1, keepdim=True)
        lse = _rows(st["lse"][..., None], iq, tq, h0, h1, group)
        lse = torch.where(lse == -math.inf, torch.zeros_like(lse), lse)
        s = q @ k.transpose(-1, -2) * scale
        p = torch.where(seen, torch.exp(s - lse), torch.zeros_like(s))
        ds = p * (do @ v.transpose(-1, -2) - delta) * scale
        _put(dq, ds @ k, iq, tq, h0, h1, group)
        _put(dk, (ds.transpose(-1, -2) @ q).sum(2, keepdim=True), ik, tk, h0, h1, 1)
        _put(dv, (p.transpose(-1, -2) @ do).sum(2, keepdim=True), ik, tk, h0, h1, 1)
    return {"q": dq, "k": dk, "v": dv}


def _plain_cache(case, st):
    page, at = (st["slots"].long() // case["page"], st["slots"].long() % case["page"])
    out = {}
    for name in ("k", "v"):
        codes, scales = _to_codes(st[name], case["bits"])
        st[name + "_codes"][page, :, at] = codes
        st[name + "_scales"][page, :, at] = scales
        out[name] = _from_codes(st[name + "_codes"][page, :, at], st[name + "_scales"][page, :, at],
                                case["bits"]).to(st[name].dtype)
    return out


def _plain_cached(case, st):
    group, scale = case["heads"] // case["kv_heads"], case["dim"] ** -0.5
    out = torch.zeros_like(st["q"])
    longest = st["table"].shape[1] * case["page"]
    step = max(1, _CELLS // (longest * case["kv_heads"] * case["dim"]))
    for b in range(0, case["batch"], step):
        pages = st["table"][b:b + step].long().clamp(min=0)
        k, v = (_from_codes(st[name + "_codes"][pages], st[name + "_scales"][pages], case["bits"])
                .transpose(1, 2).flatten(2, 3) for name in ("k", "v"))
        q = st["q"][b:b + step].float().unflatten(1, (case["kv_heads"], group))
        there = torch.arange(longest, device="cuda") < st["lengths"][b:b + step, None]
        there = there[:, None, None, :]
        s = torch.where(there, q @ k.transpose(-1, -2) * scale, -math.inf)
        top = s.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, torch.zeros_like(top), top)
        p = torch.exp(s - top)
        total = p.sum(-1, keepdim=True)
        o = p @ v / torch.where(total > 0, total, torch.ones_like(total))
        out[b:b + step] = o.flatten(1, 2).to(out.dtype)
    return {"out": out}


_PLAIN = {"rope": _plain_rope, "rope_grad": _plain_rope_grad, "attention": _plain_attention,
          "attention_grad": _plain_attention_grad, "cache": _plain_cache, "cached": _plain_cached}


def _own(case, st):
    import dlrm_embedding_bag_amd as fw
    op = case["op"]
    if op == "rope":
        q, k = fw.qk_norm_rope(st["q"], st["k"], st["positions"], st["freqs"], st["q_weight"],
                               st["k_weight"], eps=_EPS, interleaved=case["interleaved"])
        return {"q": q, "k": k}
    if op == "rope_grad":
        dq, dk, dqw, dkw = fw.qk_norm_rope_grad(
            st["grad_q"], st["grad_k"], st["q"], st["k"], st["positions"], st["freqs"],
            st["q_weight"], st["k_weight"], eps=_EPS, interleaved=case["interleaved"])
        if case["weight"]:
            return {"q_weight": dqw, "q": dq, "k_weight": dkw, "k": dk}
        return {"q": dq, "k": dk}
    if op == "attention":
        out, lse = fw.attention_packed(st["q"], st["k"], st["v"], st["offsets"], st["kv_offsets"],
                                       causal=case["causal"])
        return {"out": out, "lse": lse}
    if op == "attention_grad":
        dq, dk, dv = fw.attention_packed_grad(st["grad"], st["q"], st["k"], st["v"], st["out"],
                                              st["lse"], st["offsets"], st["kv_offsets"],
                                              causal=case["causal"])
        return {"q": dq, "k": dk, "v": dv}
    cache = fw.KVCache(st["k_codes"], st["k_scales"], st["v_codes"], st["v_scales"])
    if op == "cache":
        fw.kv_cache_write(cache, st["k"], st["v"], st["slots"])
        k, v = fw.kv_cache_read(cache, st["slots"], out_dtype=_DT[case["type"]])
        return {"k": k, "v": v}
    return {"out": fw.attention_cached(st["q"], cache, st["table"], st["lengths"])}


def run(state):
    case = state["case"]
    return _own(case, state) if own else _PLAIN[case["op"]](case, state)


# ------------------------------------------------------------------- work --
def _scores(case):
    """Scores that a mask leaves."""
    total = 0
    for n in _lengths(case):
        total += n * case["past"] + (n * (n + 1) // 2 if case["causal"] else n * n)
    return total


def work(case):
    op = case["op"]
    b = _BYTES[case["type"]]
    d = case["dim"]
    if op in ("rope", "rope_grad"):
        e = case["tokens"] * (case["heads"] + case["kv_heads"]) * d
        once = 4 * case["tokens"] + 4 * case["pairs"] + (8 * d if case["weight"] else 0)
        if op == "rope":
            return {"bytes": 2 * e * b + once, "flops": 8 * e}
        return {"bytes": 3 * e * b + once + (8 * d if case["weight"] else 0), "flops": 16 * e}
    if op in ("attention", "attention_grad"):
        lengths = _lengths(case)
        n = sum(lengths)
        m = n + case["past"] * len(lengths)
        rows, keys = n * case["heads"], m * case["kv_heads"]
        index = 4 * (len(lengths) + 1) * (2 if case["past"] else 1)
        products = 2.0 * _scores(case) * case["heads"] * d
        if op == "attention":
            return {"bytes": 2 * (rows + keys) * d * b + 4 * rows + index, "flops": 2 * products}
        return {"bytes": (4 * rows + 4 * keys) * d * b + 4 * rows + index, "flops": 5 * products}
    row = d * case["bits"] // 8 + d // _GROUP       # of codes and scales
    if op == "cache":                               # written, and read back
        t = 2 * case["tokens"] * case["kv_heads"]
        return {"bytes": t * (2 * d * b + 2 * row) + 4 * case["tokens"], "flops": 6 * t * d}
    keys = sum(_lengths(case))
    pages = sum(-(-n // case["page"]) for n in _lengths(case))
    rows = case["batch"] * case["heads"]
    return {"bytes": 2 * keys * case["kv_heads"] * row + 2 * rows * d * b + 4 * pages
            + 4 * case["batch"], "flops": 4.0 * keys * case["heads"] * d}


# ------------------------------------------------------------------ exact --
def _exact_rope(case, st):
    f64 = torch.float64
    n, p = case["tokens"], case["pairs"]
    angle = torch.outer(st["positions"].to(f64), st["freqs"].to(f64))
    # each pair as a complex number, turned by its angle
    turn = torch.complex(angle.cos(), angle.sin()).view(n, 1, p)
    grad = case["op"] == "rope_grad"
    out = {}
    for name in ("q", "k"):
        x = st[name].to(f64)
        w = st[name + "_weight"]
        w = torch.ones(case["dim"], dtype=f64, device="cuda") if w is None else w.to(f64)
        size = (x.pow(2).sum(-1, keepdim=True) / case["dim"] + _EPS).sqrt()
        y = st["grad_" + name].to(f64) if grad else x / size * w
        if case["interleaved"]:
            pair = y[..., :2 * p].reshape(*y.shape[:2], p, 2)
            z = torch.complex(pair[..., 0].contiguous(), pair[..., 1].contiguous())
            z = z * (turn.conj() if grad else turn)
            head = torch.stack((z.real, z.imag), -1).reshape(*y.shape[:2], 2 * p)
        else:
            z = torch.complex(y[..., :p].contiguous(), y[..., p:2 * p].contiguous())
            z = z * (turn.conj() if grad else turn)
            head = torch.cat((z.real, z.imag), -1)
        y = torch.cat((head, y[..., 2 * p:]), -1)
        if grad:
            unit = x / size
            if case["weight"]:
                out[name + "_weight"] = torch.einsum("thd,thd->d", y, unit)
            y = y * w
            y = (y - unit * (y * unit).sum(-1, keepdim=True) / case["dim"]) / size
        out[name] = y
    return out


def _exact_attention(case, st):
    f64 = torch.float64
    group, scale = case["heads"] // case["kv_heads"], 1.0 / math.sqrt(case["dim"])
    grad = case["op"] == "attention_grad"
    out = {name: torch.zeros(st[name].shape, dtype=f64, device="cuda")
           for name in (("q", "k", "v") if grad else ("q",))}
    lse = torch.full(st["q"].shape[:2], -math.inf, dtype=f64, device="cuda")
    for b in range(case["batch"]):
        q0, q1 = st["sums"][b], st["sums"][b + 1]
        k0, k1 = st["kv_sums"][b], st["kv_sums"][b + 1]
        if q0 == q1 or k0 == k1:
            continue
        hidden = None
        if case["causal"]:
            hidden = torch.ones(q1 - q0, k1 - k0, dtype=torch.bool, device="cuda")
            hidden = hidden.triu((k1 - k0) - (q1 - q0) + 1)
        # the short ones with all heads at once, the long ones head by head
        few = (q1 - q0) * (k1 - k0) * case["heads"] <= 1 << 24
        for h0 in range(0, case["heads"], case["heads"] if few else 1):
            h1 = h0 + (case["heads"] if few else 1)
            at = torch.arange(h0, h1, device="cuda") // group
            q = st["q"][q0:q1, h0:h1].to(f64).movedim(1, 0)
            k = st["k"][k0:k1].index_select(1, at).to(f64).movedim(1, 0)
            v = st["v"][k0:k1].index_select(1, at).to(f64).movedim(1, 0)
            s = torch.matmul(q, k.mT).mul_(scale)
            if hidden is not None:
                s.masked_fill_(hidden, -math.inf)
            if not grad:
                l = torch.logsumexp(s, -1)
                lse[q0:q1, h0:h1] = l.T
                out["q"][q0:q1, h0:h1] = torch.matmul(torch.softmax(s, -1), v).movedim(0, 1)
                continue
            do = st["grad"][q0:q1, h0:h1].to(f64).movedim(1, 0)
            o = st["out"][q0:q1, h0:h1].to(f64).movedim(1, 0)
            p = s.sub_(st["lse"][q0:q1, h0:h1].to(f64).T[..., None]).exp_()
            out["v"][k0:k1].index_add_(1, at, torch.matmul(p.mT, do).movedim(0, 1))
            p.mul_(torch.matmul(do, v.mT).sub_((do * o).sum(-1, keepdim=True))).mul_(scale)
            out["q"][q0:q1, h0:h1] = torch.matmul(p, k).movedim(0, 1)
            out["k"][k0:k1].index_add_(1, at, torch.matmul(p.mT, q).movedim(0, 1))
    return out if grad else {"out": out["q"], "lse": lse}


def _exact_cache(case, st):
    out = {}
    for name in ("k", "v"):
        x = st[name].to(torch.float64)
        g = x.reshape(-1, _GROUP)
        top = g.abs().max(1, keepdim=True).values
        unit = torch.exp2(torch.log2(top / _TOP[case["bits"]]).ceil().clamp(min=-117.0))
        # the logarithm may be off by a rounding next to a whole number
        unit = torch.where(unit * _TOP[case["bits"]] < top, unit * 2, unit)
        lower = torch.clamp(unit / 2, min=2.0 ** -117)
        unit = torch.where(lower * _TOP[case["bits"]] >= top, lower, unit)
        y = g / unit
        if case["bits"] == 4:      # steps of 1/2 below 2, of 1 below 4, of 2 above
            step = 0.5 + 0.5 * (y.abs() >= 2) + (y.abs() >= 4)
        else:                      # three bits behind the first, which is 2^-6 at least
            step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
        out[name] = ((y / step).round() * step * unit).reshape(x.shape)
    return out


def _exact_cached(case, st):
    f64 = torch.float64
    group = case["heads"] // case["kv_heads"]
    out = torch.zeros(st["q"].shape, dtype=f64, device="cuda")
    nibble = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=f64, device="cuda")
    nibble = torch.cat((nibble, -nibble))
    for b, n in enumerate(_lengths(case)):
        if n == 0:
            continue
        pages = st["table"][b, :-(-n // case["page"])].long()
        values = []
        for name in ("k", "v"):
            c = st[name + "_codes"].index_select(0, pages).movedim(1, 0).flatten(1, 2)[:, :n]
            s = st[name + "_scales"].index_select(0, pages).movedim(1, 0).flatten(1, 2)[:, :n]
            if case["bits"] == 8:
                c = c.contiguous().view(torch.float8_e4m3fn).to(f64)
            else:
                c = nibble[torch.stack((c % 16, c // 16), -1).flatten(-2).int()]
            values.append(c * torch.exp2(s.to(f64) - 127.0).repeat_interleave(_GROUP, -1))
        q = st["q"][b].to(f64).view(case["kv_heads"], group, -1)
        s = torch.matmul(q, values[0].mT) / math.sqrt(case["dim"])
        out[b] = torch.matmul(torch.softmax(s, -1), values[1]).flatten(0, 1)
    return {"out": out}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("rope", "rope_grad"):
        return _exact_rope(case, st)
    if case["op"] in ("attention", "attention_grad"):
        return _exact_attention(case, st)
    return _exact_cache(case, st) if case["op"] == "cache" else _exact_cached(case, st)
