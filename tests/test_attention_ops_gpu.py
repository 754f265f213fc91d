"""GPU tests of the attention operators against plain 64-bit forms on the host.

Tolerances count roundings.  One rounding to type t is off by at most half a
step, u(t) = finfo(t).eps / 2 relative to the value (u32 = 2^-24, bf16 2^-8).
  rotation  x u w has three roundings; sine and cosine are off by at most 4 steps
            of a value of at most 1 (8 u32) and their angle by 1 u32; two products
            and a sum follow: 14 u32 of |a| + |b| for a pair (a, b), then the
            output's type
  its gradient  the turned gradient the same; times w, minus u times a mean of
            such terms, times 1 / rms: 20 u32 of the terms' magnitudes; the
            weights' sum of c terms c u32 of the sum of magnitudes more
  attention a score of d products is off by d u32 of the sum of magnitudes, its
            exponent by 4 u32 of the largest score more, exp2 by 4 u32: e relative
            in each weight, so 2 e of sum p |v| in the quotient, n u32 for the
            sums of n terms, u(bf16) for the weights' rounding in bfloat16
"""
import math

import numpy as np
import pytest

from conftest import gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]

U32 = 2.0 ** -24
U = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
TINY = 2.0 ** -126


def _dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _np64(t):
    import torch
    return t.detach().cpu().to(torch.float64).numpy()


def _assert_within(got, want, tol, what):
    same = (got == want) | (np.isnan(got) & np.isnan(want))
    with np.errstate(invalid="ignore"):
        err = np.where(same, 0.0, np.abs(got - want))
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, first at "
                           f"{tuple(np.argwhere(bad)[0])}: {got[bad][0]!r} for {want[bad][0]!r}, "
                           f"tolerance {np.broadcast_to(tol, err.shape)[bad][0]!r}")


def _randn(g, *shape, scale=1.0):
    import torch
    return torch.randn(shape, generator=g, dtype=torch.float32) * scale


def _gen(seed):
    import torch
    return torch.Generator().manual_seed(seed)


# `layout` of (tokens, heads, dim) on the GPU: as it is; a slice of a wider row
# with other values around; or with heads outside of tokens
def _laid(t, layout):
    import torch
    if layout == "slice":
        buf = torch.full((t.shape[0], t.shape[1] + 2, t.shape[2] + 8), float("nan"), dtype=t.dtype)
        buf[:, 1:-1, :t.shape[2]] = t
        return buf.cuda()[:, 1:-1, :t.shape[2]]
    if layout == "heads":
        return t.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    return t.cuda()


# ----------------------------------------------------------- norm and rotation --
def _pairs_of(x, pairs, inter):
    if inter:
        return x[..., 0:2 * pairs:2], x[..., 1:2 * pairs:2]
    return x[..., :pairs], x[..., pairs:2 * pairs]


def _turned(y, pos, freqs, inter, sign=1.0):
    """The turned rows and, element by element, |a| + |b| of its pair."""
    pairs = len(freqs)
    angle = pos.astype(np.float64)[:, None, None] * freqs.astype(np.float64)
    out, size = y.copy(), np.abs(y)
    a, b = _pairs_of(y, pairs, inter)
    oa, ob = _pairs_of(out, pairs, inter)
    sa, sb = _pairs_of(size, pairs, inter)
    oa[...] = a * np.cos(angle) - sign * b * np.sin(angle)
    ob[...] = sign * a * np.sin(angle) + b * np.cos(angle)
    sa[...] = sb[...] = np.abs(a) + np.abs(b)
    return out, size


def _rope_inputs(n, heads, kv, dim, pairs, kind, weight, first, seed):
    import torch
    g = _gen(seed)
    q = _randn(g, n, heads, dim, scale=3.0).to(_dt(kind))
    k = _randn(g, n, kv, dim, scale=0.2).to(_dt(kind))
    pos = (torch.arange(n, dtype=torch.int64) * 37 + first).to(torch.int32)
    freqs = (10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).float()
    wq = 1.0 + _randn(g, dim, scale=0.3) if weight else None
    wk = 1.0 + _randn(g, dim, scale=0.3) if weight else None
    return q, k, pos, freqs, wq, wk


ROPES = [(1, 32, 8, 128, 64), (3, 5, 0, 64, 32), (7, 2, 2, 8, 4), (33, 3, 1, 24, 12),
         (130, 6, 2, 96, 32), (65, 1, 1, 80, 40), (5, 7, 3, 256, 128), (40, 4, 4, 120, 20),
         (1025, 2, 1, 16, 8), (2051, 1, 2, 64, 16), (1024, 5, 1, 40, 4)]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("n,heads,kv,dim,pairs", ROPES)
def test_rope(n, heads, kv, dim, pairs, inter, kind):
    import dlrm_embedding_bag_amd as fw
    weight, first = (n + dim) % 3 != 0, (0, 1000000, -5, 2**31 - 37 * n)[(n + heads) % 4]
    q, k, pos, freqs, wq, wk = _rope_inputs(n, heads, kv, dim, pairs, kind, weight, first, n + dim)
    layout = ("plain", "slice", "heads")[(n + pairs) % 3]
    got = fw.qk_norm_rope(_laid(q, layout), _laid(k, layout) if kv else None, pos.cuda(),
                          freqs.cuda(), None if wq is None else wq.cuda(),
                          None if wk is None else wk.cuda(), eps=1e-5, interleaved=inter)
    assert (got[1] is None) == (kv == 0)
    for x, w, y, what in ((q, wq, got[0], "q"), (k, wk, got[1], "k")):
        if y is None:
            continue
        x = _np64(x)
        v = x / np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5)
        if w is not None:
            v = v * _np64(w)
        want, size = _turned(v, pos.numpy(), freqs.numpy(), inter)
        _assert_within(_np64(y), want, 14 * U32 * size + U[kind] * np.abs(want) + TINY, what)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("n,heads,kv,dim,pairs", ROPES + [(4500, 3, 2, 32, 16)])
def test_rope_gradient(n, heads, kv, dim, pairs, inter, kind):
    import dlrm_embedding_bag_amd as fw
    weight, first = (n + dim) % 3 != 0, (0, 1000000, -5, 77)[(n + heads) % 4]
    q, k, pos, freqs, wq, wk = _rope_inputs(n, heads, kv, dim, pairs, kind, weight, first, n + dim)
    g = _gen(n)
    gq, gk = (_randn(g, *t.shape).to(_dt(kind)) for t in (q, k))
    layout = ("plain", "slice", "heads")[(n + pairs) % 3]

    def call():
        return fw.qk_norm_rope_grad(
            _laid(gq, layout), _laid(gk, layout) if kv else None, _laid(q, layout),
            _laid(k, layout) if kv else None, pos.cuda(), freqs.cuda(),
            None if wq is None else wq.cuda(), None if wk is None else wk.cuda(), eps=1e-5,
            interleaved=inter)

    got = call()
    for x, d, w, dx, dw, what in ((q, gq, wq, got[0], got[2], "q"), (k, gk, wk, got[1], got[3], "k")):
        if dx is None:
            assert kv == 0 and what == "k" and dw is None
            continue
        x, d = _np64(x), _np64(d)
        rms = np.sqrt((x * x).mean(-1, keepdims=True) + 1e-5)
        unit = x / rms
        dv, size = _turned(d, pos.numpy(), freqs.numpy(), inter, -1.0)
        ww = np.ones(dim) if w is None else _np64(w)
        gg = dv * ww
        want = (gg - unit * (gg * unit).mean(-1, keepdims=True)) / rms
        big = np.abs(ww) * size
        parts = (big + np.abs(unit) * (np.abs(unit) * big).mean(-1, keepdims=True)) / rms
        _assert_within(_np64(dx), want, 20 * U32 * parts + U[kind] * np.abs(want) + TINY, what)
        assert (dw is None) == (w is None)
        if dw is not None:
            terms = (np.abs(unit) * size).sum((0, 1))
            _assert_within(_np64(dw), (dv * unit).sum((0, 1)),
                           (20 + x.shape[0] * x.shape[1]) * U32 * terms + TINY, what + " weight")
    again = call()
    for a, b in zip(got, again):
        assert a is None or bool((a == b).all())


def test_rope_in_place_and_empty():
    import torch

    import dlrm_embedding_bag_amd as fw
    q, k, pos, freqs, wq, wk = (None if t is None else t.cuda()
                                for t in _rope_inputs(70, 4, 2, 64, 32, "bf16", True, 3, 1))
    for inter in (False, True):
        want = fw.qk_norm_rope(q, k, pos, freqs, wq, wk, interleaved=inter)
        a, b = q.clone(), k.clone()
        va = a._version
        out = fw.qk_norm_rope(a, b, pos, freqs, wq, wk, interleaved=inter, out_q=a, out_k=b)
        assert out[0] is a and out[1] is b and a._version > va
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])
        gq, gk = torch.randn_like(q.float()).to(q.dtype), torch.randn_like(k.float()).to(k.dtype)
        dq, dk, dwq, dwk = fw.qk_norm_rope_grad(gq, gk, q, k, pos, freqs, wq, wk, interleaved=inter)
        a, b = gq.clone(), gk.clone()
        ws = torch.empty(fw.qk_norm_rope_grad_workspace_bytes(70, 64), dtype=torch.uint8,
                         device="cuda")
        out = fw.qk_norm_rope_grad(a, b, q, k, pos, freqs, wq, wk, interleaved=inter, out_q=a,
                                   out_k=b, workspace=ws)
        assert torch.equal(a, dq) and torch.equal(b, dk)
        assert torch.equal(out[2], dwq) and torch.equal(out[3], dwk)
    none = fw.qk_norm_rope_grad(gq[:0], gk[:0], q[:0], k[:0], pos[:0], freqs, wq, wk)
    assert none[0].shape == (0, 4, 64) and not none[2].any() and not none[3].any()
    assert fw.qk_norm_rope(q[:0], k[:0], pos[:0], freqs)[0].shape == (0, 4, 64)


def test_rope_rows_that_are_not_finite_stay_alone():
    import torch

    import dlrm_embedding_bag_amd as fw
    q, k, pos, freqs, wq, wk = (None if t is None else t.cuda()
                                for t in _rope_inputs(9, 3, 1, 64, 32, "f32", True, 3, 2))
    want = fw.qk_norm_rope(q, k, pos, freqs, wq, wk)[0]
    q[4, 1, 7] = float("nan")
    q[5, 0, 9] = float("inf")
    q[6, 2] = 0.0
    q[7, 2] = 1e30              # squares beyond float32
    got = fw.qk_norm_rope(q, k, pos, freqs, wq, wk)[0]
    assert got[4, 1].isnan().any() and got[5, 0].isnan().any()
    assert not got[6, 2].any() and got[7, 2].isfinite().all() and got[7, 2].abs().max() > 0.5
    touched = torch.zeros(9, 3, dtype=torch.bool, device="cuda")
    for at in ((4, 1), (5, 0), (6, 2), (7, 2)):
        touched[at] = True
    assert torch.equal(got[~touched], want[~touched])


# ----------------------------------------------------------- packed attention --
def _sequences(lengths, past=None):
    import torch
    off = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32)
    if past is None:
        return off, None
    kv = [max(0, m + p) for m, p in zip(lengths, past)]
    return off, torch.tensor(np.concatenate([[0], np.cumsum(kv)]), dtype=torch.int32)


def _seen(nq, nk, causal):
    if not causal:
        return np.ones((nq, nk), bool)
    return np.arange(nk)[None, :] <= np.arange(nq)[:, None] + (nk - nq)


def _attention_want(q, k, v, off, koff, causal, scale, kind):
    """out, lse and their tolerances, all float64 on the host."""
    q, k, v = _np64(q), _np64(k), _np64(v)
    off = off.numpy()
    koff = off if koff is None else koff.numpy()
    n, heads, dim = q.shape
    group = heads // k.shape[1]
    out, otol = np.zeros(q.shape), np.zeros(q.shape)
    lse, ltol = np.full((n, heads), -np.inf), np.zeros((n, heads))
    for b in range(len(off) - 1):
        qs, ks = slice(off[b], off[b + 1]), slice(koff[b], koff[b + 1])
        nq, nk = off[b + 1] - off[b], koff[b + 1] - koff[b]
        if nq == 0 or nk == 0:
            continue
        seen = _seen(nq, nk, causal)
        rows = seen.any(1)
        for h in range(heads):
            kk, vv = k[ks, h // group], v[ks, h // group]
            s = np.where(seen, q[qs, h] @ kk.T * scale, -np.inf)
            size = np.where(seen, np.abs(q[qs, h]) @ np.abs(kk).T * scale, 0.0)
            top = np.where(rows, s.max(1, initial=-np.inf), 0.0)[:, None]
            p = np.exp(s - top)
            total = p.sum(1, keepdims=True)
            safe = np.where(total > 0, total, 1.0)
            e = (dim * size.max(1) + 4 * np.abs(np.where(seen, s, 0)).max(1) + 4) * U32
            out[qs, h] = p @ vv / safe
            weight = p @ np.abs(vv) / safe
            otol[qs, h] = ((2 * e[:, None] + (nk + 8) * U32
                            + (U["bf16"] if kind == "bf16" else 0.0)) * weight
                           + U[kind] * np.abs(out[qs, h]) + TINY)
            with np.errstate(divide="ignore"):
                lse[qs, h] = np.where(rows, np.log(total[:, 0]) + top[:, 0], -np.inf)
            ltol[qs, h] = e + (nk + 8 + 4 * np.abs(np.where(rows, lse[qs, h], 0))) * U32
    return out, otol, lse, ltol


# lengths, keys more than queries (None: the same), heads, key heads, dim, causal
PACKED = [
    ([1], None, 1, 1, 8, True), ([1], None, 4, 1, 128, False), ([2, 0, 1], None, 2, 2, 64, True),
    ([31, 32, 33], None, 2, 1, 64, True), ([20, 7, 0, 0, 13, 1, 19], None, 4, 4, 64, True),
    ([64, 65, 63], None, 3, 3, 40, False), ([127, 128, 129], None, 2, 1, 128, True),
    ([300], None, 2, 2, 96, True), ([257, 3, 130], None, 4, 2, 80, True),
    ([1, 1, 1, 1], [5, 64, 130, 0], 8, 2, 128, True), ([5, 40], [100, 33], 6, 3, 72, True),
    ([50, 3], [-20, -3], 2, 1, 32, True), ([50, 9], [-20, -9], 2, 2, 24, False),
    ([700, 65], [-100, 200], 2, 1, 64, True), ([90], [500], 3, 1, 104, False),
    ([3] * 150, None, 2, 1, 16, True), ([0, 0, 5], None, 2, 1, 32, False)]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("lengths,past,heads,kv,dim,causal", PACKED)
def test_attention(lengths, past, heads, kv, dim, causal, kind):
    import dlrm_embedding_bag_amd as fw
    off, koff = _sequences(lengths, past)
    n, m = int(off[-1]), int(off[-1] if koff is None else koff[-1])
    g = _gen(n + dim)
    q = _randn(g, n, heads, dim, scale=1.5).to(_dt(kind))
    k, v = (_randn(g, m, kv, dim).to(_dt(kind)) for _ in range(2))
    scale = None if dim % 16 else 0.3
    want = _attention_want(q, k, v, off, koff, causal, dim ** -0.5 if scale is None else scale, kind)
    layout = ("plain", "slice", "heads")[(n + dim // 8) % 3]
    for layout in {layout, "plain"}:
        out, lse = fw.attention_packed(_laid(q, layout), _laid(k, layout), _laid(v, layout),
                                       off.cuda(), None if koff is None else koff.cuda(),
                                       causal=causal, scale=scale)
        _assert_within(_np64(out), want[0], want[1], "out")
        _assert_within(_np64(lse), want[2], want[3], "lse")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("lengths", [[5, 9], [100, 200, 40]])
def test_attention_rows_outside_the_sequences(lengths, kind):
    """They are left as they are in given tensors and empty in new ones, and what
    they hold reaches no row."""
    import torch

    import dlrm_embedding_bag_amd as fw
    n, lead, tail = sum(lengths), 3, 200
    off = torch.tensor(lead + np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32).cuda()
    g = _gen(4)
    q, k, v = (_randn(g, n, 2, 64).to(_dt(kind)).cuda() for _ in range(3))
    want = _attention_want(q, k, v, (off - lead).cpu(), None, True, 0.125, kind)

    def wide(t):
        buf = torch.full((n + lead + tail, 2, 64), float("nan"), dtype=t.dtype, device="cuda")
        buf[lead:lead + n] = t
        return buf

    def check(out, lse):
        _assert_within(_np64(out[lead:lead + n]), want[0], want[1], "out")
        _assert_within(_np64(lse[lead:lead + n]), want[2], want[3], "lse")

    out, lse = fw.attention_packed(wide(q), wide(k), wide(v), off)
    check(out, lse)
    for part in (slice(0, lead), slice(lead + n, None)):
        assert not out[part].any() and (lse[part] == -math.inf).all()
    given, glse = torch.full_like(out, 7.0), torch.full_like(lse, 8.0)
    back = fw.attention_packed(wide(q), wide(k), wide(v), off, out=given, lse=glse)
    assert back[0] is given and back[1] is glse
    check(given, glse)
    for part in (slice(0, lead), slice(lead + n, None)):
        assert (given[part] == 7.0).all() and (glse[part] == 8.0).all()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("length,at", [(20, 11), (150, 70), (300, 299)])
def test_attention_masked_values_that_are_not_finite(length, at, bad, kind):
    """Rows before a key do not see it, whatever it and its value hold."""
    import torch

    import dlrm_embedding_bag_amd as fw
    g = _gen(length)
    q, k, v = (_randn(g, 2 * length, 2, 64).to(_dt(kind)).cuda() for _ in range(3))
    off = torch.tensor([0, length, 2 * length], dtype=torch.int32, device="cuda")
    want, wlse = fw.attention_packed(q, k, v, off)
    k[at, 0, 5] = bad
    v[at, 1, 3] = bad
    out, lse = fw.attention_packed(q, k, v, off)
    assert torch.equal(out[:at], want[:at]) and torch.equal(lse[:at], wlse[:at])
    assert torch.equal(out[length:], want[length:]) and torch.equal(lse[length:], wlse[length:])
    assert not out[at:length, 1, 3].isfinite().any()
    keep = torch.ones(64, dtype=torch.bool, device="cuda")
    keep[3] = False
    # (in float32 the careful way adds key by key)
    near = (out[at:length, 1][:, keep].float() - want[at:length, 1][:, keep].float()).abs().max()
    assert near <= (1e-5 if kind == "f32" else 2e-2)


def test_attention_extreme_scores():
    """Scores of hundreds either way, and a row whose scores are all -inf."""
    import torch

    import dlrm_embedding_bag_amd as fw
    g = _gen(3)
    q, k = _randn(g, 100, 1, 64, scale=20.0), _randn(g, 100, 1, 64, scale=20.0)
    v = _randn(g, 100, 1, 64)
    off, _ = _sequences([100])
    out, otol, lse, ltol = _attention_want(q, k, v, off, None, True, 0.125, "f32")
    got, glse = fw.attention_packed(q.cuda(), k.cuda(), v.cuda(), off.cuda())
    _assert_within(_np64(got), out, otol, "out")
    _assert_within(_np64(glse), lse, ltol, "lse")
    k[:, :, :] = 0.0
    k[:, :, 0] = -math.inf
    q[:, :, 0] = 1.0
    got, glse = fw.attention_packed(q.cuda(), k.cuda(), v.cuda(), off.cuda())
    assert not got.any() and (glse == -math.inf).all()


def test_attention_bad_offsets_stay_within_the_tensors():
    import torch

    import dlrm_embedding_bag_amd as fw
    q = torch.randn(40, 2, 64, device="cuda")
    for off in ([-5, 100], [30, 10, 60, 5], [2**31 - 1, -2**31], [0, 0, 0, 0]):
        off = torch.tensor(off, dtype=torch.int32, device="cuda")
        out, _ = fw.attention_packed(q, q, q, off)
        out, _ = fw.attention_packed(q, q, q, off, off.flip(0).contiguous())
        assert out.shape == q.shape
    torch.cuda.synchronize()


# ------------------------------------------------- gradient of packed attention --
def _gradient_want(grad, q, k, v, out, lse, off, koff, causal, scale, kind):
    """dq, dk, dv from the formula with the given out and lse, and their tolerances."""
    grad, q, k, v, out, lse = (_np64(t) for t in (grad, q, k, v, out, lse))
    off = off.numpy()
    koff = off if koff is None else koff.numpy()
    heads, dim = q.shape[1:]
    group = heads // k.shape[1]
    want = [np.zeros(t.shape) for t in (q, k, v)]
    tol = [np.zeros(t.shape) for t in (q, k, v)]
    ub = U["bf16"] if kind == "bf16" else 0.0
    for b in range(len(off) - 1):
        qs, ks = slice(off[b], off[b + 1]), slice(koff[b], koff[b + 1])
        nq, nk = off[b + 1] - off[b], koff[b + 1] - koff[b]
        if nq == 0 or nk == 0:
            continue
        seen = _seen(nq, nk, causal)
        for h in range(heads):
            g = h // group
            Q, K, V, G, O = q[qs, h], k[ks, g], v[ks, g], grad[qs, h], out[qs, h]
            s = Q @ K.T * scale
            size = np.abs(Q) @ np.abs(K).T * scale
            l = np.where(np.isinf(lse[qs, h]), 0.0, lse[qs, h])[:, None]
            p = np.where(seen, np.exp(np.where(seen, s - l, 0.0)), 0.0)
            e = (dim * size + 4 * np.abs(s) + 4 * np.abs(l) + 4) * U32     # relative, of p
            inner = G @ V.T - (G * O).sum(1, keepdims=True)
            # both inner products, their difference and the product with p
            off_inner = (dim + 2) * U32 * (np.abs(G) @ np.abs(V).T
                                           + (np.abs(G) * np.abs(O)).sum(1, keepdims=True))
            ds = p * inner
            dtol = p * off_inner + (e + ub + 2 * U32) * np.abs(ds)
            ptol = (e + ub) * p
            terms = (nq * group + nk + 8) * U32
            want[0][qs, h] += scale * ds @ K
            tol[0][qs, h] += scale * (dtol + terms * np.abs(ds)) @ np.abs(K)
            want[1][ks, g] += scale * ds.T @ Q
            tol[1][ks, g] += scale * (dtol + terms * np.abs(ds)).T @ np.abs(Q)
            want[2][ks, g] += p.T @ G
            tol[2][ks, g] += (ptol + terms * p).T @ np.abs(G)
    return want, [t + U[kind] * np.abs(w) + TINY for t, w in zip(tol, want)]


def _packed_inputs(lengths, past, heads, kv, dim, kind, seed=0):
    off, koff = _sequences(lengths, past)
    n, m = int(off[-1]), int(off[-1] if koff is None else koff[-1])
    g = _gen(n + dim + seed)
    q = _randn(g, n, heads, dim, scale=1.5).to(_dt(kind))
    k, v = (_randn(g, m, kv, dim).to(_dt(kind)) for _ in range(2))
    return off, koff, q, k, v, _randn(g, n, heads, dim).to(_dt(kind))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("lengths,past,heads,kv,dim,causal", PACKED)
def test_attention_gradient(lengths, past, heads, kv, dim, causal, kind):
    import dlrm_embedding_bag_amd as fw
    off, koff, q, k, v, grad = _packed_inputs(lengths, past, heads, kv, dim, kind)
    scale = None if dim % 16 else 0.3
    cuda = [None if t is None else t.cuda() for t in (off, koff)]
    out, lse = fw.attention_packed(q.cuda(), k.cuda(), v.cuda(), *cuda, causal=causal, scale=scale)
    want, tol = _gradient_want(grad, q, k, v, out, lse, off, koff, causal,
                               dim ** -0.5 if scale is None else scale, kind)
    layout = ("plain", "slice", "heads")[(len(q) + dim // 8) % 3]
    first = None
    for layout in ("plain", layout):
        got = fw.attention_packed_grad(_laid(grad, layout), _laid(q, layout), _laid(k, layout),
                                       _laid(v, layout), _laid(out.cpu(), layout), lse, *cuda,
                                       causal=causal, scale=scale)
        for a, w, t, what in zip(got, want, tol, "qkv"):
            _assert_within(_np64(a), w, t, what)
        if first is None:
            first = got
        for a, b in zip(first, got):      # the same sums in the same order
            assert bool((a == b).all())


@pytest.mark.parametrize("causal", [False, True])
def test_attention_gradient_against_differences(causal):
    """Of sum(out * grad), along random directions, by central differences in 64
    bits of the definition on the host."""
    import dlrm_embedding_bag_amd as fw
    off, koff, q, k, v, grad = _packed_inputs([9, 20, 1], [3, 0, 7], 4, 2, 24, "f32", 5)
    scale = 24 ** -0.5
    out, lse = fw.attention_packed(q.cuda(), k.cuda(), v.cuda(), off.cuda(), koff.cuda(),
                                   causal=causal)
    got = fw.attention_packed_grad(grad.cuda(), q.cuda(), k.cuda(), v.cuda(), out, lse, off.cuda(),
                                   koff.cuda(), causal=causal)
    base = [_np64(t) for t in (q, k, v)]
    rng = np.random.default_rng(0)
    import torch
    for i in range(3):
        d = rng.standard_normal(base[i].shape)
        h = 1e-5
        value = []
        for sign in (1, -1):
            at = [torch.from_numpy(b + sign * h * d if j == i else b) for j, b in enumerate(base)]
            o = _attention_want(*at, off, koff, causal, scale, "f32")[0]
            value.append((o * _np64(grad)).sum())
        want = (value[0] - value[1]) / (2 * h)
        # third derivatives times h^2 / 6 stay below 1e-7 here; float32 sums of
        # some 3000 terms of about 1 leave 3000 u32 of their square root's size
        assert abs((_np64(got[i]) * d).sum() - want) <= 1e-3 + 1e-5 * abs(want)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("lengths", [[5, 9], [100, 200, 40]])
def test_attention_gradient_outside_the_sequences(lengths, kind):
    import torch

    import dlrm_embedding_bag_amd as fw
    n, lead, tail = sum(lengths), 3, 200
    off = torch.tensor(lead + np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32).cuda()
    host = _packed_inputs(lengths, None, 4, 2, 64, kind)
    _, _, q, k, v, grad = (None if t is None else t.cuda() for t in host)
    out, lse = fw.attention_packed(q, k, v, off - lead)
    want, tol = _gradient_want(grad, q, k, v, out, lse, (off - lead).cpu(), None, True, 0.125, kind)

    def wide(t):
        buf = torch.full((n + lead + tail, *t.shape[1:]), float("nan"), dtype=t.dtype,
                         device="cuda")
        buf[lead:lead + n] = t
        return buf

    args = [wide(t) for t in (grad, q, k, v, out, lse)]
    got = fw.attention_packed_grad(*args, off)
    given = [torch.full_like(t, 7.0) for t in got]
    ws = torch.empty(fw.attention_packed_grad_workspace_bytes(n + lead + tail, 4),
                     dtype=torch.uint8, device="cuda")
    back = fw.attention_packed_grad(*args, off, out_q=given[0], out_k=given[1], out_v=given[2],
                                    workspace=ws)
    for a, b, c, w, t in zip(got, given, back, want, tol):
        assert c is b and torch.equal(a[lead:lead + n], b[lead:lead + n])
        _assert_within(_np64(a[lead:lead + n]), w, t, "gradient")
        for part in (slice(0, lead), slice(lead + n, None)):
            assert not a[part].any() and (b[part] == 7.0).all()


def test_attention_gradient_stays_within_its_sequence():
    """A sequence with values that are not finite leaves the others' gradients."""
    import torch

    import dlrm_embedding_bag_amd as fw
    off, _, q, k, v, grad = _packed_inputs([40, 70, 33], None, 4, 2, 64, "f32")
    off, q, k, v, grad = (t.cuda() for t in (off, q, k, v, grad))
    out, lse = fw.attention_packed(q, k, v, off)
    want = fw.attention_packed_grad(grad, q, k, v, out, lse, off)
    grad[50, 1, 3] = math.nan
    v[60, 0, 1] = math.inf
    k[70, 1, 1] = math.nan
    out, lse = fw.attention_packed(q, k, v, off)
    got = fw.attention_packed_grad(grad, q, k, v, out, lse, off)
    for a, w in zip(got, want):
        assert torch.equal(a[:40], w[:40]) and torch.equal(a[110:], w[110:])


def test_attention_gradient_without_queries_or_keys():
    import torch

    import dlrm_embedding_bag_amd as fw
    q = torch.randn(6, 2, 32, device="cuda")
    none = q[:0]
    zero = torch.zeros(3, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 2, 6], dtype=torch.int32, device="cuda")
    out, lse = fw.attention_packed(q, none, none, off, zero)
    assert not out.any() and (lse == -math.inf).all()
    dq, dk, dv = fw.attention_packed_grad(q, q, none, none, out, lse, off, zero)
    assert not dq.any() and dk.shape == dv.shape == (0, 2, 32)
    out, lse = fw.attention_packed(none, q, q, zero, off)
    dq, dk, dv = fw.attention_packed_grad(none, none, q, q, out, lse, zero, off)
    assert dq.shape == (0, 2, 32) and not dk.any() and not dv.any()
