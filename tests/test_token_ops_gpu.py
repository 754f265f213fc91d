"""GPU tests of the token operators against plain 64-bit forms on the host.

Tolerances count roundings.  One rounding to type t is off by at most half a
step, u(t) = finfo(t).eps / 2 relative to the value (u32 = 2^-24, bf16 2^-8).
  lookup    the product (u32), the output type
  gradient  a sum of c terms in float32, c u32 of the sum of magnitudes, the
            product with scale and the earlier value (2 u32), the output type
  norm      h one rounding (compared for equality with the same rounding on
            the host), the scale one rounding; a code differs by at most one,
            and only where y / scale lies within 127 * 2 u32 of a border (the
            scale's own rounding): elsewhere codes are equal
  product   the exact sum to float32, the scales' product, their product and
            the bias: 4 u32; sigmoid has a slope of at most 1/4, and expf,
            the sum, the quotient add at most 8 u32 of a value of at most 1;
            the output type
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
    return {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}[name]


def _np64(t):
    import torch
    return t.detach().cpu().to(torch.float64).numpy()


def _assert_within(got, want, tol, what):
    err = np.abs(got - want)
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, first at "
                           f"{tuple(np.argwhere(bad)[0])}: {got[bad][0]!r} for {want[bad][0]!r}, "
                           f"tolerance {np.broadcast_to(tol, err.shape)[bad][0]!r}")


def _draw_tokens(rng, n, rows, kind):
    if kind == "same":
        return np.full(n, rows // 2, np.int32)
    if kind == "none":
        return np.full(n, -1, np.int32)
    if kind == "hot":           # one row takes most of the batch, padding in between
        t = np.where(rng.random(n) < 0.7, rows // 3, rng.integers(0, rows, n))
        return np.where(rng.random(n) < 0.1, -1, t).astype(np.int32)
    if kind == "outside":       # beyond both ends
        return rng.choice([-2**31, -5, -1, 0, rows - 1, rows, rows + 7, 2**31 - 1], n).astype(np.int32)
    return rng.integers(0, rows, n).astype(np.int32)


def _view(t, pad, fill):
    """`t` as a strided view of a buffer with `pad` more columns of `fill`."""
    import torch
    buf = torch.full((t.shape[0], t.shape[1] + pad), fill, dtype=t.dtype, device="cuda")
    buf[:, :t.shape[1]] = t
    return buf, buf[:, :t.shape[1]]


# ------------------------------------------------------------------ lookup --
LOOKUPS = [(n, rows, dim, kind) for n, rows, dim, kind in [
    (1, 1, 1, "uniform"), (1, 5, 7, "uniform"), (3, 100, 8, "outside"), (33, 50, 9, "hot"),
    (257, 1000, 64, "uniform"), (64, 300, 415, "outside"), (130, 90, 1024, "hot"),
    (17, 40, 1031, "uniform"), (5, 9, 4097, "none"), (1000, 20000, 16, "outside")]]


@pytest.mark.parametrize("table,out", [("f32", "f32"), ("f32", "bf16"), ("bf16", "bf16"),
                                       ("bf16", "f32"), ("fp8", "f32"), ("fp8", "bf16")])
@pytest.mark.parametrize("n,rows,dim,kind", LOOKUPS)
def test_lookup(n, rows, dim, kind, table, out):
    import torch

    import dlrm_embedding_bag_amd as fw
    rng = np.random.default_rng(n * 7 + dim)
    tok = _draw_tokens(rng, n, rows, kind)
    tab = torch.from_numpy(rng.standard_normal((rows, dim)).astype(np.float32)).to(_dt(table))
    scale = float(np.float32(math.sqrt(dim)))
    got = fw.emb_lookup_scaled(tab.cuda(), torch.from_numpy(tok).cuda(), scale,
                               out_dtype=_dt(out))
    assert got.dtype == _dt(out) and got.shape == (n, dim)
    there = (tok >= 0) & (tok < rows)
    want = np.where(there[:, None], _np64(tab)[np.where(there, tok, 0)] * scale, 0.0)
    _assert_within(_np64(got), want, np.abs(want) * (U32 + U[out]) * (1 + U32) + TINY, "lookup")
    assert np.all(_np64(got)[~there] == 0.0)


@pytest.mark.parametrize("table,out", [("f32", "f32"), ("bf16", "bf16"), ("fp8", "bf16"),
                                       ("f32", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("n,dim", [(70001, 130), (20003, 1000), (150001, 72), (300007, 5)])
def test_lookup_of_many_tokens(n, dim, table, out):
    """Sizes at which a lane group takes one, two or four rows at once."""
    import torch

    import dlrm_embedding_bag_amd as fw
    rng = np.random.default_rng(n)
    rows = 500
    tok = torch.from_numpy(_draw_tokens(rng, n, rows, "hot"))
    tab = torch.from_numpy(rng.standard_normal((rows, dim)).astype(np.float32)).to(_dt(table))
    got = fw.emb_lookup_scaled(tab.cuda(), tok.cuda(), 0.5, out_dtype=_dt(out)).cpu()
    # halves of the table's values are exact; one rounding to the output's type
    want = torch.where((tok >= 0)[:, None], tab.float()[tok.clamp(0).long()] * 0.5, torch.zeros(()))
    assert torch.equal(got, want.to(_dt(out)))


@pytest.mark.parametrize("dim", [3, 64, 129])
def test_lookup_strides_shapes_and_infinite_rows(dim):
    import torch

    import dlrm_embedding_bag_amd as fw
    rng = np.random.default_rng(dim)
    tab = torch.from_numpy(rng.standard_normal((20, dim)).astype(np.float32))
    tab[3] = float("inf")
    tab[4] = float("nan")
    _, tv = _view(tab.cuda(), 5, 9.0)
    tok = torch.tensor([[0, 3, -1, 4], [19, 20, 1, 0]], dtype=torch.int32, device="cuda")
    got = fw.emb_lookup_scaled(tv, tok, 2.0)
    assert got.shape == (2, 4, dim)
    want = torch.where(((tok >= 0) & (tok < 20)).cpu()[..., None],
                       tab[tok.cpu().clamp(0, 19).long()] * 2.0, torch.zeros(()))
    assert torch.equal(got.cpu().nan_to_num(nan=7.0, posinf=8.0),
                       want.nan_to_num(nan=7.0, posinf=8.0))
    # a missing row stays zero under an infinite scale
    got = fw.emb_lookup_scaled(tv, tok, float("inf"))
    assert torch.all(got[0, 2] == 0) and torch.all(got[1, 1] == 0)
    # an output with padded rows: the padding is not touched
    buf = torch.full((8, dim + 3), -7.0, device="cuda")
    fw.emb_lookup_scaled(tv, tok.view(-1), 2.0, out=buf[:, :dim])
    assert torch.equal(buf[:, :dim].cpu().nan_to_num(nan=7.0, posinf=8.0),
                       want.view(8, dim).nan_to_num(nan=7.0, posinf=8.0))
    assert torch.all(buf[:, dim:] == -7.0)
    assert fw.emb_lookup_scaled(tv, tok.view(-1)[:0], 2.0).shape == (0, dim)


# ---------------------------------------------------------------- gradient --
def _grad_ref(g, tok, rows, scale, base=None):
    """Sum, sum of magnitudes and terms of each element, in 64 bits."""
    there = (tok >= 0) & (tok < rows)
    out = np.zeros((rows, g.shape[1]))
    mag = np.zeros_like(out)
    np.add.at(out, tok[there], g[there])
    np.add.at(mag, tok[there], np.abs(g[there]))
    count = np.bincount(tok[there], minlength=rows)[:, None].astype(np.float64)
    want = out * scale + (0.0 if base is None else base)
    return want, mag * abs(scale), count


def _check_grad(got, g, tok, rows, scale, out, base=None, what="gradient"):
    want, mag, count = _grad_ref(g, tok, rows, scale, base)
    tol = mag * (count + 2) * U32 * 1.01 + np.abs(want) * (U32 + U[out]) * 1.01 + TINY
    _assert_within(_np64(got), want, tol, what)
    return count[:, 0] > 0


GRADS = [(1, 1, 1, "uniform"), (1, 7, 9, "uniform"), (5, 3, 8, "same"), (160, 1000, 16, "uniform"),
         (300, 50, 415, "hot"), (1000, 100, 64, "hot"), (777, 1023, 13, "outside"),
         (64, 1024, 1031, "uniform"), (2000, 3, 520, "uniform"), (4096, 70000, 8, "uniform"),
         (4097, 1500000, 5, "uniform"), (20000, 13, 24, "hot"), (9000, 400, 40, "same"),
         (50, 11, 72, "none"), (12345, 2000, 128, "hot"), (30000, 1048576, 2, "outside")]


@pytest.mark.parametrize("grad,out", [("f32", "f32"), ("bf16", "f32"), ("f32", "bf16"),
                                      ("bf16", "bf16")])
@pytest.mark.parametrize("n,rows,dim,kind", GRADS)
def test_grad(n, rows, dim, kind, grad, out):
    import torch

    import dlrm_embedding_bag_amd as fw
    rng = np.random.default_rng(n + rows + dim)
    tok = _draw_tokens(rng, n, rows, kind)
    g = torch.from_numpy(rng.standard_normal((n, dim)).astype(np.float32)).to(_dt(grad))
    scale = float(np.float32(math.sqrt(dim)))
    td, gd = torch.from_numpy(tok).cuda(), g.cuda()
    got = fw.emb_lookup_grad(gd, td, rows, scale=scale, out_dtype=_dt(out))
    assert got.shape == (rows, dim) and got.dtype == _dt(out)
    named = _check_grad(got, _np64(g), tok, rows, scale, out)
    assert np.all(_np64(got)[~named] == 0.0)
    again = fw.emb_lookup_grad(gd, td, rows, scale=scale, out_dtype=_dt(out))
    assert torch.equal(got, again), "equal calls give equal bits"
    # added to a table: rows that no token names keep their bits
    base = torch.from_numpy(rng.standard_normal((rows, dim)).astype(np.float32)).to(_dt(out))
    t = base.cuda()
    assert fw.emb_lookup_grad(gd, td, scale=-0.25, out=t, accumulate=True) is t
    _check_grad(t, _np64(g), tok, rows, -0.25, out, _np64(base), "accumulated")
    assert torch.equal(t.cpu()[torch.from_numpy(~named)], base[torch.from_numpy(~named)])


@pytest.mark.parametrize("kind", ["hot", "same", "uniform"])
@pytest.mark.parametrize("n,rows,dim", [(63, 40, 100), (64, 5_000_000, 8), (65, 40, 72),
                                        (1023, 300, 600), (1024, 50, 16), (1025, 7, 70),
                                        (2049, 1_048_575, 3), (3000, 1_048_576, 3),
                                        (4095, 900, 33), (4096, 10, 1040), (4097, 20, 1040),
                                        (65536, 5000, 9), (65537, 5000, 9), (70000, 4_200_000, 2),
                                        (9000, 4_200_000, 2)])
def test_grad_at_the_sorts_borders(n, rows, dim, kind):
    """Sizes around those where the sort's tile, key width or launches change."""
    import torch

    import dlrm_embedding_bag_amd as fw
    rng = np.random.default_rng(n)
    tok = _draw_tokens(rng, n, rows, kind)
    g = rng.standard_normal((n, dim)).astype(np.float32)
    td, gd = torch.from_numpy(tok).cuda(), torch.from_numpy(g).cuda()
    got = fw.emb_lookup_grad(gd, td, rows)
    named = _check_grad(got, g.astype(np.float64), tok, rows, 1.0, "f32")
    assert np.all(_np64(got)[~named] == 0.0)
    assert torch.equal(got, fw.emb_lookup_grad(gd, td, rows))


def test_grad_more_tokens_than_one_merge_takes():
    """Beyond 64 tiles of 4096 tokens runs are merged twice."""
    import torch

    import dlrm_embedding_bag_amd as fw
    n, rows, dim = 2_500_001, 3000, 3
    rng = np.random.default_rng(5)
    tok = _draw_tokens(rng, n, rows, "hot")
    g = rng.standard_normal((n, dim)).astype(np.float32)
    got = fw.emb_lookup_grad(torch.from_numpy(g).cuda(), torch.from_numpy(tok).cuda(), rows)
    _check_grad(got, g.astype(np.float64), tok, rows, 1.0, "f32")


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("rows", [1, 40])
def test_grad_strides_and_broadcast(rows, accumulate):
    import torch

    import dlrm_embedding_bag_amd as fw
    rng = np.random.default_rng(rows)
    n, dim = 500, 37
    tok = _draw_tokens(rng, n, rows, "outside")
    td = torch.from_numpy(tok).cuda()
    g = torch.from_numpy(rng.standard_normal((n, dim)).astype(np.float32))
    _, gv = _view(g.cuda(), 3, float("nan"))
    base = torch.from_numpy(rng.standard_normal((rows, dim)).astype(np.float32))
    buf, ov = _view(base.cuda(), 6, -3.0)
    fw.emb_lookup_grad(gv, td, out=ov, accumulate=accumulate)
    _check_grad(ov, _np64(g), tok, rows, 1.0, "f32", _np64(base) if accumulate else None)
    assert torch.all(buf[:, dim:] == -3.0)
    # one gradient row for every token (a sum's gradient)
    one = torch.from_numpy(rng.standard_normal((1, dim)).astype(np.float32))
    got = fw.emb_lookup_grad(one.cuda().expand(n, dim), td, rows)
    _check_grad(got, np.repeat(_np64(one), n, 0), tok, rows, 1.0, "f32")


def test_grad_of_no_tokens():
    import torch

    import dlrm_embedding_bag_amd as fw
    tok = torch.empty(0, dtype=torch.int32, device="cuda")
    g = torch.empty(0, 12, device="cuda")
    out = torch.full((9, 12), 5.0, device="cuda")
    fw.emb_lookup_grad(g, tok, out=out, accumulate=True)
    assert torch.all(out == 5.0)
    buf = torch.full((9, 15), 5.0, device="cuda")
    fw.emb_lookup_grad(g, tok, out=buf[:, :12])
    assert torch.all(buf[:, :12] == 0.0) and torch.all(buf[:, 12:] == 5.0)
    fw.emb_lookup_grad(g, tok, out=out)
    assert torch.all(out == 0.0)


def test_grad_nan_stays_in_its_row():
    import torch

    import dlrm_embedding_bag_amd as fw
    tok = torch.tensor([4, -1, 2, 4, 9, 2], dtype=torch.int32, device="cuda")
    g = torch.ones(6, 20, device="cuda")
    g[0, 3], g[1, 5], g[4, 7] = float("nan"), float("nan"), float("inf")
    got = fw.emb_lookup_grad(g, tok, 9)          # token 9 is outside
    want = torch.zeros(9, 20)
    want[4], want[2], want[4, 3] = 2.0, 2.0, float("nan")
    assert torch.equal(got.cpu().nan_to_num(nan=-1.0), want.nan_to_num(nan=-1.0))


def test_grad_against_differences():
    """d/dW of sum(lookup(W) * r) by central differences, exact in the lookup's
    linearity: both sides in 64 bits apart from the kernels' own roundings."""
    import torch

    import dlrm_embedding_bag_amd as fw
    rng = np.random.default_rng(3)
    rows, dim, n, scale, step = 6, 5, 40, 2.0, 0.5
    tok = torch.from_numpy(rng.integers(-1, rows, n).astype(np.int32)).cuda()
    # small whole numbers: every product and sum below is exact in float32
    w = torch.from_numpy(rng.integers(-8, 9, (rows, dim)).astype(np.float32))
    r = torch.from_numpy(rng.integers(-4, 5, (n, dim)).astype(np.float32)).cuda()

    def loss(table):
        return float((fw.emb_lookup_scaled(table.cuda(), tok, scale).double() * r.double()).sum())

    got = fw.emb_lookup_grad(r, tok, rows, scale=scale).cpu()
    for i in range(rows):
        for j in range(dim):
            up, down = w.clone(), w.clone()
            up[i, j] += step
            down[i, j] -= step
            assert float(got[i, j]) == (loss(up) - loss(down)) / (2 * step)


# -------------------------------------------------------------------- norm --
def _norm_ref(x, res, w, eps):
    import torch
    h = x if res is None else (x.float() + res.float()).to(x.dtype)
    d = _np64(h)
    with np.errstate(all="ignore"):
        y = d / np.sqrt((d * d).mean(1, keepdims=True) + eps)
        if w is not None:
            y = y * _np64(w)
        s = np.abs(y).max(1) / 127.0
    return h, y, s


def _check_norm(h, q, s, x, res, w, eps):
    import torch
    hr, y, sr = _norm_ref(x, res, w, eps)
    assert torch.equal(h.cpu(), hr)
    _assert_within(_np64(s), sr, sr * U32 * 1.01 + TINY, "scale")
    s32 = sr.astype(np.float32).astype(np.float64)[:, None]
    with np.errstate(all="ignore"):
        v = np.where(s32 > 0, y / s32, 0.0)
    want = np.clip(np.rint(v), -127, 127)
    got = q.cpu().numpy().astype(np.float64)
    border = np.abs(v - np.floor(v) - 0.5) < 127 * 2 * U32
    diff = np.abs(got - want)
    assert np.all(diff[~border] == 0), f"{(diff[~border] != 0).sum()} codes differ"
    assert np.all(diff <= 1)


NORM_DIMS = [1, 7, 8, 63, 415, 512, 513, 1024, 2047, 2049, 4096, 4100, 8192, 8193, 20001]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("residual,weight", [(True, True), (False, True), (True, False),
                                             (False, False)])
@pytest.mark.parametrize("dim", NORM_DIMS)
def test_norm(dim, residual, weight, dtype):
    import torch

    import dlrm_embedding_bag_amd as fw
    rng = np.random.default_rng(dim)
    for m in (1, 5):
        x = torch.from_numpy(rng.standard_normal((m, dim)).astype(np.float32)).to(_dt(dtype))
        r = torch.from_numpy(2 * rng.standard_normal((m, dim)).astype(np.float32)).to(_dt(dtype))
        w = torch.from_numpy((1 + 0.1 * rng.standard_normal(dim)).astype(np.float32))
        res, wt = (r if residual else None), (w if weight else None)
        h, q, s = fw.rms_norm_residual_i8(x.cuda(), None if wt is None else wt.cuda(),
                                          None if res is None else res.cuda(), eps=1e-5)
        assert q.dtype == torch.int8 and s.dtype == torch.float32 and h.dtype == x.dtype
        _check_norm(h, q, s, x, res, wt, 1e-5)


@pytest.mark.parametrize("dim", [30, 700, 9000])
def test_norm_rows_that_are_not_finite_or_zero(dim):
    import torch

    import dlrm_embedding_bag_amd as fw
    rng = np.random.default_rng(dim)
    x = torch.from_numpy(rng.standard_normal((8, dim)).astype(np.float32))
    x[1, dim // 2] = float("inf")
    x[2, dim - 1] = float("nan")
    x[3, 0] = -float("inf")
    x[4] = 0.0
    x[5] = 1e-30               # eps dominates
    x[6] = 3e38                # squares beyond float32
    h, q, s = fw.rms_norm_residual_i8(x.cuda(), eps=1e-6)
    assert h.data_ptr() != 0 and torch.isnan(s[1:4]).all() and torch.all(q[1:5] == 0)
    assert float(s[4]) == 0.0
    keep = [0, 5, 6, 7]
    _check_norm(h[keep], q[keep], s[keep], x[keep], None, None, 1e-6)
    # eps 0 and a row of zeros: 0 / 0
    _, q, s = fw.rms_norm_residual_i8(x[4:5].cuda(), eps=0.0)
    assert torch.isnan(s).all() and torch.all(q == 0)
    # a weight that is not finite leaves no row a scale
    w = torch.ones(dim)
    w[0] = float("nan")
    _, q, s = fw.rms_norm_residual_i8(x[7:8].cuda(), w.cuda())
    assert torch.isnan(s).all() and torch.all(q == 0)
    w[0] = float("inf")
    _, q, s = fw.rms_norm_residual_i8(x[7:8].cuda(), w.cuda())
    assert torch.isnan(s).all() and torch.all(q == 0)
    # an infinity that meets a weight of zero: inf * 0
    w[0] = 0.0
    x[1, dim // 2], x[1, 0] = 1.0, float("inf")
    _, q, s = fw.rms_norm_residual_i8(x[1:2].cuda(), w.cuda())
    assert torch.isnan(s).all() and torch.all(q == 0)
    # weights of zero: zero rows
    _, q, s = fw.rms_norm_residual_i8(x[7:8].cuda(), torch.zeros(dim).cuda())
    assert float(s) == 0.0 and torch.all(q == 0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim", [33, 600, 3000, 8200])
def test_norm_strides_and_in_place(dim, dtype):
    import torch

    import dlrm_embedding_bag_amd as fw
    rng = np.random.default_rng(dim)
    m = 9
    x = torch.from_numpy(rng.standard_normal((m, dim)).astype(np.float32)).to(_dt(dtype))
    r = torch.from_numpy(rng.standard_normal((m, dim)).astype(np.float32)).to(_dt(dtype))
    _, xv = _view(x.cuda(), 3, float("nan"))
    rbuf, rv = _view(r.cuda(), 5, 2.0)
    qbuf = torch.full((m, dim + 1), 77, dtype=torch.int8, device="cuda")
    h, q, s = fw.rms_norm_residual_i8(xv, None, rv, out_h=rv, out_codes=qbuf[:, :dim])
    assert h is rv
    _check_norm(h, q, s, x, r, None, 1e-6)
    assert torch.all(rbuf[:, dim:] == 2.0) and torch.all(qbuf[:, dim:] == 77)
    # one row read for all, h over x
    one = r[:1].cuda().expand(m, dim)
    xc = x.cuda()
    h, q, s = fw.rms_norm_residual_i8(xc, None, one, out_h=xc)
    _check_norm(h, q, s, x, r[:1].expand(m, dim), None, 1e-6)
    e = fw.rms_norm_residual_i8(xv[:0], None, rv[:0])
    assert e[0].shape == (0, dim) and e[2].shape == (0,)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,dim", [(513, 700), (1000, 1024), (700, 1025), (600, 2048), (515, 4095),
                                   (514, 8192), (1001, 31), (1003, 33), (1005, 65), (1007, 200),
                                   (1009, 257)])
def test_norm_of_many_rows(m, dim, dtype):
    """Sizes at which rows share a wave, have one, or have a workgroup."""
    import torch

    import dlrm_embedding_bag_amd as fw
    rng = np.random.default_rng(m + dim)
    x = torch.from_numpy(rng.standard_normal((m, dim)).astype(np.float32)).to(_dt(dtype))
    r = torch.from_numpy(rng.standard_normal((m, dim)).astype(np.float32)).to(_dt(dtype))
    w = torch.from_numpy((1 + 0.1 * rng.standard_normal(dim)).astype(np.float32))
    x[3] = 0.0
    r[3] = 0.0
    h, q, s = fw.rms_norm_residual_i8(x.cuda(), w.cuda(), r.cuda(), eps=1e-6)
    _check_norm(h, q, s, x, r, w, 1e-6)
    # h in the residual's place
    rd = r.cuda()
    h, q2, s2 = fw.rms_norm_residual_i8(x.cuda(), w.cuda(), rd, eps=1e-6, out_h=rd)
    assert h is rd and torch.equal(q, q2) and torch.equal(s, s2)
    _check_norm(h, q2, s2, x, r, w, 1e-6)


def test_norm_products_outside_float32():
    """Products h * weight that overflow or vanish in float32 keep their codes."""
    import torch

    import dlrm_embedding_bag_amd as fw
    rng = np.random.default_rng(8)
    x = torch.from_numpy(rng.standard_normal((6, 300)).astype(np.float32))
    x[0] *= 1e30
    x[1] *= 1e-30
    x[2, ::2] *= 1e25
    for size in (1e30, 1e-30, 1.0):
        w = torch.from_numpy((rng.standard_normal(300) * size).astype(np.float32))
        h, q, s = fw.rms_norm_residual_i8(x.cuda(), w.cuda(), eps=1e-6)
        _check_norm(h, q, s, x, None, w, 1e-6)


def test_norm_many_short_rows():
    import torch

    import dlrm_embedding_bag_amd as fw
    x = torch.randn(100003, 17, generator=torch.Generator().manual_seed(1))
    h, q, s = fw.rms_norm_residual_i8(x.cuda())
    _check_norm(h, q, s, x, None, None, 1e-6)


# ----------------------------------------------------------------- product --
def _product_case(m, n, k, seed, extreme=False):
    import torch
    rng = np.random.default_rng(seed)
    a = rng.integers(-128, 128, (m, k)).astype(np.int8)
    w = rng.integers(-128, 128, (n, k)).astype(np.int8)
    if extreme:
        a[:], w[:] = -128, -128
    sa = (rng.random(m) * 0.01 + 1e-3).astype(np.float32)
    sw = (rng.random(n) * 0.01 / math.sqrt(k) + 1e-4).astype(np.float32)
    b = rng.standard_normal(n).astype(np.float32)
    return [torch.from_numpy(v) for v in (a, sa, w, sw, b)]


def _product_ref(a, sa, w, sw, bias, act):
    # whole numbers below 2^53: the float64 product is exact
    p = (_np64(a) @ _np64(w).T) * (_np64(sa)[:, None] * _np64(sw)[None, :])
    c = p + (0.0 if bias is None else _np64(bias))
    tol = (3 * np.abs(p) + np.abs(c)) * U32 * 1.01
    if act == "relu":
        c = np.maximum(c, 0.0)
    elif act == "sigmoid":
        c = 1.0 / (1.0 + np.exp(-c))
        tol = tol / 4 + 8 * U32
    return c, tol


def _check_product(got, a, sa, w, sw, bias, act, out):
    c, tol = _product_ref(a, sa, w, sw, bias, act)
    _assert_within(_np64(got), c, tol * (1 + U[out]) + np.abs(c) * U[out] * 1.01 * (out == "bf16")
                   + TINY, "product")


PRODUCTS = [(1, 1, 1), (1, 17, 15), (1, 512, 415), (3, 5, 16), (16, 33, 64), (17, 100, 129),
            (32, 64, 1024), (33, 48, 1100), (64, 130, 2049), (65, 64, 128), (65, 63, 127),
            (100, 200, 300), (128, 128, 256), (130, 257, 513), (129, 1000, 47), (300, 300, 1),
            (256, 256, 512), (257, 513, 640), (2048, 512, 415), (512, 512, 1000)]


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", PRODUCTS)
def test_product(m, n, k, out):
    import dlrm_embedding_bag_amd as fw
    a, sa, w, sw, b = _product_case(m, n, k, m + n + k)
    for bias, act in ((None, "none"), (b, "relu"), (b, "sigmoid")):
        got = fw.linear_i8_bias_act(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(),
                                    None if bias is None else bias.cuda(), act,
                                    out_dtype=_dt(out))
        assert got.shape == (m, n) and got.dtype == _dt(out)
        _check_product(got, a, sa, w, sw, bias, act, out)


@pytest.mark.parametrize("m,n,k", [(1024, 4096, 576), (4100, 2050, 1030), (2048, 2048, 2048),
                                   (5000, 1111, 384)])
def test_product_large(m, n, k):
    import dlrm_embedding_bag_amd as fw
    a, sa, w, sw, b = _product_case(m, n, k, m + n + k)
    got = fw.linear_i8_bias_act(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), b.cuda(), "relu")
    _check_product(got, a, sa, w, sw, b, "relu", "f32")


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", [
    (65, 64, 16), (100, 70, 80), (129, 1000, 48), (500, 601, 1008), (70, 4100, 1168),   # 64 x 64
    (2000, 2100, 32), (2000, 2103, 272), (1920, 2177, 576),                             # 128 x 128
    (3000, 3100, 48), (3000, 3101, 464), (2900, 3333, 320), (3073, 2817, 64 * 9)])      # 256 x 256
def test_product_of_rows_on_16_bytes(m, n, k, out):
    """Tiles of each size whose k ends before the first stage, inside one, and
    after few or many of them, and whose rows and columns end inside a tile."""
    import dlrm_embedding_bag_amd as fw
    a, sa, w, sw, b = _product_case(m, n, k, m + n + k)
    got = fw.linear_i8_bias_act(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), b.cuda(), "none",
                                out_dtype=_dt(out))
    _check_product(got, a, sa, w, sw, b, "none", out)


@pytest.mark.parametrize("m,n,k", [
    (1, 8200, 127), (16, 9000, 130), (32, 8200, 300), (50, 8195, 515), (64, 8192, 2176),  # few rows
    (65, 70, 2601), (130, 90, 4099), (100, 129, 2050), (66, 65, 2047),                    # 64 x 64
    (2000, 2100, 273), (1920, 2177, 45),                                                  # 128 x 128
    (3000, 3100, 47), (2900, 3333, 321)])                                                 # 256 x 256
def test_product_of_many_columns_and_of_rows_at_any_byte(m, n, k):
    import dlrm_embedding_bag_amd as fw
    a, sa, w, sw, b = _product_case(m, n, k, m + n + k)
    for out in ("f32", "bf16"):
        got = fw.linear_i8_bias_act(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), b.cuda(), "relu",
                                    out_dtype=_dt(out))
        _check_product(got, a, sa, w, sw, b, "relu", out)


@pytest.mark.parametrize("m", [1, 40, 200])
def test_product_longest_sum(m):
    """k at its limit with every product at its largest: 2^14 * 131071 < 2^31."""
    import dlrm_embedding_bag_amd as fw
    a, sa, w, sw, b = _product_case(m, 70, 131071, m, extreme=True)
    got = fw.linear_i8_bias_act(a.cuda(), sa.cuda(), w.cuda(), sw.cuda())
    _check_product(got, a, sa, w, sw, None, "none", "f32")


@pytest.mark.parametrize("m,n,k", [(5, 40, 100), (64, 96, 272), (200, 150, 300), (1024, 2048, 160)])
def test_product_strides(m, n, k):
    import torch

    import dlrm_embedding_bag_amd as fw
    a, sa, w, sw, b = _product_case(m, n, k, 9)
    for pad in (16, 3):
        _, av = _view(a.cuda(), pad, 55)
        _, wv = _view(w.cuda(), 2 * pad, 66)
        for out in ("f32", "bf16"):
            buf = torch.full((m, n + pad), -5.0, dtype=_dt(out), device="cuda")
            fw.linear_i8_bias_act(av, sa.cuda(), wv, sw.cuda(), b.cuda(), out=buf[:, :n])
            _check_product(buf[:, :n], a, sa, w, sw, b, "none", out)
            assert torch.all(buf[:, n:] == -5.0)
    # one row for all
    got = fw.linear_i8_bias_act(a[:1].cuda().expand(m, k), sa.cuda(), w.cuda(), sw.cuda())
    _check_product(got, a[:1].expand(m, k), sa, w, sw, None, "none", "f32")
    # operands that start at an odd byte
    flat = torch.zeros(m * k + 1, dtype=torch.int8, device="cuda")
    flat[1:] = a.cuda().view(-1)
    got = fw.linear_i8_bias_act(flat[1:].view(m, k), sa.cuda(), w.cuda(), sw.cuda())
    _check_product(got, a, sa, w, sw, None, "none", "f32")
    assert fw.linear_i8_bias_act(a[:0].cuda(), sa[:0].cuda(), w.cuda(), sw.cuda()).shape == (0, n)


@pytest.mark.parametrize("m,n,k", [(3, 40, 100), (200, 130, 300)])
def test_product_rows_without_a_scale(m, n, k):
    """A row that the norm could not scale (NaN) stays visible after every act,
    and its neighbours are not affected."""
    import torch

    import dlrm_embedding_bag_amd as fw
    a, sa, w, sw, b = _product_case(m, n, k, 11)
    a[1], sa[1] = 0, float("nan")
    keep = [i for i in range(m) if i != 1]
    for act in ("none", "relu", "sigmoid"):
        got = fw.linear_i8_bias_act(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), b.cuda(), act)
        assert torch.isnan(got[1]).all()
        _check_product(got[keep], a[keep], sa[keep], w, sw, b, act, "f32")


# ------------------------------------------------- offsets beyond 32 bits --
def test_lookup_and_gradient_far_into_a_table():
    """A table of 2.2 billion elements: its last rows lie beyond 2^31 elements
    and 2^32 bytes."""
    import torch

    import dlrm_embedding_bag_amd as fw
    rows, dim = 1_100_000, 2048
    table = torch.zeros(rows, dim, dtype=torch.bfloat16, device="cuda")
    tok = torch.tensor([rows - 1, 0, -1, rows - 2, 1_048_577, rows], dtype=torch.int32,
                       device="cuda")
    there = [0, 1, 3, 4]
    values = torch.randn(len(there), dim, device="cuda").bfloat16()
    table[tok[there].long()] = values
    got = fw.emb_lookup_scaled(table, tok, 2.0)
    assert torch.equal(got[there], values * 2.0)
    assert torch.all(got[[2, 5]] == 0)
    grad = torch.randn(6, dim, device="cuda").bfloat16()
    fw.emb_lookup_grad(grad, tok, scale=1.0, out=table, accumulate=True)
    assert torch.equal(table[tok[there].long()],
                       (values.float() + grad[there].float()).bfloat16())
    assert torch.all(table[rows - 3] == 0) and torch.all(table[1] == 0)
    many = tok[:1].repeat(5000)      # the launches for many tokens
    one = torch.full((1, dim), 0.5, device="cuda").expand(5000, dim)
    out = table.zero_()
    fw.emb_lookup_grad(one, many, scale=2.0 ** -10, out=out)
    assert torch.all(out[rows - 1] == torch.tensor(5000 * 0.5 / 1024.0).bfloat16().cuda())
    assert torch.all(out[rows - 2] == 0)


@pytest.mark.parametrize("m", [1, 100])
def test_product_far_into_the_weight(m):
    import torch

    import dlrm_embedding_bag_amd as fw
    n, k = 70_016, 32_768            # 2.3 billion bytes
    g = torch.Generator(device="cuda").manual_seed(m)
    w = torch.randint(-128, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    a = torch.randint(-128, 128, (m, k), generator=g, device="cuda", dtype=torch.int8)
    sa = torch.rand(m, generator=g, device="cuda") * 0.01
    sw = torch.rand(n, generator=g, device="cuda") * 1e-4
    got = fw.linear_i8_bias_act(a, sa, w, sw)
    cols = torch.tensor([0, 1, 65_535, 65_536, n - 2, n - 1], device="cuda")
    _check_product(got[:, cols], a, sa, w[cols], sw[cols], None, "none", "f32")


# ------------------------------------------------------- streams and graphs --
def _chain(fw, table, tok, res, wn, w8, sw, grad, rows):
    x = fw.emb_lookup_scaled(table, tok, 3.0)
    h, q, s = fw.rms_norm_residual_i8(x, wn, res)
    y = fw.linear_i8_bias_act(q, s, w8, sw, None, "relu")
    d = fw.emb_lookup_grad(grad, tok, rows, scale=3.0)
    return x, h, q, s, y, d


def _chain_state(n, rows, dim, out, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    tok = torch.randint(-1, rows, (n,), generator=g, device="cuda", dtype=torch.int32)
    w8 = torch.randint(-127, 128, (out, dim), generator=g, device="cuda").to(torch.int8)
    return [rn(rows, dim), tok, rn(n, dim), rn(dim), w8, rn(out).abs(), rn(n, dim)]


@pytest.mark.parametrize("n,rows,dim,out", [(1, 50, 64, 32), (700, 3000, 130, 96),
                                            (6000, 2000, 256, 256)])
def test_graph_replays_equal_eager(n, rows, dim, out):
    import torch

    import dlrm_embedding_bag_amd as fw
    bufs = _chain_state(n, rows, dim, out, 0)
    for _ in range(2):
        _chain(fw, *bufs, rows)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _chain(fw, *bufs, rows)
    noise = torch.randn(1 << 18, device="cuda")
    for it in range(1, 5):
        new = _chain_state(n, rows, dim, out, it)
        for b, v in zip(bufs, new):
            b.copy_(v)
        want = [t.clone() for t in _chain(fw, *new, rows)]
        (noise * 2).sum()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), (it, i)


def test_calls_on_another_stream():
    import torch

    import dlrm_embedding_bag_amd as fw
    bufs = _chain_state(900, 500, 200, 64, 3)
    want = _chain(fw, *bufs, 500)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    table, tok, res, wn, w8, sw, grad = bufs
    x = fw.emb_lookup_scaled(table, tok, 3.0, stream=side)
    h, q, s = fw.rms_norm_residual_i8(x, wn, res, stream=side)
    y = fw.linear_i8_bias_act(q, s, w8, sw, None, "relu", stream=side.cuda_stream)
    d = fw.emb_lookup_grad(grad, tok, 500, scale=3.0, stream=side)
    side.synchronize()
    for a, b in zip((x, h, q, s, y, d), want):
        assert torch.equal(a, b)


def test_given_workspace_and_refusals():
    import torch

    import dlrm_embedding_bag_amd as fw
    table, tok, res, wn, w8, sw, grad = _chain_state(300, 40, 24, 16, 4)
    many, tok_many = grad.repeat(20, 1), tok.repeat(20)
    need = fw.emb_lookup_grad_workspace_bytes(6000, 40, 24)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")   # content does not matter
    got = fw.emb_lookup_grad(many, tok_many, 40, workspace=ws)
    assert torch.equal(got, fw.emb_lookup_grad(many, tok_many, 40))
    with pytest.raises(fw.DlrmError) as e:
        fw.emb_lookup_grad(many, tok_many, 40, workspace=ws[:-1])
    assert e.value.name == "DLRM_ERR_WORKSPACE"
    with pytest.raises(ValueError):
        fw.emb_lookup_grad(grad, tok)                                  # no rows, no out
    with pytest.raises(ValueError):
        fw.emb_lookup_grad(grad, tok, 40, accumulate=True)             # nothing to add to
    with pytest.raises(ValueError):
        fw.emb_lookup_grad(grad[:-1], tok, 40)
    with pytest.raises(ValueError):
        fw.emb_lookup_grad(grad, tok, 41, out=torch.zeros(40, 24, device="cuda"))
    with pytest.raises(TypeError):
        fw.emb_lookup_grad(grad, tok.long(), 40)
    with pytest.raises(TypeError):
        fw.emb_lookup_grad(grad.double(), tok, 40)
    with pytest.raises(TypeError):
        fw.emb_lookup_scaled(table, tok, out_dtype=torch.float16)
    with pytest.raises(ValueError):
        fw.emb_lookup_scaled(table.t(), tok)
    with pytest.raises(ValueError):
        fw.emb_lookup_scaled(table, tok, out=torch.zeros(299, 24, device="cuda"))
    with pytest.raises(ValueError):
        fw.rms_norm_residual_i8(res, wn[:-1])
    with pytest.raises(ValueError):
        fw.rms_norm_residual_i8(res, wn, res[:-1])
    with pytest.raises(TypeError):
        fw.rms_norm_residual_i8(res, wn, res.bfloat16())
    with pytest.raises(fw.DlrmError):
        fw.rms_norm_residual_i8(res, wn, eps=-1.0)
    _, q, s = fw.rms_norm_residual_i8(res, wn)
    with pytest.raises(ValueError):
        fw.linear_i8_bias_act(q, s[:-1], w8, sw)
    with pytest.raises(ValueError):
        fw.linear_i8_bias_act(q, s, w8[:, :-1], sw)
    with pytest.raises(TypeError):
        fw.linear_i8_bias_act(q.float(), s, w8, sw)
    with pytest.raises(KeyError):
        fw.linear_i8_bias_act(q, s, w8, sw, act="tanh")
