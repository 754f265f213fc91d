"""GPU tests of the token operators at the edges of their ranges.  The references
and the counting of roundings are those of test_token_ops_gpu.py."""
import numpy as np
import pytest

from conftest import gpu_available
from test_token_ops_gpu import TINY, U, U32, _check_grad, _draw_tokens, _dt, _np64

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]


@pytest.mark.parametrize("n", [65536 * 64, 65536 * 64 + 1, 5_000_003])
def test_grad_more_tokens_than_merging_workgroups_take_at_once(n):
    """65536 workgroups of 64 tokens: the last of them, one token more, and
    workgroups that take a second turn."""
    import torch

    import dlrm_embedding_bag_amd as fw
    rng = np.random.default_rng(n)
    rows, dim = 3000, 2
    tok = _draw_tokens(rng, n, rows, "hot")
    g = rng.standard_normal((n, dim)).astype(np.float32)
    td, gd = torch.from_numpy(tok).cuda(), torch.from_numpy(g).cuda()
    got = fw.emb_lookup_grad(gd, td, rows)
    _check_grad(got, g.astype(np.float64), tok, rows, 1.0, "f32")
    assert torch.equal(got, fw.emb_lookup_grad(gd, td, rows))


def _codes_of(h, w, eps, scale):
    """y, and y / scale with the returned scale, in 64 bits."""
    d = _np64(h)
    y = d / np.sqrt((d * d).mean(1, keepdims=True) + eps)
    if w is not None:
        y = y * _np64(w)
    s = _np64(scale)[:, None]
    return y, np.divide(y, s, out=np.zeros_like(y), where=s > 0)


def _check_codes(q, v, border=1e-11):
    """Codes equal round(v), ties to even, within +-127.  v is off by a few
    2^-53 of at most 191 on either side, far below `border`: within that of a
    half either neighbour will do."""
    got = q.cpu().numpy().astype(np.float64)
    near = np.abs(v - np.floor(v) - 0.5) < border
    want = np.clip(np.rint(v), -127, 127)
    assert np.all((got == want) | (near & (np.abs(got - want) <= 1))), \
        f"{(got != want).sum()} codes of {got.size} differ"


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,dim", [(40, 17), (40, 64), (40, 300), (600, 1000), (20, 3000),
                                   (600, 4096), (9, 8192), (9, 9000)])
def test_norm_scale_below_float32s_normal_range(m, dim, dtype):
    """Such a scale has few bits, so max|y| / scale may lie well beyond 127: codes
    stop there and keep their sign."""
    import torch

    import dlrm_embedding_bag_amd as fw
    rng = np.random.default_rng(dim)
    x = torch.from_numpy(rng.standard_normal((m, dim)).astype(np.float32))
    ones = rng.choice([-1.0, 1.0], dim) * (1 + 0.1 * rng.standard_normal(dim))
    # (size of x, size of the weight, eps): the scale is some 1 to 10^5 steps of 2^-149
    for size, small, eps in ((1e20, 1e-42, 1e-6), (1e15, 3e-41, 1e-6), (1.0, 1e-38, 1e-6),
                             (1.0, 1.0, 1e84), (1.0, 1.0, 1e80), (1e10, 1e-3, 1e96)):
        xt = (x * size).to(_dt(dtype))
        w = torch.from_numpy((ones * small).astype(np.float32))
        _, q, s = fw.rms_norm_residual_i8(xt.cuda(), w.cuda(), eps=eps)
        y, v = _codes_of(xt, w, eps, s)
        top = np.abs(y).max(1) / 127.0
        # one rounding: half a step of 2^-149, or u32 of the value
        assert np.all(np.abs(_np64(s) - top) <= np.maximum(2.0 ** -150, top * U32) * 1.01)
        assert np.any((_np64(s) > 0) & (_np64(s) < TINY))
        _check_codes(q, v)


@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("m,n,k", [(1, 70, 4096), (30, 8200, 300), (64, 130, 2049),    # few rows
                                   (100, 129, 2050), (2000, 2100, 273),                # any byte
                                   (200, 150, 1024), (2000, 2100, 272), (3000, 3100, 464)])
def test_product_of_scales_beyond_float32(m, n, k, out):
    """a_scale * w_scale leaves float32's normal range, upwards or downwards, and
    the outputs do not: their errors are those of other scales.  A sum of zero
    takes no overflow from its scales."""
    import torch

    import dlrm_embedding_bag_amd as fw
    rng = np.random.default_rng(m + n + k)
    a = rng.integers(-128, 128, (m, k)).astype(np.int8)
    w = rng.integers(-128, 128, (n, k)).astype(np.int8)
    a[m // 2] = 0
    sizes_a = np.array([1e-22, 1e25, 1e-3, 0.0, 1e-38, 3e-44, 1e30])
    sizes_w = np.array([1e-20, 1e-3, 1e20, -1e-5, 0.0])
    sa = (sizes_a[np.arange(m) % 7] * (1 + rng.random(m))).astype(np.float32)
    sw = (sizes_w[np.arange(n) % 5] * (1 + rng.random(n))).astype(np.float32)
    sa[m // 2] = 1e30
    b = (rng.standard_normal(n) * 1e-30).astype(np.float32)
    ta, tw, tsa, tsw, tb = [torch.from_numpy(v).cuda() for v in (a, w, sa, sw, b)]
    # (whole numbers below 2^31: a float64 product on the GPU is exact)
    sums = (ta.double() @ tw.double().t()).cpu().numpy()
    p = sums * (sa.astype(np.float64)[:, None] * sw.astype(np.float64)[None, :])
    for bias in (None, tb):
        c = p + (0.0 if bias is None else b.astype(np.float64))
        got = _np64(fw.linear_i8_bias_act(ta, tsa, tw, tsw, bias, out_dtype=_dt(out)))
        high = np.abs(c) >= 2.0 ** 128
        assert np.array_equal(got[high], np.sign(c[high]) * np.inf)
        tol = (3 * np.abs(p) + np.abs(c)) * U32 * 1.01
        tol = tol * (1 + U[out]) + np.abs(c) * U[out] * 1.01 * (out == "bf16") + TINY
        bad = ~high & ~(np.abs(got - c) <= tol)
        assert not bad.any(), (f"{bad.sum()} of {bad.size} off, first at {tuple(np.argwhere(bad)[0])}: "
                               f"{got[bad][0]!r} for {c[bad][0]!r}")
        assert np.array_equal(got[m // 2], np.zeros(n) if bias is None else
                              _np64(bias.to(_dt(out))))


@pytest.mark.parametrize("m,n,k", [(40, 70, 300), (100, 129, 330), (200, 150, 1024),
                                   (2000, 2100, 272), (3000, 3100, 464), (2900, 3333, 321)])
def test_product_rows_do_not_see_their_neighbours_scales(m, n, k):
    """Equal bits of a row, whatever the scales of the rows around it."""
    import torch

    import dlrm_embedding_bag_amd as fw
    g = torch.Generator(device="cuda").manual_seed(m)
    a = torch.randint(-128, 128, (m, k), generator=g, device="cuda", dtype=torch.int8)
    w = torch.randint(-128, 128, (n, k), generator=g, device="cuda", dtype=torch.int8)
    sa = torch.rand(m, generator=g, device="cuda") * 0.01
    sw = torch.rand(n, generator=g, device="cuda") * 1e-3
    want = fw.linear_i8_bias_act(a, sa, w, sw, act="relu")
    other = sa.clone()
    other[::3] = 0.0
    other[1::9] = 1e36
    other[4::9] = float("nan")
    keep = other == sa
    got = fw.linear_i8_bias_act(a, other, w, sw, act="relu")
    assert torch.equal(got[keep], want[keep])
    assert torch.all(got[::3] == 0) and torch.isnan(got[4::9]).all()


def _row_next_to_borders(dim, dtype, seed):
    """A row and weights whose y / scale lies next to k + 1/2 for all codes k: the
    weight that meets a value is the float32 next to where the border would be,
    so the distances are of the size of float32's steps, 1e-9 to 1e-5."""
    import torch
    rng = np.random.default_rng(seed)
    x = torch.from_numpy((1 + rng.random((1, dim))).astype(np.float32)).to(_dt(dtype))
    h = _np64(x)[0]
    w = np.ones(dim, np.float32)
    w[0] = 200.0 / h[0]                       # the largest product
    r = 1.0 / np.sqrt((h * h).mean() + 1e-6)
    scale = float(np.float32(h[0] * np.float64(w[0]) * r / 127.0))
    k = rng.integers(-127, 127, dim - 1)
    w[1:] = ((k + 0.5) * scale / r / h[1:]).astype(np.float32)
    return x, torch.from_numpy(w)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("m,dim", [(1, 31), (600, 60), (600, 130), (1, 250), (1, 500), (600, 1000),
                                   (1, 2000), (600, 2000), (1, 4000), (600, 4000), (2, 8000),
                                   (2, 9001)])
def test_norm_codes_next_to_borders(m, dim, dtype):
    """Each code is the one that 64 bits decide, which float32 does not tell."""
    import torch

    import dlrm_embedding_bag_amd as fw
    told = 0
    for seed in range(4):
        x, w = _row_next_to_borders(dim, dtype, seed)
        _, q, s = fw.rms_norm_residual_i8(x.cuda().expand(m, dim), w.cuda(), eps=1e-6)
        _, v = _codes_of(x, w, 1e-6, s[:1])
        away = np.abs(np.abs(v - np.floor(v)) - 0.5)
        assert np.median(away[0, 1:]) < 1e-5
        # the same in float32: product, factor, rounded product
        d = _np64(x)
        f = np.float32(1.0 / np.sqrt((d * d).mean() + 1e-6) / float(s[0]))
        rough = np.rint((x.float().numpy() * w.numpy()).astype(np.float64) * np.float64(f))
        told += int((rough != np.rint(v)).sum())
        for i in {0, m // 2, m - 1}:
            _check_codes(q[i:i + 1], v)
        assert torch.equal(q, q[:1].expand(m, dim)) and torch.equal(s, s[:1].expand(m))
    assert told > 0, "float32 alone would do for these inputs"


@pytest.mark.parametrize("kind", ["hot", "same", "uniform"])
@pytest.mark.parametrize("n,rows,dim", [
    (2047, 900, 33), (2048, 900, 33), (2048, 20, 1040), (2049, 900, 33),   # one launch's last
    (1024, 4_194_303, 3), (1024, 4_194_304, 3),      # few tokens: rows of 32-bit values and beyond
    (1025, 2_097_151, 3), (1025, 2_097_152, 3), (2048, 3_000_000, 3),      # many tokens, likewise
    (2049, 2_097_151, 3), (2049, 2_097_152, 3),      # tiles, likewise
    (65536, 2_097_152, 2), (65537, 2_097_151, 2)])   # one merge's last, and two
def test_grad_at_the_sorts_own_borders(n, rows, dim, kind):
    """Up to 2048 tokens take one launch and 32 tiles of 2048 one merge; rows below
    2^22 (up to 1024 tokens) or 2^21 (beyond) sort as 32-bit values."""
    import torch

    import dlrm_embedding_bag_amd as fw
    rng = np.random.default_rng(n)
    tok = _draw_tokens(rng, n, rows, kind)
    if kind == "uniform":
        tok[::7] = rows - 1
        tok[5::97] = rows
    g = rng.standard_normal((n, dim)).astype(np.float32)
    td, gd = torch.from_numpy(tok).cuda(), torch.from_numpy(g).cuda()
    got = fw.emb_lookup_grad(gd, td, rows)
    named = _check_grad(got, g.astype(np.float64), tok, rows, 1.0, "f32")
    assert not got.cpu()[torch.from_numpy(~named)].any()
    assert torch.equal(got, fw.emb_lookup_grad(gd, td, rows))


def test_given_outputs_count_as_modified():
    """A value that autograd saved is not used after a call wrote over it; outputs
    and tensors that were only read keep their versions."""
    import torch

    import dlrm_embedding_bag_amd as fw
    leaf = torch.randn(30, 16, device="cuda", requires_grad=True)
    table = leaf * 1.0
    tok = torch.arange(20, dtype=torch.int32, device="cuda")
    grad = torch.randn(20, 16, device="cuda")
    loss = table.square().sum()                      # saves table
    before = table._version
    rows = fw.emb_lookup_scaled(table, tok)
    assert not rows.requires_grad and table._version == before
    fw.emb_lookup_grad(grad, tok, out=table.detach(), accumulate=True)
    assert table._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    codes = torch.zeros(20, 16, dtype=torch.int8, device="cuda")
    scale, h = torch.zeros(20, device="cuda"), torch.zeros(20, 16, device="cuda")
    y = torch.zeros(20, 8, device="cuda")
    w = torch.ones(8, 16, dtype=torch.int8, device="cuda")
    ws = torch.ones(8, device="cuda")
    reads = [grad, tok, rows, w, ws]
    versions = [t._version for t in reads]
    fw.rms_norm_residual_i8(rows, None, grad, out_h=h, out_codes=codes, out_scale=scale)
    fw.linear_i8_bias_act(codes, scale, w, ws, out=y)
    lookup = torch.zeros(20, 16, device="cuda")
    fw.emb_lookup_scaled(table, tok, out=lookup)
    assert all(t._version == 1 for t in (h, codes, scale, y, lookup))
    assert [t._version for t in reads] == versions
    with torch.inference_mode():                     # tensors without a version
        fw.emb_lookup_scaled(table, tok, out=torch.zeros(20, 16, device="cuda"))


@pytest.mark.parametrize("dtype", [None, "f32"])
def test_outputs_that_are_not_gpu_tensors_are_refused(dtype):
    import torch

    import dlrm_embedding_bag_amd as fw
    table = torch.zeros(5, 8, device="cuda")
    tok = torch.zeros(3, dtype=torch.int32, device="cuda")
    codes, scale = table.to(torch.int8), torch.ones(5, device="cuda")
    kind = {} if dtype is None else {"out_dtype": _dt(dtype)}
    for out, error in (([0.0], TypeError), (torch.zeros(3, 8), ValueError)):
        with pytest.raises(error, match="out must be"):
            fw.emb_lookup_scaled(table, tok, out=out, **kind)
        with pytest.raises(error, match="out must be"):
            fw.emb_lookup_grad(table[:3], tok, out=out, **kind)
        with pytest.raises(error, match="out must be"):
            fw.linear_i8_bias_act(codes, scale, codes, scale, out=out, **kind)
        with pytest.raises(error, match="out_h must be"):
            fw.rms_norm_residual_i8(table, None, table, out_h=out)


@pytest.mark.parametrize("dim", [40_001, 1 << 20])
@pytest.mark.parametrize("n", [7, 2049])
def test_lookup_and_gradient_of_the_widest_rows(n, dim):
    """Whole numbers whose products and sums float32 holds: equal to any order's."""
    import torch

    import dlrm_embedding_bag_amd as fw
    rows = 3
    g = torch.Generator(device="cuda").manual_seed(n)
    table = torch.randint(-50, 51, (rows, dim), generator=g, device="cuda").float()
    tok = torch.randint(-1, rows + 1, (n,), generator=g, device="cuda", dtype=torch.int32)
    few = tok[:7].contiguous()
    there = ((few >= 0) & (few < rows))[:, None]
    got = fw.emb_lookup_scaled(table, few, 2.0)
    assert torch.equal(got, torch.where(there, table[few.clamp(0, rows - 1).long()] * 2.0, 0.0))
    # one gradient row for all tokens
    row = torch.randint(-9, 10, (1, dim), generator=g, device="cuda").float()
    count = torch.stack([(tok == r).sum() for r in range(rows)])[:, None].float()
    got = fw.emb_lookup_grad(row.expand(n, dim), tok, rows, scale=0.5)
    assert torch.equal(got, count * row * 0.5)
    want = table - count * row
    assert torch.equal(fw.emb_lookup_grad(row.expand(n, dim), tok, scale=-1.0, out=table,
                                          accumulate=True), want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_of_the_widest_rows(dtype):
    import torch

    import dlrm_embedding_bag_amd as fw
    rng = np.random.default_rng(20)
    dim = 1 << 20
    x = torch.from_numpy(rng.standard_normal((2, dim)).astype(np.float32)).to(_dt(dtype))
    w = torch.from_numpy((1 + 0.1 * rng.standard_normal(dim)).astype(np.float32))
    _, q, s = fw.rms_norm_residual_i8(x.cuda(), w.cuda(), eps=1e-6)
    y, v = _codes_of(x, w, 1e-6, s)
    top = np.abs(y).max(1) / 127.0
    assert np.all(np.abs(_np64(s) - top) <= top * U32 * 1.01)
    _check_codes(q, v, border=1e-9)     # sums of 2^20 squares: 2^20 2^-53 of 127 at most
    # a scale beyond float32: no codes (one value whose norm is 1024, a weight of 1e38)
    x = torch.zeros(1, dim)
    x[0, 5] = 1.0
    w = torch.full((dim,), 1e38)
    _, q, s = fw.rms_norm_residual_i8(x.cuda(), w.cuda(), eps=0.0)
    assert torch.isinf(s).all() and not q.any()


@pytest.mark.parametrize("dim,rows", [(1, 1 << 27), (300, 1 << 23), (1030, 1 << 22), (4097, 1 << 21)])
def test_norm_of_more_rows_than_one_launch_has_workgroups_for(dim, rows):
    """Workgroups that take a second turn: rows of a few lanes, a wave, two, eight."""
    import torch

    import dlrm_embedding_bag_amd as fw
    m = rows + 1001
    g = torch.Generator(device="cuda").manual_seed(dim)
    base = torch.randn(977, dim, generator=g, device="cuda").bfloat16()
    x = torch.empty(m, dim, dtype=torch.bfloat16, device="cuda")
    whole = m // 977 * 977
    x[:whole].view(-1, 977, dim).copy_(base[None])
    x[whole:] = base[:m - whole]
    _, q, s = fw.rms_norm_residual_i8(x)
    _, q1, s1 = fw.rms_norm_residual_i8(base)
    assert torch.equal(q[:whole].view(-1, 977, dim), q1.expand(whole // 977, 977, dim))
    assert torch.equal(s[:whole].view(-1, 977), s1.expand(whole // 977, 977))
    assert torch.equal(q[whole:], q1[:m - whole]) and torch.equal(s[whole:], s1[:m - whole])


def test_sizes_beyond_32_bits_are_refused():
    """A size that a 32-bit argument would be narrowed from, to one that is
    accepted, is refused."""
    import torch

    import dlrm_embedding_bag_amd as fw
    wide, tok = (1 << 32) + 8, torch.zeros(1, dtype=torch.int32, device="cuda")

    def row(dtype):
        return torch.empty(1, wide, dtype=dtype, device="cuda")

    assert fw.emb_lookup_grad_workspace_bytes(5000, 10, wide) == 0
    with pytest.raises(ValueError, match="columns"):
        fw.emb_lookup_scaled(row(torch.float8_e4m3fn), tok, out_dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="columns"):
        fw.emb_lookup_grad(row(torch.bfloat16), tok, 1)
    with pytest.raises(ValueError, match="columns"):
        fw.rms_norm_residual_i8(row(torch.bfloat16))
    codes, one = row(torch.int8), torch.ones(1, device="cuda")
    with pytest.raises(ValueError, match="columns"):
        fw.linear_i8_bias_act(codes, one, codes, one)
    many = torch.ones(1, 16, dtype=torch.int8, device="cuda").expand(wide, 16)
    with pytest.raises(ValueError, match="rows"):
        fw.linear_i8_bias_act(many, one, codes[:, :16], one)
    with pytest.raises(ValueError, match="rows"):
        fw.linear_i8_bias_act(codes[:, :16], one, many, one)
