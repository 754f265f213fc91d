"""GPU tests of the quantised cache and of attention over it against plain forms
in 64 bits on the host.

Codes and scales are decided by comparisons of exact values (a power of two
scales without rounding), so what is written and read back is compared for
equality.  Tolerances of attention are those of attention over packed sequences:
a score of d products is off by d u32 of the sum of magnitudes, its exponent by
4 u32 of the largest score more, exp2 by 4 u32; 2 e of sum p |v| in the quotient,
n u32 for sums of n terms, u(bf16) for the weights' rounding in bfloat16, and the
output's type.
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
TOP = {8: 448.0, 4: 6.0}
E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])


def _dt(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _np64(t):
    import torch
    return t.detach().cpu().to(torch.float64).numpy()


def _grid(bits):
    """The magnitudes that codes stand for, in the order of their codes."""
    if bits == 4:
        return E2M1
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e > 0, (8 + m) * 2.0 ** (e - 10), m * 2.0 ** -9)


def _quantised(x, bits):
    """Codes, scale bytes and values of float64 rows, group by group."""
    g = x.reshape(-1, 32)
    codes = np.zeros(g.shape, np.int64)
    scales = np.zeros(len(g), np.int64)
    grid = _grid(bits)
    for i, row in enumerate(g):
        if not np.isfinite(row).all():
            scales[i] = 255
            continue
        top = np.abs(row).max()
        e = -117
        if top > 0:
            e = max(-117, int(math.floor(math.log2(top))) - (12 if bits == 8 else 6))
            while TOP[bits] * 2.0 ** e < top:
                e += 1
            e = min(e, 119 if bits == 8 else 125)       # beyond it values are clipped
        scales[i] = e + 127
        y = np.abs(row) * 2.0 ** -e
        lo = np.clip(np.searchsorted(grid, y, side="right") - 1, 0, len(grid) - 1)
        hi = np.minimum(lo + 1, len(grid) - 1)
        up, down = grid[hi] - y, y - grid[lo]
        c = np.where(up < down, hi, np.where(up > down, lo, np.where(lo % 2 == 0, lo, hi)))
        codes[i] = c + np.signbit(row) * (128 if bits == 8 else 8)
    sign = np.where(codes >= (128 if bits == 8 else 8), -1.0, 1.0)
    with np.errstate(invalid="ignore"):
        values = sign * grid[codes & (127 if bits == 8 else 7)] * 2.0 ** (scales[:, None] - 127.0)
    values = np.where(scales[:, None] == 255, np.nan, values)
    rows = codes.reshape(*x.shape)
    if bits == 4:
        rows = rows[..., 0::2] | rows[..., 1::2] << 4
    return rows.astype(np.uint8), scales.reshape(*x.shape[:-1], -1).astype(np.uint8), \
        values.reshape(x.shape)


def _values(n, heads, dim, kind, seed):
    """Rows of many magnitudes, borders between codes and groups of zeros among them."""
    import torch
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, heads, dim, generator=g) * torch.exp2(
        torch.randint(-20, 20, (n, heads, 1), generator=g).float())
    x[0::5] = torch.randint(-64, 65, x[0::5].shape, generator=g) * 0.125
    x[1::7] = 0.0
    x[2::7, :, ::3] = -0.0
    x[3::7] *= 2.0 ** -118
    x[4::7] = torch.where(torch.rand(x[4::7].shape, generator=g) < 0.5, 448.0 * 3, 6.0 * 5)
    if n > 9:
        x[5, 0, :4] = torch.tensor([3e38, -3e38, 1.0, 0.0])
        x[6, 0, 1] = float("nan")
        x[8, 0, 2] = float("-inf")
    return x.to(_dt(kind))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("n,heads,dim,pages,page", [
    (1, 1, 32, 1, 16), (40, 3, 64, 5, 16), (70, 2, 128, 2, 64), (129, 1, 32, 3, 256),
    (33, 5, 128, 7, 32)])
def test_cache_holds_the_nearest_codes(n, heads, dim, pages, page, bits, kind):
    import torch

    import dlrm_embedding_bag_amd as fw
    k, v = _values(n, heads, dim, kind, 1), _values(n, heads, dim, kind, 2)
    rng = np.random.default_rng(n)
    slots = rng.permutation(pages * page)[:n].astype(np.int32)
    skipped = rng.random(n) < 0.2
    slots = np.where(skipped, rng.choice([-1, -2**31, pages * page, 2**31 - 1], n), slots)
    cache = fw.kv_cache(pages, page, heads, dim, bits)
    for t in cache:
        t.fill_(0x5a)
    on = torch.from_numpy(slots.astype(np.int32)).cuda()
    strided = torch.full((n, heads + 1, dim + 8), float("nan"), dtype=_dt(kind))
    strided[:, 1:, 8:] = k
    fw.kv_cache_write(cache, strided.cuda()[:, 1:, 8:], v.transpose(0, 1).contiguous().cuda()
                      .transpose(0, 1), on)
    want = [np.full(t.shape, 0x5a, np.uint8) for t in cache]
    values = []
    for i, x in enumerate((k, v)):
        codes, scales, val = _quantised(_np64(x), bits)
        values.append(np.where(skipped[:, None, None], 0.0, val))
        for t in np.flatnonzero(~skipped):
            want[2 * i][slots[t] // page, :, slots[t] % page] = codes[t]
            want[2 * i + 1][slots[t] // page, :, slots[t] % page] = scales[t]
    for got, w, what in zip(cache, want, cache._fields):
        bad = got.cpu().numpy() != w
        assert not bad.any(), f"{what}: {bad.sum()} of {bad.size}, first {np.argwhere(bad)[0]}"
    for out in ("f32", "bf16"):
        back = fw.kv_cache_read(cache, on, out_dtype=_dt(out))
        for got, w, what in zip(back, values, "kv"):
            assert got.dtype == _dt(out)
            np.testing.assert_array_equal(_np64(got), w, err_msg=what)
    buf = torch.full((n, heads + 1, dim + 8), 7.0, dtype=_dt(kind), device="cuda")
    view = buf[:, 1:, 8:]
    back = fw.kv_cache_read(cache, on, out_k=view)
    assert back[0] is view and (buf[:, 0] == 7).all() and (buf[:, :, :8] == 7).all()
    np.testing.assert_array_equal(_np64(view), values[0])


def test_cache_of_no_tokens():
    import torch

    import dlrm_embedding_bag_amd as fw
    cache = fw.kv_cache(2, 16, 1, 32)
    none = torch.empty(0, 1, 32, device="cuda")
    slots = torch.empty(0, dtype=torch.int32, device="cuda")
    fw.kv_cache_write(cache, none, none, slots)
    assert fw.kv_cache_read(cache, slots)[0].shape == (0, 1, 32)
    assert not any(bool(t.any()) for t in cache)


# ------------------------------------------------------------ attention over it --
def _filled(pages, page, heads, dim, bits, seed):
    """A cache whose every row was written, and the values that it holds."""
    import torch

    import dlrm_embedding_bag_amd as fw
    g = torch.Generator().manual_seed(seed)
    n = pages * page
    k, v = (torch.randn(n, heads, dim, generator=g).cuda() for _ in range(2))
    cache = fw.kv_cache(pages, page, heads, dim, bits)
    slots = torch.arange(n, dtype=torch.int32, device="cuda")
    fw.kv_cache_write(cache, k, v, slots)
    return cache, [_np64(t) for t in fw.kv_cache_read(cache, slots, out_dtype=torch.float32)]


def _cached_want(q, k, v, table, lengths, page, pages, scale, kind):
    q = _np64(q)
    batch, heads, dim = q.shape
    group = heads // k.shape[1]
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(batch):
        j = np.arange(max(0, min(lengths[b], table.shape[1] * page)))
        names = table[b, j // page]
        there = (names >= 0) & (names < pages)
        rows = (names.astype(np.int64) * page + j % page)[there]
        if not len(rows):
            continue
        for h in range(heads):
            kk, vv = k[rows, h // group], v[rows, h // group]
            s = kk @ q[b, h] * scale
            size = np.abs(kk) @ np.abs(q[b, h]) * scale
            p = np.exp(s - s.max())
            e = (dim * size.max() + 4 * np.abs(s).max() + 4) * U32
            out[b, h] = p @ vv / p.sum()
            weight = p @ np.abs(vv) / p.sum()
            tol[b, h] = (2 * e + (len(rows) + 8) * U32
                         + (U["bf16"] if kind == "bf16" else 0.0)) * weight \
                + U[kind] * np.abs(out[b, h]) + TINY
    return out, tol


def _assert_within(got, want, tol, what):
    err = np.abs(got - want)
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {bad.sum()} of {bad.size} off, first at "
                           f"{tuple(np.argwhere(bad)[0])}: {got[bad][0]!r} for {want[bad][0]!r}, "
                           f"tolerance {np.broadcast_to(tol, err.shape)[bad][0]!r}")


CACHED = [  # lengths, heads, kv_heads, dim, page, columns of the table
    ([1], 1, 1, 32, 16, 1), ([0, 1, 15, 16, 17], 4, 2, 64, 16, 3), ([63, 64, 65, 0], 8, 1, 128, 32, 3),
    ([257, 3], 16, 1, 64, 64, 5), ([130, 129], 34, 2, 128, 16, 9), ([700], 6, 3, 32, 256, 3),
    ([5, 300, 1000, 2], 4, 4, 128, 64, 16), ([2100], 3, 1, 64, 16, 140), ([50] * 70, 2, 2, 32, 16, 4),
    ([1, 4000], 20, 1, 128, 128, 32)]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("lengths,heads,kv,dim,page,columns", CACHED)
def test_cached_attention(lengths, heads, kv, dim, page, columns, bits, kind):
    import torch

    import dlrm_embedding_bag_amd as fw
    rng = np.random.default_rng(sum(lengths) + dim)
    pages = 40 if page < 128 else 20
    cache, (k, v) = _filled(pages, page, kv, dim, bits, dim)
    # pages are shared between sequences, and repeat; some entries name none
    table = rng.integers(0, pages, (len(lengths), columns)).astype(np.int32)
    table[rng.random(table.shape) < 0.1] = rng.choice([-1, pages, 2**31 - 1, -2**31])
    lens = np.array(lengths, np.int32)
    g = torch.Generator().manual_seed(dim)
    q = (torch.randn(len(lengths), heads, dim, generator=g) * 1.5).to(_dt(kind))
    scale = None if dim == 64 else 0.2
    want, tol = _cached_want(q, k, v, table, lens, page, pages, dim ** -0.5 if scale is None else
                             scale, kind)
    t, n = torch.from_numpy(table).cuda(), torch.from_numpy(lens).cuda()
    out = fw.attention_cached(q.cuda(), cache, t, n, scale=scale)
    _assert_within(_np64(out), want, tol, "out")
    # strides, a wider table, given outputs and workspace
    wide = torch.full((len(lengths), columns + 3), 2**30, dtype=torch.int32, device="cuda")
    wide[:, :columns] = t
    sq = torch.full((len(lengths), heads + 1, dim + 8), float("nan"), dtype=_dt(kind),
                    device="cuda")
    sq[:, 1:, 1:dim + 1] = q.cuda()
    so = torch.full((heads, len(lengths), dim), 3.0, dtype=_dt(kind), device="cuda")
    ws = torch.full((max(1, fw.attention_cached_workspace_bytes(len(lengths), heads, kv, dim, columns,
                                                                 page)),), 255, dtype=torch.uint8,
                    device="cuda")
    back = fw.attention_cached(sq[:, 1:, 1:dim + 1], cache, wide[:, :columns], n, scale=scale,
                               out=so.transpose(0, 1), workspace=ws)
    assert torch.equal(back, out)


@pytest.mark.parametrize("bits", [4, 8])
def test_cached_attention_follows_lengths_and_capacity(bits):
    """Lengths beyond the table, below zero, and groups of NaN that lie behind the
    last key, or within."""
    import torch

    import dlrm_embedding_bag_amd as fw
    cache, (k, v) = _filled(6, 32, 2, 64, bits, 3)
    q = torch.randn(4, 4, 64, generator=torch.Generator().manual_seed(1))
    table = np.array([[0, 1, 2]] * 4, np.int32)
    for lens in ([96, 97, 2**31 - 1, -7], [64, 70, 1, 0]):
        want, tol = _cached_want(q, k, v, table, np.array(lens), 32, 6, 0.125, "f32")
        out = fw.attention_cached(q.cuda(), cache, torch.from_numpy(table).cuda(),
                                  torch.tensor(lens, dtype=torch.int32, device="cuda"))
        _assert_within(_np64(out), want, tol, "out")
    bad = torch.full((1, 2, 64), float("nan"), device="cuda")
    fw.kv_cache_write(cache, bad, bad, torch.tensor([70], dtype=torch.int32, device="cuda"))
    lens = torch.tensor([70, 64, 71, 0], dtype=torch.int32, device="cuda")
    again = fw.attention_cached(q.cuda(), cache, torch.from_numpy(table).cuda(), lens)
    want, tol = _cached_want(q, k, v, table, np.array([70, 64, 70, 0]), 32, 6, 0.125, "f32")
    _assert_within(_np64(again)[[0, 1, 3]], want[[0, 1, 3]], tol[[0, 1, 3]], "out")
    assert again[2].isnan().all()
