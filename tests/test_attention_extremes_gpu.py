"""GPU tests of the attention operators at the ends of what they accept: rows and
eps far from 1, scales at the limit, rows that repeat with values that are not
finite, batches of unlike sequences.  References and the counting of roundings are
those of test_attention_ops_gpu.py."""
import math

import numpy as np
import pytest

from conftest import gpu_available
from test_attention_ops_gpu import (TINY, U, U32, _assert_within, _attention_want, _dt, _gen,
                                    _gradient_want, _np64, _packed_inputs, _randn, _turned)

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]


# ----------------------------------------------------------- norm and rotation --
SIZES = (1e-44, 3e-39, 2e-38, 1e-30, 1.0, 1e30, 8e37, 3e38)   # of rows; float32 reaches 3.4e38


def _far_rows(sizes, heads, dim, kind, seed):
    """One token for each size, elements of 0.25 to 1 times it."""
    import torch
    u = torch.rand(len(sizes), heads, dim, generator=_gen(seed), dtype=torch.float64) * 1.5 - 0.75
    u = u + torch.where(u < 0, -0.25, 0.25)
    return (u * torch.tensor(sizes, dtype=torch.float64)[:, None, None]).to(_dt(kind))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("dim,pairs", [(64, 32), (24, 4), (256, 128)])
@pytest.mark.parametrize("eps,sizes", [(0.0, SIZES), (1e-80, (0.0, *SIZES)), (1e-300, (0.0, 1.0)),
                                       (5e-324, (0.0, 0.0, 1e-44))])
def test_rope_of_rows_and_eps_far_from_one(eps, sizes, dim, pairs, inter, kind):
    """Where 1 / rms is beyond float32, or below its normal numbers."""
    import torch

    import dlrm_embedding_bag_amd as fw
    if kind == "bf16":     # (which holds no 1e-44)
        sizes = [1e-39 if size == 1e-44 else size for size in sizes]
    n = len(sizes)
    pos = torch.arange(n, dtype=torch.int32) * 1001
    freqs = (10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / pairs)).float()
    xs = [_far_rows(sizes, h, dim, kind, h) for h in (3, 1)]
    ws = [1.0 + _randn(_gen(h), dim, scale=0.3) for h in (3, 1)]
    rms = [np.sqrt((_np64(x) ** 2).mean(-1, keepdims=True) + eps) for x in xs]
    # gradients whose products with 1 / rms stay within float32
    ds = [(_randn(_gen(5 + i), *x.shape).double() * torch.from_numpy(np.minimum(1e3, r * 1e36)))
          .to(_dt(kind)) for i, (x, r) in enumerate(zip(xs, rms))]
    cuda = [t.cuda() for t in (*xs, pos, freqs, *ws)]
    got = fw.qk_norm_rope(*cuda, eps=eps, interleaved=inter)
    back = fw.qk_norm_rope_grad(ds[0].cuda(), ds[1].cuda(), *cuda, eps=eps, interleaved=inter)
    for i, what in enumerate("qk"):
        unit, w = _np64(xs[i]) / rms[i], _np64(ws[i])
        want, size = _turned(unit * w, pos.numpy(), freqs.numpy(), inter)
        _assert_within(_np64(got[i]), want, 14 * U32 * size + U[kind] * np.abs(want) + TINY, what)
        dv, size = _turned(_np64(ds[i]), pos.numpy(), freqs.numpy(), inter, -1.0)
        g, big = dv * w, np.abs(w) * size
        want = (g - unit * (g * unit).mean(-1, keepdims=True)) / rms[i]
        parts = (big + np.abs(unit) * (np.abs(unit) * big).mean(-1, keepdims=True)) / rms[i]
        _assert_within(_np64(back[i]), want, 20 * U32 * parts + U[kind] * np.abs(want) + TINY,
                       what + " gradient")
        terms = (np.abs(unit) * size).sum((0, 1))
        _assert_within(_np64(back[2 + i]), (dv * unit).sum((0, 1)),
                       (20 + unit.shape[0] * unit.shape[1]) * U32 * terms + TINY, what + " weight")


# ----------------------------------------------------------- packed attention --
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_attention_with_a_scale_next_to_the_limit(kind):
    """Scores of up to 128 of products of 2^-120, all of them powers of two or so."""
    import torch

    import dlrm_embedding_bag_amd as fw
    q, k = torch.zeros(30, 1, 8), torch.zeros(30, 1, 8)
    g = _gen(1)
    q[:, 0, 3] = 2.0 ** -60 * (0.5 + torch.rand(30, generator=g) / 2)
    k[:, 0, 3] = 2.0 ** -60 * (0.5 + torch.rand(30, generator=g) / 2)
    q, k, v = (t.to(_dt(kind)) for t in (q, k, _randn(g, 30, 1, 8)))
    off = torch.tensor([0, 30], dtype=torch.int32)
    want = _attention_want(q, k, v, off, None, True, 2.0 ** 127, kind)
    out, lse = fw.attention_packed(q.cuda(), k.cuda(), v.cuda(), off.cuda(), scale=2.0 ** 127)
    _assert_within(_np64(out), want[0], want[1], "out")
    _assert_within(_np64(lse), want[2], want[3], "lse")
    with pytest.raises(fw.DlrmError, match="attention"):
        fw.attention_packed(q.cuda(), k.cuda(), v.cuda(), off.cuda(), scale=2.4e38)


# Lengths and heads that go to lone waves of 16 and of 32 rows, to two groups of waves
# and to four waves; none fills its last tile of keys.
KINDS = [([20, 7], 2), ([100, 90], 2), ([301], 2), ([4100], 16)]


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("lengths,heads", KINDS)
def test_attention_of_repeated_values_that_are_not_finite(lengths, heads, causal, kind):
    """One row of values for all keys (stride 0), and rows that overlap, as the same
    rows one after another: behind the last key there is none of them."""
    import torch

    import dlrm_embedding_bag_amd as fw
    off, _, q, k, _, _ = (None if t is None else t.cuda()
                          for t in _packed_inputs(lengths, None, heads, heads, 32, kind))
    n = len(q)
    row = _randn(_gen(2), 1, heads, 32).to(_dt(kind)).cuda()
    row[0, 0, 5], row[0, 1, 6], row[0, 1, 7] = math.inf, -math.inf, math.nan
    same = row.expand(n, -1, -1)
    out, lse = fw.attention_packed(q, k, same, off, causal=causal)
    want, wlse = fw.attention_packed(q, k, same.contiguous(), off, causal=causal)
    assert torch.equal(lse, wlse) and torch.equal(torch.nan_to_num(out), torch.nan_to_num(want))
    assert (out[:, 0, 5] == math.inf).all() and (out[:, 1, 6] == -math.inf).all()
    assert torch.equal(out.isnan(), same.isnan())

    flat = _randn(_gen(3), 8 * n + 24).to(_dt(kind)).cuda()
    flat[-1], flat[-30] = math.inf, -math.inf          # of the last row, of the last four
    over = flat.as_strided((n, 1, 32), (8, 32, 1)).expand(-1, heads, -1)
    out, lse = fw.attention_packed(q, k, over, off, causal=causal)
    want, wlse = fw.attention_packed(q, k, over.contiguous(), off, causal=causal)
    assert torch.equal(lse, wlse) and torch.equal(torch.nan_to_num(out), torch.nan_to_num(want))
    assert not out.isnan().any() and out.isinf().any()


def _after_junk(value, kind, call, times):
    """`call` after one that leaves `value` all over LDS: its results and its times in us."""
    import torch

    import dlrm_embedding_bag_amd as fw
    junk = torch.full((4000, 32, 64), value, dtype=_dt(kind), device="cuda")
    off = torch.tensor([0, 4000], dtype=torch.int32, device="cuda")
    out, us = [], []
    for _ in range(times):
        fw.attention_packed(junk, junk, junk, off, causal=False)
        begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        begin.record()
        out.append(call())
        end.record()
        end.synchronize()
        us.append(begin.elapsed_time(end) * 1e3)
    return out, us


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("lengths", [[330, 40, 64, 1], [129, 300, 65, 160], [148] * 4])
def test_attention_of_sequences_that_leave_a_group_without_a_tile(lengths, kind):
    """Of two groups of waves one finds no keys in some rounds; what its part of LDS
    holds then, here the NaN of another call, is nobody's."""
    import dlrm_embedding_bag_amd as fw
    off, _, q, k, v, _ = _packed_inputs(lengths, None, 2, 2, 64, kind)
    want = _attention_want(q, k, v, off, None, True, 0.125, kind)
    args = [t.cuda() for t in (q, k, v, off)]
    for out, lse in _after_junk(math.nan, kind, lambda: fw.attention_packed(*args), 3)[0]:
        _assert_within(_np64(out), want[0], want[1], "out")
        _assert_within(_np64(lse), want[2], want[3], "lse")


def test_attention_takes_no_longer_for_what_others_left_in_lds():
    """(Taken for values that are not finite, it made a call of 10 us one of 62.)"""
    import dlrm_embedding_bag_amd as fw
    off, _, q, k, v, _ = _packed_inputs([148] * 4, None, 8, 8, 64, "bf16")
    args = [t.cuda() for t in (q, k, v, off)]
    times = [np.median(_after_junk(value, "bf16", lambda: fw.attention_packed(*args), 20)[1])
             for value in (1.0, math.nan)]
    assert times[1] < 3 * times[0], times


def test_attention_refuses_logarithms_that_are_no_tensor():
    import torch

    import dlrm_embedding_bag_amd as fw
    off, _, q, k, v, _ = (None if t is None else t.cuda()
                          for t in _packed_inputs([20], None, 2, 2, 64, "f32"))
    for lse in ([0.0] * 20, np.zeros((20, 2), np.float32)):
        with pytest.raises(TypeError, match="lse"):
            fw.attention_packed(q, k, v, off, lse=lse)
    with pytest.raises(ValueError, match="lse"):
        fw.attention_packed(q, k, v, off, lse=torch.zeros(20, 2))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("lengths,heads", [([1] * 40 + [900] + [2] * 30, 8), ([1] * 9 + [900], 8),
                                           ([0] * 200 + [700, 0, 3], 2), ([3000] + [10] * 99, 1)])
def test_attention_of_one_long_sequence_among_short_ones(lengths, heads, kind):
    import dlrm_embedding_bag_amd as fw
    off, _, q, k, v, grad = _packed_inputs(lengths, None, heads, max(1, heads // 4), 64, kind)
    out, lse = fw.attention_packed(q.cuda(), k.cuda(), v.cuda(), off.cuda())
    want = _attention_want(q, k, v, off, None, True, 0.125, kind)
    _assert_within(_np64(out), want[0], want[1], "out")
    _assert_within(_np64(lse), want[2], want[3], "lse")
    got = fw.attention_packed_grad(grad.cuda(), q.cuda(), k.cuda(), v.cuda(), out, lse, off.cuda())
    want, tol = _gradient_want(grad, q, k, v, out, lse, off, None, True, 0.125, kind)
    for a, w, t, what in zip(got, want, tol, "qkv"):
        _assert_within(_np64(a), w, t, what)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("lengths", [[20, 7], [100, 90], [301]])
def test_attention_without_its_logarithms(lengths, kind):
    """lse may be NULL for the C entry point, fill asking for it or not."""
    import torch

    import dlrm_embedding_bag_amd as fw
    off, _, q, k, v, _ = (None if t is None else t.cuda()
                          for t in _packed_inputs(lengths, None, 2, 2, 64, kind))
    n = len(q)
    off = torch.cat((off, off[-1:] + 0))[1:].contiguous()     # rows before the first sequence
    want, _ = fw.attention_packed(q, k, v, off)
    for fill in (0, 1, 2, 3):
        out = torch.full_like(q, 7.0)
        row = (128, 64)
        status = fw.load().attention_packed(
            n, n, len(off) - 1, 2, 2, 64, 0 if kind == "f32" else 1, q.data_ptr(), *row,
            k.data_ptr(), *row, v.data_ptr(), *row, off.data_ptr(), None, 1, 0.125, fill,
            out.data_ptr(), *row, None, torch.cuda.current_stream().cuda_stream)
        assert status == 0
        first = int(off[0])
        assert torch.equal(out[first:], want[first:])
        assert (out[:first] == (0.0 if fill & 1 else 7.0)).all()
