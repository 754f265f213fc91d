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
