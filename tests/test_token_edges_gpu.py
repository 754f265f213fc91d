"""GPU tests of the token operators at the edges of their ranges.  The references
and the counting of roundings are those of test_token_ops_gpu.py."""
import numpy as np
import pytest

from conftest import gpu_available
from test_token_ops_gpu import TINY, U32, _check_grad, _draw_tokens, _dt, _np64

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
