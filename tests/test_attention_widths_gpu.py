"""GPU tests of packed attention and its gradient in every width that sequences call
for: many of few rows, some of about a hundred, few long ones of few heads, and enough
rows and heads for the widest workgroups; and of the rotation of few heads.  References and the counting of roundings
are those of test_attention_ops_gpu.py."""
import pytest

import test_attention_ops_gpu as ops
from conftest import gpu_available
from test_attention_ops_gpu import (_assert_within, _attention_want, _dt, _gen, _gradient_want,
                                    _laid, _np64, _packed_inputs, _randn)

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]

# lengths, keys more than queries, heads, key heads
SHORT = [([0, 1, 15, 16, 17, 33, 2, 0, 5, 14], None, 3, 1),
         ([16] * 5 + [1] * 7, [0, 3, 16, -9, 40, 0, 1, 31, 0, 0, -1, 100], 2, 2),
         ([1] * 40, [0, 5, 15, 16] * 10, 8, 2), ([32, 0, 0, 0], [0, 7, 0, 20], 5, 5)]
SOME = [([40, 60, 90, 33], None, 3, 1), ([100, 50], [-60, 70], 2, 2)]
LONG = [([1, 8, 0, 20], [700, 300, 400, 1200], 4, 2), ([3, 60], [600, 290], 3, 1),
        ([5] * 300, [270] * 300, 2, 1)]
FEW = [([129, 300], None, 3, 1), ([260, 131], [-140, 63], 2, 2), ([513], [64], 1, 1)]


def _check(lengths, past, heads, kv, dim, causal, kind, pick=None):
    import dlrm_embedding_bag_amd as fw
    off, koff, q, k, v, grad = _packed_inputs(lengths, past, heads, kv, dim, kind)
    cuda = [None if t is None else t.cuda() for t in (off, koff)]
    out, lse = fw.attention_packed(q.cuda(), k.cuda(), v.cuda(), *cuda, causal=causal)
    got = fw.attention_packed_grad(grad.cuda(), q.cuda(), k.cuda(), v.cuda(), out, lse, *cuda,
                                   causal=causal)
    rows = list(range(heads)) if pick is None else [h for j in pick for h in
                                                    range(j * heads // kv, (j + 1) * heads // kv)]
    keys = list(range(kv)) if pick is None else pick
    q, k, v, grad, out, lse = q[:, rows], k[:, keys], v[:, keys], grad[:, rows], out[:, rows], lse[:, rows]
    want = _attention_want(q, k, v, off, koff, causal, dim ** -0.5, kind)
    _assert_within(_np64(out), want[0], want[1], f"out of {dim}")
    _assert_within(_np64(lse), want[2], want[3], f"lse of {dim}")
    want, tol = _gradient_want(grad, q, k, v, out, lse, off, koff, causal, dim ** -0.5, kind)
    for a, w, t, what, at in zip(got, want, tol, "qkv", (rows, keys, keys)):
        _assert_within(_np64(a[:, at]), w, t, f"{what} of {dim}")


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lengths,past,heads,kv", SHORT + SOME + LONG + FEW)
def test_widths(lengths, past, heads, kv, causal, kind):
    for dim in (8, 32, 40, 64, 88, 96, 104, 128) if len(lengths) < 100 else (64,):
        _check(lengths, past, heads, kv, dim, causal, kind)


@pytest.mark.parametrize("dim", [32, 56, 96, 128])
@pytest.mark.parametrize("kind,tokens", [("f32", 1030), ("bf16", 520)])
def test_many_rows_of_many_heads(kind, tokens, dim):
    """(8 or 4 times 128 rows of 64 heads)"""
    _check([tokens - 130, 130], [65, 0], 64, 4, dim, True, kind, pick=[0, 3])


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lengths,past", [([300, 0, 77, 129, 1, 200], None),
                                          ([200, 64, 0, 300], [-150, 500, 9, -300]),
                                          ([40] * 17, None)])
def test_rows_outside_sequences_of_many_heads(lengths, past, causal, kind):
    """Rows before the first sequence and behind the last, with tiles enough that
    workgroups go out by their work: each row is written once, as it should be."""
    import torch

    import dlrm_embedding_bag_amd as fw
    lead, tail, heads, kv = 150, 200, 40, 20
    off, koff, q, k, v, grad = _packed_inputs(lengths, past, heads, kv, 64, kind)
    n = int(off[-1])
    wide = [torch.cat([torch.full((a, *t.shape[1:]), float("nan"), dtype=t.dtype), t,
                       torch.full((b, *t.shape[1:]), float("nan"), dtype=t.dtype)]).cuda()
            for t, a, b in ((q, lead, tail), (grad, lead, tail))]
    if past is None:
        wk, wv = (torch.cat([torch.full((lead, kv, 64), float("nan"), dtype=t.dtype), t,
                             torch.full((tail, kv, 64), float("nan"), dtype=t.dtype)]).cuda()
                  for t in (k, v))
    else:
        wk, wv = k.cuda(), v.cuda()
    offs = ((off + lead).cuda(), None if koff is None else koff.cuda())
    out, lse = fw.attention_packed(wide[0], wk, wv, *offs, causal=causal)
    pick = [0, 19]
    rows = [0, 1, 38, 39]
    inside = slice(lead, lead + n)
    want = _attention_want(q[:, rows], k[:, pick], v[:, pick], off, koff, causal, 0.125, kind)
    _assert_within(_np64(out[inside, rows]), want[0], want[1], "out")
    _assert_within(_np64(lse[inside, rows]), want[2], want[3], "lse")
    got = fw.attention_packed_grad(wide[1], wide[0], wk, wv, out, lse, *offs, causal=causal)
    want, tol = _gradient_want(grad[:, rows], q[:, rows], k[:, pick], v[:, pick], out[inside, rows],
                               lse[inside, rows], off, koff, causal, 0.125, kind)
    keys = inside if past is None else slice(None)
    for a, w, t, what, at in zip((got[0][inside], got[1][keys], got[2][keys]), want, tol, "qkv",
                                 (rows, pick, pick)):
        _assert_within(_np64(a[:, at]), w, t, what)
    for part in (slice(0, lead), slice(lead + n, None)):
        assert not out[part].any() and (lse[part] == float("-inf")).all() and not got[0][part].any()
        if past is None:
            assert not got[1][part].any() and not got[2][part].any()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("layout", ["slice", "heads"])
@pytest.mark.parametrize("lengths", [[3, 16, 7, 0, 18], [60, 70], [257, 60]])
def test_layouts(lengths, layout, kind):
    import torch

    import dlrm_embedding_bag_amd as fw
    off, _, q, k, v, grad = _packed_inputs(lengths, None, 4, 2, 72, kind)
    off = off.cuda()
    want = fw.attention_packed(q.cuda(), k.cuda(), v.cuda(), off)
    out, lse = fw.attention_packed(_laid(q, layout), _laid(k, layout), _laid(v, layout), off)
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    want = fw.attention_packed_grad(grad.cuda(), q.cuda(), k.cuda(), v.cuda(), out, lse, off)
    got = fw.attention_packed_grad(_laid(grad, layout), _laid(q, layout), _laid(k, layout),
                                   _laid(v, layout), _laid(out.cpu(), layout), lse, off)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("length,at,heads", [(40, 17, 2), (40, 0, 2), (100, 70, 2), (129, 128, 2),
                                             (260, 3, 2), (530, 300, 64)])
def test_masked_values_that_are_not_finite(length, at, heads, bad, kind):
    """Rows before a key do not see it, whatever it and its value hold, and of rows
    that do only those elements change."""
    import torch

    import dlrm_embedding_bag_amd as fw
    g = _gen(length)
    q, k, v = (_randn(g, 2 * length, heads, 64).to(_dt(kind)).cuda() for _ in range(3))
    off = torch.tensor([0, length, 2 * length], dtype=torch.int32, device="cuda")
    want, wlse = fw.attention_packed(q, k, v, off)
    v[at, 1, 3] = bad
    out, lse = fw.attention_packed(q, k, v, off)
    assert torch.equal(lse, wlse)
    assert torch.equal(out[:at], want[:at]) and torch.equal(out[length:], want[length:])
    assert not out[at:length, 1, 3].isfinite().any()
    out[at:length, 1, 3] = want[at:length, 1, 3]
    # (the careful way adds the same products in the same order, but for these)
    assert torch.equal(out, want)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("n,heads,kv,dim,pairs", [(4100, 1, 1, 64, 32), (8207, 2, 0, 8, 4),
                                                  (33000, 1, 2, 8, 4), (5000, 3, 1, 128, 64)])
def test_rotation_of_many_tokens_of_few_heads(n, heads, kv, dim, pairs, kind):
    """(several tokens a workgroup, the last of them not whole)"""
    ops.test_rope(n, heads, kv, dim, pairs, False, kind)
    ops.test_rope_gradient(n, heads, kv, dim, pairs, True, kind)


def test_offsets_that_decrease_stay_within_the_tensors():
    """Bad offsets give rows of no meaning, but no access outside the tensors: what
    lies around them stays as it was, and calls after them are right."""
    import torch

    import dlrm_embedding_bag_amd as fw
    g = _gen(3)
    n = 90
    for off in ([0, 50, 20, 90], [-7, 30, 2**31 - 1, 10], [90, 0, 0, 0]):
        off = torch.tensor(off, dtype=torch.int32, device="cuda")
        for batch in (3, 1):
            o = off[:batch + 1].contiguous()
            q, k, v, grad = (_randn(g, n, 2, 64).cuda() for _ in range(4))
            wide = torch.full((n + 400, 2, 64), 7.0, device="cuda")
            out, lse = fw.attention_packed(q, k, v, o, out=wide[200:200 + n])
            assert (wide[:200] == 7.0).all() and (wide[200 + n:] == 7.0).all()
            got = [torch.full((n + 400, 2, 64), 7.0, device="cuda") for _ in range(3)]
            fw.attention_packed_grad(grad, q, k, v, out, lse, o, out_q=got[0][200:200 + n],
                                     out_k=got[1][200:200 + n], out_v=got[2][200:200 + n])
            for t in got:
                assert (t[:200] == 7.0).all() and (t[200 + n:] == 7.0).all()
    _check([20, 30], None, 2, 1, 64, True, "f32")
