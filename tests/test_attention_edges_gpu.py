"""GPU tests of the attention operators at the edges of their use: other streams,
captured graphs, memory beyond 32-bit offsets, many heads, the Python functions'
refusals.  References and the counting of roundings are those of
test_attention_ops_gpu.py and test_attention_cache_gpu.py."""
import math

import numpy as np
import pytest

from conftest import gpu_available
from test_attention_cache_gpu import _cached_want, _filled
from test_attention_ops_gpu import (_assert_within, _attention_want, _dt, _gen, _gradient_want,
                                    _np64, _packed_inputs, _randn)

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]


def _calls(kind="bf16"):
    """Each operator as (inputs to be refilled, call)."""
    import torch

    import dlrm_embedding_bag_amd as fw
    g = _gen(7)
    off, _, q, k, v, grad = _packed_inputs([70, 3, 0, 150], None, 8, 2, 64, kind, 3)
    off, q, k, v, grad = (t.cuda() for t in (off, q, k, v, grad))
    pos = torch.arange(len(q), dtype=torch.int32, device="cuda")
    freqs = (10000.0 ** (-torch.arange(32) / 32)).cuda()
    w = 1.0 + _randn(g, 64, scale=0.1).cuda()
    out, lse = fw.attention_packed(q, k, v, off)
    cache, _ = _filled(20, 16, 2, 64, 8, 1)
    slots = torch.randperm(320, generator=g)[:len(q)].to(torch.int32).cuda()
    table = torch.randperm(20, generator=g).view(4, 5).to(torch.int32).cuda()
    lengths = torch.tensor([80, 33, 0, 17], dtype=torch.int32, device="cuda")
    few = q[:4].clone()

    def cached():
        fw.kv_cache_write(cache, k, v, slots)
        return (*fw.kv_cache_read(cache, slots, out_dtype=_dt(kind)),
                fw.attention_cached(few, cache, table, lengths))

    return {
        "rope": ((q, k), lambda: fw.qk_norm_rope(q, k, pos, freqs, w, w)),
        "rope gradient": ((q, k, grad), lambda: fw.qk_norm_rope_grad(grad, k, q, k, pos, freqs, w, w)),
        "attention": ((q, k, v), lambda: fw.attention_packed(q, k, v, off)),
        "attention gradient": ((q, k, v, grad),
                               lambda: fw.attention_packed_grad(grad, q, k, v, out, lse, off)),
        "cache": ((k, v, few), cached)}


@pytest.mark.parametrize("name", ["rope", "rope gradient", "attention", "attention gradient", "cache"])
def test_replays_of_a_captured_call_follow_its_inputs(name):
    """Two graphs of one call, replayed in turn with the program's own calls and
    synchronizations between, each equal to the eager result on the same inputs."""
    import torch
    inputs, call = _calls()[name]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs.append((graph, call()))
    for turn in range(4):
        g = torch.Generator(device="cuda").manual_seed(turn)
        for t in inputs:
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        want = [t.clone() for t in call()]
        for graph, got in graphs if turn % 2 else graphs[::-1]:
            graph.replay()
            if turn == 2:
                torch.cuda.synchronize()
            for a, b in zip(got, want):
                assert torch.equal(a, b), (turn, name)


@pytest.mark.parametrize("name", ["rope", "rope gradient", "attention", "attention gradient", "cache"])
def test_calls_on_another_stream(name):
    """Given as an argument or made current, while the default stream works."""
    import torch
    inputs, call = _calls("f32")[name]
    want = [t.clone() for t in call()]
    torch.cuda.synchronize()
    busy = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    for _ in range(3):
        busy = busy @ busy * 1e-3
        with torch.cuda.stream(side):
            got = call()
        side.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_stream_argument():
    import torch

    import dlrm_embedding_bag_amd as fw
    off, _, q, k, v, grad = (None if t is None else t.cuda()
                             for t in _packed_inputs([70, 150], None, 4, 2, 64, "f32"))
    out, lse = fw.attention_packed(q, k, v, off)
    want = fw.attention_packed_grad(grad, q, k, v, out, lse, off)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o2, l2 = fw.attention_packed(q, k, v, off, stream=side)
    got = fw.attention_packed_grad(grad, q, k, v, o2, l2, off, stream=side)
    side.synchronize()
    assert torch.equal(out, o2) and torch.equal(lse, l2)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_calls_at_once():
    """On two streams, each with its own workspace."""
    import torch

    import dlrm_embedding_bag_amd as fw
    sets = []
    for seed in range(2):
        off, _, q, k, v, grad = (None if t is None else t.cuda() for t in
                                 _packed_inputs([400, 90], None, 8, 2, 64, "bf16", seed))
        out, lse = fw.attention_packed(q, k, v, off)
        want = fw.attention_packed_grad(grad, q, k, v, out, lse, off)
        sets.append(((grad, q, k, v, out, lse, off), want, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for args, _, stream in sets:
            with torch.cuda.stream(stream):
                got.append(fw.attention_packed_grad(*args))
        torch.cuda.synchronize()
        for (_, want, _), g in zip(sets, got):
            assert all(torch.equal(a, b) for a, b in zip(g, want))


def test_packed_rows_beyond_32_bit_offsets():
    """Sequences behind 2^31 elements and 2^32 bytes of rows that no sequence holds."""
    import torch

    import dlrm_embedding_bag_amd as fw
    n, heads, dim = 1_200_000, 16, 128
    lengths = [200, 57]
    first = n - sum(lengths)
    off = torch.tensor(first + np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32)
    g = _gen(1)
    small = [_randn(g, sum(lengths), h, dim).to(_dt("bf16")) for h in (heads, heads, heads, heads)]
    big = []
    for t in small:
        b = torch.zeros(n, heads, dim, dtype=t.dtype, device="cuda")
        b[first:] = t.cuda()
        big.append(b)
    q, k, v, grad = big
    out, lse = fw.attention_packed(q, k, v, off.cuda())
    want = _attention_want(*small[:3], off - first, None, True, dim ** -0.5, "bf16")
    _assert_within(_np64(out[first:]), want[0], want[1], "out")
    _assert_within(_np64(lse[first:]), want[2], want[3], "lse")
    assert not out[:first].any() and (lse[:first] == -math.inf).all()
    got = fw.attention_packed_grad(grad, q, k, v, out, lse, off.cuda())
    want, tol = _gradient_want(small[3], *small[:3], out[first:], lse[first:], off - first, None, True,
                               dim ** -0.5, "bf16")
    for a, w, t, what in zip(got, want, tol, "qkv"):
        _assert_within(_np64(a[first:]), w, t, what)
        assert not a[:first].any()


def test_cache_beyond_32_bit_offsets():
    """Pages behind 2^32 bytes of codes."""
    import torch

    import dlrm_embedding_bag_amd as fw
    pages, page, heads, dim = 40_000, 128, 8, 128
    cache = fw.KVCache(*(torch.empty(pages, heads, page, n, dtype=torch.uint8, device="cuda")
                         for n in (dim, dim // 32) * 2))
    g = _gen(2)
    n = 300
    k, v = (_randn(g, n, heads, dim) for _ in range(2))
    names = np.array([pages - 1, 3, pages - 2], np.int32)
    slots = torch.from_numpy(np.array([names[j // page] * page + j % page for j in range(n)],
                                      np.int32)).cuda()
    fw.kv_cache_write(cache, k.cuda(), v.cuda(), slots)
    kr, vr = fw.kv_cache_read(cache, slots, out_dtype=torch.float32)
    # (codes of 8 bits are off by at most half of 2^-3 of their magnitude, or of
    # the smallest step, 2^-9 of a group's scale, which is below its largest / 224)
    for a, b in ((kr, k), (vr, v)):
        far = (a.cpu() - b).abs() - b.abs() / 16 - b.abs().amax() / 224 / 1024
        assert (far <= 0).all()
    q = _randn(g, 1, 16, dim)
    out = fw.attention_cached(q.cuda(), cache, torch.from_numpy(names[None]).cuda(),
                              torch.tensor([n], dtype=torch.int32, device="cuda"))
    # rows named 0, 1, 2 in the reference's small cache
    kk, vv = (np.zeros((3 * page, heads, dim)) for _ in range(2))
    kk[:n], vv[:n] = _np64(kr), _np64(vr)
    want, tol = _cached_want(q, kk, vv, np.array([[0, 1, 2]], np.int32), np.array([n]), page, 3,
                             dim ** -0.5, "f32")
    _assert_within(_np64(out), want, tol, "out")


def test_rope_rows_beyond_32_bit_offsets():
    import torch

    import dlrm_embedding_bag_amd as fw
    n, heads, dim = 70_000, 256, 128
    q = torch.zeros(n, heads, dim, dtype=torch.bfloat16, device="cuda")
    tail = _randn(_gen(3), 5, heads, dim).to(torch.bfloat16).cuda()
    q[-5:] = tail
    pos = torch.arange(n, dtype=torch.int32, device="cuda")
    freqs = (10000.0 ** (-torch.arange(64) / 64)).cuda()
    want, _ = fw.qk_norm_rope(tail, None, pos[-5:].clone(), freqs)
    got, _ = fw.qk_norm_rope(q, None, pos, freqs, out_q=q)
    assert torch.equal(got[-5:], want) and not got[:-5].any()


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv,lengths", [(64, 1, [33, 130]), (7, 7, [300]), (48, 2, [200, 260, 1]),
                                              (3, 1, [400, 129])])
def test_group_sizes(heads, kv, lengths, kind):
    """Groups of odd sizes and of one, for the two halves that share a key tile."""
    import dlrm_embedding_bag_amd as fw
    off, _, q, k, v, grad = _packed_inputs(lengths, None, heads, kv, 64, kind)
    out, lse = fw.attention_packed(q.cuda(), k.cuda(), v.cuda(), off.cuda())
    want = _attention_want(q, k, v, off, None, True, 0.125, kind)
    _assert_within(_np64(out), want[0], want[1], "out")
    got = fw.attention_packed_grad(grad.cuda(), q.cuda(), k.cuda(), v.cuda(), out, lse, off.cuda())
    want, tol = _gradient_want(grad, q, k, v, out, lse, off, None, True, 0.125, kind)
    for a, w, t, what in zip(got, want, tol, "qkv"):
        _assert_within(_np64(a), w, t, what)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("causal", [False, True])
def test_many_keys_of_few_heads(causal, kind):
    """Enough tiles of keys for the widest workgroups, in every width of heads."""
    import dlrm_embedding_bag_amd as fw
    for dim, kv in ((32, 40), (64, 40), (96, 36), (128, 36)):
        off, koff, q, k, v, grad = _packed_inputs([300, 641], [7, 0], kv, kv, dim, kind)
        out, lse = fw.attention_packed(q.cuda(), k.cuda(), v.cuda(), off.cuda(), koff.cuda(),
                                       causal=causal)
        got = fw.attention_packed_grad(grad.cuda(), q.cuda(), k.cuda(), v.cuda(), out, lse,
                                       off.cuda(), koff.cuda(), causal=causal)
        pick = [0, kv // 2, kv - 1]
        args = [t[:, pick] for t in (grad, q, k, v)]
        want, tol = _gradient_want(*args, out.cpu()[:, pick], lse.cpu()[:, pick], off, koff, causal,
                                   dim ** -0.5, kind)
        for a, w, t, what in zip(got, want, tol, "qkv"):
            _assert_within(_np64(a)[:, pick], w, t, f"{what} of {dim}")


def test_repeated_rows():
    """Inputs whose rows or heads repeat (stride 0), as one key for all heads."""
    import torch

    import dlrm_embedding_bag_amd as fw
    off, _, q, k, v, grad = (None if t is None else t.cuda()
                             for t in _packed_inputs([40, 100], None, 4, 4, 64, "f32"))
    k1, v1 = k[:, :1].expand(-1, 4, -1), v[:1].expand(140, -1, -1)
    a = fw.attention_packed(q, k1, v1, off)
    b = fw.attention_packed(q, k1.contiguous(), v1.contiguous(), off)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    x = fw.attention_packed_grad(grad[:1].expand(140, -1, -1), q, k1, v1, *a, off)
    y = fw.attention_packed_grad(grad[:1].expand(140, -1, -1).contiguous(), q, k1.contiguous(),
                                 v1.contiguous(), *b, off)
    assert all(torch.equal(s, t) for s, t in zip(x, y))


def test_python_refusals():
    import torch

    import dlrm_embedding_bag_amd as fw
    q = torch.zeros(6, 4, 64, device="cuda")
    k = torch.zeros(6, 2, 64, device="cuda")
    i = torch.zeros(6, dtype=torch.int32, device="cuda")
    off = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    freqs = torch.ones(32, device="cuda")
    out, lse = fw.attention_packed(q, k, k, off)
    cache = fw.kv_cache(4, 16, 2, 64)
    table = torch.zeros(6, 2, dtype=torch.int32, device="cuda")
    for error, match, call in (
            (TypeError, "int32", lambda: fw.qk_norm_rope(q, k, i.long(), freqs)),
            (ValueError, "elements", lambda: fw.qk_norm_rope(q, k, i[:5], freqs)),
            (TypeError, "float32", lambda: fw.qk_norm_rope(q, k, i, freqs.bfloat16())),
            (fw.DlrmError, "attention|rope", lambda: fw.qk_norm_rope(q, k, i, freqs[:30])),
            (ValueError, "tokens", lambda: fw.qk_norm_rope(q, k[:5], i, freqs)),
            (TypeError, "k must be", lambda: fw.qk_norm_rope(q, k.bfloat16(), i, freqs)),
            (ValueError, "out_k", lambda: fw.qk_norm_rope(q, None, i, freqs, out_k=k)),
            (ValueError, "out_q", lambda: fw.qk_norm_rope(q, k, i, freqs, out_q=k)),
            (ValueError, "shapes", lambda: fw.qk_norm_rope_grad(q, q, q, k, i, freqs)),
            (ValueError, "unit stride", lambda: fw.attention_packed(q.transpose(1, 2), k, k, off)),
            (ValueError, "same tokens", lambda: fw.attention_packed(q, k, q, off)),
            (ValueError, "q's tokens", lambda: fw.attention_packed(q[:5], k, k, off)),
            (fw.DlrmError, "attention|rope", lambda: fw.attention_packed(q, torch.zeros(6, 3, 64, device="cuda"),
                                                           torch.zeros(6, 3, 64, device="cuda"), off)),
            (fw.DlrmError, "attention|rope", lambda: fw.attention_packed(q, k, k, off[:1])),
            (fw.DlrmError, "attention|rope", lambda: fw.attention_packed(q[:, :, 2:50], k[:, :, 2:50],
                                                           k[:, :, 2:50], off)),
            (ValueError, "lse", lambda: fw.attention_packed(q, k, k, off, lse=lse.T)),
            (ValueError, "q's shape", lambda: fw.attention_packed_grad(q[:5], q, k, k, out, lse, off)),
            (ValueError, "lse", lambda: fw.attention_packed_grad(q, q, k, k, out, lse[:5], off)),
            (TypeError, "workspace", lambda: fw.attention_packed_grad(q, q, k, k, out, lse, off,
                                                                      workspace=freqs)),
            (fw.DlrmError, "attention|rope", lambda: fw.attention_packed_grad(
                q, q, k, k, out, lse, off, workspace=torch.zeros(8, dtype=torch.uint8, device="cuda"))),
            (ValueError, "cache's heads", lambda: fw.kv_cache_write(cache, q, q, i)),
            (TypeError, "uint8", lambda: fw.kv_cache_read(cache._replace(v_codes=freqs), i)),
            (ValueError, "same pages", lambda: fw.kv_cache_read(
                cache._replace(v_scales=cache.v_scales[:3]), i)),
            (TypeError, "out_dtype", lambda: fw.kv_cache_read(cache, i, out_dtype=torch.float16)),
            (ValueError, "dim", lambda: fw.attention_cached(q[:, :, :32], cache, table, i)),
            (ValueError, "table", lambda: fw.attention_cached(q, cache, table[:5], i)),
            (ValueError, "elements", lambda: fw.attention_cached(q, cache, table, i[:5])),
            (TypeError, "table", lambda: fw.attention_cached(q, cache, table.long(), i))):
        with pytest.raises(error, match=match):
            call()


def test_outputs_count_as_modified():
    import torch

    import dlrm_embedding_bag_amd as fw
    q = torch.randn(6, 4, 64, device="cuda")
    off = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(6, 4, device="cuda")
    given = [torch.empty_like(q) for _ in range(3)]
    cache = fw.kv_cache(1, 16, 4, 64)
    slots = torch.arange(6, dtype=torch.int32, device="cuda")
    before = [t._version for t in (out, lse, *given, *cache)]
    fw.attention_packed(q, q, q, off, out=out, lse=lse)
    fw.attention_packed_grad(q, q, q, q, out, lse, off, out_q=given[0], out_k=given[1],
                             out_v=given[2])
    fw.kv_cache_write(cache, q, q, slots)
    assert all(t._version > v for t, v in zip((out, lse, *given, *cache), before))
    x = q.clone().requires_grad_()
    assert not fw.attention_packed(x, x, x, off)[0].requires_grad
