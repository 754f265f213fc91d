"""GPU test of examples/attention_step.py: the attention operators run together
with the token operators as a training step and as serving calls."""
import importlib.util
import os

import pytest

from conftest import ROOT, gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]


def _example():
    spec = importlib.util.spec_from_file_location(
        "attention_step", os.path.join(ROOT, "examples", "attention_step.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _plain_probabilities(model, w, tokens, positions, offsets):
    """The model in float64 on the host, with autograd."""
    import torch
    x = w["table"][tokens.long()] * model.scale
    qkv = (x @ w["qkv"]).view(len(tokens), -1, model.head)
    q, k, v = qkv.split((model.heads, model.kv_heads, model.kv_heads), 1)

    def turned(t, weight):
        t = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6) * weight
        a = positions.double()[:, None, None] * model.freqs.cpu().double()
        lo, hi = t.chunk(2, -1)
        return torch.cat((lo * a.cos() - hi * a.sin(), lo * a.sin() + hi * a.cos()), -1)

    q, k = turned(q, w["q_norm"]), turned(k, w["k_norm"])
    group = model.heads // model.kv_heads
    k, v = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
    a = []
    for b in range(len(offsets) - 1):
        s = slice(offsets[b], offsets[b + 1])
        score = torch.einsum("ihd,jhd->hij", q[s], k[s]) * model.head ** -0.5
        score = score.masked_fill(torch.ones_like(score, dtype=torch.bool).triu(1), -torch.inf)
        a.append(torch.einsum("hij,jhd->ihd", score.softmax(-1), v[s]))
    y = x + torch.cat(a).reshape(len(x), -1) @ w["out"]
    return torch.sigmoid(y @ w["classes"])


def test_gradients_equal_the_formulas_in_64_bits():
    """Eight stages in float32, each a sum of at most 256 terms off by 256 u32 of
    their magnitudes: 2^11 u32 together, of magnitudes that lie within 2^4 of the
    largest gradient."""
    import torch
    ex = _example()
    model = ex.AttentionModel(rows=300, classes=40)
    batch = ex.batch_of(model, 30, 20, 40)
    loss, grads = model.gradients(*batch)
    w = {n: t.detach().cpu().double().requires_grad_() for n, t in model.weights.items()}
    tokens, positions, offsets, target = (t.cpu() for t in batch)
    p = _plain_probabilities(model, w, tokens, positions, offsets.tolist())
    want = torch.nn.functional.binary_cross_entropy(p, target.double())
    want.backward()
    assert abs(loss.item() - want.item()) <= 2.0 ** -13 * want.item()
    assert set(grads) == set(w)
    for name, g in grads.items():
        far = (g.cpu().double() - w[name].grad).abs().max()
        assert far <= 2.0 ** (15 - 24) * w[name].grad.abs().max(), name
    before = {n: t.clone() for n, t in model.weights.items()}
    model.step(*batch, rate=0.5)
    for name, g in grads.items():
        assert torch.equal(model.weights[name], before[name].sub(g, alpha=0.5)), name


@pytest.mark.parametrize("bits", [4, 8])
def test_serving_reads_what_it_wrote(bits):
    """Each call equals attention in 64 bits over the values that the cache holds."""
    import torch

    import dlrm_embedding_bag_amd as fw
    ex = _example()
    model = ex.AttentionModel(rows=300, classes=40)
    batch, longest = 5, 37
    server = ex.Server(model, batch, longest, bits=bits)
    g = torch.Generator(device="cuda").manual_seed(3)
    w = {n: t.cpu().double() for n, t in model.weights.items()}
    for step in range(longest):
        tokens = torch.randint(0, 300, (batch,), generator=g, device="cuda", dtype=torch.int32)
        p = server.next(tokens)
        if step not in (0, 1, 15, 16, 36):
            continue
        at = torch.full((batch,), step, dtype=torch.int32, device="cuda")
        x, _, _, _, qn, _ = model._heads(tokens, at)
        for b in range(batch):
            j = torch.arange(step + 1, device="cuda")
            slots = (server.table[b][j // 16] * 16 + j % 16).to(torch.int32)
            k, v = (t.cpu().double().repeat_interleave(2, 1)
                    for t in fw.kv_cache_read(server.cache, slots, out_dtype=torch.float32))
            s = torch.einsum("hd,jhd->hj", qn[b].cpu().double(), k) * model.head ** -0.5
            a = torch.einsum("hj,jhd->hd", s.softmax(-1), v).reshape(-1)
            y = x[b].cpu().double() + a @ w["out"]
            want = torch.sigmoid(y @ w["classes"])
            # sums of at most 128 terms in three products, and a slope of 1/4
            assert (p[b].cpu().double() - want).abs().max() <= 2.0 ** -14, (step, b)


def test_example_runs(capsys):
    _example().main(3)
    out = capsys.readouterr().out
    assert "step 0: loss" in out and "served (8, 64)" in out
