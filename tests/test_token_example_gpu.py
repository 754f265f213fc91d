"""GPU test of examples/token_step.py: the token operators run together as a
training step and as a serving call."""
import importlib.util
import os

import pytest

from conftest import ROOT, gpu_available

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not gpu_available(), reason="needs an MI355X GPU")]


def _example():
    spec = importlib.util.spec_from_file_location(
        "token_step", os.path.join(ROOT, "examples", "token_step.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_step_learns_and_touches_the_named_rows_only():
    import torch
    ex = _example()
    model = ex.HistoryModel(rows=3000, dim=72, length=9, classes=40)
    tokens, target = ex.batch_of(model, 64)
    before = model.table.clone()
    losses = [model.step(tokens, target, rate=1000.0).item() for _ in range(20)]
    assert losses[-1] < 0.8 * losses[0], losses
    named = torch.zeros(model.rows, dtype=torch.bool, device="cuda")
    named[tokens[tokens >= 0].long()] = True
    assert torch.equal(model.table[~named], before[~named])
    assert not torch.equal(model.table[named], before[named])


def test_step_equals_the_formulas_in_64_bits():
    """One step against the same step in float64 from the same codes' inputs:
    the update of a row is a sum of c terms in float32 whose rows were computed
    in float32 over dim and classes terms, each at most u of the magnitudes."""
    import torch
    ex = _example()
    model = ex.HistoryModel(rows=200, dim=40, length=6, classes=24, seed=3)
    tokens, target = ex.batch_of(model, 32, seed=4)
    p, h = model.forward(tokens)
    w = (model.w8.double() * model.w_scale.double()[:, None]).cpu()
    dy = ((p - target).double().cpu() / p.numel()) @ w * model.weight.double().cpu()
    h64 = h.double().cpu()
    r = 1.0 / torch.sqrt((h64 * h64).mean(1, keepdim=True) + ex.EPS)
    # d/dh of h r(h): r dy - h r^3 mean(h dy)
    want = r * dy - h64 * r ** 3 * (h64 * dy).mean(1, keepdim=True)
    table = model.table.double().cpu()
    flat = tokens.view(-1).long().cpu()
    there = flat >= 0
    rate = 100.0
    change = torch.zeros_like(table).index_add_(0, flat[there], want[there] * -rate * model.scale)
    size = torch.zeros_like(table).index_add_(0, flat[there],
                                              want[there].abs() * rate * model.scale)
    model.step(tokens, target, rate)
    u = 2.0 ** -24
    # each gradient element: sums over 24 classes and 40 columns of terms of
    # the row's own size; the row's largest element stands for their magnitude
    row = size.amax(1, keepdim=True)
    tol = row * (24 + 40 + 32 * 6) * 8 * u + table.abs() * 2 * u
    err = (model.table.double().cpu() - (table + change)).abs()
    assert (err <= tol).all(), (err / tol.clamp_min(1e-300)).max()


def test_serving_equals_the_first_position_of_the_forward():
    import torch
    ex = _example()
    model = ex.HistoryModel(rows=500, dim=64, length=4, classes=32)
    tokens, _ = ex.batch_of(model, 16)
    p, _ = model.forward(tokens)
    got = model.serve(tokens[:, 0].contiguous(), 0)
    assert torch.equal(got, p.view(16, 4, -1)[:, 0])
