"""Host checks of the token operators: the C entry points refuse bad sizes,
types, strides and pointers before any work is enqueued, and the Python
functions refuse tensors that are not what they document.  No GPU needed."""
import os

import pytest

from dlrm_embedding_bag_amd import abi

FAKE = 0x10000  # never dereferenced: every call below fails validation first
F32, BF16, FP8 = 0, 1, 2
OK, NULL, SHAPE, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(abi.LIB_PATH):
        from dlrm_embedding_bag_amd import build
        build.build()
    return abi.load()


def _lookup(lib, n=4, rows=10, dim=8, table=FAKE, ldt=8, tdt=F32, tok=FAKE, out=FAKE, ldo=8,
            odt=F32):
    return lib.emb_lookup_scaled(n, rows, dim, table, ldt, tdt, tok, 1.0, out, ldo, odt, None)


def test_lookup_refusals(lib):
    assert _lookup(lib, n=-1) == SHAPE
    assert _lookup(lib, n=2**31) == SHAPE
    assert _lookup(lib, rows=0) == SHAPE
    assert _lookup(lib, rows=2**31 - 1) == SHAPE
    assert _lookup(lib, dim=0) == SHAPE
    assert _lookup(lib, dim=(1 << 20) + 1, ldt=1 << 21, ldo=1 << 21) == SHAPE
    assert _lookup(lib, tdt=3) == SHAPE
    assert _lookup(lib, odt=FP8) == SHAPE
    assert _lookup(lib, ldt=7) == SHAPE
    assert _lookup(lib, ldt=-8) == SHAPE
    assert _lookup(lib, ldo=7) == SHAPE
    assert _lookup(lib, ldo=0) == SHAPE
    assert _lookup(lib, table=None) == NULL
    assert _lookup(lib, tok=None) == NULL
    assert _lookup(lib, out=None) == NULL
    assert _lookup(lib, n=0, table=None, tok=None, out=None) == OK


def _grad(lib, n=4, rows=10, dim=8, grad=FAKE, ldg=8, gdt=F32, tok=FAKE, acc=0, out=FAKE, ldo=8,
          odt=F32, ws=FAKE, wsb=1 << 30):
    return lib.emb_lookup_grad(n, rows, dim, grad, ldg, gdt, tok, 1.0, acc, out, ldo, odt, ws,
                               wsb, None)


def test_grad_refusals(lib):
    assert _grad(lib, n=-1) == SHAPE
    assert _grad(lib, n=2**31) == SHAPE
    assert _grad(lib, rows=0) == SHAPE
    assert _grad(lib, dim=0) == SHAPE
    assert _grad(lib, gdt=FP8) == SHAPE
    assert _grad(lib, odt=FP8) == SHAPE
    assert _grad(lib, ldg=7) == SHAPE
    assert _grad(lib, ldo=0) == SHAPE
    assert _grad(lib, acc=2) == SHAPE
    assert _grad(lib, grad=None) == NULL
    assert _grad(lib, tok=None) == NULL
    assert _grad(lib, out=None) == NULL
    n = 100000
    need = lib.emb_lookup_grad_workspace_bytes(n, 10, 8)
    assert need > 0
    assert _grad(lib, n=n, ws=None) == WORKSPACE
    assert _grad(lib, n=n, wsb=need - 1) == WORKSPACE
    assert _grad(lib, n=n, ws=FAKE + 8) == WORKSPACE
    # no tokens and nothing to write
    assert _grad(lib, n=0, acc=1, grad=None, tok=None, out=None, ws=None, wsb=0) == OK


def test_grad_workspace_sizes(lib):
    f = lib.emb_lookup_grad_workspace_bytes
    assert f(0, 10, 8) == 0
    assert f(-1, 10, 8) == 0
    assert f(4, 0, 8) == 0
    assert f(4, 10, 0) == 0
    last = 0
    for n in (1, 100, 4096, 4097, 100000, 3 << 20, 1 << 28):
        assert f(n, 1000, 64) >= last
        last = f(n, 1000, 64)
    # the sorted copies of the tokens and their positions at least
    assert f(1 << 28, 1000, 64) >= 16 << 28


def _norm(lib, m=4, dim=8, x=FAKE, ldx=8, r=FAKE, ldr=8, dt=F32, w=FAKE, eps=1e-6, h=FAKE, ldh=8,
          q=FAKE, ldq=8, s=FAKE):
    return lib.rms_norm_residual_i8(m, dim, x, ldx, r, ldr, dt, w, eps, h, ldh, q, ldq, s, None)


def test_norm_refusals(lib):
    assert _norm(lib, m=-1) == SHAPE
    assert _norm(lib, dim=0) == SHAPE
    assert _norm(lib, dim=(1 << 20) + 1) == SHAPE
    assert _norm(lib, dt=FP8) == SHAPE
    for eps in (-1e-9, float("nan"), float("inf")):
        assert _norm(lib, eps=eps) == SHAPE
    assert _norm(lib, ldx=7) == SHAPE
    assert _norm(lib, ldr=7) == SHAPE
    assert _norm(lib, ldh=0) == SHAPE
    assert _norm(lib, ldq=7) == SHAPE
    assert _norm(lib, x=None) == NULL
    assert _norm(lib, h=None) == NULL
    assert _norm(lib, q=None) == NULL
    assert _norm(lib, s=None) == NULL
    assert _norm(lib, m=0, x=None, r=None, h=None, q=None, s=None) == OK


def _linear(lib, m=4, n=8, k=16, a=FAKE, lda=16, s=FAKE, w=FAKE, ldw=16, ws=FAKE, b=None, act=0,
            c=FAKE, ldc=8, odt=F32):
    return lib.linear_i8_bias_act(m, n, k, a, lda, s, w, ldw, ws, b, act, c, ldc, odt, None)


def test_linear_refusals(lib):
    assert _linear(lib, m=-1) == SHAPE
    assert _linear(lib, n=0) == SHAPE
    assert _linear(lib, k=0) == SHAPE
    assert _linear(lib, act=3) == SHAPE
    assert _linear(lib, odt=FP8) == SHAPE
    assert _linear(lib, lda=15) == SHAPE
    assert _linear(lib, ldw=15) == SHAPE
    assert _linear(lib, ldw=0) == SHAPE
    assert _linear(lib, ldc=7) == SHAPE
    assert _linear(lib, k=131072, lda=131072, ldw=131072) == UNSUPPORTED
    assert _linear(lib, m=(1 << 26) + 1) == UNSUPPORTED
    assert _linear(lib, n=(1 << 26) + 1, ldc=(1 << 26) + 1) == UNSUPPORTED
    for name in ("a", "s", "w", "ws", "c"):
        assert _linear(lib, **{name: None}) == NULL
    assert _linear(lib, m=0, a=None, s=None, w=None, ws=None, c=None) == OK


def test_python_refuses_what_is_not_a_gpu_tensor():
    import torch

    import dlrm_embedding_bag_amd as fw
    x = torch.zeros(4, 8)
    t = torch.zeros(4, dtype=torch.int32)
    q = torch.zeros(4, 8, dtype=torch.int8)
    s = torch.zeros(4)
    with pytest.raises(ValueError, match="GPU tensor"):
        fw.emb_lookup_scaled(x, t)
    with pytest.raises(ValueError, match="GPU tensor"):
        fw.emb_lookup_grad(x, t, 10)
    with pytest.raises(ValueError, match="GPU tensor"):
        fw.rms_norm_residual_i8(x)
    with pytest.raises(ValueError, match="GPU tensor"):
        fw.linear_i8_bias_act(q, s, q, s)
    with pytest.raises(TypeError):
        fw.emb_lookup_scaled([1.0], t)
    with pytest.raises(TypeError):
        fw.rms_norm_residual_i8(None)
