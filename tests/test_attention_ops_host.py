"""Host checks of the attention operators: the C entry points refuse bad sizes,
types, strides, alignments and pointers before any work is enqueued, their
launches hold fewer than 2^32 threads and none follows one that failed, and the
Python functions refuse tensors that are not what they document.  No GPU needed."""
import os

import pytest

from dlrm_embedding_bag_amd import abi
from test_token_launches_host import launches  # noqa: F401  (a fixture)

FAKE = 0x10000  # never dereferenced: every call below fails validation first
F32, BF16, FP8 = 0, 1, 2
OK, NULL, SHAPE, UNSUPPORTED, WORKSPACE, HIP = 0, 1, 2, 3, 4, 5
INT32_MAX = 2**31 - 1
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(abi.LIB_PATH):
        from dlrm_embedding_bag_amd import build
        build.build()
    return abi.load()


def _rope(n=4, h=4, kv=2, dim=64, dt=F32, q=FAKE, qt=256, qh=64, k=FAKE, kt=128, kh=64, pos=FAKE,
          freqs=FAKE, pairs=32, inter=0, qw=FAKE, kw=None, eps=1e-6, oq=FAKE, oqt=256, oqh=64,
          ok=FAKE, okt=128, okh=64):
    return ["qk_norm_rope", [n, h, kv, dim, dt, q, qt, qh, k, kt, kh, pos, freqs, pairs, inter, qw,
                             kw, eps, oq, oqt, oqh, ok, okt, okh, None]]


def _rope_grad(n=4, h=4, kv=2, dim=64, dt=F32, gq=FAKE, gk=FAKE, q=FAKE, qt=256, k=FAKE, kt=128,
               pos=FAKE, freqs=FAKE, pairs=32, inter=0, eps=1e-6, oq=FAKE, oqt=256, ok=FAKE,
               okt=128, okh=64, dqw=FAKE, dkw=FAKE, ws=FAKE, wsb=1 << 40):
    hd = dim
    return ["qk_norm_rope_grad",
            [n, h, kv, dim, dt, gq, qt, hd, gk, kt, hd, q, qt, hd, k, kt, hd, pos, freqs, pairs,
             inter, FAKE, FAKE, eps, oq, oqt, hd, ok, okt, okh, dqw, dkw, ws, wsb, None]]


def _packed(n=10, m=10, b=2, h=4, kv=2, dim=64, dt=F32, q=FAKE, qt=256, qh=64, k=FAKE, kt=128,
            kh=64, v=FAKE, vt=128, vh=64, off=FAKE, koff=None, causal=1, scale=0.1, fill=0,
            out=FAKE, ot=256, oh=64, lse=FAKE):
    return ["attention_packed", [n, m, b, h, kv, dim, dt, q, qt, qh, k, kt, kh, v, vt, vh, off, koff,
                                 causal, scale, fill, out, ot, oh, lse, None]]


def _packed_grad(n=10, m=10, b=2, h=4, kv=2, dim=64, dt=F32, g=FAKE, gt=256, q=FAKE, qt=256, k=FAKE,
                 kt=128, v=FAKE, vt=128, o=FAKE, lse=FAKE, off=FAKE, koff=None, causal=1, scale=0.1,
                 fill=0, dq=FAKE, dqt=256, dk=FAKE, dkt=128, dv=FAKE, ws=FAKE, wsb=1 << 62):
    d = dim
    return ["attention_packed_grad",
            [n, m, b, h, kv, dim, dt, g, gt, d, q, qt, d, k, kt, d, v, vt, d, o, qt, d, lse, off,
             koff, causal, scale, fill, dq, dqt, d, dk, dkt, d, dv, dkt, d, ws, wsb, None]]


def _write(n=4, h=2, dim=64, dt=F32, k=FAKE, kt=128, kh=64, v=FAKE, slots=FAKE, pages=8, page=16,
           bits=8, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE):
    return ["kv_cache_write", [n, h, dim, dt, k, kt, kh, v, kt, kh, slots, pages, page, bits, kc, ks,
                               vc, vs, None]]


def _read(n=4, h=2, dim=64, dt=F32, k=FAKE, kt=128, kh=64, v=FAKE, slots=FAKE, pages=8, page=16,
          bits=8, kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE):
    return ["kv_cache_read", [n, h, dim, dt, slots, pages, page, bits, kc, ks, vc, vs, k, kt, kh, v,
                              kt, kh, None]]


def _cached(b=4, h=4, kv=2, dim=64, dt=F32, q=FAKE, qt=256, qh=64, pages=8, page=16, bits=8,
            kc=FAKE, ks=FAKE, vc=FAKE, vs=FAKE, table=FAKE, ldt=8, most=8, lengths=FAKE, scale=0.1,
            out=FAKE, ot=256, oh=64, ws=FAKE, wsb=1 << 62):
    return ["attention_cached", [b, h, kv, dim, dt, q, qt, qh, pages, page, bits, kc, ks, vc, vs,
                                 table, ldt, most, lengths, scale, out, ot, oh, ws, wsb, None]]


def _status(lib, call):
    return getattr(lib, call[0])(*call[1])


def test_rope_refusals(lib):
    for bad in (dict(n=-1), dict(n=2**31), dict(h=-1), dict(h=65537), dict(h=0, kv=0),
                dict(kv=65537), dict(dim=0), dict(dim=4), dict(dim=60), dict(dim=264, qh=264),
                dict(dt=FP8), dict(pairs=0), dict(pairs=6), dict(pairs=36), dict(inter=2),
                dict(eps=-1e-9), dict(eps=NAN), dict(eps=INF), dict(qt=-256), dict(kh=-1),
                dict(oqt=255), dict(oqh=63), dict(okt=64), dict(oqt=0), dict(okh=0)):
        assert _status(lib, _rope(**bad)) == SHAPE, bad
    for name in ("q", "k", "pos", "freqs", "oq", "ok"):
        assert _status(lib, _rope(**{name: None})) == NULL, name
    assert _status(lib, _rope(n=0, q=None, k=None, pos=None, freqs=None, oq=None, ok=None)) == OK


def test_rope_gradient_refusals(lib):
    for bad in (dict(n=-1), dict(dim=60), dict(dt=FP8), dict(pairs=2), dict(inter=-1),
                dict(eps=NAN), dict(qt=-1), dict(oqt=255), dict(okt=127), dict(okh=63)):
        assert _status(lib, _rope_grad(**bad)) == SHAPE, bad
    for name in ("gq", "gk", "q", "k", "pos", "freqs", "oq", "ok"):
        assert _status(lib, _rope_grad(**{name: None})) == NULL, name
    need = lib.qk_norm_rope_grad_workspace_bytes(4, 64)
    assert need > 0
    for bad in (dict(ws=None), dict(wsb=need - 1), dict(ws=FAKE + 8)):
        assert _status(lib, _rope_grad(**bad)) == WORKSPACE, bad
    f = lib.qk_norm_rope_grad_workspace_bytes
    assert f(-1, 64) == f(2**31, 64) == f(4, 0) == f(4, 512) == 0
    assert f(INT32_MAX, 256) >= f(5000, 256) >= f(4, 256)
    assert _status(lib, _rope_grad(n=0, gq=None, q=None, pos=None, freqs=None, dqw=None, dkw=None,
                                   ws=None, wsb=0)) == OK


def test_packed_refusals(lib):
    for bad in (dict(n=-1), dict(n=2**31), dict(m=-1), dict(m=9), dict(koff=FAKE, m=2**31),
                dict(b=0), dict(b=INT32_MAX), dict(h=0), dict(h=65538, kv=2), dict(kv=0),
                dict(kv=3), dict(kv=8), dict(dim=0), dict(dim=60), dict(dt=FP8), dict(causal=2),
                dict(scale=0.0), dict(scale=-1.0), dict(scale=NAN), dict(scale=INF), dict(fill=4),
                dict(fill=-1), dict(qt=-256), dict(kh=-64), dict(ot=255), dict(oh=60), dict(ot=0)):
        assert _status(lib, _packed(**bad)) == SHAPE, bad
    for bad in (dict(dim=136, qh=136, ot=544, oh=136), dict(q=FAKE + 4), dict(k=FAKE + 8),
                dict(v=FAKE + 2), dict(out=FAKE + 4), dict(qt=258), dict(kt=130), dict(vh=66),
                dict(ot=258), dict(dt=BF16, kt=132), dict(kt=(1 << 22) + 8), dict(vt=1 << 23),
                dict(qt=1 << 22), dict(ot=1 << 22)):
        assert _status(lib, _packed(**bad)) == UNSUPPORTED, bad
    for name in ("q", "k", "v", "off", "out"):
        assert _status(lib, _packed(**{name: None})) == NULL, name
    assert _status(lib, _packed(n=0, m=0, q=None, k=None, v=None, off=None, out=None)) == OK


def test_packed_gradient_refusals(lib):
    for bad in (dict(n=-1), dict(m=9), dict(b=0), dict(kv=3), dict(dim=60), dict(dt=FP8),
                dict(causal=-1), dict(scale=0.0), dict(fill=8), dict(gt=-8), dict(dqt=255),
                dict(dkt=127)):
        assert _status(lib, _packed_grad(**bad)) == SHAPE, bad
    for bad in (dict(dim=136, dqt=544, dkt=272), dict(g=FAKE + 4), dict(q=FAKE + 8), dict(k=FAKE + 4),
                dict(v=FAKE + 4), dict(o=FAKE + 4), dict(dq=FAKE + 4), dict(dk=FAKE + 8),
                dict(dv=FAKE + 8), dict(gt=258), dict(gt=1 << 23), dict(kt=1 << 23),
                dict(dqt=1 << 22), dict(dkt=1 << 22)):
        assert _status(lib, _packed_grad(**bad)) == UNSUPPORTED, bad
    for name in ("g", "q", "k", "v", "o", "lse", "off", "dq", "dk", "dv"):
        assert _status(lib, _packed_grad(**{name: None})) == NULL, name
    need = lib.attention_packed_grad_workspace_bytes(10, 4)
    assert need > 0
    for bad in (dict(ws=None), dict(wsb=need - 1), dict(ws=FAKE + 8)):
        assert _status(lib, _packed_grad(**bad)) == WORKSPACE, bad
    f = lib.attention_packed_grad_workspace_bytes
    assert f(0, 4) == f(-1, 4) == f(2**31, 4) == f(4, 0) == f(4, 65537) == 0
    assert f(INT32_MAX, 65536) >= 8 * INT32_MAX * 65536


@pytest.mark.parametrize("make", [_write, _read])
def test_cache_refusals(lib, make):
    for bad in (dict(n=-1), dict(n=2**31), dict(dt=FP8), dict(h=0), dict(h=65537), dict(dim=0),
                dict(pages=0), dict(page=0), dict(pages=1 << 27), dict(kt=-1)):
        assert _status(lib, make(**bad)) == SHAPE, bad
    for bad in (dict(bits=5), dict(bits=16), dict(dim=96), dict(dim=256), dict(page=8),
                dict(page=24), dict(page=8192), dict(kc=FAKE + 8), dict(ks=FAKE + 4),
                dict(vc=FAKE + 1), dict(vs=FAKE + 2)):
        assert _status(lib, make(**bad)) == UNSUPPORTED, bad
    for name in ("k", "v", "slots", "kc", "ks", "vc", "vs"):
        assert _status(lib, make(**{name: None})) == NULL, name
    if make is _read:
        assert _status(lib, make(kt=64)) == SHAPE
    assert _status(lib, make(n=0, k=None, v=None, slots=None, kc=None)) == OK


def test_cached_refusals(lib):
    for bad in (dict(b=-1), dict(b=2**31), dict(h=0), dict(kv=0), dict(kv=3), dict(kv=8),
                dict(dt=FP8), dict(most=-1), dict(most=2**31), dict(ldt=-1), dict(scale=0.0),
                dict(scale=NAN), dict(pages=0), dict(pages=1 << 27), dict(qt=-1), dict(ot=255),
                dict(oh=63)):
        assert _status(lib, _cached(**bad)) == SHAPE, bad
    for bad in (dict(bits=2), dict(dim=96), dict(page=48), dict(kc=FAKE + 4), dict(vs=FAKE + 8)):
        assert _status(lib, _cached(**bad)) == UNSUPPORTED, bad
    for name in ("q", "kc", "ks", "vc", "vs", "table", "lengths", "out"):
        assert _status(lib, _cached(**{name: None})) == NULL, name
    f = lib.attention_cached_workspace_bytes
    need = f(4, 4, 2, 64, 1000, 16)
    assert need > 0 and f(4, 4, 2, 64, 1, 16) == 0
    for bad in (dict(ws=None), dict(wsb=need - 1), dict(ws=FAKE + 8)):
        assert _status(lib, _cached(most=1000, ldt=1000, **bad)) == WORKSPACE, bad
    assert f(0, 4, 2, 64, 10, 16) == f(4, 4, 3, 64, 10, 16) == f(4, 4, 2, 96, 10, 16) == 0
    assert f(4, 4, 2, 64, -1, 16) == f(4, 4, 2, 64, 10, 24) == 0
    assert _status(lib, _cached(b=0, q=None, kc=None, table=None, lengths=None, out=None)) == OK


def _made(launches, calls):  # noqa: F811
    for call, (status, made) in zip(calls, launches([[*c, -1] for c in calls])):
        assert status == OK, call
        assert made, call
        for x, y, z, block in made:
            assert 0 < x < 2**32 and 0 < y < 2**32 and 0 < z < 2**32, (call, made)
            assert x * y * z < 2**32 and 0 < block <= 1024, (call, made)


def test_launches_hold_fewer_than_2_to_32_threads(launches):  # noqa: F811
    calls = []
    for n in (1, 1023, 1024, 1 << 20, INT32_MAX):
        for h, kv in ((1, 0), (4, 2), (65536, 65536)):
            for dim, pairs in ((8, 4), (64, 32), (256, 128)):
                t, kt = h * dim, max(kv, 1) * dim
                calls.append(_rope(n=n, h=h, kv=kv, dim=dim, pairs=pairs, qt=t, qh=dim, kt=kt, kh=dim,
                                   oqt=t, oqh=dim, okt=kt, okh=dim))
                calls.append(_rope_grad(n=n, h=h, kv=kv, dim=dim, pairs=pairs, qt=t, kt=kt, oqt=t,
                                        okt=kt, okh=dim))
    for n in (1, 1000, 1 << 24, INT32_MAX):
        for b in (1, 1000, INT32_MAX - 1):
            for h, kv in ((1, 1), (32, 8), (65536, 1), (16384, 16384)):
                for dim in (8, 40, 96, 128):
                    for dt in (F32, BF16):
                        t, kt = h * dim, kv * dim
                        if t <= 1 << 21:
                            calls.append(_packed(n=n, m=n, b=b, h=h, kv=kv, dim=dim, dt=dt, qt=t,
                                                 qh=dim, kt=kt, kh=dim, vt=kt, vh=dim, ot=t, oh=dim))
                            calls.append(_packed_grad(n=n, m=n, b=b, h=h, kv=kv, dim=dim, dt=dt, gt=t,
                                                      qt=t, kt=kt, vt=kt, dqt=t, dkt=kt))
                        else:     # rows of so many heads lie head by head
                            calls.append(_packed(n=n, m=n, b=b, h=h, kv=kv, dim=dim, dt=dt, qt=dim,
                                                 qh=n * dim, kt=dim, kh=n * dim, vt=dim, vh=n * dim,
                                                 ot=dim, oh=n * dim))
    for n in (1, 1000, INT32_MAX):
        for h in (1, 8, 65536):
            for dim in (32, 128):
                calls += [make(n=n, h=h, dim=dim, kt=h * dim, kh=dim, pages=1 << 20)
                          for make in (_write, _read)]
    for b in (1, 64, INT32_MAX):
        for h, kv in ((1, 1), (32, 8), (65536, 1), (65536, 65536)):
            for most in (0, 1, 1000, INT32_MAX):
                calls.append(_cached(b=b, h=h, kv=kv, qt=h * 64, ot=h * 64, most=most, ldt=most))
    _made(launches, calls)


def test_no_launch_after_one_that_failed(launches):  # noqa: F811
    """What follows reads what it should have written."""
    for call in (_rope_grad(n=5000), _packed_grad(), _packed_grad(n=4000, m=4000, b=1),
                 _cached(most=1000, ldt=1000)):
        (status, made), = launches([[*call, -1]])
        assert status == OK and len(made) == 2, call
        for i, (status, first) in enumerate(launches([[*call, i] for i in range(2)])):
            assert status == HIP, (call, i)
            assert first == made[:i + 1], (call, i)


def test_python_refuses_what_is_not_a_gpu_tensor():
    import torch

    import dlrm_embedding_bag_amd as fw
    x = torch.zeros(4, 2, 32)
    i = torch.zeros(4, dtype=torch.int32)
    f = torch.zeros(8)
    cache = fw.KVCache(*(torch.zeros(1, 2, 16, n, dtype=torch.uint8) for n in (32, 1, 32, 1)))
    for call in (lambda: fw.qk_norm_rope(x, x, i, f), lambda: fw.qk_norm_rope_grad(x, x, x, x, i, f),
                 lambda: fw.attention_packed(x, x, x, i),
                 lambda: fw.attention_packed_grad(x, x, x, x, x, x[..., 0], i),
                 lambda: fw.kv_cache_write(cache, x, x, i), lambda: fw.kv_cache_read(cache, i),
                 lambda: fw.attention_cached(x, cache, i[:, None], i)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    for call in (lambda: fw.qk_norm_rope(x.half(), None, i, f), lambda: fw.attention_packed(1, x, x, i),
                 lambda: fw.kv_cache_write(cache, x.int(), x, i)):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(ValueError):
        fw.kv_cache(4, 16, 2, 96)
    with pytest.raises(ValueError):
        fw.kv_cache(4, 16, 2, 64, bits=6)
