"""Attention operators: norm and rotation of query and key heads and attention
over packed sequences, with their gradients; a paged cache of keys and values in
8 or 4 bits, and attention of single tokens over it.

Argument marshalling only, as in token_ops.py: every function has the name of
the C entry point it calls (include/dlrm_embedding_bag.h says what it computes),
checks its tensors, allocates the outputs and workspace that it is not given on
the stream the call runs on, and raises on refusal.  There is no CPU path, and
no graph is recorded for autograd: the gradients are calls of their own.  A
tensor given as an output counts as modified in place.

Queries, keys and values are (tokens, heads, dim) tensors whose heads are
contiguous; tokens and heads may have any stride, so slices of a joint product
and transposed views go in as they are.
"""
from __future__ import annotations

from typing import Any, NamedTuple

from .abi import _check, load
from .token_ops import _CODES, _INT_MAX, _device, _handle, _on, _torch, _vector
from .token_ops import _new as _new_flat


def _heads(torch, t, what, dtype, dev):
    """(rows, heads, dim, row stride, head stride) of a (rows, heads, dim)
    tensor with unit stride within a head.  A dimension of one element has
    whatever stride it was made with, which no access uses."""
    _on(torch, t, what, dev)
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype} (got {t.dtype})")
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or (stride[2] != 1 and shape[2] != 1):
        raise ValueError(f"{what} must be (rows, heads, dim) with unit stride within a head")
    n, h, d = shape
    if n > _INT_MAX or h > _INT_MAX or d > _INT_MAX:
        raise ValueError(f"{what} has a dimension above {_INT_MAX}")
    sh = stride[1] if h > 1 else max(d, 1)
    return n, h, d, stride[0] if n > 1 else max(h, 1) * sh, sh


def _dtype_of(torch, t, what):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a torch.Tensor")
    if t.dtype is not torch.float32 and t.dtype is not torch.bfloat16:
        raise TypeError(f"{what} must be torch.float32 or torch.bfloat16 (got {t.dtype})")
    return t.dtype


def _new(torch, shape, like, stream, dtype):
    """A new contiguous tensor."""
    if len(shape) < 3:
        return _new_flat(torch, shape, like, stream, dtype)
    if stream is None:
        return torch.empty_strided(shape, (shape[1] * shape[2], shape[2], 1), dtype=dtype,
                                   device=like.device)
    return _new_flat(torch, (shape[0], shape[1] * shape[2]), like, stream, dtype).view(shape)


def _rows_out(torch, out, what, shape, like, stream, dtype, dev):
    """An output of (rows, heads, dim), new if it is not given: it, its strides."""
    if out is None:
        return _new(torch, shape, like, stream, dtype), shape[1] * shape[2], shape[2]
    n, h, d, st, sh = _heads(torch, out, what, dtype, dev)
    if (n, h, d) != tuple(shape):
        raise ValueError(f"{what} must be {tuple(shape)}")
    return out, st, sh


def _ints(torch, t, what, n, dev):
    _on(torch, t, what, dev)
    if t.dtype is not torch.int32:
        raise TypeError(f"{what} must be torch.int32 (got {t.dtype})")
    if not t.is_contiguous() or (n is not None and t.numel() != n):
        raise ValueError(f"{what} must be contiguous" + ("" if n is None else f" with {n} elements"))
    return t.data_ptr()


def _mark(torch, given):
    given = [t for t in given if t is not None]
    if given:
        torch.autograd.graph.increment_version(given)


def _scratch(torch, workspace, size, like, stream, dev):
    """The workspace of a call: (pointer, bytes) and the tensor that holds it."""
    if workspace is None:
        if not size:
            return None, 0, None
        workspace = _new(torch, (size,), like, stream, torch.uint8)
    else:
        _on(torch, workspace, "workspace", dev)
        if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise TypeError("workspace must be a contiguous uint8 tensor")
    return workspace.data_ptr(), workspace.numel(), workspace


def _sides(torch, q, k, dtype, dev, names=("q", "k")):
    """Pointer and strides of queries and keys (None: no heads), their tokens,
    heads, key heads and dim."""
    out, n, heads, dim = [], None, [0, 0], None
    for i, t in enumerate((q, k)):
        if t is None:
            out.append((None, 0, 0))
            continue
        m, h, d, st, sh = _heads(torch, t, names[i], dtype, dev)
        if n is not None and (m != n or d != dim):
            raise ValueError(f"{names[1]} must have {names[0]}'s tokens and dim")
        n, dim, heads[i] = m, d, h
        out.append((t.data_ptr(), st, sh))
    return out[0], out[1], n, heads[0], heads[1], dim


def qk_norm_rope(q, k, positions, freqs, q_weight=None, k_weight=None, eps=1e-6,
                 interleaved=False, out_q=None, out_k=None, stream=None):
    """(q, k) of (tokens, heads, dim) with each head's row normed by its RMS,
    times weight, and its pairs turned by positions * freqs: int32 (tokens,),
    float32 (pairs,).  Pairs are elements (i, i + pairs), or (2i, 2i + 1) if
    interleaved; elements from 2 * pairs on are only normed.  k may be None.
    out_q and out_k may be q and k themselves."""
    torch = _torch()
    lib = load()
    dtype = _dtype_of(torch, q, "q")
    dev = _device(torch, q, "q")
    qr, kr, n, heads, kv_heads, dim = _sides(torch, q, k, dtype, dev)
    pos = _ints(torch, positions, "positions", n, dev)
    pairs = freqs.numel() if isinstance(freqs, torch.Tensor) else 0
    fp = _vector(torch, freqs, "freqs", pairs, dev)
    qw = None if q_weight is None else _vector(torch, q_weight, "q_weight", dim, dev)
    kw = None if k_weight is None else _vector(torch, k_weight, "k_weight", dim, dev)
    given = (out_q, out_k)
    out_q, oqt, oqh = _rows_out(torch, out_q, "out_q", (n, heads, dim), q, stream, dtype, dev)
    okp, okt, okh = None, 0, 0
    if k is None:
        if out_k is not None:
            raise ValueError("out_k needs k")
    else:
        out_k, okt, okh = _rows_out(torch, out_k, "out_k", (n, kv_heads, dim), q, stream, dtype,
                                    dev)
        okp = out_k.data_ptr()
    status = lib.qk_norm_rope(n, heads, kv_heads, dim, _CODES[dtype], *qr, *kr, pos, fp, pairs,
                              1 if interleaved else 0, qw, kw, eps, out_q.data_ptr(), oqt, oqh,
                              okp, okt, okh, _handle(torch, stream, dev))
    if status:
        _check(status, "qk_norm_rope")
    _mark(torch, given)
    return out_q, out_k


def qk_norm_rope_grad_workspace_bytes(tokens, dim):
    """Bytes of workspace that qk_norm_rope_grad takes for these sizes."""
    return load().qk_norm_rope_grad_workspace_bytes(tokens, min(dim, _INT_MAX))


def qk_norm_rope_grad(grad_q, grad_k, q, k, positions, freqs, q_weight=None, k_weight=None,
                      eps=1e-6, interleaved=False, out_q=None, out_k=None, workspace=None,
                      stream=None):
    """Gradients of qk_norm_rope: (of q, of k, of q_weight, of k_weight) from
    those of its outputs and its inputs; None for what it was not given.
    `workspace` is a uint8 tensor of at least qk_norm_rope_grad_workspace_bytes;
    without it one is allocated for the call."""
    torch = _torch()
    lib = load()
    dtype = _dtype_of(torch, q, "q")
    dev = _device(torch, q, "q")
    qr, kr, n, heads, kv_heads, dim = _sides(torch, q, k, dtype, dev)
    gq, gk, gn, gheads, gkv, gdim = _sides(torch, grad_q, grad_k, dtype, dev,
                                           ("grad_q", "grad_k"))
    if (gn, gheads, gkv, gdim) != (n, heads, kv_heads, dim):
        raise ValueError("grad_q and grad_k must have the shapes of q and k")
    pos = _ints(torch, positions, "positions", n, dev)
    pairs = freqs.numel() if isinstance(freqs, torch.Tensor) else 0
    fp = _vector(torch, freqs, "freqs", pairs, dev)
    qw = kw = dqw = dkw = dqp = dkp = None
    given = (out_q, out_k)
    if q_weight is not None:
        qw = _vector(torch, q_weight, "q_weight", dim, dev)
        dqw = _new(torch, (dim,), q, stream, torch.float32)
        dqp = dqw.data_ptr()
    if k_weight is not None and k is not None:
        kw = _vector(torch, k_weight, "k_weight", dim, dev)
        dkw = _new(torch, (dim,), q, stream, torch.float32)
        dkp = dkw.data_ptr()
    out_q, oqt, oqh = _rows_out(torch, out_q, "out_q", (n, heads, dim), q, stream, dtype, dev)
    okp, okt, okh = None, 0, 0
    if k is None:
        if out_k is not None:
            raise ValueError("out_k needs k")
    else:
        out_k, okt, okh = _rows_out(torch, out_k, "out_k", (n, kv_heads, dim), q, stream, dtype,
                                    dev)
        okp = out_k.data_ptr()
    size = lib.qk_norm_rope_grad_workspace_bytes(n, dim) if dqp or dkp else 0
    ws, size, _hold = _scratch(torch, workspace, size, q, stream, dev)
    status = lib.qk_norm_rope_grad(n, heads, kv_heads, dim, _CODES[dtype], *gq, *gk, *qr, *kr, pos,
                                   fp, pairs, 1 if interleaved else 0, qw, kw, eps,
                                   out_q.data_ptr(), oqt, oqh, okp, okt, okh, dqp, dkp, ws, size,
                                   _handle(torch, stream, dev))
    if status:
        _check(status, "qk_norm_rope_grad")
    _mark(torch, given)
    return out_q, out_k, dqw, dkw


def _packed(torch, q, k, v, offsets, kv_offsets, scale, dev, dtype):
    """What the packed calls share: the leading arguments of the C call, the
    pointers and strides of q, k and v, and the offsets."""
    n, heads, dim, qt, qh = _heads(torch, q, "q", dtype, dev)
    m, kv_heads, kdim, kt, kh = _heads(torch, k, "k", dtype, dev)
    vm, vh, vdim, vt, vhs = _heads(torch, v, "v", dtype, dev)
    if kdim != dim or vdim != dim or vm != m or vh != kv_heads:
        raise ValueError("k and v must have the same tokens and heads, and q's dim")
    off = _ints(torch, offsets, "offsets", None, dev)
    batch = offsets.numel() - 1
    if kv_offsets is None:
        if m != n:
            raise ValueError("without kv_offsets, k and v must have q's tokens")
        koff = None
    else:
        koff = _ints(torch, kv_offsets, "kv_offsets", batch + 1, dev)
    if scale is None:
        scale = dim ** -0.5 if dim else 1.0
    return ((n, m, batch, heads, kv_heads, dim, _CODES[dtype]),
            (q.data_ptr(), qt, qh, k.data_ptr(), kt, kh, v.data_ptr(), vt, vhs), off, koff, scale)


def attention_packed(q, k, v, offsets, kv_offsets=None, causal=True, scale=None, out=None,
                     lse=None, stream=None):
    """(out, lse) of attention over packed sequences: sequence b holds rows
    offsets[b]:offsets[b + 1] of q and kv_offsets[b]:kv_offsets[b + 1] of k and v
    (offsets again without kv_offsets); both int32 (sequences + 1,).  Heads of q
    share those of k and v in equal groups.  With causal a sequence's last query
    sees all its keys, the one before it all but the last.  `scale` is
    dim ** -0.5 unless given.  lse, (tokens, heads) float32, is what the gradient
    needs.  Rows outside all sequences are 0 (and -inf in lse) in new tensors,
    and left as they are in given ones."""
    torch = _torch()
    lib = load()
    dtype = _dtype_of(torch, q, "q")
    dev = _device(torch, q, "q")
    sizes, rows, off, koff, scale = _packed(torch, q, k, v, offsets, kv_offsets, scale, dev, dtype)
    given = (out, lse)
    fill = (1 if out is None else 0) | (2 if lse is None else 0)
    n, heads, dim = sizes[0], sizes[3], sizes[5]
    out, ot, oh = _rows_out(torch, out, "out", (n, heads, dim), q, stream, dtype, dev)
    if lse is None:
        lse = _new(torch, (n, heads), q, stream, torch.float32)
    else:
        _on(torch, lse, "lse", dev)
        if lse.shape != (n, heads):
            raise ValueError("lse must be (tokens, heads)")
    status = lib.attention_packed(*sizes, *rows, off, koff, 1 if causal else 0, scale, fill,
                                  out.data_ptr(), ot, oh,
                                  _vector(torch, lse, "lse", n * heads, dev),
                                  _handle(torch, stream, dev))
    if status:
        _check(status, "attention_packed")
    _mark(torch, given)
    return out, lse


def attention_packed_grad_workspace_bytes(tokens, heads):
    """Bytes of workspace that attention_packed_grad takes for these sizes."""
    return load().attention_packed_grad_workspace_bytes(tokens, min(heads, _INT_MAX))


def attention_packed_grad(grad, q, k, v, out, lse, offsets, kv_offsets=None, causal=True,
                          scale=None, out_q=None, out_k=None, out_v=None, workspace=None,
                          stream=None):
    """Gradients (of q, of k, of v) of attention_packed's out, from that of out,
    its inputs and both its outputs.  Rows outside all sequences are 0 in new
    tensors and left as they are in given ones.  `workspace` is a uint8 tensor of
    at least attention_packed_grad_workspace_bytes; without it one is allocated
    for the call."""
    torch = _torch()
    lib = load()
    dtype = _dtype_of(torch, q, "q")
    dev = _device(torch, q, "q")
    sizes, rows, off, koff, scale = _packed(torch, q, k, v, offsets, kv_offsets, scale, dev, dtype)
    n, m, _, heads, kv_heads, dim, _ = sizes
    gn, gh, gd, gt, ghs = _heads(torch, grad, "grad", dtype, dev)
    on, oh, od, ot, ohs = _heads(torch, out, "out", dtype, dev)
    if (gn, gh, gd) != (n, heads, dim) or (on, oh, od) != (n, heads, dim):
        raise ValueError("grad and out must have q's shape")
    if not isinstance(lse, torch.Tensor) or lse.shape != (n, heads):
        raise ValueError("lse must be (tokens, heads)")
    lp = _vector(torch, lse, "lse", n * heads, dev)
    given = (out_q, out_k, out_v)
    fill = sum(1 << i for i, t in enumerate(given) if t is None)
    out_q, qt, qh = _rows_out(torch, out_q, "out_q", (n, heads, dim), q, stream, dtype, dev)
    out_k, kt, kh = _rows_out(torch, out_k, "out_k", (m, kv_heads, dim), q, stream, dtype, dev)
    out_v, vt, vh = _rows_out(torch, out_v, "out_v", (m, kv_heads, dim), q, stream, dtype, dev)
    size = lib.attention_packed_grad_workspace_bytes(n, heads)
    ws, size, _hold = _scratch(torch, workspace, size, q, stream, dev)
    status = lib.attention_packed_grad(*sizes, grad.data_ptr(), gt, ghs, *rows, out.data_ptr(), ot,
                                       ohs, lp, off, koff, 1 if causal else 0, scale, fill,
                                       out_q.data_ptr(), qt, qh, out_k.data_ptr(), kt, kh,
                                       out_v.data_ptr(), vt, vh, ws, size,
                                       _handle(torch, stream, dev))
    if status:
        _check(status, "attention_packed_grad")
    _mark(torch, given)
    return out_q, out_k, out_v


class KVCache(NamedTuple):
    """A paged cache's uint8 tensors: codes (pages, heads, page, dim * bits / 8)
    and scales (pages, heads, page, dim / 32) of keys and of values."""
    k_codes: Any
    k_scales: Any
    v_codes: Any
    v_scales: Any


def kv_cache(pages, page, heads, dim, bits=8, device=None):
    """A new KVCache of `pages` pages of `page` rows on `device` (the current
    GPU), all of it zeros."""
    torch = _torch()
    if bits not in (4, 8) or dim not in (32, 64, 128):
        raise ValueError("bits must be 4 or 8, and dim 32, 64 or 128")
    if device is None:
        device = torch.device("cuda", torch.cuda.current_device())
    return KVCache(*(torch.zeros((pages, heads, page, n), dtype=torch.uint8, device=device)
                     for n in (dim * bits // 8, dim // 32) * 2))


def _cache(torch, cache, dev):
    """pages, page, bits and pointers of a cache, its heads and dim."""
    kc, ks, vc, vs = cache
    u8 = torch.uint8
    for i, t in enumerate((kc, ks, vc, vs)):
        if not isinstance(t, torch.Tensor) or t.get_device() != dev:
            _on(torch, t, KVCache._fields[i], dev)
        if t.dtype is not u8:
            raise TypeError(f"{KVCache._fields[i]} must be torch.uint8 (got {t.dtype})")
        if not t.is_contiguous():
            raise ValueError(f"{KVCache._fields[i]} must be contiguous (pages, heads, page, bytes)")
    codes, scales = kc.shape, ks.shape
    if len(codes) != 4 or len(scales) != 4:
        raise ValueError("codes and scales must be (pages, heads, page, bytes)")
    pages, heads, page, row = codes
    if vc.shape != codes or vs.shape != scales or scales != (pages, heads, page, scales[3]):
        raise ValueError("codes and scales of keys and values must have the same pages, heads, "
                         "page and dim")
    dim = scales[3] * 32
    if row == dim and dim:
        bits = 8
    elif row * 2 == dim and dim:
        bits = 4
    else:
        raise ValueError("codes must have 32 or 16 bytes for each byte of the scales")
    if pages > _INT_MAX or heads > _INT_MAX or page > _INT_MAX or dim > _INT_MAX:
        raise ValueError(f"the cache has a dimension above {_INT_MAX}")
    return (pages, page, bits, kc.data_ptr(), ks.data_ptr(), vc.data_ptr(), vs.data_ptr()), heads, dim


def kv_cache_write(cache, k, v, slots, stream=None):
    """Token t's keys and values, (tokens, heads, dim) float32 or bfloat16, into
    row slots[t] of the cache, int32: row slot % page of page slot // page.
    Tokens whose slot is outside the cache are not written."""
    torch = _torch()
    lib = load()
    dtype = _dtype_of(torch, k, "k")
    dev = _device(torch, k, "k")
    n, heads, dim, kt, kh = _heads(torch, k, "k", dtype, dev)
    vn, vh, vd, vt, vhs = _heads(torch, v, "v", dtype, dev)
    places, cheads, cdim = _cache(torch, cache, dev)
    if (vn, vh, vd) != (n, heads, dim) or (cheads, cdim) != (heads, dim):
        raise ValueError("k and v must have the same shape, and the cache's heads and dim")
    status = lib.kv_cache_write(n, heads, dim, _CODES[dtype], k.data_ptr(), kt, kh, v.data_ptr(),
                                vt, vhs, _ints(torch, slots, "slots", n, dev), *places,
                                _handle(torch, stream, dev))
    if status:
        _check(status, "kv_cache_write")
    _mark(torch, cache)


def kv_cache_read(cache, slots, out_dtype=None, out_k=None, out_v=None, stream=None):
    """(k, v): the values that the cache's rows slots[t] stand for, as (tokens,
    heads, dim) of out_dtype (bfloat16 unless given; float32); zeros for a slot
    outside the cache."""
    torch = _torch()
    lib = load()
    dev = _device(torch, cache[0], "k_codes")
    places, heads, dim = _cache(torch, cache, dev)
    pos = _ints(torch, slots, "slots", None, dev)
    n = slots.numel()
    given = (out_k, out_v)
    for t in given:
        if t is not None and out_dtype is None:
            out_dtype = _dtype_of(torch, t, "out_k or out_v")
    if out_dtype is None:
        out_dtype = torch.bfloat16
    if out_dtype is not torch.float32 and out_dtype is not torch.bfloat16:
        raise TypeError(f"out_dtype must be torch.float32 or torch.bfloat16 (got {out_dtype})")
    out_k, kt, kh = _rows_out(torch, out_k, "out_k", (n, heads, dim), cache[0], stream, out_dtype,
                              dev)
    out_v, vt, vh = _rows_out(torch, out_v, "out_v", (n, heads, dim), cache[0], stream, out_dtype,
                              dev)
    status = lib.kv_cache_read(n, heads, dim, _CODES[out_dtype], pos, *places, out_k.data_ptr(), kt,
                               kh, out_v.data_ptr(), vt, vh, _handle(torch, stream, dev))
    if status:
        _check(status, "kv_cache_read")
    _mark(torch, given)
    return out_k, out_v


def attention_cached_workspace_bytes(batch, heads, kv_heads, dim, max_pages, page):
    """Bytes of workspace that attention_cached takes for these sizes."""
    return load().attention_cached_workspace_bytes(batch, min(heads, _INT_MAX),
                                                   min(kv_heads, _INT_MAX), min(dim, _INT_MAX),
                                                   max_pages, min(page, _INT_MAX))


def attention_cached(q, cache, table, lengths, scale=None, out=None, workspace=None, stream=None):
    """Attention of one query for each sequence, q (batch, heads, dim), over its
    first lengths[b] keys and values in the cache: key j lies in row j % page of
    page table[b, j // page].  table is int32 (batch, max_pages), lengths int32
    (batch,); heads of q share those of the cache in equal groups.  `scale` is
    dim ** -0.5 unless given.  `workspace` is a uint8 tensor of at least
    attention_cached_workspace_bytes; without it one is allocated for the call."""
    torch = _torch()
    lib = load()
    dtype = _dtype_of(torch, q, "q")
    dev = _device(torch, q, "q")
    n, heads, dim, qt, qh = _heads(torch, q, "q", dtype, dev)
    places, kv_heads, cdim = _cache(torch, cache, dev)
    if cdim != dim:
        raise ValueError("q must have the cache's dim")
    _on(torch, table, "table", dev)
    if table.dtype is not torch.int32:
        raise TypeError(f"table must be torch.int32 (got {table.dtype})")
    if table.dim() != 2 or table.shape[0] != n or (table.shape[1] > 1 and table.stride(1) != 1):
        raise ValueError("table must be (batch, max_pages) with unit column stride")
    most = table.shape[1]
    if most > _INT_MAX:
        raise ValueError(f"table has more than {_INT_MAX} columns")
    lp = _ints(torch, lengths, "lengths", n, dev)
    if scale is None:
        scale = dim ** -0.5
    given = (out,)
    out, ot, oh = _rows_out(torch, out, "out", (n, heads, dim), q, stream, dtype, dev)
    size = lib.attention_cached_workspace_bytes(n, heads, kv_heads, dim, most, places[1])
    ws, size, _hold = _scratch(torch, workspace, size, q, stream, dev)
    status = lib.attention_cached(n, heads, kv_heads, dim, _CODES[dtype], q.data_ptr(), qt, qh,
                                  *places, table.data_ptr(), table.stride(0) if n > 1 else most,
                                  most, lp, scale, out.data_ptr(), ot, oh, ws, size,
                                  _handle(torch, stream, dev))
    if status:
        _check(status, "attention_cached")
    _mark(torch, given)
    return out
