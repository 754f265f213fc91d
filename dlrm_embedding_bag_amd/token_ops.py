"""Token operators: embedding lookup with a scale and its gradient, RMS norm
to int8 codes, and the int8 product with a scale for each token and channel.

Argument marshalling only, as in abi.py: every function has the name of the C
entry point it calls (include/dlrm_embedding_bag.h says what it computes),
checks its tensors, allocates the outputs and workspace that it is not given
on the stream the call runs on, and raises on refusal.  There is no CPU path.

They work on the tensors' memory and record no graph for autograd: an output
does not require a gradient, whatever the inputs do, and a table's gradient is
what emb_lookup_grad gives for the rows' gradient.  A tensor given as an output
counts as modified in place, so autograd refuses to use a value of it that was
saved before.
"""
from __future__ import annotations

from .abi import ACTS, _check, _empty, load

# One call of a short operator is as long as its marshalling, so each tensor's
# shape and strides are read once, the device is asked for once a call, and the
# current stream is taken as the raw handle that the C entry point wants.
_CODES = {}    # torch dtype -> dlrm_dtype, filled on the first call (torch is imported late)
_MODULE = None
_FLOATS = ()   # float32, bfloat16
_TABLES = ()   # and the table's FP8
_INT8 = ()
_INT_MAX = 2**31 - 1  # of a C int32 argument, to which ctypes narrows without a word


def _torch():
    global _MODULE, _FLOATS, _TABLES, _INT8
    if _MODULE is None:
        import torch
        _CODES.update({torch.float32: 0, torch.bfloat16: 1, torch.float8_e4m3fn: 2})
        _FLOATS = (torch.float32, torch.bfloat16)
        _TABLES = (*_FLOATS, torch.float8_e4m3fn)
        _INT8 = (torch.int8,)
        _MODULE = torch
    return _MODULE


def _device(torch, t, what):
    """The device of a call's first tensor, which is the current one."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a GPU tensor (got {t.device}); there is no CPU path")
    dev = t.get_device()
    if dev != torch.cuda.current_device():
        raise ValueError(f"{what} is on {t.device}, not on the current device")
    return dev


def _on(torch, t, what, dev):
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        _device(torch, t, what)  # says what is wrong
        raise ValueError(f"{what} is on {t.device}, not on the current device")


def _rows(torch, t, what, dtypes, dev):
    """Rows, columns and row stride of a 2-D tensor of one of `dtypes` with
    unit column stride.  A tensor of one row has whatever stride it was made
    with, which no access uses."""
    _on(torch, t, what, dev)
    if t.dtype not in dtypes:
        raise TypeError(f"{what} must be {' or '.join(str(d) for d in dtypes)} (got {t.dtype})")
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or (stride[1] != 1 and shape[1] != 1):
        raise ValueError(f"{what} must be 2-D with unit column stride")
    m, n = shape
    if n > _INT_MAX:
        raise ValueError(f"{what} has more than {_INT_MAX} columns")
    return m, n, stride[0] if m > 1 else max(n, 1)


def _vector(torch, t, what, n, dev):
    _on(torch, t, what, dev)
    if t.dtype is not torch.float32:
        raise TypeError(f"{what} must be torch.float32 (got {t.dtype})")
    if t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous with {n} elements")
    return t.data_ptr()


def _new(torch, shape, like, stream, dtype):
    """A new contiguous tensor of one or two dimensions.  (With its strides
    named, torch makes one in 1.3 us; new_empty takes 1.6.)"""
    if stream is None:
        strides = (shape[1], 1) if len(shape) == 2 else (1,)
        return torch.empty_strided(shape, strides, dtype=dtype, device=like.device)
    return _empty(shape, like.device, stream, dtype)


def _handle(torch, stream, dev):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(dev)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _tokens(torch, tokens, dev):
    _on(torch, tokens, "tokens", dev)
    if tokens.dtype is not torch.int32:
        raise TypeError(f"tokens must be torch.int32 (got {tokens.dtype})")
    if not tokens.is_contiguous():
        raise ValueError("tokens must be contiguous")
    return tokens.numel()


def _token_rows(torch, t, what, tokens, dim, dtypes, dev):
    """Row stride of one row of `dim` for each token: (n, dim), or contiguous
    with the tokens' shape and dim."""
    if t.dim() != 2:
        if t.shape != (*tokens.shape, dim) or not t.is_contiguous():
            raise ValueError(f"{what} must be (tokens, dim), or contiguous with the tokens' "
                             "shape and dim")
        t = t.view(-1, dim)
    m, n, ld = _rows(torch, t, what, dtypes, dev)
    if m != tokens.numel() or n != dim:
        raise ValueError(f"{what} must have a row of {dim} for each of {tokens.numel()} tokens")
    return ld


def _out_dtype(out_dtype):
    if out_dtype not in _FLOATS:
        raise TypeError(f"out_dtype must be torch.float32 or torch.bfloat16 (got {out_dtype})")
    return out_dtype


def emb_lookup_scaled(table, tokens, scale=1.0, out_dtype=None, out=None, stream=None):
    """scale * table[tokens]: one row for each token (any shape of int32
    tokens), zeros for a token outside [0, rows).  `table` is (rows, dim)
    float32, bfloat16 or float8_e4m3fn; the output is float32 or bfloat16
    (`out_dtype`; the table's type if that is one of them, else float32)."""
    torch = _torch()
    lib = load()
    dev = _device(torch, table, "table")
    rows, dim, ld = _rows(torch, table, "table", _TABLES, dev)
    n = _tokens(torch, tokens, dev)
    given = out is not None
    if not given:
        if out_dtype is None:
            out_dtype = table.dtype if table.dtype in _FLOATS else torch.float32
        out = _new(torch, (n, dim), table, stream, _out_dtype(out_dtype))
        if tokens.dim() != 1:
            out = out.view(*tokens.shape, dim)
        ld_out = dim
    else:
        _on(torch, out, "out", dev)
        if out_dtype is not None and out.dtype != out_dtype:
            raise TypeError("out and out_dtype disagree")
        ld_out = _token_rows(torch, out, "out", tokens, dim, _FLOATS, dev)
    status = lib.emb_lookup_scaled(n, rows, dim, table.data_ptr(), ld, _CODES[table.dtype],
                                   tokens.data_ptr(), scale, out.data_ptr(), ld_out,
                                   _CODES[out.dtype], _handle(torch, stream, dev))
    if status:
        _check(status, "emb_lookup_scaled")
    if given:
        torch.autograd.graph.increment_version(out)
    return out


def emb_lookup_grad_workspace_bytes(num_tokens, rows, dim):
    """Bytes of workspace that emb_lookup_grad takes for these sizes."""
    return load().emb_lookup_grad_workspace_bytes(num_tokens, rows, min(dim, _INT_MAX))


def emb_lookup_grad(grad, tokens, rows=None, scale=1.0, out_dtype=None, out=None,
                    accumulate=False, workspace=None, stream=None):
    """Gradient of emb_lookup_scaled with respect to its table: (rows, dim)
    with scale * the sum of the grad rows of each row's tokens, in `out` or a
    new tensor of `out_dtype` (the gradient's type unless given).  With
    accumulate=True it is added to `out`, whose other rows are not touched.
    `workspace` is a uint8 tensor of at least emb_lookup_grad_workspace_bytes;
    without it one is allocated for the call."""
    torch = _torch()
    lib = load()
    if not isinstance(grad, torch.Tensor) or grad.dim() < 1:
        raise TypeError("grad must be a torch.Tensor with a row for each token")
    dev = _device(torch, grad, "grad")
    n = _tokens(torch, tokens, dev)
    dim = grad.shape[-1]
    ld = _token_rows(torch, grad, "grad", tokens, dim, _FLOATS, dev)
    given = out is not None
    if not given:
        if accumulate:
            raise ValueError("accumulate needs out")
        if rows is None:
            raise ValueError("rows is required without out")
        out = _new(torch, (rows, dim), grad, stream,
                   grad.dtype if out_dtype is None else _out_dtype(out_dtype))
        ld_out = dim
    else:
        out_rows, out_dim, ld_out = _rows(torch, out, "out", _FLOATS, dev)
        if out_dtype is not None and out.dtype != out_dtype:
            raise TypeError("out and out_dtype disagree")
        if out_dim != dim or (rows is not None and out_rows != rows):
            raise ValueError("out must be (rows, dim)")
        rows = out_rows
    if workspace is None:
        size = lib.emb_lookup_grad_workspace_bytes(n, rows, dim)
        if size:
            workspace = _new(torch, (size,), grad, stream, torch.uint8)
    else:
        _on(torch, workspace, "workspace", dev)
        if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise TypeError("workspace must be a contiguous uint8 tensor")
        size = workspace.numel()
    status = lib.emb_lookup_grad(n, rows, dim, grad.data_ptr(), ld, _CODES[grad.dtype],
                                 tokens.data_ptr(), scale, 1 if accumulate else 0,
                                 out.data_ptr(), ld_out, _CODES[out.dtype],
                                 workspace.data_ptr() if workspace is not None else None, size,
                                 _handle(torch, stream, dev))
    if status:
        _check(status, "emb_lookup_grad")
    if given:
        torch.autograd.graph.increment_version(out)
    return out


def rms_norm_residual_i8(x, weight=None, residual=None, eps=1e-6, out_h=None, out_codes=None,
                         out_scale=None, stream=None):
    """(h, codes, scale): h = x + residual (x itself without one), and the RMS
    norm of h times weight as int8 codes with a float32 scale for each row.
    `out_h` may be x or residual."""
    torch = _torch()
    lib = load()
    dev = _device(torch, x, "x")
    m, dim, ldx = _rows(torch, x, "x", _FLOATS, dev)
    dtype = x.dtype
    given = [t for t in (out_h, out_codes, out_scale) if t is not None]
    wp = None if weight is None else _vector(torch, weight, "weight", dim, dev)
    rp, ldr, hp, ldh = None, 0, None, 0
    if residual is None:
        if out_h is not None:
            raise ValueError("out_h needs a residual (without one, h is x)")
        h = x
    else:
        rm, rdim, ldr = _rows(torch, residual, "residual", (dtype,), dev)
        if rm != m or rdim != dim:
            raise ValueError("residual must have x's shape")
        if out_h is None:
            h, ldh = _new(torch, (m, dim), x, stream, dtype), dim
        else:
            h = out_h
            hm, hdim, ldh = _rows(torch, h, "out_h", (dtype,), dev)
            if hm != m or hdim != dim:
                raise ValueError("out_h must have x's shape")
        rp, hp = residual.data_ptr(), h.data_ptr()
    if out_codes is None:
        out_codes, ldq = _new(torch, (m, dim), x, stream, torch.int8), dim
    else:
        qm, qdim, ldq = _rows(torch, out_codes, "out_codes", _INT8, dev)
        if qm != m or qdim != dim:
            raise ValueError("out_codes must have x's shape")
    if out_scale is None:
        out_scale = _new(torch, (m,), x, stream, torch.float32)
        sp = out_scale.data_ptr()
    else:
        sp = _vector(torch, out_scale, "out_scale", m, dev)
    status = lib.rms_norm_residual_i8(m, dim, x.data_ptr(), ldx, rp, ldr, _CODES[dtype], wp, eps,
                                      hp, ldh, out_codes.data_ptr(), ldq, sp,
                                      _handle(torch, stream, dev))
    if status:
        _check(status, "rms_norm_residual_i8")
    if given:
        torch.autograd.graph.increment_version(given)
    return h, out_codes, out_scale


def linear_i8_bias_act(a, a_scale, w, w_scale, bias=None, act="none", out_dtype=None, out=None,
                       stream=None):
    """act((a @ w.T) * a_scale[:, None] * w_scale + bias) of int8 `a` (M, K)
    and `w` (N, K), as (M, N) float32 or bfloat16 (`out_dtype`, float32 unless
    given)."""
    torch = _torch()
    lib = load()
    dev = _device(torch, a, "a")
    m, k, lda = _rows(torch, a, "a", _INT8, dev)
    n, kw, ldw = _rows(torch, w, "w", _INT8, dev)
    if kw != k:
        raise ValueError("w must be (N, K) with a's K")
    if m > _INT_MAX or n > _INT_MAX:
        raise ValueError(f"a or w has more than {_INT_MAX} rows")
    ap = _vector(torch, a_scale, "a_scale", m, dev)
    wp = _vector(torch, w_scale, "w_scale", n, dev)
    bp = None if bias is None else _vector(torch, bias, "bias", n, dev)
    given = out is not None
    if not given:
        out = _new(torch, (m, n), a, stream,
                   torch.float32 if out_dtype is None else _out_dtype(out_dtype))
        ldc = n
    else:
        om, on, ldc = _rows(torch, out, "out", _FLOATS, dev)
        if out_dtype is not None and out.dtype != out_dtype:
            raise TypeError("out and out_dtype disagree")
        if om != m or on != n:
            raise ValueError("out must be (M, N)")
    status = lib.linear_i8_bias_act(m, n, k, a.data_ptr(), lda, ap, w.data_ptr(), ldw, wp, bp,
                                    ACTS[act] if isinstance(act, str) else int(act),
                                    out.data_ptr(), ldc, _CODES[out.dtype],
                                    _handle(torch, stream, dev))
    if status:
        _check(status, "linear_i8_bias_act")
    if given:
        torch.autograd.graph.increment_version(out)
    return out
