"""Token operators: embedding lookup with a scale and its gradient, RMS norm
to int8 codes, and the int8 product with a scale for each token and channel.

Argument marshalling only, as in abi.py: every function has the name of the C
entry point it calls (include/dlrm_embedding_bag.h says what it computes),
checks its tensors, allocates the outputs and workspace that it is not given
on the stream the call runs on, and raises on refusal.  There is no CPU path.
"""
from __future__ import annotations

from .abi import ACTS, _check, _empty, _stream, load

_CODES = {}   # torch dtype -> dlrm_dtype, filled on the first call (torch is imported late)


def _torch():
    import torch
    if not _CODES:
        _CODES.update({torch.float32: 0, torch.bfloat16: 1, torch.float8_e4m3fn: 2})
    return torch


def _gpu(torch, t, what):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a GPU tensor (got {t.device}); there is no CPU path")
    if t.get_device() != torch.cuda.current_device():
        raise ValueError(f"{what} is on {t.device}, not on the current device")
    return t


def _rows(torch, t, what, dtypes):
    """A 2-D tensor of one of `dtypes` with unit column stride."""
    _gpu(torch, t, what)
    if t.dtype not in dtypes:
        raise TypeError(f"{what} must be {' or '.join(str(d) for d in dtypes)} (got {t.dtype})")
    if t.dim() != 2 or (t.stride(1) != 1 and t.shape[1] != 1):
        raise ValueError(f"{what} must be 2-D with unit column stride")
    return t


def _vector(torch, t, what, n, dtype=None):
    _gpu(torch, t, what)
    if t.dtype != (dtype or torch.float32):
        raise TypeError(f"{what} must be {dtype or torch.float32} (got {t.dtype})")
    if not t.is_contiguous() or t.numel() != n:
        raise ValueError(f"{what} must be contiguous with {n} elements")
    return t


def _ld(t):
    """Row stride of a 2-D tensor; a tensor of one row has whatever stride it
    was made with, which no access uses."""
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _new(torch, shape, like, stream, dtype):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    return _empty(shape, like.device, stream, dtype)


def _tokens(torch, tokens):
    _gpu(torch, tokens, "tokens")
    if tokens.dtype != torch.int32:
        raise TypeError(f"tokens must be torch.int32 (got {tokens.dtype})")
    if not tokens.is_contiguous():
        raise ValueError("tokens must be contiguous")
    return tokens


def _token_rows(torch, t, what, tokens, dim, dtypes):
    """One row of `dim` for each token: (n, dim), or contiguous with the
    tokens' shape and dim."""
    if t.dim() != 2:
        if t.shape != (*tokens.shape, dim) or not t.is_contiguous():
            raise ValueError(f"{what} must be (tokens, dim), or contiguous with the tokens' "
                             "shape and dim")
        t = t.view(-1, dim)
    _rows(torch, t, what, dtypes)
    if t.shape != (tokens.numel(), dim):
        raise ValueError(f"{what} must have a row of {dim} for each of {tokens.numel()} tokens")
    return t


def emb_lookup_scaled(table, tokens, scale=1.0, out_dtype=None, out=None, stream=None):
    """scale * table[tokens]: one row for each token (any shape of int32
    tokens), zeros for a token outside [0, rows).  `table` is (rows, dim)
    float32, bfloat16 or float8_e4m3fn; the output is float32 or bfloat16
    (`out_dtype`; the table's type if that is one of them, else float32)."""
    torch = _torch()
    lib = load()
    _rows(torch, table, "table", (torch.float32, torch.bfloat16, torch.float8_e4m3fn))
    _tokens(torch, tokens)
    rows, dim = table.shape
    if out is None:
        if out_dtype is None:
            out_dtype = torch.float32 if table.dtype == torch.float8_e4m3fn else table.dtype
        if out_dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"out_dtype must be torch.float32 or torch.bfloat16 (got {out_dtype})")
        out = _new(torch, (*tokens.shape, dim), table, stream, out_dtype)
        ld_out = dim
    else:
        if out_dtype is not None and out.dtype != out_dtype:
            raise TypeError("out and out_dtype disagree")
        ld_out = _ld(_token_rows(torch, out, "out", tokens, dim, (torch.float32, torch.bfloat16)))
    _check(lib.emb_lookup_scaled(tokens.numel(), rows, dim, table.data_ptr(), _ld(table),
                                 _CODES[table.dtype], tokens.data_ptr(), scale, out.data_ptr(),
                                 ld_out, _CODES[out.dtype], _stream(stream)),
           "emb_lookup_scaled")
    return out


def emb_lookup_grad_workspace_bytes(num_tokens, rows, dim):
    """Bytes of workspace that emb_lookup_grad takes for these sizes."""
    return load().emb_lookup_grad_workspace_bytes(num_tokens, rows, dim)


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
    types = (torch.float32, torch.bfloat16)
    _tokens(torch, tokens)
    if not isinstance(grad, torch.Tensor) or grad.dim() < 1:
        raise TypeError("grad must be a torch.Tensor with a row for each token")
    grad2 = _token_rows(torch, grad, "grad", tokens, grad.shape[-1], types)
    dim = grad2.shape[1]
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        if rows is None:
            raise ValueError("rows is required without out")
        if out_dtype is None:
            out_dtype = grad2.dtype
        if out_dtype not in types:
            raise TypeError(f"out_dtype must be torch.float32 or torch.bfloat16 (got {out_dtype})")
        out = _new(torch, (rows, dim), grad2, stream, out_dtype)
    else:
        _rows(torch, out, "out", types)
        if out_dtype is not None and out.dtype != out_dtype:
            raise TypeError("out and out_dtype disagree")
        if out.shape[1] != dim or (rows is not None and out.shape[0] != rows):
            raise ValueError("out must be (rows, dim)")
        rows = out.shape[0]
    n = tokens.numel()
    if workspace is None:
        workspace = _new(torch, (lib.emb_lookup_grad_workspace_bytes(n, rows, dim),), grad2,
                         stream, torch.uint8)
    else:
        _gpu(torch, workspace, "workspace")
        if workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise TypeError("workspace must be a contiguous uint8 tensor")
    _check(lib.emb_lookup_grad(n, rows, dim, grad2.data_ptr(), _ld(grad2), _CODES[grad2.dtype],
                               tokens.data_ptr(), scale, 1 if accumulate else 0, out.data_ptr(),
                               _ld(out), _CODES[out.dtype], workspace.data_ptr(),
                               workspace.numel(), _stream(stream)), "emb_lookup_grad")
    return out


def rms_norm_residual_i8(x, weight=None, residual=None, eps=1e-6, out_h=None, out_codes=None,
                         out_scale=None, stream=None):
    """(h, codes, scale): h = x + residual (x itself without one), and the RMS
    norm of h times weight as int8 codes with a float32 scale for each row.
    `out_h` may be x or residual."""
    torch = _torch()
    lib = load()
    types = (torch.float32, torch.bfloat16)
    _rows(torch, x, "x", types)
    m, dim = x.shape
    wp = None if weight is None else _vector(torch, weight, "weight", dim).data_ptr()
    rp, ldr, hp, ldh = None, 0, None, 0
    if residual is None:
        if out_h is not None:
            raise ValueError("out_h needs a residual (without one, h is x)")
        h = x
    else:
        _rows(torch, residual, "residual", (x.dtype,))
        if residual.shape != x.shape:
            raise ValueError("residual must have x's shape")
        if out_h is None:
            h = _new(torch, (m, dim), x, stream, x.dtype)
        else:
            h = _rows(torch, out_h, "out_h", (x.dtype,))
            if h.shape != x.shape:
                raise ValueError("out_h must have x's shape")
        rp, ldr, hp, ldh = residual.data_ptr(), _ld(residual), h.data_ptr(), _ld(h)
    if out_codes is None:
        out_codes = _new(torch, (m, dim), x, stream, torch.int8)
    elif _rows(torch, out_codes, "out_codes", (torch.int8,)).shape != x.shape:
        raise ValueError("out_codes must have x's shape")
    if out_scale is None:
        out_scale = _new(torch, (m,), x, stream, torch.float32)
    else:
        _vector(torch, out_scale, "out_scale", m)
    _check(lib.rms_norm_residual_i8(m, dim, x.data_ptr(), _ld(x), rp, ldr, _CODES[x.dtype], wp,
                                    eps, hp, ldh, out_codes.data_ptr(), _ld(out_codes),
                                    out_scale.data_ptr(), _stream(stream)),
           "rms_norm_residual_i8")
    return h, out_codes, out_scale


def linear_i8_bias_act(a, a_scale, w, w_scale, bias=None, act="none", out_dtype=None, out=None,
                       stream=None):
    """act((a @ w.T) * a_scale[:, None] * w_scale + bias) of int8 `a` (M, K)
    and `w` (N, K), as (M, N) float32 or bfloat16 (`out_dtype`, float32 unless
    given)."""
    torch = _torch()
    lib = load()
    _rows(torch, a, "a", (torch.int8,))
    _rows(torch, w, "w", (torch.int8,))
    m, k = a.shape
    n = w.shape[0]
    if w.shape[1] != k:
        raise ValueError("w must be (N, K) with a's K")
    _vector(torch, a_scale, "a_scale", m)
    _vector(torch, w_scale, "w_scale", n)
    bp = None if bias is None else _vector(torch, bias, "bias", n).data_ptr()
    if out is None:
        if out_dtype is None:
            out_dtype = torch.float32
        if out_dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"out_dtype must be torch.float32 or torch.bfloat16 (got {out_dtype})")
        out = _new(torch, (m, n), a, stream, out_dtype)
    else:
        _rows(torch, out, "out", (torch.float32, torch.bfloat16))
        if out_dtype is not None and out.dtype != out_dtype:
            raise TypeError("out and out_dtype disagree")
        if out.shape != (m, n):
            raise ValueError("out must be (M, N)")
    _check(lib.linear_i8_bias_act(m, n, k, a.data_ptr(), _ld(a), a_scale.data_ptr(), w.data_ptr(),
                                  _ld(w), w_scale.data_ptr(), bp,
                                  ACTS[act] if isinstance(act, str) else int(act), out.data_ptr(),
                                  _ld(out), _CODES[out.dtype], _stream(stream)),
           "linear_i8_bias_act")
    return out
