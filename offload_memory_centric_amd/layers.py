"""What a training step runs on the device around the tiled block, for torch tensors.

Layer norm with the residual sum, the token embedding and its gradient, each
in its forward and its backward call, and the orthogonalised update of a
weight, over caller-owned outputs; every step runs in libzi.so.  Calls enqueue on ``stream`` (a torch stream or a handle such
as ``Context.streams[0]``; by default torch's current stream) and return at
once.  As with any stream, tensors made on another one must be complete
before, and be kept until the work is done.  A call's tensors and stream are of
one device, which need not be the current one.
"""
from __future__ import annotations

import torch

from . import zi

_CODES = {torch.float16: zi.ZI_F16, torch.bfloat16: zi.ZI_BF16, torch.float32: zi.ZI_F32}


def workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """Device memory for a call's workspace; one per stream that may run such calls."""
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def _code(t, name: str) -> int:
    code = _CODES.get(t.dtype)
    if code is None:
        raise TypeError("%s has dtype %s, expected float16, bfloat16 or float32" % (name, t.dtype))
    return code


def _on(t, name: str) -> int:
    """The index of the device that holds t, the first of a call's tensors that is looked at."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("%s must be a device tensor" % name)
    return dev


def _elsewhere(t, name: str, dev: int) -> ValueError:
    return ValueError("%s is on %s, the call's other tensors on cuda:%d" % (name, t.device, dev))


def _ld(t, cols: int, name: str) -> int:
    """The row stride of a matrix whose rows are contiguous."""
    if t.is_contiguous():
        return cols
    if cols > 1 and t.stride(1) != 1:
        raise ValueError("the rows of %s must be contiguous" % name)
    ld = t.stride(0)
    if ld < cols:
        raise ValueError("the rows of %s overlap" % name)
    return ld


def _rows(t, rows: int, cols: int, name: str, dev: int, dtype=None) -> int:
    """The row stride of a [rows, cols] tensor on device dev whose rows are contiguous."""
    if dtype is not None and t.dtype is not dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.get_device() != dev:
        raise _elsewhere(t, name, dev)
    if t.shape != (rows, cols):
        raise ValueError("%s has shape %s, expected (%d, %d)" % (name, tuple(t.shape), rows, cols))
    return _ld(t, cols, name)


def _vector(t, n: int, name: str, dev: int, dtype=None) -> None:
    if dtype is not None and t.dtype is not dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.get_device() != dev:
        raise _elsewhere(t, name, dev)
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError("%s must be a contiguous vector of %d elements" % (name, n))


def _bytes(work, dev: int) -> int:
    if work is None:
        return 0
    if work.get_device() != dev:
        raise _elsewhere(work, "work", dev)
    if not work.is_contiguous():
        raise ValueError("work must be contiguous")
    return work.numel() * work.element_size()


# The handle of torch's current stream, and the current device; the public calls
# take longer than the rest of a small call's checks.
_current = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev))
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _run(dev: int, stream, call, *args) -> None:
    """call(*args, stream) with dev, the tensors' device, as the current one."""
    if stream is None:
        stream = _current(dev)
    else:
        of = getattr(stream, "device", None)
        if of is not None and of.index != dev:
            raise ValueError("the stream is of %s, the tensors are on cuda:%d" % (of, dev))
    if _device() == dev:
        call(*args, stream)
    else:
        with torch.cuda.device(dev):
            call(*args, stream)


def _matrix(t, name: str):
    if t.dim() != 2:
        raise ValueError("%s must be a matrix" % name)
    return t.shape


def _params(gamma, beta, D: int, dev: int) -> int:
    """The type of gamma and beta, of which either may be None."""
    given = beta if gamma is None else gamma
    if given is None:
        return zi.ZI_F32
    if gamma is not None:
        _vector(gamma, D, "gamma", dev)
    if beta is not None:
        _vector(beta, D, "beta", dev, given.dtype)
    return _code(given, "gamma" if given is gamma else "beta")


def layer_norm_fwd(X, gamma, beta, Y, mean=None, rstd=None, eps: float = 1e-5, R=None, S=None, stream=None) -> None:
    """S = X + R (S = X without R), Y = (S - mean) * rstd * gamma + beta over rows (zi_layer_norm_fwd).

    X and S, the residual stream, share a dtype; R and Y, the block's side, another: the two are equal or one
    of them is fp32.  gamma, beta, mean, rstd and S (with R) may be None."""
    (T, D), dev = _matrix(X, "X"), _on(X, "X")
    ldx, ldy = _ld(X, D, "X"), _rows(Y, T, D, "Y", dev)
    ldr = 0 if R is None else _rows(R, T, D, "R", dev, Y.dtype)
    lds = 0 if S is None else _rows(S, T, D, "S", dev, X.dtype)
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        if t is not None:
            _vector(t, T, name, dev, torch.float32)
    norm = zi.zi_norm(T, D, ldx, ldr, lds, ldy, _code(X, "X"), _code(Y, "Y"), _params(gamma, beta, D, dev), eps)
    _run(dev, stream, zi.zi_layer_norm_fwd, norm, X, R, gamma, beta, S, Y, mean, rstd)


def layer_norm_bwd_bytes(T: int, D: int) -> int:
    """Workspace bytes of layer_norm_bwd."""
    return zi.zi_layer_norm_bwd_bytes(T, D)


def layer_norm_bwd(dY, S, gamma, mean, rstd, dX, dgamma, dbeta, work, dS=None, stream=None) -> None:
    """dX, dgamma and dbeta of layer_norm_fwd's Y, plus dS, the gradient that reaches S past the norm
    (zi_layer_norm_bwd).  dgamma and dbeta are fp32 and overwritten; both None: not formed, and work unused."""
    (T, D), dev = _matrix(S, "S"), _on(S, "S")
    lds, ldy, ldx = _ld(S, D, "S"), _rows(dY, T, D, "dY", dev), _rows(dX, T, D, "dX", dev, S.dtype)
    ldr = 0 if dS is None else _rows(dS, T, D, "dS", dev, S.dtype)
    _vector(mean, T, "mean", dev, torch.float32)
    _vector(rstd, T, "rstd", dev, torch.float32)
    for t, name in ((dgamma, "dgamma"), (dbeta, "dbeta")):
        if t is not None:
            _vector(t, D, name, dev, torch.float32)
    norm = zi.zi_norm(T, D, ldx, ldr, lds, ldy, _code(S, "S"), _code(dY, "dY"), _params(gamma, None, D, dev), 0.0)
    _run(dev, stream, zi.zi_layer_norm_bwd, norm, dY, S, gamma, mean, rstd, dS, dX, dgamma, dbeta, work, _bytes(work, dev))


def _embedding(ids, W, X, scale, accumulate, names):
    """The problem, and the tensors' device."""
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError("ids has dtype %s, expected int32 or int64" % ids.dtype)
    (V, D), T, dev = _matrix(W, names[0]), ids.numel(), _on(W, names[0])
    _vector(ids, T, "ids", dev)
    return zi.zi_embedding(T, V, D, _ld(W, D, names[0]), _rows(X, T, D, names[1], dev), _code(W, names[0]),
                           _code(X, names[1]), ids.dtype == torch.int64, scale, accumulate), dev


def embedding_fwd(ids, W, X, scale: float = 1.0, stream=None) -> None:
    """X[t] = scale * W[ids[t]] (zi_embedding_fwd); an id outside the table gives a zero row."""
    emb, dev = _embedding(ids, W, X, scale, False, ("W", "X"))
    _run(dev, stream, zi.zi_embedding_fwd, emb, ids, W, X)


def embedding_bwd_bytes(T: int, V: int, D: int) -> int:
    """Workspace bytes of embedding_bwd."""
    return zi.zi_embedding_bwd_bytes(T, V, D)


def embedding_bwd(ids, dX, dW, work, scale: float = 1.0, accumulate: bool = False, stream=None) -> None:
    """dW[v] = scale * sum of dX[t] over ids[t] == v, added to dW with ``accumulate`` (zi_embedding_bwd)."""
    emb, dev = _embedding(ids, dW, dX, scale, accumulate, ("dW", "dX"))
    _run(dev, stream, zi.zi_embedding_bwd, emb, ids, dX, dW, work, _bytes(work, dev))


def orthogonalize_bytes(M: int, K: int) -> int:
    """Workspace bytes of orthogonalize."""
    return zi.zi_orthogonalize_bytes(M, K)


def orthogonalize(G, O, work, steps: int = 5, coeffs=(3.4445, -4.7750, 2.0315), eps: float = 1e-7,
                  stream=None) -> None:
    """O (bf16) = the update G with its singular values driven towards one by `steps` Newton-Schulz steps
    (zi_orthogonalize)."""
    (M, K), dev = _matrix(G, "G"), _on(G, "G")
    a, b, c = coeffs
    orth = zi.zi_orth(M, K, _ld(G, K, "G"), _rows(O, M, K, "O", dev, torch.bfloat16), _code(G, "G"), steps, a, b, c,
                      eps)
    _run(dev, stream, zi.zi_orthogonalize, orth, G, O, work, _bytes(work, dev))
