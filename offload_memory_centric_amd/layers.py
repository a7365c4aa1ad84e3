"""What a training step runs on the device around the tiled block, for torch tensors.

Layer norm with the residual sum, the token embedding and its gradient, each
in its forward and its backward call, and the orthogonalised update of a
weight; for a block that is a mixture of experts the router, the products
grouped by expert and the combination, and low-rank adapters beside the tiled
linear, forward and backward; over caller-owned outputs; every step runs in
libzi.so.  Calls enqueue on ``stream`` (a torch stream or a handle such as
``Context.streams[0]``; by default torch's current stream) and return at once.  As with any stream, tensors made on another one must be complete
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


def _index(t, shape, name: str, dev: int) -> None:
    """An int32 tensor of the given shape, contiguous."""
    if t.dtype is not torch.int32:
        raise TypeError("%s has dtype %s, expected int32" % (name, t.dtype))
    if t.get_device() != dev:
        raise _elsewhere(t, name, dev)
    if t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be contiguous, of shape %s" % (name, tuple(shape)))


def _dense(t, shape, name: str, dev: int, dtype) -> None:
    """A contiguous tensor of the given shape and type."""
    if t.dtype is not dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if t.get_device() != dev:
        raise _elsewhere(t, name, dev)
    if t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be contiguous, of shape %s" % (name, tuple(shape)))


def route_fwd_bytes(T: int, E: int, k: int) -> int:
    """Workspace bytes of route_fwd."""
    return zi.zi_route_fwd_bytes(T, E, k)


def route_fwd(logits, ids, weights, offsets, rows, slots, work, normalize: bool = True, stream=None) -> None:
    """The k experts of each of T tokens and their softmax weights, and the choices grouped by expert (zi_route_fwd).

    logits [T, E]; ids, weights (fp32) and slots [T, k], offsets [E + 1], rows [T k], all but weights int32.
    Expert e's places are offsets[e] .. offsets[e + 1] - 1; rows names the token at each place (-1 past the last:
    rows are the ids for embedding_fwd), slots the place of each choice (-1: none).  work may be None for 64 tokens
    or fewer."""
    (T, E), dev = _matrix(logits, "logits"), _on(logits, "logits")
    k = _matrix(ids, "ids")[1]
    for t, shape, name in ((ids, (T, k), "ids"), (slots, (T, k), "slots"), (offsets, (E + 1,), "offsets"),
                           (rows, (T * k,), "rows")):
        _index(t, shape, name, dev)
    _dense(weights, (T, k), "weights", dev, torch.float32)
    route = zi.zi_route(T, _ld(logits, E, "logits"), 0, E, k, _code(logits, "logits"), normalize)
    _run(dev, stream, zi.zi_route_fwd, route, logits, ids, weights, offsets, rows, slots, work, _bytes(work, dev))


def route_bwd(logits, ids, weights, dweights, dlogits, normalize: bool = True, stream=None) -> None:
    """dlogits from dweights, the gradient of route_fwd's weights (zi_route_bwd)."""
    (T, E), dev = _matrix(logits, "logits"), _on(logits, "logits")
    k = _matrix(ids, "ids")[1]
    _index(ids, (T, k), "ids", dev)
    _dense(weights, (T, k), "weights", dev, torch.float32)
    _dense(dweights, (T, k), "dweights", dev, torch.float32)
    ldd = _rows(dlogits, T, E, "dlogits", dev, logits.dtype)
    route = zi.zi_route(T, _ld(logits, E, "logits"), ldd, E, k, _code(logits, "logits"), normalize)
    _run(dev, stream, zi.zi_route_bwd, route, logits, ids, weights, dweights, dlogits)


def _weights(W, name: str):
    """Shape and strides (of a row, of a group) of the groups' weights."""
    if W.dim() != 3:
        raise ValueError("%s must be [E, M, K]" % name)
    E, M, K = W.shape
    if W.is_contiguous():
        return E, M, K, K, M * K
    if K > 1 and W.stride(2) != 1:
        raise ValueError("the rows of %s must be contiguous" % name)
    ldw = W.stride(1) if M > 1 else K
    ldg = W.stride(0) if E > 1 else (M - 1) * ldw + K + -K % 8
    if ldw < K or ldg < (M - 1) * ldw + K:
        raise ValueError("the rows of %s overlap" % name)
    return E, M, K, ldw, ldg


def _like(t, name: str, dtype) -> None:
    if t.dtype is not dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))


def grouped_fwd(X, W, offsets, Y, A=None, gelu: bool = False, stream=None) -> None:
    """Y = X W_e^T over the rows offsets[e] .. offsets[e + 1] - 1 of every group e (zi_grouped_fwd).

    X [R, K] and W [E, M, K] of one 16-bit type, Y [R, M] of that type or fp32, offsets int32 [E + 1].  With gelu, or
    A [R, M] given: Y = GeLU(X W_e^T), and A keeps X W_e^T for the backward."""
    (R, K), dev = _matrix(X, "X"), _on(X, "X")
    E, M, _, ldw, ldg = _weights(W, "W")
    _index(offsets, (E + 1,), "offsets", dev)
    _like(W, "W", X.dtype)
    if W.get_device() != dev:
        raise _elsewhere(W, "W", dev)
    if W.shape[2] != K:
        raise ValueError("W has rows of %d elements, X of %d" % (W.shape[2], K))
    ldx, ldy = _ld(X, K, "X"), _rows(Y, R, M, "Y", dev)
    lda = 0 if A is None else _rows(A, R, M, "A", dev, X.dtype)
    grouped = zi.zi_grouped(R, K, M, ldx, ldy, lda, ldw, ldg, E, _code(X, "X"), _code(Y, "Y"), gelu or A is not None, 0)
    _run(dev, stream, zi.zi_grouped_fwd, grouped, X, W, offsets, Y, A)


def grouped_dx(dY, W, offsets, dX, A=None, stream=None) -> None:
    """dX = dY W_e of grouped_fwd; with A [R, K], the input of the GeLU that made X, times GeLU'(A)
    (zi_grouped_dx)."""
    (R, M), dev = _matrix(dY, "dY"), _on(dY, "dY")
    E, _, K, ldw, ldg = _weights(W, "W")
    _index(offsets, (E + 1,), "offsets", dev)
    _like(W, "W", dY.dtype)
    if W.get_device() != dev:
        raise _elsewhere(W, "W", dev)
    if W.shape[1] != M:
        raise ValueError("W has %d rows a group, dY rows of %d elements" % (W.shape[1], M))
    ldy, ldx = _ld(dY, M, "dY"), _rows(dX, R, K, "dX", dev)
    lda = 0 if A is None else _rows(A, R, K, "A", dev, dY.dtype)
    grouped = zi.zi_grouped(R, K, M, ldx, ldy, lda, ldw, ldg, E, _code(dY, "dY"), _code(dX, "dX"), 0, 0)
    _run(dev, stream, zi.zi_grouped_dx, grouped, dY, W, offsets, A, dX)


def grouped_dw(X, dY, offsets, dW, accumulate: bool = False, stream=None) -> None:
    """dW_e = dY_e^T X_e of grouped_fwd, in X's type or fp32, added to an fp32 dW with ``accumulate``
    (zi_grouped_dw)."""
    (R, K), dev = _matrix(X, "X"), _on(X, "X")
    E, M, _, ldw, ldg = _weights(dW, "dW")
    _index(offsets, (E + 1,), "offsets", dev)
    if dW.get_device() != dev:
        raise _elsewhere(dW, "dW", dev)
    if dW.shape[2] != K:
        raise ValueError("dW has rows of %d elements, X of %d" % (dW.shape[2], K))
    ldx, ldy = _ld(X, K, "X"), _rows(dY, R, M, "dY", dev, X.dtype)
    grouped = zi.zi_grouped(R, K, M, ldx, ldy, 0, ldw, ldg, E, _code(X, "X"), _code(dW, "dW"), 0, accumulate)
    _run(dev, stream, zi.zi_grouped_dw, grouped, X, dY, offsets, dW)


def combine_fwd(Z, slots, weights, Y, stream=None) -> None:
    """Y[t] = sum_j weights[t][j] Z[slots[t][j]] (zi_combine_fwd); a slot outside Z's rows stands for none."""
    (R, D), dev = _matrix(Z, "Z"), _on(Z, "Z")
    T, k = _matrix(slots, "slots")
    _index(slots, (T, k), "slots", dev)
    _dense(weights, (T, k), "weights", dev, torch.float32)
    combine = zi.zi_combine(T, R, D, _ld(Z, D, "Z"), _rows(Y, T, D, "Y", dev, Z.dtype), 0, k, _code(Z, "Z"))
    _run(dev, stream, zi.zi_combine_fwd, combine, Z, slots, weights, Y)


def combine_bwd(dY, Z, slots, weights, dZ, dweights, stream=None) -> None:
    """dZ and dweights of combine_fwd (zi_combine_bwd); the slots are distinct."""
    (R, D), dev = _matrix(Z, "Z"), _on(Z, "Z")
    T, k = _matrix(slots, "slots")
    _index(slots, (T, k), "slots", dev)
    _dense(weights, (T, k), "weights", dev, torch.float32)
    _dense(dweights, (T, k), "dweights", dev, torch.float32)
    ldz, ldy, lddz = _ld(Z, D, "Z"), _rows(dY, T, D, "dY", dev, Z.dtype), _rows(dZ, R, D, "dZ", dev, Z.dtype)
    combine = zi.zi_combine(T, R, D, ldz, ldy, lddz, k, _code(Z, "Z"))
    _run(dev, stream, zi.zi_combine_bwd, combine, dY, Z, slots, weights, dZ, dweights)


def adapters_fwd_bytes(T: int, r: int) -> int:
    """Workspace bytes of adapters_fwd."""
    return zi.zi_adapters_fwd_bytes(T, r)


def _adapters(X, A, B, offsets, ids, scales, dev):
    """T, K, M, S, N, r."""
    (T, K), (S,) = _matrix(X, "X"), ids.shape
    if A.dim() != 3 or B.dim() != 3:
        raise ValueError("A must be [N, r, K], B [N, r, M]")
    (N, r, _), M = A.shape, B.shape[2]
    _dense(A, (N, r, K), "A", dev, X.dtype)
    _dense(B, (N, r, M), "B", dev, X.dtype)
    _index(ids, (S,), "ids", dev)
    _index(offsets, (S + 1,), "offsets", dev)
    _vector(scales, N, "scales", dev, torch.float32)
    return T, K, M, S, N, r


def adapters_fwd(X, A, B, offsets, ids, scales, Y, work, Y0=None, U=None, stream=None) -> None:
    """Y = Y0 + scales[n] (X A_n^T) B_n, n = ids[s] for the rows of segment s (zi_adapters_fwd).

    X [T, K], A [N, r, K] and B [N, r, M] of one 16-bit type; Y and Y0 [T, M] of that type or fp32 (Y0 may be Y:
    what the tiled linear left there; None: zero); offsets [S + 1] and ids [S] int32, scales [N] fp32.  U [r, T]
    (fp32) keeps A_n X^T for the backward.  Rows without an adapter get Y0, and zeros in U."""
    dev = _on(X, "X")
    T, K, M, S, N, r = _adapters(X, A, B, offsets, ids, scales, dev)
    ldx, ldy = _ld(X, K, "X"), _rows(Y, T, M, "Y", dev)
    ldy0 = 0 if Y0 is None else _rows(Y0, T, M, "Y0", dev, Y.dtype)
    if U is not None:
        _dense(U, (r, T), "U", dev, torch.float32)
    adapters = zi.zi_adapters(T, K, M, ldx, 0, 0, ldy, ldy0, S, N, r, _code(X, "X"), _code(Y, "Y"), 0)
    _run(dev, stream, zi.zi_adapters_fwd, adapters, X, A, B, offsets, ids, scales, Y0, Y, U, work, _bytes(work, dev))


def adapters_bwd_bytes(T: int, r: int) -> int:
    """Workspace bytes of adapters_bwd."""
    return zi.zi_adapters_bwd_bytes(T, r)


def adapters_bwd(X, dY, U, A, B, offsets, ids, scales, dA, dB, work, dX=None, dX0=None, accumulate: bool = False,
                 stream=None) -> None:
    """dA [N, r, K], dB [N, r, M] (fp32, overwritten, or added to with ``accumulate``) and dX of adapters_fwd, from
    its U (zi_adapters_bwd).  dX and dX0 [T, K] are of X's type or fp32; dX0, such as the tiled linear's dX, is
    added, and may be dX; without dX it is not formed."""
    dev = _on(X, "X")
    T, K, M, S, N, r = _adapters(X, A, B, offsets, ids, scales, dev)
    ldx, ldy = _ld(X, K, "X"), _rows(dY, T, M, "dY", dev, X.dtype)
    _dense(U, (r, T), "U", dev, torch.float32)
    _dense(dA, (N, r, K), "dA", dev, torch.float32)
    _dense(dB, (N, r, M), "dB", dev, torch.float32)
    lddx = 0 if dX is None else _rows(dX, T, K, "dX", dev)
    lddx0 = 0 if dX0 is None else _rows(dX0, T, K, "dX0", dev, None if dX is None else dX.dtype)
    out = X if dX is None else dX
    adapters = zi.zi_adapters(T, K, M, ldx, lddx, lddx0, ldy, 0, S, N, r, _code(X, "X"), _code(out, "dX"), accumulate)
    _run(dev, stream, zi.zi_adapters_bwd, adapters, X, dY, U, A, B, offsets, ids, scales, dX0, dX, dA, dB, work,
         _bytes(work, dev))
