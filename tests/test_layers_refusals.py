"""Refusals of the operators next to the block: they come before anything is
enqueued, so they are tested without a GPU, with addresses that nothing reads."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def zi():
    from offload_memory_centric_amd import zi as m
    return m


A = 1 << 20  # a 256-byte aligned address


def norm(zi, **kw):
    d = dict(T=4, D=16, ldx=0, ldr=0, lds=0, ldy=0, x_dtype=zi.ZI_F16, y_dtype=zi.ZI_F16, p_dtype=zi.ZI_F32, eps=1e-5)
    d.update(kw)
    return zi.zi_norm(*[d[k] for k, _ in zi.zi_norm._fields_])


def emb(zi, **kw):
    d = dict(T=4, V=10, D=16, ldw=0, ldx=0, w_dtype=zi.ZI_F16, x_dtype=zi.ZI_F16, ids64=1, scale=1.0, accumulate=0)
    d.update(kw)
    return zi.zi_embedding(*[d[k] for k, _ in zi.zi_embedding._fields_])


def refused(zi, status, f, *args):
    with pytest.raises(zi.ZiError) as e:
        f(*args)
    assert e.value.status == getattr(zi, status), str(e.value)
    assert zi.zi_last_error()


NORM_BAD = [
    (dict(T=-1), "ZI_ERR_SHAPE"), (dict(T=1 << 31), "ZI_ERR_SHAPE"), (dict(D=0), "ZI_ERR_SHAPE"),
    (dict(D=1 << 31), "ZI_ERR_SHAPE"), (dict(ldx=15), "ZI_ERR_SHAPE"), (dict(ldr=-1), "ZI_ERR_SHAPE"),
    (dict(lds=1), "ZI_ERR_SHAPE"), (dict(ldy=15), "ZI_ERR_SHAPE"),
    (dict(x_dtype=0), "ZI_ERR_ARG"), (dict(y_dtype=4), "ZI_ERR_ARG"), (dict(p_dtype=-1), "ZI_ERR_ARG"),
    (dict(x_dtype=1, y_dtype=2), "ZI_ERR_ARG"), (dict(eps=-1.0), "ZI_ERR_ARG"),
    (dict(eps=float("nan")), "ZI_ERR_ARG"), (dict(eps=float("inf")), "ZI_ERR_ARG"),
]


@pytest.mark.parametrize("bad,status", NORM_BAD)
def test_norm_problem(zi, bad, status):
    n = norm(zi, **bad)
    refused(zi, status, zi.zi_layer_norm_fwd, n, A, A, A, A, A, A, A, A)
    refused(zi, status, zi.zi_layer_norm_bwd, n, A, A, A, A, A, A, A, A, A, A, 1 << 30)


def test_norm_pointers(zi):
    n = norm(zi)
    refused(zi, "ZI_ERR_ARG", zi.zi_layer_norm_fwd, n, None, None, A, A, None, A, A, A)
    refused(zi, "ZI_ERR_ARG", zi.zi_layer_norm_fwd, n, A, None, A, A, None, None, A, A)
    refused(zi, "ZI_ERR_ARG", zi.zi_layer_norm_fwd, n, A, None, A, A, A, A, A, A)  # S without R
    fwd = [A, A, A, A, A, A, A, A]
    for k, off in ((0, 1), (1, 1), (2, 2), (3, 2), (4, 1), (5, 1), (6, 2), (7, 2)):
        args = list(fwd)
        args[k] += off
        refused(zi, "ZI_ERR_ALIGN", zi.zi_layer_norm_fwd, n, *args)
    bwd = [A] * 10
    for k in (0, 1, 3, 4, 6):  # dY, S, mean, rstd, dX
        args = list(bwd)
        args[k] = None
        refused(zi, "ZI_ERR_ARG", zi.zi_layer_norm_bwd, n, *args[:9], A, 1 << 30)
    for k in range(9):
        args = list(bwd)
        args[k] += 1
        refused(zi, "ZI_ERR_ALIGN", zi.zi_layer_norm_bwd, n, *args[:9], A, 1 << 30)


def test_norm_workspace(zi):
    n = norm(zi)
    need = zi.zi_layer_norm_bwd_bytes(4, 16)
    assert need == 4 * 2 * 16 * 4
    assert zi.zi_layer_norm_bwd_bytes(0, 16) == 0 and zi.zi_layer_norm_bwd_bytes(-1, 16) == 0
    refused(zi, "ZI_ERR_BUDGET", zi.zi_layer_norm_bwd, n, A, A, A, A, A, A, A, A, A, A, need - 1)
    refused(zi, "ZI_ERR_BUDGET", zi.zi_layer_norm_bwd, n, A, A, A, A, A, A, A, A, None, None, need)
    refused(zi, "ZI_ERR_ALIGN", zi.zi_layer_norm_bwd, n, A, A, A, A, A, A, A, A, A, A + 16, need)


def test_null_problem(zi):
    null = ctypes.POINTER(zi.zi_norm)()
    assert zi._lib.zi_layer_norm_fwd(null, A, A, A, A, A, A, A, A, None) == zi.ZI_ERR_ARG
    assert zi._lib.zi_layer_norm_bwd(null, A, A, A, A, A, A, A, A, A, A, 0, None) == zi.ZI_ERR_ARG
    null = ctypes.POINTER(zi.zi_embedding)()
    assert zi._lib.zi_embedding_fwd(null, A, A, A, None) == zi.ZI_ERR_ARG
    assert zi._lib.zi_embedding_bwd(null, A, A, A, A, 0, None) == zi.ZI_ERR_ARG


EMB_BAD = [
    (dict(T=-1), "ZI_ERR_SHAPE"), (dict(T=(1 << 27) + 1), "ZI_ERR_SHAPE"), (dict(V=0), "ZI_ERR_SHAPE"),
    (dict(V=1 << 31), "ZI_ERR_SHAPE"), (dict(D=0), "ZI_ERR_SHAPE"), (dict(D=65535 * 2048 + 1), "ZI_ERR_SHAPE"),
    (dict(ldw=8), "ZI_ERR_SHAPE"), (dict(ldx=-16), "ZI_ERR_SHAPE"), (dict(w_dtype=0), "ZI_ERR_ARG"),
    (dict(x_dtype=9), "ZI_ERR_ARG"), (dict(scale=float("nan")), "ZI_ERR_ARG"), (dict(scale=float("inf")), "ZI_ERR_ARG"),
]


@pytest.mark.parametrize("bad,status", EMB_BAD)
def test_embedding_problem(zi, bad, status):
    p = emb(zi, **bad)
    refused(zi, status, zi.zi_embedding_fwd, p, A, A, A)
    refused(zi, status, zi.zi_embedding_bwd, p, A, A, A, A, 1 << 40)


def test_embedding_pointers(zi):
    p = emb(zi)
    for k in range(3):
        args = [A, A, A]
        args[k] = None
        refused(zi, "ZI_ERR_ARG", zi.zi_embedding_fwd, p, *args)
        refused(zi, "ZI_ERR_ARG", zi.zi_embedding_bwd, p, *args, A, 1 << 30)
        args = [A, A, A]
        args[k] += 4 if k == 0 else 1
        refused(zi, "ZI_ERR_ALIGN", zi.zi_embedding_fwd, p, *args)
        refused(zi, "ZI_ERR_ALIGN", zi.zi_embedding_bwd, p, *args, A, 1 << 30)


def test_embedding_workspace(zi):
    p = emb(zi)
    need = zi.zi_embedding_bwd_bytes(4, 10, 16)
    assert need > 0 and zi.zi_embedding_bwd_bytes(0, 10, 16) == 0
    refused(zi, "ZI_ERR_BUDGET", zi.zi_embedding_bwd, p, A, A, A, A, need - 1)
    refused(zi, "ZI_ERR_BUDGET", zi.zi_embedding_bwd, p, A, A, A, None, need)
    refused(zi, "ZI_ERR_ALIGN", zi.zi_embedding_bwd, p, A, A, A, A + 128, need)


def orth(zi, **kw):
    d = dict(M=100, K=40, ldg=0, ldo=0, dtype=zi.ZI_BF16, steps=5, a=3.4445, b=-4.775, c=2.0315, eps=1e-7)
    d.update(kw)
    return zi.zi_orth(*[d[k] for k, _ in zi.zi_orth._fields_])


ORTH_BAD = [
    (dict(M=0), "ZI_ERR_SHAPE"), (dict(K=0), "ZI_ERR_SHAPE"), (dict(M=262145), "ZI_ERR_SHAPE"),
    (dict(K=262145), "ZI_ERR_SHAPE"), (dict(ldg=39), "ZI_ERR_SHAPE"), (dict(ldo=-1), "ZI_ERR_SHAPE"),
    (dict(dtype=0), "ZI_ERR_ARG"), (dict(dtype=4), "ZI_ERR_ARG"), (dict(steps=0), "ZI_ERR_ARG"),
    (dict(steps=101), "ZI_ERR_ARG"), (dict(a=float("nan")), "ZI_ERR_ARG"), (dict(b=float("inf")), "ZI_ERR_ARG"),
    (dict(c=float("inf")), "ZI_ERR_ARG"), (dict(eps=-1e-7), "ZI_ERR_ARG"), (dict(eps=float("nan")), "ZI_ERR_ARG"),
]


@pytest.mark.parametrize("bad,status", ORTH_BAD)
def test_orth_problem(zi, bad, status):
    refused(zi, status, zi.zi_orthogonalize, orth(zi, **bad), A, A, A, 1 << 40)


def test_orth_pointers_and_workspace(zi):
    o = orth(zi)
    need = zi.zi_orthogonalize_bytes(100, 40)
    assert need > 0 and zi.zi_orthogonalize_bytes(0, 40) == 0 and zi.zi_orthogonalize_bytes(40, 262145) == 0
    refused(zi, "ZI_ERR_ARG", zi.zi_orthogonalize, o, None, A, A, need)
    refused(zi, "ZI_ERR_ARG", zi.zi_orthogonalize, o, A, None, A, need)
    refused(zi, "ZI_ERR_ALIGN", zi.zi_orthogonalize, o, A + 1, A, A, need)
    refused(zi, "ZI_ERR_ALIGN", zi.zi_orthogonalize, o, A, A + 1, A, need)
    refused(zi, "ZI_ERR_ALIGN", zi.zi_orthogonalize, o, A, A, A + 128, need)
    refused(zi, "ZI_ERR_BUDGET", zi.zi_orthogonalize, o, A, A, A, need - 1)
    refused(zi, "ZI_ERR_BUDGET", zi.zi_orthogonalize, o, A, A, None, need)
    null = ctypes.POINTER(zi.zi_orth)()
    assert zi._lib.zi_orthogonalize(null, A, A, A, need, None) == zi.ZI_ERR_ARG


def test_nothing_to_do(zi):
    """No rows: no launch, so these pass without a GPU."""
    zi.zi_layer_norm_fwd(norm(zi, T=0), None, None, None, None, None, None, None, None)
    zi.zi_layer_norm_bwd(norm(zi, T=0), None, None, None, None, None, None, None, None, None, None, 0)
    zi.zi_embedding_fwd(emb(zi, T=0), None, A, None)
    zi.zi_embedding_bwd(emb(zi, T=0, accumulate=1), None, None, A, None, 0)


def test_torch_layer(zi):
    from offload_memory_centric_amd import layers
    X = torch.zeros((4, 16), dtype=torch.float16)
    v = torch.zeros(16)
    with pytest.raises(ValueError):  # not on the device
        layers.layer_norm_fwd(X, v, v, X)
    with pytest.raises(ValueError):
        layers.layer_norm_fwd(X[0], v, v, X)
    with pytest.raises(TypeError):
        layers.embedding_fwd(torch.zeros(4), X, X)
    with pytest.raises(ValueError):
        layers.embedding_fwd(torch.zeros(4, dtype=torch.int64), X, X)


def test_structs_match_the_header(zi, tmp_path):
    import os
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("needs gcc")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    structs = ["zi_norm", "zi_embedding", "zi_orth"]
    body = ""
    for name in structs:
        body += 'printf("%s . %%zu\\n", sizeof(%s));' % (name, name)
        for field, _ in getattr(zi, name)._fields_:
            body += 'printf("%s %s %%zu\\n", offsetof(%s, %s));' % (name, field, name, field)
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "zi.h"\nint main(void) {%s return 0;}\n' % body)
    exe = str(tmp_path / "layout")
    subprocess.run(["gcc", "-std=c11", "-I", os.path.join(root, "include"), str(src), "-o", exe], check=True)
    out = subprocess.run([exe], capture_output=True, text=True, check=True).stdout
    for line in out.strip().split("\n"):
        name, field, value = line.split()
        cls = getattr(zi, name)
        assert (ctypes.sizeof(cls) if field == "." else getattr(cls, field).offset) == int(value), line
