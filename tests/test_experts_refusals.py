"""Refusals of the router, the grouped products, the combination and the adapters: they come before anything is
enqueued, so they are tested without a GPU, with addresses that nothing reads."""
import contextlib
import ctypes

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode


@pytest.fixture(scope="module")
def zi():
    from offload_memory_centric_amd import zi as m
    return m


A = 1 << 20  # a 256-byte aligned address
BIG = 1 << 40

DEFAULTS = {
    "zi_route": dict(T=100, ldl=0, ldd=0, E=16, k=2, dtype=1, normalize=1),
    "zi_grouped": dict(R=64, K=32, M=48, ldx=0, ldy=0, lda=0, ldw=0, ldg=0, E=4, dtype=1, out_dtype=1, gelu=1, accumulate=0),
    "zi_combine": dict(T=10, R=20, D=24, ldz=0, ldy=0, lddz=0, k=2, dtype=1),
    "zi_adapters": dict(T=100, K=32, M=48, ldx=0, lddx=0, lddx0=0, ldy=0, ldy0=0, S=4, N=3, r=8, dtype=1, out_dtype=1,
                        accumulate=0),
}


def make(zi, name, **kw):
    d = dict(DEFAULTS[name], **kw)
    cls = getattr(zi, name)
    assert set(d) == {f for f, _ in cls._fields_}
    return cls(*[d[f] for f, _ in cls._fields_])


def calls(zi, name):
    """The entry points that take this problem, each with the number of pointers before the workspace."""
    return {"zi_route": [(zi.zi_route_fwd, 6, True), (zi.zi_route_bwd, 5, False)],
            "zi_grouped": [(zi.zi_grouped_fwd, 5, False), (zi.zi_grouped_dx, 5, False), (zi.zi_grouped_dw, 4, False)],
            "zi_combine": [(zi.zi_combine_fwd, 4, False), (zi.zi_combine_bwd, 6, False)],
            "zi_adapters": [(zi.zi_adapters_fwd, 9, True), (zi.zi_adapters_bwd, 12, True)]}[name]


def refused(zi, status, f, *args):
    with pytest.raises(zi.ZiError) as e:
        f(*args)
    assert e.value.status == getattr(zi, status), str(e.value)
    assert zi.zi_last_error()


def call(f, problem, pointers, work, need=BIG):
    f(problem, *pointers, *((A, need) if work else ()))


BAD = [
    ("zi_route", dict(T=-1), "ZI_ERR_SHAPE"), ("zi_route", dict(T=1 << 30), "ZI_ERR_SHAPE"), ("zi_route", dict(E=0), "ZI_ERR_SHAPE"),
    ("zi_route", dict(E=1025), "ZI_ERR_SHAPE"), ("zi_route", dict(k=0), "ZI_ERR_SHAPE"), ("zi_route", dict(k=17), "ZI_ERR_SHAPE"),
    ("zi_route", dict(E=100, k=33), "ZI_ERR_SHAPE"), ("zi_route", dict(ldl=15), "ZI_ERR_SHAPE"),
    ("zi_route", dict(ldd=-1), "ZI_ERR_SHAPE"), ("zi_route", dict(dtype=0), "ZI_ERR_ARG"),
    ("zi_grouped", dict(R=-1), "ZI_ERR_SHAPE"), ("zi_grouped", dict(R=(1 << 30) + 1), "ZI_ERR_SHAPE"),
    ("zi_grouped", dict(K=12), "ZI_ERR_SHAPE"), ("zi_grouped", dict(M=0), "ZI_ERR_SHAPE"), ("zi_grouped", dict(M=20), "ZI_ERR_SHAPE"),
    ("zi_grouped", dict(K=(1 << 20) + 8), "ZI_ERR_SHAPE"), ("zi_grouped", dict(E=0), "ZI_ERR_SHAPE"),
    ("zi_grouped", dict(E=4097), "ZI_ERR_SHAPE"), ("zi_grouped", dict(ldx=24), "ZI_ERR_SHAPE"), ("zi_grouped", dict(ldx=36), "ZI_ERR_SHAPE"),
    ("zi_grouped", dict(ldy=40), "ZI_ERR_SHAPE"), ("zi_grouped", dict(ldw=-8), "ZI_ERR_SHAPE"),
    ("zi_grouped", dict(lda=(1 << 20) + 8), "ZI_ERR_SHAPE"), ("zi_grouped", dict(ldg=48 * 32 - 8), "ZI_ERR_SHAPE"),
    ("zi_grouped", dict(ldg=48 * 32 + 4), "ZI_ERR_SHAPE"), ("zi_grouped", dict(dtype=3, out_dtype=3), "ZI_ERR_ARG"),
    ("zi_grouped", dict(out_dtype=2), "ZI_ERR_ARG"),
    ("zi_combine", dict(T=-1), "ZI_ERR_SHAPE"), ("zi_combine", dict(T=1 << 30), "ZI_ERR_SHAPE"), ("zi_combine", dict(R=-1), "ZI_ERR_SHAPE"),
    ("zi_combine", dict(R=1 << 31), "ZI_ERR_SHAPE"), ("zi_combine", dict(D=0), "ZI_ERR_SHAPE"), ("zi_combine", dict(k=0), "ZI_ERR_SHAPE"),
    ("zi_combine", dict(k=1025), "ZI_ERR_SHAPE"), ("zi_combine", dict(ldz=23), "ZI_ERR_SHAPE"), ("zi_combine", dict(dtype=9), "ZI_ERR_ARG"),
    ("zi_adapters", dict(T=-1), "ZI_ERR_SHAPE"), ("zi_adapters", dict(T=(1 << 23) + 1), "ZI_ERR_SHAPE"),
    ("zi_adapters", dict(K=4), "ZI_ERR_SHAPE"), ("zi_adapters", dict(M=50), "ZI_ERR_SHAPE"), ("zi_adapters", dict(N=0), "ZI_ERR_SHAPE"),
    ("zi_adapters", dict(N=65536), "ZI_ERR_SHAPE"), ("zi_adapters", dict(r=0), "ZI_ERR_SHAPE"), ("zi_adapters", dict(r=257), "ZI_ERR_SHAPE"),
    ("zi_adapters", dict(S=-1), "ZI_ERR_SHAPE"), ("zi_adapters", dict(ldx=24), "ZI_ERR_SHAPE"), ("zi_adapters", dict(ldy=52), "ZI_ERR_SHAPE"),
    ("zi_adapters", dict(lddx=24), "ZI_ERR_SHAPE"), ("zi_adapters", dict(lddx0=-8), "ZI_ERR_SHAPE"),
    ("zi_adapters", dict(dtype=3, out_dtype=3), "ZI_ERR_ARG"), ("zi_adapters", dict(dtype=1, out_dtype=2), "ZI_ERR_ARG"),
]


@pytest.mark.parametrize("name,bad,status", BAD)
def test_problem(zi, name, bad, status):
    for f, n, work in calls(zi, name):
        refused(zi, status, call, f, make(zi, name, **bad), [A] * n, work)


# entry point: its required pointers, and those that must be aligned to 16 bytes
REQUIRED = {"zi_route_fwd": (range(6), ()), "zi_route_bwd": ((1, 2, 3, 4), ()),
            "zi_grouped_fwd": ((0, 1, 2, 3), (0, 1, 3, 4)), "zi_grouped_dx": ((0, 1, 2, 4), (0, 1, 3, 4)),
            "zi_grouped_dw": ((0, 1, 2, 3), (0, 1, 3)), "zi_combine_fwd": (range(4), ()), "zi_combine_bwd": (range(6), ()),
            "zi_adapters_fwd": ((0, 1, 2, 3, 4, 5, 7), (0, 1, 2, 6, 7)),
            "zi_adapters_bwd": ((0, 1, 2, 3, 4, 5, 6, 7, 10, 11), (0, 1, 3, 4, 8, 9, 10, 11))}


@pytest.mark.parametrize("name", list(DEFAULTS))
def test_pointers(zi, name):
    for f, n, work in calls(zi, name):
        required, wide = REQUIRED[f.__name__]
        # distinct addresses: an output that is an input has a meaning of its own
        at = [A + 4096 * i for i in range(n)]
        problem = make(zi, name)
        for i in required:
            refused(zi, "ZI_ERR_ARG", call, f, problem, at[:i] + [None] + at[i + 1:], work)
        for i in range(n):
            refused(zi, "ZI_ERR_ALIGN", call, f, problem, at[:i] + [at[i] + 1] + at[i + 1:], work)
        for i in wide:
            refused(zi, "ZI_ERR_ALIGN", call, f, problem, at[:i] + [at[i] + 8] + at[i + 1:], work)


def test_combinations(zi):
    # a normalised router's gradient needs the weights, the other the logits
    refused(zi, "ZI_ERR_ARG", zi.zi_route_bwd, make(zi, "zi_route", normalize=1), A, A, None, A, A)
    refused(zi, "ZI_ERR_ARG", zi.zi_route_bwd, make(zi, "zi_route", normalize=0), None, A, A, A, A)
    # A belongs to GeLU, GeLU to 16-bit outputs
    refused(zi, "ZI_ERR_ARG", zi.zi_grouped_fwd, make(zi, "zi_grouped", gelu=0), A, A, A, A, A)
    refused(zi, "ZI_ERR_ARG", zi.zi_grouped_fwd, make(zi, "zi_grouped", out_dtype=3), A, A, A, A, None)
    refused(zi, "ZI_ERR_ARG", zi.zi_grouped_dx, make(zi, "zi_grouped", out_dtype=3), A, A, A, A, A)
    refused(zi, "ZI_ERR_SHAPE", zi.zi_grouped_fwd, make(zi, "zi_grouped", lda=40), A, A, A, A, A)
    refused(zi, "ZI_ERR_SHAPE", zi.zi_grouped_dx, make(zi, "zi_grouped", lda=24), A, A, A, A, A)
    refused(zi, "ZI_ERR_ARG", zi.zi_grouped_dw, make(zi, "zi_grouped", accumulate=1), A, A, A, A)
    # an output in place has its input's stride
    p = make(zi, "zi_adapters", ldy=56, ldy0=48)
    refused(zi, "ZI_ERR_SHAPE", zi.zi_adapters_fwd, p, A, A, A, A, A, A, A, A, A, A, BIG)
    p = make(zi, "zi_adapters", lddx=40, lddx0=32)
    refused(zi, "ZI_ERR_SHAPE", zi.zi_adapters_bwd, p, *[A] * 12, A, BIG)
    refused(zi, "ZI_ERR_ARG", zi.zi_adapters_bwd, make(zi, "zi_adapters"), *[A] * 8, A, None, A, A, A, BIG)
    for f in (zi.zi_route_fwd, zi.zi_route_bwd, zi.zi_grouped_fwd, zi.zi_grouped_dx, zi.zi_grouped_dw, zi.zi_combine_fwd,
              zi.zi_combine_bwd, zi.zi_adapters_fwd, zi.zi_adapters_bwd):
        name = f.__name__
        lib = getattr(zi._lib, name)
        assert lib(None, *[0] * (len(lib.argtypes) - 1)) == zi.ZI_ERR_ARG


def test_workspaces(zi):
    p = make(zi, "zi_route")
    need = zi.zi_route_fwd_bytes(100, 16, 2)
    assert need > 0
    refused(zi, "ZI_ERR_BUDGET", zi.zi_route_fwd, p, *[A] * 6, A, need - 1)
    refused(zi, "ZI_ERR_BUDGET", zi.zi_route_fwd, p, *[A] * 6, None, BIG)
    refused(zi, "ZI_ERR_ALIGN", zi.zi_route_fwd, p, *[A] * 6, A + 128, BIG)
    at = [A + 4096 * i for i in range(12)]
    p = make(zi, "zi_adapters")
    for f, n, size in ((zi.zi_adapters_fwd, 9, zi.zi_adapters_fwd_bytes), (zi.zi_adapters_bwd, 12, zi.zi_adapters_bwd_bytes)):
        need = size(100, 8)
        refused(zi, "ZI_ERR_BUDGET", f, p, *at[:n], A, need - 1)
        refused(zi, "ZI_ERR_BUDGET", f, p, *at[:n], None, BIG)
        refused(zi, "ZI_ERR_ALIGN", f, p, *at[:n], A + 128, BIG)


def test_workspaces_of_more_rows_serve_fewer(zi):
    rows = [0, 1, 2, 3, 63, 64, 65, 100, 127, 128, 129, 511, 512, 513, 1000, 2047, 2048, 2049, 4096, 30000, 32767, 32768, 32769,
            65536, 65537, 100000, 131073, 1 << 20, 1 << 23]
    sizes = [lambda T: zi.zi_route_fwd_bytes(T, 256, 4), lambda T: zi.zi_adapters_fwd_bytes(T, 16),
             lambda T: zi.zi_adapters_bwd_bytes(T, 64)]
    for size in sizes:
        got = [size(T) for T in rows]
        assert got == sorted(got)


def test_nothing_to_do(zi):
    """No rows: no launch, so these pass without a GPU."""
    zi.zi_route_bwd(make(zi, "zi_route", T=0), None, None, None, None, None)
    zi.zi_grouped_fwd(make(zi, "zi_grouped", R=0), None, None, None, None, None)
    zi.zi_grouped_dx(make(zi, "zi_grouped", R=0), None, None, None, None, None)
    zi.zi_grouped_dw(make(zi, "zi_grouped", R=0, out_dtype=3, accumulate=1), None, None, A, A)
    zi.zi_combine_fwd(make(zi, "zi_combine", T=0), None, None, None, None)
    zi.zi_combine_bwd(make(zi, "zi_combine", T=0), None, None, None, None, None, None)
    zi.zi_adapters_fwd(make(zi, "zi_adapters", T=0), *[None] * 9, None, 0)
    zi.zi_adapters_bwd(make(zi, "zi_adapters", T=0, accumulate=1), *[None] * 10, A, A, None, 0)


def test_structs_match_the_header(zi, tmp_path):
    import os
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("needs gcc")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    body = 'printf("experts . %d\\n", ZI_ROUTE_EXPERTS); printf("groups . %d\\n", ZI_GROUPS_MOST);'
    for name in DEFAULTS:
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
        if name in ("experts", "groups"):
            assert int(value) == (zi.ZI_ROUTE_EXPERTS if name == "experts" else zi.ZI_GROUPS_MOST)
            continue
        cls = getattr(zi, name)
        assert (ctypes.sizeof(cls) if field == "." else getattr(cls, field).offset) == int(value), line


# ---- the torch layer -------------------------------------------------------------------------

T, E, K, M, N, S, r, k = 6, 4, 16, 24, 3, 2, 8, 2
F16, BF16, F32, U8, I32, I64 = torch.float16, torch.bfloat16, torch.float32, torch.uint8, torch.int32, torch.int64
ADAPTERS = dict(A=((N, r, K), F16), B=((N, r, M), F16), offsets=((S + 1,), I32), ids=((S,), I32), scales=((N,), F32))
# entry point: its tensors, in order
CALLS = {
    "route_fwd": dict(logits=((T, E), BF16), ids=((T, k), I32), weights=((T, k), F32), offsets=((E + 1,), I32),
                      rows=((T * k,), I32), slots=((T, k), I32), work=((4096,), U8)),
    "route_bwd": dict(logits=((T, E), BF16), ids=((T, k), I32), weights=((T, k), F32), dweights=((T, k), F32),
                      dlogits=((T, E), BF16)),
    "grouped_fwd": dict(X=((T, K), F16), W=((E, M, K), F16), offsets=((E + 1,), I32), Y=((T, M), F16), A=((T, M), F16)),
    "grouped_dx": dict(dY=((T, M), F16), W=((E, M, K), F16), offsets=((E + 1,), I32), dX=((T, K), F16), A=((T, K), F16)),
    "grouped_dw": dict(X=((T, K), F16), dY=((T, M), F16), offsets=((E + 1,), I32), dW=((E, M, K), F32)),
    "combine_fwd": dict(Z=((T * k, K), F16), slots=((T, k), I32), weights=((T, k), F32), Y=((T, K), F16)),
    "combine_bwd": dict(dY=((T, K), F16), Z=((T * k, K), F16), slots=((T, k), I32), weights=((T, k), F32),
                        dZ=((T * k, K), F16), dweights=((T, k), F32)),
    "adapters_fwd": dict(X=((T, K), F16), **ADAPTERS, Y=((T, M), F32), work=((1 << 20,), U8), Y0=((T, M), F32), U=((r, T), F32)),
    "adapters_bwd": dict(X=((T, K), F16), dY=((T, M), F16), U=((r, T), F32), **ADAPTERS, dA=((N, r, K), F32),
                         dB=((N, r, M), F32), work=((1 << 20,), U8), dX=((T, K), F16), dX0=((T, K), F16)),
}


@pytest.fixture(scope="module")
def layers():
    from offload_memory_centric_amd import layers as m
    return m


def tensors(name, device="cuda:0", **other):
    """Tensors without memory; `other`: shape, dtype or device of some of them."""
    with FakeTensorMode():
        return {n: torch.empty(other.get(n, {}).get("shape", shape), dtype=other.get(n, {}).get("dtype", dtype),
                               device=other.get(n, {}).get("device", device)) for n, (shape, dtype) in CALLS[name].items()}


@pytest.fixture
def made(layers, monkeypatch):
    """The library calls that are made, each with the device that is current then."""
    got, current = [], [0]

    @contextlib.contextmanager
    def device(index):
        before, current[0] = current[0], index
        yield
        current[0] = before

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(layers, "_device", lambda: current[0], raising=False)
    monkeypatch.setattr(layers, "_current", lambda index: 1000 + index)
    for name in CALLS:
        monkeypatch.setattr(layers.zi, "zi_" + name, lambda *a: got.append((current[0], a[-1])))
    return got


@pytest.mark.parametrize("name,moved", [(c, n) for c in CALLS for n in CALLS[c]])
@pytest.mark.parametrize("device", ["cuda:1", "cpu"])
def test_one_device(layers, made, name, moved, device):
    with pytest.raises(ValueError):
        getattr(layers, name)(**tensors(name, **{moved: dict(device=device)}))
    assert not made


@pytest.mark.parametrize("name", CALLS)
def test_current_device(layers, made, name):
    getattr(layers, name)(**tensors(name, "cuda:1"))
    getattr(layers, name)(**tensors(name, "cuda:0"), stream=77)
    assert made == [(1, 1001), (0, 77)]


@pytest.mark.parametrize("name,wrong", [(c, n) for c in CALLS for n in CALLS[c] if n != "work"])
def test_types_and_shapes(layers, made, name, wrong):
    shape, _ = CALLS[name][wrong]
    with pytest.raises(TypeError):
        getattr(layers, name)(**tensors(name, **{wrong: dict(dtype=I64)}))
    # a tensor that gives a size is contradicted by the others
    for at in range(len(shape)):
        if (name, wrong, at) == ("combine_fwd", "Z", 0):
            continue  # any number of rows
        with pytest.raises(ValueError):
            getattr(layers, name)(**tensors(name, **{wrong: dict(shape=shape[:at] + (shape[at] + 8,) + shape[at + 1:])}))
    with pytest.raises(ValueError):
        getattr(layers, name)(**tensors(name, **{wrong: dict(shape=shape + (1,))}))
    assert not made


def test_strides(layers, made):
    with FakeTensorMode():
        t = {n: torch.empty(s, dtype=d, device="cuda:0") for n, (s, d) in CALLS["grouped_fwd"].items()}
        for W in (torch.empty((E, K, M), dtype=F16, device="cuda:0").transpose(1, 2),
                  torch.empty((M, K), dtype=F16, device="cuda:0").expand(E, M, K)):
            with pytest.raises(ValueError):
                layers.grouped_fwd(**dict(t, W=W))
        layers.grouped_fwd(**dict(t, W=torch.empty((E, 2 * M, K), dtype=F16, device="cuda:0")[:, :M]))
        layers.grouped_fwd(**dict(t, W=torch.empty((E, M, 2 * K), dtype=F16, device="cuda:0")[:, :, :K]))
    assert len(made) == 2


# ---- the assembly check of builtin MFMAs ------------------------------------------------------

def test_early_reads_of_a_result():
    """A result read too soon is found along the listing and behind a branch; one read in time is not."""
    from offload_memory_centric_amd import asm_check

    def findings(*lines):
        return asm_check.early_reads(list(enumerate(lines, 1)))

    mfma = "\tv_mfma_f32_16x16x32_f16 a[0:3], v[0:3], v[4:7], a[0:3]"
    read = "\tds_write_b128 v8, a[0:3]"
    assert findings(mfma, read)
    assert findings(mfma, "\ts_nop 5", read)
    assert not findings(mfma, "\ts_nop 6", read)
    assert findings(".LBB0_1:", mfma, "\ts_cbranch_vccnz .LBB0_1", read)
    assert findings(".LBB0_1:", read, "\ts_nop 7", mfma, "\ts_cbranch_vccnz .LBB0_1", "\ts_endpgm")
    assert not findings(".LBB0_1:", "\ts_nop 6", read, mfma, "\ts_cbranch_vccnz .LBB0_1", "\ts_nop 6", read)
    assert not findings(mfma, mfma, "\tv_add_f32 v8, v9, v10")
    copy = ["\ts_mov_b32 m0, s3", "\tbuffer_load_dwordx4 v1, s[4:7], 0 offen lds"]
    assert not findings(*copy) and findings(copy[0], mfma) and findings("\tv_mov_b32 v1, m0")
    slow = "\tv_mfma_f32_16x16x4_f32 a[0:3], v0, v1, a[0:3]"
    assert findings(slow, "\ts_nop 6", read) and not findings(slow, "\ts_nop 7", "\ts_nop 1", read)


def test_built_sources_have_none():
    import os
    from offload_memory_centric_amd import asm_check, build
    for src in build.BUILTIN_SOURCES:
        path = build.device_asm(src)
        if not os.path.exists(path):
            pytest.skip("no kept assembly")
        found = asm_check.check_file(path, check=asm_check.early_reads)
        assert found and not any(found.values()), {k: v for k, v in found.items() if v}
