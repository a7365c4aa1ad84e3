"""The torch layer's operators on several devices: a call's tensors and stream are of one device, and the call is
made with that device as the current one.  Tensors without memory stand in for those of the devices."""
import contextlib
import types

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode


@pytest.fixture(scope="module")
def layers():
    from offload_memory_centric_amd import layers as m
    return m


T, D, V = 4, 16, 10
F16, BF16, F32, U8, I64 = torch.float16, torch.bfloat16, torch.float32, torch.uint8, torch.int64
# entry point: its tensors, in order
CALLS = {
    "layer_norm_fwd": dict(X=((T, D), F16), gamma=((D,), F32), beta=((D,), F32), Y=((T, D), F16), mean=((T,), F32),
                           rstd=((T,), F32), R=((T, D), F16), S=((T, D), F16)),
    "layer_norm_bwd": dict(dY=((T, D), F32), S=((T, D), F16), gamma=((D,), F32), mean=((T,), F32), rstd=((T,), F32),
                           dX=((T, D), F16), dgamma=((D,), F32), dbeta=((D,), F32), work=((4096,), U8), dS=((T, D), F16)),
    "embedding_fwd": dict(ids=((T,), I64), W=((V, D), F16), X=((T, D), F16)),
    "embedding_bwd": dict(ids=((T,), I64), dX=((T, D), F16), dW=((V, D), F32), work=((4096,), U8)),
    "orthogonalize": dict(G=((T, D), F16), O=((T, D), BF16), work=((4096,), U8)),
}


def tensors(call, device, other=None, moved=None):
    with FakeTensorMode():
        return {k: torch.empty(shape, dtype=dtype, device=moved if k == other else device)
                for k, (shape, dtype) in CALLS[call].items()}


@pytest.fixture
def calls(layers, monkeypatch):
    """The library calls that are made, each with the device that is current then."""
    made, current = [], [0]

    @contextlib.contextmanager
    def device(index):
        before, current[0] = current[0], index
        yield
        current[0] = before

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(layers, "_device", lambda: current[0], raising=False)
    monkeypatch.setattr(layers, "_current", lambda index: 1000 + index)
    for call in CALLS:
        monkeypatch.setattr(layers.zi, "zi_" + call, lambda *a: made.append((current[0], a[-1])))
    return made


@pytest.mark.parametrize("call,name", [(c, n) for c in CALLS for n in CALLS[c]])
@pytest.mark.parametrize("moved", ["cuda:1", "cpu"])
def test_one_device(layers, calls, call, name, moved):
    with pytest.raises(ValueError):
        getattr(layers, call)(**tensors(call, "cuda:0", name, moved))
    assert not calls


@pytest.mark.parametrize("call", list(CALLS))
@pytest.mark.parametrize("index", [0, 1])
def test_current_device(layers, calls, call, index):
    args = tensors(call, "cuda:%d" % index)
    getattr(layers, call)(**args)
    getattr(layers, call)(**args, stream=77)  # a handle says nothing of its device
    assert calls == [(index, 1000 + index), (index, 77)]
    assert layers._device() == 0


@pytest.mark.parametrize("call", list(CALLS))
def test_stream_of_another_device(layers, calls, call):
    args = tensors(call, "cuda:1")
    with pytest.raises(ValueError):
        getattr(layers, call)(**args, stream=types.SimpleNamespace(device=torch.device("cuda:0"), cuda_stream=5))
    assert not calls
    mine = types.SimpleNamespace(device=torch.device("cuda:1"), cuda_stream=5)
    getattr(layers, call)(**args, stream=mine)
    assert calls == [(1, mine)]
