"""The workspaces of the norm's backward and of the embedding's gradient: what holds the largest batch and the widest
rows holds every smaller one's."""
import pytest


@pytest.fixture(scope="module")
def zi():
    from offload_memory_centric_amd import zi as m
    return m


TS = [0, 1, 2, 15, 16, 17, 63, 64, 255, 256, 257, 511, 512, 513, 1023, 1024, 1025, 4096, 4097, 8000, 8191, 8192, 8193, 10000,
      16384, 16385, 32768, 32769, 100000, 1 << 27]
DS = [1, 7, 8, 100, 511, 512, 513, 514, 600, 1024, 1025, 4095, 4096, 4097, 5000, 8191, 8192, 8193, 9000, 16384, 16385, 25600,
      32768, 32769, 100000]


def falls(size, xs):
    return [(a, b, size(a), size(b)) for a, b in zip(xs, xs[1:]) if size(a) > size(b)]


@pytest.mark.parametrize("D", DS)
def test_embedding_in_tokens(zi, D):
    assert not falls(lambda T: zi.zi_embedding_bwd_bytes(T, 1000, D), TS)


@pytest.mark.parametrize("T", TS)
def test_embedding_in_columns(zi, T):
    assert not falls(lambda D: zi.zi_embedding_bwd_bytes(T, 1000, D), DS)


@pytest.mark.parametrize("D", DS)
def test_norm_in_rows(zi, D):
    assert not falls(lambda T: zi.zi_layer_norm_bwd_bytes(T, D), TS)


@pytest.mark.parametrize("T", TS)
def test_norm_in_columns(zi, T):
    assert not falls(lambda D: zi.zi_layer_norm_bwd_bytes(T, D), DS)
