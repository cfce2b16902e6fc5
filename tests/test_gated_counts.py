"""Streams and channels beyond what the kernels count in 32 bits are refused on the host (a search among 2^30 or
more streams adds two of their numbers; a block adds up to 255 to a channel's)."""
import pytest

from tests.test_gated_refusals import A, ARG, COUNT, CUDA, backward, conv, lib, scan, step  # noqa: F401

BIG = 2 ** 62


@pytest.fixture(autouse=True)
def injected(monkeypatch):
    monkeypatch.setenv("LA_FAULT_INJECT", "launch")  # behind the checks: nothing runs


@pytest.mark.parametrize("call", [scan, backward, conv])
def test_streams(lib, call):  # noqa: F811
    far = dict(wsb=BIG) if call is not backward else dict(wsb=BIG, sb=BIG, dx=1 << 50, dab=1 << 51)
    assert call(lib, B=2 ** 30 - 1, **far) == CUDA
    for B in (2 ** 30, 2 ** 31 - 1):
        assert call(lib, B=B, **far) == COUNT and str(2 ** 30 - 1) in lib.last_error()


def test_streams_of_a_step(lib):  # noqa: F811
    far = dict(maxb=2 ** 31 - 1, C=8, xs=8, abs=16, ys=8, x=1 << 40, ab=1 << 41, y=1 << 42)
    assert step(lib, B=2 ** 30 - 1, **far) == CUDA
    assert step(lib, B=2 ** 30, **far) == COUNT and step(lib, B=2 ** 31 - 1, **far) == COUNT


def test_channels(lib):  # noqa: F811
    most = 2 ** 31 - 1024
    one = dict(T=1, maxt=1, B=1, dtype=0)
    far = dict(x=1 << 40, ab=1 << 41, y=1 << 42)
    assert scan(lib, C=most, xs=most, abs=2 * most, ys=most, wsb=BIG, **far, **one) == CUDA
    assert step(lib, C=most, xs=most, abs=2 * most, ys=most, B=1, dtype=0, **far) == CUDA
    for C in (most + 4, 2 ** 31 - 4):
        assert scan(lib, C=C, xs=C, abs=2 * C, ys=C, wsb=BIG, **far, **one) == COUNT
        assert step(lib, C=C, xs=C, abs=2 * C, ys=C, B=1, dtype=0, **far) == COUNT
        assert backward(lib, C=C, xs=C, abs=2 * C, dys=C, dxs=C, dabs=2 * C, wsb=BIG, sb=BIG, **one) == COUNT
    blocks = 65535 * 512  # of the conv's grid
    far = dict(x=1 << 40, dout=1 << 41, dx=1 << 42)
    assert conv(lib, C=blocks, xs=blocks, dos=blocks, dxs=blocks, wsb=BIG, **far, **one) == CUDA
    assert conv(lib, C=blocks + 4, xs=blocks + 4, dos=blocks + 4, dxs=blocks + 4, wsb=BIG, **far, **one) == COUNT
