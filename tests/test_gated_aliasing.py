"""Outputs of the gated recurrence, the conv's backward pass and the 4-bit products that share memory with their
inputs: refused on the host before any launch, wherever in the input they lie; columns of one buffer are not
(fake aligned addresses, with an injected launch failure behind the checks: nothing is dereferenced)."""
import pytest

from tests.test_gated_refusals import A, ARG, CUDA, backward, conv, lib, matvec, scan, step  # noqa: F401

T, C = 40, 64  # of the fake calls: rows of 128 bytes, of ab 256
X, AB, DY = A, 2 * A, 6 * A


@pytest.fixture(autouse=True)
def injected(monkeypatch):
    monkeypatch.setenv("LA_FAULT_INJECT", "launch")


def into(base, rows, width):
    """Addresses at which an output of 128-byte rows touches `rows` rows of `width` bytes, and two that do not."""
    end = base + rows * width
    return [base, base + 16, base + width, end - width, end - 16, base - 128 * rows + 16, base - 16], [end, base - 128 * rows]


def test_scan(lib):  # noqa: F811
    for base, width in ((X, 128), (AB, 256)):
        hit, miss = into(base, T, width)
        for y in hit:
            assert scan(lib, y=y) == ARG and "alias" in lib.last_error(), hex(y - base)
        for y in miss:
            assert scan(lib, y=y) == CUDA


def test_scan_of_columns_of_one_buffer(lib):  # noqa: F811
    wide = dict(x=A, ab=A + 128, xs=256, abs=256, ys=256)  # x | a | b | y, 64 columns each
    assert scan(lib, y=A + 384, **wide) == CUDA
    for col in (0, 8, 56, 64, 128, 184, 200, 248):  # y reaches into x, a, b or the next row's x
        assert scan(lib, y=A + 2 * col, **wide) == ARG, col
    # the same columns, rows further on: still those columns
    assert scan(lib, y=A + 384 + 512 * 5, **wide) == CUDA and scan(lib, y=A + 128 + 512 * 5, **wide) == ARG
    assert scan(lib, x=A + 384, ab=A, y=A + 256, xs=256, abs=256, ys=256) == CUDA  # y before x
    assert scan(lib, x=A + 384, ab=A, y=A + 264, xs=256, abs=256, ys=256) == ARG
    assert scan(lib, y=A + 384, **{**wide, "ys": 264}) == ARG  # another stride in the same place
    one = dict(T=1, maxt=1, B=1, cu=None)  # a single row's stride says nothing
    assert scan(lib, x=A, ab=A + 128, y=A + 384, xs=64, abs=128, ys=64, **one) == CUDA
    assert scan(lib, x=A, ab=A + 128, y=A + 368, xs=64, abs=128, ys=64, **one) == ARG


def test_scan_backward(lib):  # noqa: F811
    for out, key in ((7 * A, "dx"), (8 * A, "dab")):
        for base, width in ((X, 128), (AB, 256), (DY, 128)):
            for at in into(base, T, width)[0][:5]:
                assert backward(lib, **{key: at}) == ARG and "alias" in lib.last_error()
        assert backward(lib, **{key: 5 * A + 16}) == ARG  # inside what the forward pass saved
    assert backward(lib, dab=7 * A + 64) == ARG and backward(lib, dx=8 * A + 256) == ARG
    assert backward(lib, dx=A, dab=A + 128, x=9 * A, dxs=192, dabs=192) == CUDA  # dx | da | db
    assert backward(lib, dx=A, dab=A + 112, x=9 * A, dxs=192, dabs=192) == ARG
    assert backward(lib) == CUDA


def test_step(lib):  # noqa: F811
    for base, width in ((X, 128), (AB, 256)):
        hit, miss = into(base, 4, width)
        assert all(step(lib, y=y) == ARG for y in hit) and step(lib, y=miss[0]) == CUDA
    assert step(lib, x=A, ab=A + 128, y=A + 384, xs=256, abs=256, ys=256) == CUDA
    assert step(lib, x=A, ab=A + 128, y=A + 256, xs=256, abs=256, ys=256) == ARG  # over b


def test_conv_backward(lib):  # noqa: F811
    for base in (A, 2 * A):
        hit, miss = into(base, T, 128)
        assert all(conv(lib, dx=p) == ARG for p in hit) and conv(lib, dx=miss[0]) == CUDA
    assert conv(lib, x=A, dout=A + 128, dx=A + 256, xs=192, dos=192, dxs=192) == CUDA
    assert conv(lib, x=A, dout=A + 128, dx=A + 240, xs=192, dos=192, dxs=192) == ARG


def test_products(lib):  # noqa: F811
    side = dict(M=4, N=10, K=256, ldx=272, ldy=272)
    assert matvec(lib, x=A, y=A + 512, **side) == CUDA  # x | y in rows of 272
    assert matvec(lib, x=A + 32, y=A, **side) == CUDA   # y | x: ten outputs of two bytes before x
    assert matvec(lib, x=A, y=A + 510, **side) == ARG and matvec(lib, x=A, y=A + 526, **side) == ARG
    assert matvec(lib, x=A + 16, y=A, **side) == ARG
    assert matvec(lib, x=A, y=A + 512, **{**side, "ldy": 280}) == ARG
    assert matvec(lib, x=A, y=A + 512, M=1, N=10, K=256, ldx=256, ldy=10) == CUDA
    assert matvec(lib, x=A, y=A + 510, M=1, N=10, K=256, ldx=256, ldy=10) == ARG
