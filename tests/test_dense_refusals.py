"""What the layer norm, the products with an epilogue and the gated feed-forward block refuse on the host, before
any CUDA call (fake aligned addresses; nothing is dereferenced), and what the binding refuses."""
import pytest
import torch

A = 0x10000000  # fake buffers lie this far apart
COUNT, ARG, UNSUPPORTED, CUDA = 2, 1, 3, 4
MOST = 2 ** 31 - 1024


@pytest.fixture(scope="module")
def lib(built_lib):
    import linear_attention_chunked_conv1d_gb300 as la
    la._load()
    return la


def norm(lib, **kw):
    a = dict(x=A, w=2 * A, b=3 * A, y=4 * A, stats=5 * A, rows=10, width=60, ldx=64, ldy=64, eps=1e-5, dtype=1)
    a.update(kw)
    return lib._load().la_layernorm_rows(a["x"], a["w"], a["b"], a["y"], a["stats"], a["rows"], a["width"], a["ldx"],
                                         a["ldy"], a["eps"], a["dtype"], 0)


def norm_backward(lib, **kw):
    a = dict(x=A, w=2 * A, stats=5 * A, dy=6 * A, dskip=7 * A, dx=8 * A, dw=9 * A, db=10 * A, rows=10, width=60, ldx=64,
             lddy=64, ldskip=64, lddx=64, dtype=1, ws=11 * A, wsb=1 << 20)
    a.update(kw)
    return lib._load().la_layernorm_rows_backward(
        a["x"], a["w"], a["stats"], a["dy"], a["dskip"], a["dx"], a["dw"], a["db"], a["rows"], a["width"], a["ldx"], a["lddy"],
        a["ldskip"], a["lddx"], a["dtype"], a["ws"], a["wsb"], 0)


def linear(lib, **kw):
    a = dict(x=A, w=2 * A, bias=3 * A, residual=4 * A, y=5 * A, saved=6 * A, sb=1 << 20, M=10, N=60, K=70, ldx=72, ldw=72,
             ldr=64, ldy=64, act=2)
    a.update(kw)
    return lib._load().la_linear(a["x"], a["w"], a["bias"], a["residual"], a["y"], a["saved"], a["sb"], a["M"], a["N"], a["K"],
                                 a["ldx"], a["ldw"], a["ldr"], a["ldy"], a["act"], 0)


def linear_backward(lib, **kw):
    a = dict(x=A, w=2 * A, saved=6 * A, sb=1 << 20, dy=7 * A, dx=8 * A, dw=9 * A, dbias=10 * A, M=10, N=60, K=70, ldx=72,
             ldw=72, lddy=64, lddx=72, lddw=72, act=2, ws=11 * A, wsb=1 << 20)
    a.update(kw)
    return lib._load().la_linear_backward(
        a["x"], a["w"], a["saved"], a["sb"], a["dy"], a["dx"], a["dw"], a["dbias"], a["M"], a["N"], a["K"], a["ldx"], a["ldw"],
        a["lddy"], a["lddx"], a["lddw"], a["act"], a["ws"], a["wsb"], 0)


def ffn(lib, **kw):
    a = dict(x=A, w=2 * A, w_up=3 * A, h=5 * A, saved=6 * A, sb=1 << 20, M=10, N=60, K=70, ldx=72, ldw=72, ldu=72, ldh=64, act=4)
    a.update(kw)
    return lib._load().la_gated_ffn(a["x"], a["w"], a["w_up"], a["h"], a["saved"], a["sb"], a["M"], a["N"], a["K"], a["ldx"],
                                    a["ldw"], a["ldu"], a["ldh"], a["act"], 0)


def ffn_backward(lib, **kw):
    a = dict(x=A, w=2 * A, w_up=3 * A, saved=6 * A, sb=1 << 20, dh=7 * A, dx=8 * A, dw=9 * A, dw_up=10 * A, M=10, N=60, K=70,
             ldx=72, ldw=72, ldu=72, lddh=64, lddx=72, lddw=72, lddu=72, act=4, ws=11 * A, wsb=1 << 20)
    a.update(kw)
    return lib._load().la_gated_ffn_backward(
        a["x"], a["w"], a["w_up"], a["saved"], a["sb"], a["dh"], a["dx"], a["dw"], a["dw_up"], a["M"], a["N"], a["K"], a["ldx"],
        a["ldw"], a["ldu"], a["lddh"], a["lddx"], a["lddw"], a["lddu"], a["act"], a["ws"], a["wsb"], 0)


@pytest.fixture(autouse=True)
def no_launch(monkeypatch):
    """What passes the checks ends in the injected failure, so every refusal below is the check's own."""
    monkeypatch.setenv("LA_FAULT_INJECT", "launch")


@pytest.mark.parametrize("call", [norm, norm_backward, linear, linear_backward, ffn, ffn_backward])
def test_the_plain_call_passes(lib, call):
    assert call(lib) == CUDA


@pytest.mark.parametrize("call", [norm, norm_backward])
def test_norm_sizes(lib, call):
    assert call(lib, rows=0) == COUNT and call(lib, rows=-1) == COUNT and call(lib, rows=MOST + 1) == COUNT
    assert call(lib, width=0) == UNSUPPORTED and call(lib, width=8193, ldx=8200, ldy=8200) == UNSUPPORTED
    assert call(lib, dtype=2) == ARG and call(lib, dtype=-1) == ARG
    assert call(lib, x=None) == ARG and call(lib, x=A + 8) == ARG and call(lib, w=None) == ARG and call(lib, w=A + 2) == ARG
    assert call(lib, ldx=56) == ARG and call(lib, ldx=66) == ARG
    assert call(lib, dtype=0, ldx=62) == ARG


def test_norm(lib):
    assert norm(lib, b=None) == CUDA and norm(lib, stats=None) == CUDA and norm(lib, b=3 * A + 2) == ARG
    assert norm(lib, y=None) == ARG and norm(lib, y=4 * A + 8) == ARG and norm(lib, stats=5 * A + 8) == ARG
    assert norm(lib, ldy=56) == ARG and norm(lib, eps=-1.0) == ARG and norm(lib, eps=float("nan")) == ARG
    assert norm(lib, y=A) == CUDA  # in place
    assert norm(lib, y=A, ldy=72) == ARG and norm(lib, y=A + 128) == ARG  # neither the same rows nor others
    assert norm(lib, y=2 * A) == ARG and norm(lib, y=3 * A) == ARG and norm(lib, y=5 * A) == ARG
    assert norm(lib, stats=A) == ARG and norm(lib, stats=2 * A) == ARG
    assert norm(lib, ldx=128, ldy=128, y=A + 128) == CUDA  # columns of its own beside x
    assert norm(lib, ldx=128, ldy=128, y=A + 112) == ARG


def test_norm_backward(lib):
    assert norm_backward(lib, db=None) == CUDA and norm_backward(lib, dskip=None) == CUDA
    for name in ("stats", "dy", "dx", "dw", "ws"):
        assert norm_backward(lib, **{name: None}) == ARG and norm_backward(lib, **{name: 20 * A + 4}) == ARG
    assert norm_backward(lib, db=10 * A + 4) == ARG and norm_backward(lib, dskip=7 * A + 2) == ARG
    for name in ("lddy", "lddx", "ldskip"):
        assert norm_backward(lib, **{name: 56}) == ARG and norm_backward(lib, **{name: 63}) == ARG
    assert norm_backward(lib, dskip=None, ldskip=0) == CUDA
    assert norm_backward(lib, wsb=100) == ARG
    assert "workspace" in lib.last_error()
    assert norm_backward(lib, dx=6 * A) == CUDA and norm_backward(lib, dx=7 * A) == CUDA  # dy's or dskip's rows
    assert norm_backward(lib, dx=6 * A, lddx=72) == ARG and norm_backward(lib, dx=6 * A + 128) == ARG
    for out in ("dx", "dw", "db", "ws"):
        for taken in (A, 2 * A, 5 * A):
            assert norm_backward(lib, **{out: taken}) == ARG
    for out in ("dw", "db", "ws"):
        for taken in (6 * A, 7 * A, 8 * A):
            assert norm_backward(lib, **{out: taken}) == ARG
    assert norm_backward(lib, db=9 * A) == ARG and norm_backward(lib, ws=9 * A) == ARG


@pytest.mark.parametrize("call", [linear, linear_backward, ffn, ffn_backward])
def test_product_sizes(lib, call):
    for name in "MNK":
        assert call(lib, **{name: 0}) == COUNT and call(lib, **{name: -5}) == COUNT and call(lib, **{name: MOST + 1}) == COUNT
    assert call(lib, M=MOST, N=MOST) == COUNT  # more values than the buffers' bytes can be counted for
    assert call(lib, act=-1) == UNSUPPORTED and call(lib, act=5) == UNSUPPORTED
    assert call(lib, x=None) == ARG and call(lib, x=A + 2) == ARG and call(lib, w=None) == ARG and call(lib, w=A + 8) == ARG
    assert call(lib, ldx=64) == ARG and call(lib, ldx=76) == ARG and call(lib, ldw=64) == ARG and call(lib, ldw=74) == ARG
    assert call(lib, sb=100) == ARG
    assert "saved" in lib.last_error()
    assert call(lib, saved=6 * A + 2) == ARG


def test_linear(lib):
    assert linear(lib, bias=None, residual=None, saved=None, sb=0) == CUDA
    assert linear(lib, act=0, saved=6 * A, sb=0) == CUDA  # nothing is kept without an activation
    assert linear(lib, bias=3 * A + 2) == ARG and linear(lib, residual=4 * A + 2) == ARG and linear(lib, y=None) == ARG
    assert linear(lib, ldy=56) == ARG and linear(lib, ldy=62) == ARG and linear(lib, ldr=56) == ARG
    assert linear(lib, residual=None, ldr=0) == CUDA
    assert linear(lib, y=4 * A) == CUDA  # the residual's rows
    assert linear(lib, y=4 * A, ldy=72) == ARG and linear(lib, y=4 * A + 128) == ARG
    for taken in (A, 2 * A, 3 * A):
        assert linear(lib, y=taken) == ARG and linear(lib, saved=taken) == ARG
    assert linear(lib, saved=4 * A) == ARG and linear(lib, saved=5 * A) == ARG
    assert linear(lib, ldx=144, ldy=144, y=A + 144) == CUDA and linear(lib, ldx=144, ldy=144, y=A + 128) == ARG


def test_linear_backward(lib):
    assert linear_backward(lib, dx=None) == CUDA and linear_backward(lib, dw=None) == CUDA and linear_backward(lib, dbias=None) == CUDA
    assert linear_backward(lib, dx=None, dw=None) == CUDA and linear_backward(lib, dx=None, dw=None, dbias=None) == ARG
    assert linear_backward(lib, saved=None) == ARG and linear_backward(lib, saved=None, sb=0, act=0) == CUDA
    for name in ("dx", "dw", "dbias", "dy", "ws"):
        assert linear_backward(lib, **{name: 20 * A + 2}) == ARG
    assert linear_backward(lib, dy=None) == ARG and linear_backward(lib, ws=None) == ARG and linear_backward(lib, wsb=64) == ARG
    for name in ("lddy", "lddx", "lddw"):
        assert linear_backward(lib, **{name: 56}) == ARG and linear_backward(lib, **{name: 76}) == ARG
    for out in ("dx", "dw", "dbias", "ws"):
        for taken in (A, 2 * A, 6 * A, 7 * A):
            assert linear_backward(lib, **{out: taken}) == ARG
    assert linear_backward(lib, dw=8 * A) == ARG and linear_backward(lib, dbias=9 * A) == ARG and linear_backward(lib, ws=8 * A) == ARG


def test_ffn(lib):
    assert ffn(lib, saved=None, sb=0) == CUDA
    assert ffn(lib, w_up=None) == ARG and ffn(lib, w_up=3 * A + 2) == ARG and ffn(lib, h=None) == ARG
    assert ffn(lib, ldu=64) == ARG and ffn(lib, ldh=56) == ARG and ffn(lib, ldh=60) == ARG
    for taken in (A, 2 * A, 3 * A):
        assert ffn(lib, h=taken) == ARG and ffn(lib, saved=taken) == ARG
    assert ffn(lib, saved=5 * A) == ARG
    assert ffn(lib, w_up=2 * A + 60 * 72 * 2) == CUDA and ffn(lib, w_up=2 * A) == CUDA  # one packed weight; one weight twice


def test_ffn_backward(lib):
    assert ffn_backward(lib, dx=None) == CUDA and ffn_backward(lib, dw=None, dw_up=None) == CUDA
    assert ffn_backward(lib, dw=None) == ARG and ffn_backward(lib, dw_up=None) == ARG
    assert ffn_backward(lib, dx=None, dw=None, dw_up=None) == ARG
    assert ffn_backward(lib, saved=None) == ARG and ffn_backward(lib, dh=None) == ARG and ffn_backward(lib, ws=None) == ARG
    assert ffn_backward(lib, wsb=64) == ARG
    for name in ("lddh", "lddx", "lddw", "lddu"):
        assert ffn_backward(lib, **{name: 56}) == ARG and ffn_backward(lib, **{name: 76}) == ARG
    for out in ("dx", "dw", "dw_up", "ws"):
        for taken in (A, 2 * A, 3 * A, 6 * A, 7 * A):
            assert ffn_backward(lib, **{out: taken}) == ARG
    assert ffn_backward(lib, dw_up=9 * A) == ARG and ffn_backward(lib, ws=10 * A) == ARG
    assert ffn_backward(lib, dw_up=9 * A + 60 * 72 * 2) == CUDA  # halves of one packed gradient


def test_sizes_of_buffers(lib):
    assert lib.linear_saved_bytes(10, 60, "gelu") == 10 * 64 * 2 and lib.linear_saved_bytes(10, 60) == 0
    assert lib.gated_ffn_saved_bytes(10, 61) == 10 * 128 * 3 and lib.gated_ffn_backward_workspace_bytes(10, 61, 7) == 10 * 128 * 2
    for call in (lib._load().la_linear_saved_bytes, lib._load().la_layernorm_rows_backward_workspace_bytes):
        assert call(0, 5, 1) == 0 and call(5, 0, 1) == 0
    assert lib._load().la_gated_ffn_saved_bytes(0, 5) == 0 and lib._load().la_linear_backward_workspace_bytes(5, 5, 0, 1) == 0


def test_binding(lib):
    t = lambda *s, dtype=torch.bfloat16: torch.zeros(*s, dtype=dtype)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        lib.layernorm_rows(t(4, 8), t(8))
    with pytest.raises(ValueError, match="CUDA"):
        lib.linear(t(4, 8), t(8, 8), t(4, 8))
    with pytest.raises(ValueError, match="CUDA"):
        lib.gated_ffn(t(4, 8), t(8, 8), t(8, 8), t(4, 8))
    with pytest.raises(ValueError, match="CUDA"):
        lib.linear_backward(t(4, 8), t(8, 8), None, t(4, 8), t(4, 8))
    with pytest.raises(ValueError, match="activation"):
        lib.linear_saved_bytes(4, 8, "tanh")
