"""What the gated recurrence, the conv's backward pass and the 4-bit products refuse on the host, before
any CUDA call (fake aligned addresses; nothing is dereferenced), and what the binding refuses."""
import pytest
import torch

A = 0x100000


@pytest.fixture(scope="module")
def lib(built_lib):
    import linear_attention_chunked_conv1d_gb300 as la
    la._load()
    return la


def scan(lib, **kw):
    a = dict(h=A, x=A, ab=2 * A, y=3 * A, saved=None, sb=0, cu=A, B=2, T=40, maxt=40, C=64, xs=64, abs=128, ys=64,
             dtype=1, ws=4 * A, wsb=1 << 24)
    a.update(kw)
    return lib._load().la_gated_scan(a["h"], a["x"], a["ab"], a["y"], a["saved"], a["sb"], a["cu"], a["B"], a["T"],
                                     a["maxt"], a["C"], a["xs"], a["abs"], a["ys"], a["dtype"], a["ws"], a["wsb"], 0)


def backward(lib, **kw):
    a = dict(x=A, ab=2 * A, saved=5 * A, sb=1 << 24, dy=6 * A, fin=A, dx=7 * A, dab=8 * A, dh0=2 * A, cu=A, B=2, T=40,
             maxt=40, C=64, xs=64, abs=128, dys=64, dxs=64, dabs=128, dtype=1, ws=4 * A, wsb=1 << 24)
    a.update(kw)
    return lib._load().la_gated_scan_backward(
        a["x"], a["ab"], a["saved"], a["sb"], a["dy"], a["fin"], a["dx"], a["dab"], a["dh0"], a["cu"], a["B"], a["T"],
        a["maxt"], a["C"], a["xs"], a["abs"], a["dys"], a["dxs"], a["dabs"], a["dtype"], a["ws"], a["wsb"], 0)


def step(lib, **kw):
    a = dict(cs=A, h=A, x=A, ab=2 * A, w=A, bias=None, K=4, y=3 * A, B=4, maxb=4, C=64, xs=64, abs=128, ys=64, dtype=1)
    a.update(kw)
    return lib._load().la_gated_scan_step(a["cs"], a["h"], a["x"], a["ab"], a["w"], a["bias"], a["K"], a["y"], a["B"],
                                          a["maxb"], a["C"], a["xs"], a["abs"], a["ys"], a["dtype"], 0)


def conv(lib, **kw):
    a = dict(st=A, x=A, w=A, bias=None, dout=2 * A, fin=A, dx=3 * A, dw=A, db=None, dst=2 * A, cu=A, B=2, T=40, maxt=40,
             C=64, K=4, xs=64, dos=64, dxs=64, dtype=1, ws=4 * A, wsb=1 << 24)
    a.update(kw)
    return lib._load().la_conv1d_silu_backward(
        a["st"], a["x"], a["w"], a["bias"], a["dout"], a["fin"], a["dx"], a["dw"], a["db"], a["dst"], a["cu"], a["B"],
        a["T"], a["maxt"], a["C"], a["K"], a["xs"], a["dos"], a["dxs"], a["dtype"], a["ws"], a["wsb"], 0)


def matvec(lib, **kw):
    a = dict(x=A, q=2 * A, s=3 * A, y=4 * A, M=4, N=10, K=256, g=64, ldx=256, ldy=10)
    a.update(kw)
    return lib._load().la_w4_matvec(a["x"], a["q"], a["s"], a["y"], a["M"], a["N"], a["K"], a["g"], a["ldx"], a["ldy"], 0)


def quantize(lib, **kw):
    a = dict(w=A, q=2 * A, s=3 * A, N=10, K=256, g=64, ldw=256)
    a.update(kw)
    return lib._load().la_w4_quantize(a["w"], a["q"], a["s"], a["N"], a["K"], a["g"], a["ldw"], 0)


COUNT, ARG, UNSUPPORTED, CUDA = 2, 1, 3, 4


@pytest.mark.parametrize("call", [scan, backward, conv])
def test_packed_calls(lib, call):
    assert call(lib, T=0) == COUNT and call(lib, T=-1) == COUNT
    assert call(lib, T=41) == COUNT
    assert "max_tokens" in lib.last_error()
    most = 2 ** 31 - 1024  # the kernels add a tile's tokens to a token's number
    assert call(lib, T=most + 1, maxt=2 ** 31 - 1, wsb=2 ** 62, sb=2 ** 62) == COUNT
    assert str(most) in lib.last_error()
    assert call(lib, T=2 ** 31 - 1, maxt=2 ** 31 - 1, wsb=2 ** 62, sb=2 ** 62) == COUNT
    assert call(lib, T=most, maxt=most, C=8, xs=8, wsb=8) == ARG
    assert call(lib, dtype=2) == ARG
    assert call(lib, B=0) == ARG
    assert call(lib, cu=None, B=3) == ARG  # 40 tokens are not 3 equal streams
    assert call(lib, C=0) == ARG and call(lib, C=60) == ARG
    assert call(lib, dtype=0, C=66) == ARG
    assert call(lib, x=None) == ARG and call(lib, x=A + 8) == ARG
    assert call(lib, xs=56) == ARG and call(lib, xs=68) == ARG
    assert call(lib, wsb=8) == ARG
    assert "workspace" in lib.last_error()
    assert call(lib, ws=None) == ARG and call(lib, ws=A + 4) == ARG


def test_scan(lib):
    assert scan(lib, ab=None) == ARG and scan(lib, y=A + 2) == ARG
    assert scan(lib, abs=120) == ARG and scan(lib, ys=32) == ARG
    assert scan(lib, y=A) == ARG and scan(lib, y=2 * A) == ARG
    assert scan(lib, saved=5 * A, sb=100) == ARG
    assert "saved" in lib.last_error()
    assert scan(lib, saved=5 * A + 4, sb=1 << 24) == ARG


def test_scan_backward(lib):
    assert backward(lib, saved=None) == ARG and backward(lib, sb=100) == ARG
    assert backward(lib, dy=None) == ARG and backward(lib, dx=A + 4) == ARG and backward(lib, dab=None) == ARG
    for out in ("dx", "dab"):
        for taken in (A, 2 * A, 5 * A, 6 * A):
            assert backward(lib, **{out: taken}) == ARG
    assert backward(lib, dab=7 * A) == ARG  # dx
    assert backward(lib, dh0=A) == ARG  # dh_final
    assert backward(lib, dabs=64) == ARG and backward(lib, dys=60) == ARG and backward(lib, dxs=0) == ARG


def test_step(lib):
    assert step(lib, B=0) == COUNT and step(lib, B=5) == COUNT
    assert step(lib, K=5) == UNSUPPORTED and step(lib, K=-1) == UNSUPPORTED
    assert step(lib, h=None) == ARG and step(lib, cs=None) == ARG and step(lib, w=None) == ARG
    assert step(lib, w=A + 2) == ARG and step(lib, bias=A + 2) == ARG
    assert step(lib, C=20) == ARG and step(lib, dtype=3) == ARG
    assert step(lib, y=A) == ARG and step(lib, y=2 * A) == ARG
    assert step(lib, abs=64) == ARG and step(lib, ys=8) == ARG


def test_conv_backward(lib):
    assert conv(lib, K=0) == UNSUPPORTED and conv(lib, K=5) == UNSUPPORTED
    assert conv(lib, st=None) == ARG and conv(lib, dout=None) == ARG and conv(lib, dw=None) == ARG
    assert conv(lib, dw=A + 4) == ARG and conv(lib, db=A + 4) == ARG and conv(lib, w=A + 4) == ARG
    assert conv(lib, dx=A) == ARG and conv(lib, dx=2 * A) == ARG
    assert conv(lib, dst=A) == ARG  # the gradients of the final windows
    assert conv(lib, dos=32) == ARG and conv(lib, dxs=60) == ARG


def test_w4(lib):
    assert matvec(lib, M=0) == COUNT and matvec(lib, M=33) == COUNT and matvec(lib, N=0) == COUNT
    assert lib.LA_W4_MAX_ROWS == 32
    assert matvec(lib, N=2 ** 31 - 1023, ldy=2 ** 31) == COUNT and matvec(lib, K=2 ** 31 - 512, ldx=2 ** 31) == COUNT
    assert matvec(lib, g=48) == UNSUPPORTED and quantize(lib, g=256) == UNSUPPORTED
    assert matvec(lib, K=224, g=64) == ARG and quantize(lib, K=100, g=32) == ARG
    assert matvec(lib, x=A + 2) == ARG and matvec(lib, q=None) == ARG and matvec(lib, s=None) == ARG
    assert matvec(lib, s=3 * A + 2) == ARG
    assert matvec(lib, ldx=128) == ARG and matvec(lib, ldy=9) == ARG and matvec(lib, ldx=260) == ARG
    assert matvec(lib, y=A + 64) == ARG  # overlaps x
    assert matvec(lib, y=4 * A + 1) == ARG
    assert quantize(lib, N=0) == COUNT
    assert quantize(lib, w=None) == ARG and quantize(lib, ldw=128) == ARG and quantize(lib, q=A + 1) == ARG


def test_injected_launch_failure(lib, monkeypatch):
    monkeypatch.setenv("LA_FAULT_INJECT", "launch")
    for call in (scan, backward, step, conv, matvec, quantize):
        assert call(lib) == CUDA, call
        assert "injected launch failure" in lib.last_error()
    assert scan(lib, T=0) == COUNT  # the checks come first
    monkeypatch.setenv("LA_FAULT_INJECT", "alloc")
    for call in (scan, backward, conv):  # these report bad offsets through the status word
        assert call(lib) == CUDA and "injected allocation failure" in lib.last_error()


def test_sizes(lib):
    for fn in (lib.gated_scan_workspace_bytes, lib.gated_scan_saved_bytes):
        assert fn(0, 10, 64, torch.bfloat16) == 0 and fn(1, 0, 64, torch.bfloat16) == 0
        assert 0 < fn(1, 10, 64, torch.bfloat16) <= fn(1, 1000, 64, torch.bfloat16) <= fn(3, 1000, 128, torch.float32)
    # no 32-bit product on the way
    assert lib.gated_scan_saved_bytes(1, 1 << 30, 8192, torch.bfloat16) > 1 << 33
    assert lib.conv1d_silu_backward_workspace_bytes(1, 1 << 30, 8192, 4, torch.bfloat16) > 1 << 33
    assert lib.conv1d_silu_backward_workspace_bytes(2, 100, 64, 0, torch.float32) == 0


def test_binding_refuses_host_tensors(lib):
    x, ab = torch.zeros(4, 8), torch.zeros(4, 16)
    with pytest.raises(ValueError, match="CUDA"):
        lib.gated_scan(None, x, ab, x.clone())
    with pytest.raises(ValueError, match="CUDA"):
        lib.w4_matvec(x.bfloat16(), torch.zeros(1, 4, dtype=torch.uint8), torch.zeros(1, 1, dtype=torch.bfloat16))


def test_binding_checks(lib):
    """The helpers that look at every tensor, on host tensors (the device only has to agree)."""
    dev = -1  # as get_device says of the host
    t = torch.zeros(4, 8)
    assert lib._matrix("t", t, 4, 8, torch.float32, dev) == 8
    assert lib._matrix("t", torch.zeros(4, 24)[:, 8:16], 4, 8, torch.float32, dev) == 24
    for bad in (t.t(), torch.zeros(8, 4).t(), torch.zeros(3, 8), torch.zeros(4, 16)[:, ::2]):
        with pytest.raises(ValueError, match="name"):
            lib._matrix("name", bad, 4, 8, torch.float32, dev)
    with pytest.raises(ValueError, match="name"):
        lib._matrix("name", t, 4, 8, torch.float32, 0)
    with pytest.raises(TypeError, match="name"):
        lib._matrix("name", t, 4, 8, torch.bfloat16, dev)
    with pytest.raises(ValueError, match="name"):
        lib._dense("name", torch.zeros(4, 16)[:, :8], (4, 8), torch.float32, dev)
    with pytest.raises(ValueError, match="name"):
        lib._ptrs("name", torch.zeros(3, dtype=torch.int64), 4, dev)
    with pytest.raises(TypeError, match="name"):
        lib._ptrs("name", torch.zeros(4), 4, dev)
    with pytest.raises(ValueError, match="B = 3"):
        lib._streams(torch.zeros(3, dtype=torch.int32), 3, dev)
    with pytest.raises(TypeError, match="cu_seqlens"):
        lib._streams(torch.zeros(3, dtype=torch.int64), None, dev)
