"""The gated recurrence where streams start and end on the edges of the kernels' tiles (256 tokens forward in
bf16, 128 in fp32 and backward), inside a chain of tiles: such a tile's incoming state is known without a
search of its chain, and what it leaves is published without a map. There are more streams than sections of
the rows (at most 8), so that chains go on over such an edge. Against the 64-bit form, with the running
bounds of test_gpu_gated_scan."""
import numpy as np
import pytest
import torch

import linear_attention_chunked_conv1d_gb300 as la
from tests.helpers import f64
from tests.test_gpu_gated_scan import backward, close, forward, gpu_pass, make

pytestmark = pytest.mark.gpu

EDGES = {
    "24 of 256": [256] * 24,
    "12 of 512": [512] * 12,
    "30 of 128": [128] * 30,
    "one off": [256, 255, 257, 128, 127, 129, 256, 0, 1, 255, 384, 128, 512, 0, 256, 257, 255, 640, 127, 129, 256, 128, 128],
    "one token over": [256, 257, 256, 255, 513, 511, 256, 1, 255, 256, 128, 129, 127, 256] * 2,
}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("name,C", [(n, c) for n in EDGES for c in (8, 72)] + [("12 of 512", 2056)])
def test_streams_that_meet_on_tile_edges(cuda, name, C, dtype):
    lengths = EDGES[name]
    inp = make(lengths, C, dtype, seed=40 + C + len(lengths), slow=6.0)
    x, ab, dy = (f64(inp[n]) for n in ("x", "ab", "dy"))
    a, b = ab[:, :C], ab[:, C:]
    y_r, before, fin, err, err_b, fin_err = forward(x, a, b, f64(inp["h"]), lengths)
    dx_r, dab_r, dh0_r = backward(x, a, b, before, err_b, dy, f64(inp["dfinal"]), lengths)
    outs = [gpu_pass(cuda, inp, lengths)]
    if len(set(lengths)) == 1:
        outs.append(gpu_pass(cuda, inp, lengths, packed=False))
    for y, h, dx, dab, dh0 in outs:
        close(y, y_r, err, dtype)
        close(h, fin, fin_err)
        close(dx, *dx_r, dtype)
        close(dab, *dab_r, dtype)
        close(dh0, *dh0_r)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_edges_repeat_bit_for_bit(cuda, dtype):
    """8 equal streams of a training batch, eight tiles each: the same bits every time."""
    lengths = [2048] * 8
    inp = make(lengths, 2048, dtype, seed=41, slow=6.0)
    first = gpu_pass(cuda, inp, lengths, packed=False)
    for _ in range(5):
        for u, v in zip(first, gpu_pass(cuda, inp, lengths, packed=False)):
            assert torch.equal(u, v)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_gates_that_are_nan_stay_in_their_stream(cuda, dtype):
    """NaN and infinite gates, on both sides of tile edges and inside tiles, reach no other stream or channel."""
    lengths, C = [256, 30, 226, 256, 0, 64, 320, 128, 128, 5, 256, 512], 24
    inp = make(lengths, C, dtype, seed=42)
    clean = gpu_pass(cuda, inp, lengths)
    ends = np.cumsum([0] + lengths)
    bad, inf = {0, 3, 5, 8, 10}, float("inf")
    for s in bad:
        ab = inp["ab"][ends[s]:ends[s + 1]]
        ab[:, :8] = ab[:, C:C + 8] = float("nan")
        ab[::2, 8:16], ab[1::2, C + 8:C + 16] = inf, -inf
    got = gpu_pass(cuda, inp, lengths)
    for s in range(len(lengths)):
        rows, chans = slice(ends[s], ends[s + 1]), slice(16, C) if s in bad else slice(0, C)
        for i in (0, 2):
            assert torch.equal(got[i][rows, chans], clean[i][rows, chans]), (s, i)
        for half in (0, C):
            part = slice(chans.start + half, chans.stop + half)
            assert torch.equal(got[3][rows, part], clean[3][rows, part]), s
        for i in (1, 4):
            assert torch.equal(got[i][s, chans], clean[i][s, chans]), (s, i)
        if s in bad:
            assert bool(torch.isnan(got[0][rows, :8]).all())
            assert bool(torch.isfinite(got[0][rows, 8:16]).all())


@pytest.mark.parametrize("M", [1, 7, 32])
def test_products_into_columns_beside_their_rows(cuda, M):
    """x | gap | y in one wide buffer: the products are those into a tensor of their own, the rest stays."""
    N, K = 200, 256
    g = torch.Generator().manual_seed(43)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).to(cuda)  # noqa: E731
    q, s = la.w4_quantize((r(N, K) / 16).contiguous(), group=64)
    wide = torch.full((M, K + N + 32), 5.0, dtype=torch.bfloat16, device=cuda)
    x, y = wide[:, :K], wide[:, K + 16:K + 16 + N]
    x.copy_(r(M, K))
    want = la.w4_matvec(x.contiguous(), q, s)
    before = x.clone()
    la.w4_matvec(x, q, s, y)
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(x, before)
    assert torch.all(wide[:, K:K + 16] == 5.0) and torch.all(wide[:, K + 16 + N:] == 5.0)


def test_step_refuses_taps_that_are_none(cuda):
    """conv_w [C][0] is no layer without a convolution: x would have entered without bias and SiLU."""
    B, C = 2, 16
    bf = dict(dtype=torch.bfloat16, device=cuda)
    h, y = torch.zeros(B, C, device=cuda), torch.full((B, C), 5.0, **bf)
    args = la.pointer_array(list(h)), torch.zeros(B, C, **bf), torch.zeros(B, 2 * C, **bf), y
    with pytest.raises(ValueError, match="taps"):
        la.gated_scan_step(*args, conv_w=torch.zeros(C, 0, **bf), conv_bias=torch.zeros(C, **bf))
    torch.cuda.synchronize()
    assert torch.all(y == 5.0)
    la.gated_scan_step(*args)
    torch.cuda.synchronize()
    assert torch.all(y == 0.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_nan_of_every_bit_set(cuda, dtype):
    """The pattern by which a chain's word says that nobody has written it is a NaN, too: in states, inputs, gates
    and gradients it comes out as a NaN, and no tile waits for it."""
    lengths, C = [900, 256, 700], 72
    inp = make(lengths, C, dtype, seed=44)
    clean = gpu_pass(cuda, inp, lengths)
    bits = torch.int32 if dtype == "f32" else torch.int16
    chans = {"x": slice(0, 8), "h": slice(8, 16), "ab": slice(16, 24), "dy": slice(24, 32), "dfinal": slice(32, 40)}
    for n, at in chans.items():
        v = inp[n]
        v[(slice(3, 4) if n in ("x", "ab") else slice(890, 891) if n == "dy" else slice(0, 1)), at] = float("nan")
        v.view(torch.int32 if v.dtype == torch.float32 else bits)[torch.isnan(v)] = -1
    y, h, dx, dab, dh0 = gpu_pass(cuda, inp, lengths)  # la_device_status() is 0
    for at in (chans["x"], chans["h"], chans["ab"]):
        assert bool(torch.isnan(y[3:900, at]).all()) and bool(torch.isnan(h[0, at]).all())
    for at in (chans["dy"], chans["dfinal"]):
        assert bool(torch.isnan(dx[:890, at]).all()) and bool(torch.isnan(dh0[0, at]).all())
    rest = slice(40, C)
    for got, want in zip((y, h, dx, dh0), (clean[0], clean[1], clean[2], clean[4])):
        assert torch.equal(got[:, rest], want[:, rest])
    assert torch.equal(y[900:], clean[0][900:]) and torch.equal(dx[900:], clean[2][900:])
