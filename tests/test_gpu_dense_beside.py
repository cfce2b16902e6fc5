"""Calls whose last few rows are a second kernel's, beside the first one's last round: everything that they read is written
by the kernel directly ahead of them, over values that the call before has read at the same addresses. The second kernel
must not find those older values. Results are compared bit for bit with calls that the device was waited for between."""
import math

import pytest
import torch

import linear_attention_chunked_conv1d_gb300 as la
from tests.test_gpu_dense import out_rows, rows

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("which", ["residual", "bias", "x", "w"])
@pytest.mark.parametrize("m,n,k", [(777, 5001, 2048), (1030, 8192, 2048)])
def test_what_the_kernel_ahead_wrote_is_read(cuda, m, n, k, which):
    g = torch.Generator().manual_seed(m)
    steps = 24
    make = {"residual": lambda: rows((m, n), BF16, cuda, g), "bias": lambda: torch.randn(n, generator=g).to(BF16).to(cuda),
            "x": lambda: rows((m, k), BF16, cuda, g), "w": lambda: rows((n, k), BF16, cuda, g, 1 / math.sqrt(k))}
    args = {name: f() for name, f in make.items()}
    values = [make[which]() for _ in range(3)]
    if which == "bias":
        values = [v.clone() for v in values]
    ys = [out_rows((m, n), BF16, cuda) for _ in range(steps)]
    last = slice(m // 256 * 256, m)

    def call(y):
        la.linear(args["x"], args["w"], y, bias=args["bias"], residual=args["residual"], act="gelu")
    want = []
    for v in values:
        args[which].copy_(v)
        torch.cuda.synchronize()
        call(ys[0])
        torch.cuda.synchronize()
        want.append(ys[0].clone())
    assert not any(torch.equal(a[last], b[last]) for a, b in zip(want, want[1:]))

    def chain():
        for i, y in enumerate(ys):
            args[which].copy_(values[i % 3])
            call(y)
    for _ in range(4):
        for y in ys:
            y.fill_(7.0)
        chain()
        assert all(torch.equal(y, want[i % 3]) for i, y in enumerate(ys))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for _ in range(4):
        for y in ys:
            y.fill_(7.0)
        graph.replay()
        assert all(torch.equal(y, want[i % 3]) for i, y in enumerate(ys))
    assert la.device_status() == 0


@pytest.mark.parametrize("m,f,k", [(777, 2500, 2048), (1030, 4096, 2048)])
def test_a_chain_of_the_library_s_own_kernels(cuda, m, f, k):
    """norm -> gated block -> projection back onto the residual stream, round after round in the same buffers: every call's
    inputs are those of a kernel that may still be ending when the next one is let start."""
    g = torch.Generator().manual_seed(f)
    nw = (1 + 0.2 * torch.randn(k, generator=g)).to(BF16).to(cuda)
    wg, wu, wd = (rows(s, BF16, cuda, g, 1 / math.sqrt(s[1])) for s in ((f, k), (f, k), (k, f)))
    x0 = rows((m, k), BF16, cuda, g)
    x, n, h = rows((m, k), BF16, cuda, g), out_rows((m, k), BF16, cuda), out_rows((m, f), BF16, cuda)

    def chain(after=lambda: None):
        x.copy_(x0)
        for _ in range(6):
            la.layernorm_rows(x, nw, y=n)
            after()
            la.gated_ffn(n, wg, wu, h)
            after()
            la.linear(h, wd, x, residual=x)
            after()
        return x.clone()
    want = chain(torch.cuda.synchronize)
    assert bool(want.isfinite().all())
    for _ in range(8):
        assert torch.equal(chain(), want)
    assert la.device_status() == 0
