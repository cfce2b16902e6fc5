"""The dense half next to the recurrent half: a layer of both, forward and backward, on one stream and on several at
once, against the same calls with the device waited for after each of them. Kernels of both halves start while the one
ahead ends, share SMs, tensor memory and shared memory; none of that may show in a result, so all comparisons are exact."""
import math

import pytest
import torch

import linear_attention_chunked_conv1d_gb300 as la
from linear_attention_chunked_conv1d_gb300.path import FeedForward, GatedDecode, GatedPass

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


class Layer:
    """x -> gated pass -> projection with residual -> feed-forward block; gradients back through all of it."""

    def __init__(self, cuda, seed, T=777, C=512, D=520, F=1104, B=5):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s, sd=1.0: (torch.randn(*s, generator=g) * sd).to(BF16).to(cuda)  # noqa: E731
        cuts = sorted(torch.randint(0, T + 1, (B - 1,), generator=g).tolist())
        self.start = dict(conv_state=r(B, 3, C), h=torch.randn(B, C, generator=g).to(cuda))
        self.inp = dict(x=r(T, C), ab=r(T, 2 * C), conv_w=r(C, 4, sd=0.5), conv_bias=r(C, sd=0.1),
                        conv_state=self.start["conv_state"].clone(), h=self.start["h"].clone(),
                        cu_seqlens=torch.tensor([0, *cuts, T], dtype=torch.int32, device=cuda))
        self.w_out, self.hidden, self.dy = r(D, C, sd=C ** -0.5), r(T, D), r(T, D)
        self.rec = GatedPass(self.inp, train=True)
        self.ffn = FeedForward(T, r(D), r(D, sd=0.1), r(F, D, sd=D ** -0.5), r(F, D, sd=D ** -0.5), r(D, F, sd=F ** -0.5), train=True)
        self.mid, self.du, self.dw = torch.empty(T, D, dtype=BF16, device=cuda), torch.empty(T, C, dtype=BF16, device=cuda), torch.empty_like(self.w_out)
        self.ws = torch.empty(la.linear_backward_workspace_bytes(T, D, C), dtype=torch.uint8, device=cuda)
        torch.cuda.synchronize()

    def run(self, stream=None, after=lambda: None):
        with torch.cuda.stream(stream):
            for name, t in self.start.items():
                self.inp[name].copy_(t)
            u = self.rec.forward(stream)
            after()
            la.linear(u, self.w_out, self.mid, residual=self.hidden, act="silu", stream=stream)
            after()
            y = self.ffn.forward(self.mid, stream)
            after()
            g = self.ffn.backward(self.dy, stream)
            after()
            la.linear_backward(u, self.w_out, None, g["x"], self.du, self.dw, workspace=self.ws, stream=stream)
            after()
            back = self.rec.backward(self.du, stream=stream)
            after()
        return [y, self.dw, self.du] + [t for t in (*g.values(), *back.values()) if t is not None]


def test_a_layer_of_both_halves(cuda):
    layer = Layer(cuda, 1)
    want = [t.clone() for t in layer.run(after=torch.cuda.synchronize)]
    assert all(bool(t.isfinite().all()) for t in want)
    for _ in range(4):
        assert all(torch.equal(a, b) for a, b in zip(layer.run(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer.run(torch.cuda.current_stream())
    for _ in range(4):
        for t in got:
            t.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert la.device_status() == 0


def test_layers_on_several_streams(cuda):
    """Three layers at once, next to projections by the other tensor-core kernel; then the same from one stream."""
    layers = [Layer(cuda, 2), Layer(cuda, 3, T=2500, D=264, F=704), Layer(cuda, 4, T=40, C=1024, D=1024, F=2048, B=40)]
    want = [[t.clone() for t in q.run(after=torch.cuda.synchronize)] for q in layers]
    a, w = torch.randn(2000, 520, device=cuda).to(BF16), torch.randn(1000, 520, device=cuda).to(BF16)
    ref, out = la.gemm_bf16(a, w), torch.empty(2000, 1000, dtype=BF16, device=cuda)
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [q.run(s) for q, s in zip(layers, streams)]
        la.gemm_bf16(a, w, out, stream=streams[3])
    torch.cuda.synchronize()
    assert torch.equal(out, ref)
    for g, r in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(g, r))
    assert la.device_status() == 0


def test_decode_steps_of_both_halves(cuda):
    """Decode steps of the recurrent and the dense half in a row: as with the device waited for between them."""
    g = torch.Generator().manual_seed(5)
    B, C, D, F = 7, 512, 392, 1000
    r = lambda *s, sd=1.0: (torch.randn(*s, generator=g) * sd).to(BF16).to(cuda)  # noqa: E731
    weights = dict(norm_w=r(D), w_in=r(3 * C, D, sd=D ** -0.5), w_out=r(D, C, sd=C ** -0.5), conv_w=r(C, 4, sd=0.5), conv_bias=r(C, sd=0.1))
    state, h = r(B, 3, C), torch.randn(B, C, generator=g).to(cuda)
    dense = [r(D), None, r(F, D, sd=D ** -0.5), r(F, D, sd=D ** -0.5), r(D, F, sd=F ** -0.5)]
    x0 = r(B, D)

    def steps(after):
        window, carried = state.clone(), h.clone()  # the layer has their addresses only
        rec = GatedDecode(**weights, conv_state=window, h=carried)
        ffn = FeedForward(B, *dense)
        x = x0.clone()
        torch.cuda.synchronize()
        for _ in range(6):
            y = rec.run(x)
            after()
            x.copy_(ffn.forward(y))
            after()
        torch.cuda.synchronize()
        del window, carried
        return x
    want = steps(torch.cuda.synchronize)
    assert bool(want.isfinite().all())
    for _ in range(3):
        assert torch.equal(steps(lambda: None), want)
    assert la.device_status() == 0 and math.isfinite(float(want.float().norm()))
