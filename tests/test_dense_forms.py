"""How near the dense half's gradients have to be to their forms in 64 bits (tests/dense_forms.py) is near enough to see a
mistake: on the CPU, results that are rounded as stated pass, and those with a planted mistake do not, at each size at which
the kernels are held to it."""
import math

import pytest
import torch

from tests.dense_forms import BF16, U, block, gated_gradients, linear_gradients, off, r16

# many rows and a small weight, whose sums the kernels may cut in parts; tiles with ragged edges; few rows; few outputs
SIZES = [(16384, 520, 392), (30001, 257, 264), (8192, 256, 256), (12000, 1001, 513), (40000, 8, 72),
         (2500, 1300, 264), (1030, 2100, 136), (777, 1001, 520), (300, 520, 200), (64, 640, 1000), (33, 130, 1000), (5, 520, 264)]
BLOCKS = [(37, 200, 333, "gelu"), (600, 1000, 1500, "silu"), (3000, 264, 700, "gelu_tanh"), (8, 64, 128, "silu")]


def inputs(m, n, k, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, sd=1.0: (torch.randn(*s, generator=g) * sd).to(BF16)  # noqa: E731
    return dict(x=r(m, k), w=r(n, k, sd=1 / math.sqrt(k)), w_up=r(n, k, sd=1 / math.sqrt(k)), bias=r(n), dy=r(m, n))


def block_inputs(m, D, F):
    g = torch.Generator().manual_seed(m + D)
    r = lambda *s, sd=1.0: (torch.randn(*s, generator=g) * sd).to(BF16)  # noqa: E731
    return dict(x=r(m, D), norm_w=r(D, sd=0.2) + 1, norm_b=r(D, sd=0.2), w_gate=r(F, D, sd=D ** -0.5), w_up=r(F, D, sd=D ** -0.5),
                w_down=r(D, F, sd=F ** -0.5), dy=r(m, D))


def planted(t, without):
    """A gradient's wrong forms: nothing, an eighth of its sum left out, one value off by the usual, a row and a column of a
    matrix by a 16th."""
    yield "zero", torch.zeros_like(t)
    yield "without an eighth of the sum", (t - without)
    for name, at in (("value", (0,) * t.dim()), ("row", (t.shape[0] - 1,)), ("column", (..., t.shape[-1] - 1)))[:1 if t.dim() == 1 else 3]:
        wrong = t.clone()
        wrong[at] = wrong[at] + (t.double().square().mean().sqrt() if name == "value" else wrong[at] / 16)
        yield name, wrong


def check(name, want, terms, without):
    want, term = want[name], terms[name]
    assert off(want.to(BF16), want, term) <= 1, name
    for what, wrong in planted(want, without):
        assert off(wrong.to(BF16), want, term) > 1, (name, what)


@pytest.mark.parametrize("m,n,k", SIZES)
def test_a_mistake_in_a_gradient_is_seen(m, n, k):
    c = inputs(m, n, k, m)
    rows, outs = slice(0, max(1, m // 8)), slice(0, max(1, n // 8))
    for act in ("gelu", "none"):
        want, d, terms = linear_gradients(c["x"], c["w"], c["bias"], c["dy"], act)
        X, W = c["x"].double(), c["w"].double()
        check("dx", want, terms, d[:, outs] @ W[outs])
        check("dw", want, terms, d[rows].T @ X[rows])
        check("dbias", want, terms, d[rows].sum(0))
    want, (dg, du), terms = gated_gradients(c["x"], c["w"], c["w_up"], c["dy"], "silu")
    check("dx", want, terms, dg[:, outs] @ W[outs] + du[:, outs] @ c["w_up"].double()[outs])
    check("dw", want, terms, dg[rows].T @ X[rows])
    check("dw_up", want, terms, du[rows].T @ X[rows])


@pytest.mark.parametrize("m,D,F,act", BLOCKS)
def test_a_mistake_in_the_block_is_seen(m, D, F, act):
    c = block_inputs(m, D, F)
    want = block(**c, act=act)
    for name, t in want.items():
        assert off(t.to(torch.float32 if name.startswith("norm") else BF16), t) <= 1, name
    # what passes the norm by left out; without a mean; a norm's weight, the residual or h of another rounding forgotten
    x, dy, nw = (c[n].double() for n in ("x", "dy", "norm_w"))
    var, mean = torch.var_mean(x, 1, unbiased=False, keepdim=True)
    rstd = 1 / torch.sqrt(var + 1e-5)
    plain = want["x"] - dy  # of the norm alone
    u_mean = (want["x"] - dy).mean(1, keepdim=True)
    assert float(u_mean.abs().max()) < 1e-9  # its rows sum to 0: the mean is what is taken off
    dn = r16(gated_gradients(r16((x - mean) * rstd * nw + c["norm_b"].double()), c["w_gate"], c["w_up"], r16(dy @ c["w_down"].double()), act)[0]["dx"])
    u = dn * nw
    xh = (x - mean) * rstd
    for what, wrong in (("dskip", plain), ("mean(u)", want["x"] + rstd * u.mean(1, keepdim=True)),
                        ("mean(u xh)", want["x"] + rstd * xh * (u * xh).mean(1, keepdim=True)), ("w", want["x"] - plain + plain / nw)):
        assert off(wrong.to(BF16), want["x"]) > 1, what
    assert off((want["y"] - x).to(BF16), want["y"]) > 1
    for name in ("norm_w", "norm_b"):
        assert off((want[name] * (1 + U)).float(), want[name]) > 1, name
    for name in ("w_gate", "w_up", "w_down"):
        assert off((want[name] * (1 + 3 * U)).to(BF16), want[name]) > 1, name
