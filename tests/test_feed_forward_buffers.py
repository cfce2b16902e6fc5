"""path.FeedForward on host tensors, its kernels replaced by records of their names: which tensors of its own it takes as x
and dy, and what it does after a call that was refused (no kernel runs). On the GPU: the places that it takes."""
import pytest
import torch

from linear_attention_chunked_conv1d_gb300 import path

BF = torch.bfloat16
KERNELS = ("layernorm_rows", "gated_ffn", "linear", "linear_backward", "gated_ffn_backward", "layernorm_rows_backward")
ROWS, D, F = 16, 16, 16  # so that every matrix of the object's has the shape of x


@pytest.fixture
def calls(monkeypatch, built_lib):
    made = []
    for name in KERNELS:
        monkeypatch.setattr(path, name, lambda *a, _n=name, **k: made.append(_n))
    return made


def block(train, bias=True):
    w = lambda *s: torch.zeros(*s, dtype=BF)  # noqa: E731
    return path.FeedForward(ROWS, w(D), w(D) if bias else None, w(F, D), w(F, D), w(D, F), train=train)


def rows_of(t):
    """The first bytes of a buffer as rows of x."""
    return t.view(-1).view(torch.uint8)[:ROWS * D * 2].view(BF).view(ROWS, D)


def test_x_is_not_written_before_it_was_last_read(calls):
    """In training x is read by the last call of backward(); without it by linear, which takes y in the residual's place."""
    b = block(False)
    b.forward(b.y)
    b.forward(torch.zeros(ROWS, D, dtype=BF))
    assert calls == list(KERNELS[:3]) * 2
    t = block(True)
    own = [t.normed, t.h, t.y, t.dh, t.dnormed, rows_of(t.saved), rows_of(t.workspace)] + [t.grads[n] for n in ("x", "w_gate", "w_up", "w_down")]
    del calls[:]
    for q, taken in [(b, b.normed), (b, b.h)] + [(t, v) for v in own]:
        for x in (taken, taken[1:], taken[:, 8:], taken[:1, :8]):
            with pytest.raises(ValueError, match="x shares memory"):
                q.forward(x)
    assert not calls and t.x is None
    t.forward(b.y)  # another object's
    t.backward(t.y)
    assert calls == list(KERNELS)


def test_dy_is_not_written_before_it_was_last_read(calls):
    t = block(True)
    t.forward(torch.zeros(ROWS, D, dtype=BF))
    del calls[:]
    for taken in [t.dh, t.dnormed, rows_of(t.workspace)] + [t.grads[n] for n in ("w_gate", "w_up", "w_down")]:
        for dy in (taken, taken[1:], taken[:1, :8]):
            with pytest.raises(ValueError, match="dy shares memory"):
                t.backward(dy)
    assert not calls
    for dy in (t.grads["x"], t.y, t.normed, t.h, t.x):  # what is read only, and x's gradient, which may stand in dy's place
        t.backward(dy)
    assert calls == list(KERNELS[3:]) * 5
    q = block(True, bias=False)
    q.forward(torch.zeros(ROWS, D, dtype=BF))
    q.backward(torch.zeros(ROWS, D, dtype=BF))


@pytest.mark.parametrize("refused", KERNELS[:3])
def test_backward_after_a_forward_that_was_refused(calls, monkeypatch, refused):
    """The calls before the refused one have written over what the last whole pass kept: its gradients cannot be had."""
    t, x = block(True), torch.zeros(ROWS, D, dtype=BF)
    t.forward(x)
    t.backward(x.clone())

    def refuse(*a, **k):
        raise ValueError("refused")
    with monkeypatch.context() as m:
        m.setattr(path, refused, refuse)
        with pytest.raises(ValueError, match="refused"):
            t.forward(torch.ones(ROWS, D, dtype=BF))
    del calls[:]
    with pytest.raises(RuntimeError, match="forward"):
        t.backward(x.clone())
    assert not calls
    t.forward(x)
    t.backward(x.clone())
    assert calls == list(KERNELS)


@pytest.mark.gpu
def test_the_places_that_are_taken_give_the_same_bits(cuda):
    """x in y's place without train, and dy in the place of x's gradient, as with tensors of their own."""
    g = torch.Generator().manual_seed(1)
    m, d, f = 300, 200, 333
    r = lambda *s, sd=1.0: (torch.randn(*s, generator=g) * sd).to(BF).to(cuda)  # noqa: E731
    pad = lambda t: torch.nn.functional.pad(t, (0, -t.shape[1] % 8))[:, :t.shape[1]]  # noqa: E731
    weights = (r(d), r(d), r(f, d, sd=d ** -0.5), r(f, d, sd=d ** -0.5), pad(r(d, f, sd=f ** -0.5)))
    x, dy = r(m, d), r(m, d)
    b = path.FeedForward(m, *weights)
    want = b.forward(b.forward(x).clone()).clone()
    assert torch.equal(b.forward(b.forward(x)), want)
    t = path.FeedForward(m, *weights, train=True)
    t.forward(x)
    want = {n: v.clone() for n, v in t.backward(dy).items()}
    t.grads["x"].copy_(dy)
    got = t.backward(t.grads["x"])
    assert all(torch.equal(got[n], v) for n, v in want.items())
    with pytest.raises(ValueError, match="x shares memory"):
        t.forward(t.y)
