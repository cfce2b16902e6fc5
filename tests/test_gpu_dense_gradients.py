"""Gradients of the dense half against 64-bit forms that are rounded on the way as the calls state (tests/dense_forms.py says
how near they have to be and why; tests/test_dense_forms.py that a mistake would be seen). Inputs are the same as there."""
import pytest
import torch

import linear_attention_chunked_conv1d_gb300 as la
from linear_attention_chunked_conv1d_gb300.path import FeedForward
from tests.dense_forms import BF16, block, gated_gradients, linear_gradients, off
from tests.test_dense_forms import BLOCKS, SIZES, block_inputs, inputs

pytestmark = pytest.mark.gpu


def aligned(t, cuda):
    """The same values in rows that start on 16 bytes."""
    if t.dim() == 1:
        return t.to(cuda)
    return torch.nn.functional.pad(t, (0, -t.shape[1] % 8)).to(cuda)[:, :t.shape[1]]


def like(t):
    """A matrix of NaN whose rows start on 16 bytes."""
    return torch.full((t.shape[0], (t.shape[1] + 7) // 8 * 8), float("nan"), dtype=BF16, device=t.device)[:, :t.shape[1]]


def nan(nbytes, cuda):
    return torch.full((nbytes // 4 + 4,), float("nan"), device=cuda).view(torch.uint8)


@pytest.mark.parametrize("act", ["gelu", "silu", "none"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_linear_gradients(cuda, m, n, k, act):
    c = {q: aligned(t, cuda) for q, t in inputs(m, n, k, m).items()}
    saved, ws = nan(la.linear_saved_bytes(m, n, act), cuda), nan(la.linear_backward_workspace_bytes(m, n, k, act), cuda)
    la.linear(c["x"], c["w"], bias=c["bias"], act=act, saved=saved)
    want, _, terms = linear_gradients(c["x"], c["w"], c["bias"], c["dy"], act)
    for which in (("dx", "dw", "dbias"), ("dw",), ("dx",)):
        got = dict(dx=like(c["x"]), dw=like(c["w"]), dbias=torch.full((n,), float("nan"), dtype=BF16, device=cuda))
        ws.fill_(255)
        la.linear_backward(c["x"], c["w"], saved if act != "none" else None, c["dy"], *(got[q] if q in which else None for q in ("dx", "dw")),
                           dbias=got["dbias"] if "dbias" in which else None, act=act, workspace=ws)
        for q in which:
            assert off(got[q], want[q], terms[q]) <= 1, (q, which, off(got[q], want[q], terms[q]))
    assert la.device_status() == 0


@pytest.mark.parametrize("act", ["gelu_tanh", "silu"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_gated_gradients(cuda, m, n, k, act):
    c = {q: aligned(t, cuda) for q, t in inputs(m, n, k, m).items()}
    saved, ws = nan(la.gated_ffn_saved_bytes(m, n), cuda), nan(la.gated_ffn_backward_workspace_bytes(m, n, k), cuda)
    la.gated_ffn(c["x"], c["w"], c["w_up"], act=act, saved=saved)
    want, _, terms = gated_gradients(c["x"], c["w"], c["w_up"], c["dy"], act)
    for which in (("dx", "dw", "dw_up"), ("dw", "dw_up"), ("dx",)):
        got = dict(dx=like(c["x"]), dw=like(c["w"]), dw_up=like(c["w"]))
        ws.fill_(255)
        la.gated_ffn_backward(c["x"], c["w"], c["w_up"], saved, c["dy"], *(got[q] if q in which else None for q in ("dx", "dw", "dw_up")),
                              act=act, workspace=ws)
        for q in which:
            assert off(got[q], want[q], terms[q]) <= 1, (q, which, off(got[q], want[q], terms[q]))
    assert la.device_status() == 0


@pytest.mark.parametrize("m,D,F,act", BLOCKS)
def test_block(cuda, m, D, F, act):
    c = {q: aligned(t, cuda) for q, t in block_inputs(m, D, F).items()}
    b = FeedForward(m, *(c[q] for q in ("norm_w", "norm_b", "w_gate", "w_up", "w_down")), act=act, train=True)
    got = dict(y=b.forward(c["x"]).clone(), **b.backward(c["dy"]))
    for q, t in block(**c, act=act).items():
        assert off(got[q], t) <= 1, (q, off(got[q], t))
    assert la.device_status() == 0
