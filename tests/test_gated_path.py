"""path.GatedPass, path.GatedDecode and path.project on host tensors: which call a weight goes to, and what the
objects refuse when they are made or run (no kernel runs)."""
import pytest
import torch

from linear_attention_chunked_conv1d_gb300 import path

BF = torch.bfloat16


@pytest.fixture
def calls(monkeypatch, built_lib):
    """The kernels' calls, replaced by records of their names."""
    made = []
    for name in ("gemm_bf16", "w4_matvec", "rmsnorm_rows", "gated_scan_step", "gated_scan", "gated_scan_backward",
                 "conv1d_silu_prefill_varlen", "conv1d_silu_backward"):
        monkeypatch.setattr(path, name, lambda *a, _n=name, **k: made.append((_n, a)))
    return made


def quantized(n, k, group=32):
    return torch.zeros(n, k // 2, dtype=torch.uint8), torch.zeros(n, k // group, dtype=BF)


@pytest.mark.parametrize("kind", [tuple, list])
def test_a_pair_is_a_4_bit_weight_whatever_holds_it(calls, kind):
    y, w = torch.zeros(3, 64, dtype=BF), kind(quantized(24, 64))
    path.project(y, w)
    path.project(y, torch.zeros(24, 64, dtype=BF))
    assert [n for n, _ in calls] == ["w4_matvec", "gemm_bf16"]
    assert calls[0][1][1] is w[0] and calls[0][1][2] is w[1]
    assert path._outputs(w) == 24 and path._outputs(torch.zeros(7, 64)) == 7


def decode(B=3, C=16, D=64, K=4, **kw):
    a = dict(norm_w=torch.zeros(D, dtype=BF), w_in=torch.zeros(3 * C, D, dtype=BF), w_out=torch.zeros(D, C, dtype=BF),
             conv_w=torch.zeros(C, K, dtype=BF), conv_bias=torch.zeros(C, dtype=BF),
             conv_state=torch.zeros(B, K - 1, C, dtype=BF), h=torch.zeros(B, C))
    a.update(kw)
    return path.GatedDecode(**a)


def test_decode_refuses_more_streams_than_4_bit_rows_when_it_is_made(calls):
    C, D = 32, 64
    most = path.LA_W4_MAX_ROWS
    four = dict(w_in=quantized(3 * C, D), w_out=quantized(D, C))
    decode(B=most, C=C, D=D, **four)
    decode(B=most + 1, C=C, D=D)  # bf16 weights: any number
    for given in (four, dict(w_in=four["w_in"]), dict(w_out=four["w_out"])):
        with pytest.raises(ValueError, match="33 streams"):
            decode(B=most + 1, C=C, D=D, **given)


def test_decode_refuses_what_does_not_fit_when_it_is_made(calls):
    B, C, D, K = 3, 16, 64, 4
    decode()
    decode(K=1)
    decode(conv_bias=None)
    # states that are parts of larger pools, one stream's dense each
    decode(conv_state=torch.zeros(B, 2, K - 1, C, dtype=BF)[:, 1], h=torch.zeros(B, 2 * C)[:, C:])
    for bad in (dict(norm_w=torch.zeros(D)), dict(w_in=torch.zeros(3 * C, D + 8, dtype=BF)), dict(w_in=torch.zeros(3 * C - 8, D, dtype=BF)),
                dict(w_in=quantized(3 * C, D + 64)), dict(w_in=quantized(2 * C, D)), dict(w_out=quantized(D, 2 * C)),
                dict(w_out=torch.zeros(D, 2 * C, dtype=BF)), dict(w_out=torch.zeros(D, C)), dict(conv_w=torch.zeros(2 * C, K, dtype=BF)),
                dict(conv_w=torch.zeros(K, C, dtype=BF).t()), dict(conv_bias=torch.zeros(2 * C, dtype=BF)),
                dict(conv_state=torch.zeros(B, K, C, dtype=BF)), dict(conv_state=torch.zeros(B - 1, K - 1, C, dtype=BF)),
                dict(conv_state=torch.zeros(B, C, K - 1, dtype=BF).transpose(1, 2)), dict(h=torch.zeros(B, C, dtype=BF)),
                dict(h=torch.zeros(C, B).t()), dict(h=torch.zeros(B * C + 1)[1:].view(B, C)), dict(h=torch.zeros(B, C + 1)[:, :C])):
        with pytest.raises(ValueError, match=next(iter(bad))):
            decode(**bad)


def test_decode_refuses_hidden_rows_that_do_not_fit(calls):
    """More rows than streams would be written past the normed rows, fewer would leave old ones in them."""
    layer = decode(B=3, D=64)
    layer.run(torch.zeros(3, 64, dtype=BF))
    layer.run(torch.zeros(3, 80, dtype=BF)[:, :64])
    assert [n for n, _ in calls] == ["rmsnorm_rows", "gemm_bf16", "gated_scan_step", "gemm_bf16"] * 2
    del calls[:]
    for bad in (torch.zeros(4, 64, dtype=BF), torch.zeros(2, 64, dtype=BF), torch.zeros(3, 72, dtype=BF), torch.zeros(3, 64),
                torch.zeros(64, 3, dtype=BF).t()):
        with pytest.raises(ValueError, match="hidden"):
            layer.run(bad)
    assert not calls


def inputs(T=10, C=16, B=2, K=4, dtype=torch.float32, **kw):
    a = dict(x=torch.zeros(T, C, dtype=dtype), ab=torch.zeros(T, 2 * C, dtype=dtype), conv_w=torch.zeros(C, K, dtype=dtype),
             conv_bias=torch.zeros(C, dtype=dtype), conv_state=torch.zeros(B, K - 1, C, dtype=dtype), h=torch.zeros(B, C),
             cu_seqlens=torch.zeros(B + 1, dtype=torch.int32))
    a.update(kw)
    return a


def test_pass_refuses_what_does_not_fit_when_it_is_made(calls):
    T, C, B, K = 10, 16, 2, 4
    for ok in (inputs(), inputs(dtype=BF), inputs(K=1), inputs(conv_bias=None), inputs(x=torch.zeros(T, 3 * C)[:, C:2 * C]),
               inputs(conv_state=torch.zeros(B, 2, K - 1, C)[:, 1], h=torch.zeros(B, 2 * C)[:, C:])):
        for train in (False, True):
            path.GatedPass(ok, train=train).forward()
    for bad in (dict(ab=torch.zeros(T, C)), dict(ab=torch.zeros(T + 1, 2 * C)), dict(ab=torch.zeros(T, 2 * C, dtype=BF)),
                dict(conv_w=torch.zeros(C + 4, K)), dict(conv_w=torch.zeros(K, C).t()), dict(conv_bias=torch.zeros(C + 4)),
                dict(conv_state=torch.zeros(B, K, C)), dict(conv_state=torch.zeros(B, K - 1, C, dtype=BF)),
                dict(conv_state=torch.zeros(B, C, K - 1).transpose(1, 2)), dict(h=torch.zeros(C, B).t()),
                dict(h=torch.zeros(B, C, dtype=torch.float64)), dict(cu_seqlens=torch.zeros(B + 1, dtype=torch.int64)),
                dict(cu_seqlens=torch.zeros(B, dtype=torch.int32)), dict(x=torch.zeros(C, T).t())):
        with pytest.raises(ValueError, match=next(iter(bad))):
            path.GatedPass(inputs(**bad))


def test_backward_needs_a_forward(calls):
    """Before it there is nothing to go back through but what the buffers happen to hold."""
    p, dy = path.GatedPass(inputs(), train=True), torch.zeros(10, 16)
    with pytest.raises(RuntimeError, match="forward"):
        p.backward(dy)
    assert not calls
    p.forward()
    p.backward(dy)
    assert [n for n, _ in calls][-2:] == ["gated_scan_backward", "conv1d_silu_backward"]
