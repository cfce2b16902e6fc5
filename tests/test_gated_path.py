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
