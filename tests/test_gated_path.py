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
