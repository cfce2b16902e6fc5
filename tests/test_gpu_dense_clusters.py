"""Products of few rows at the numbers of tiles where one more changes how many blocks share a sum (36 clusters of eight, 46
of six and so on are resident at one time): each call against 64 bits, and the same bits each time, alone and in a row."""
import math

import pytest
import torch

import linear_attention_chunked_conv1d_gb300 as la
from tests.test_gpu_dense import F32, U, close, rows

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.mark.parametrize("tiles", [30, 32, 33, 36, 37, 38, 39, 46, 47, 49, 50, 58, 59, 74, 75, 97, 98, 152, 153])
def test_few_rows(cuda, tiles):
    g = torch.Generator().manual_seed(tiles)
    k, n = 2056, 128 * tiles - 3
    w = rows((n, k), BF16, cuda, g, 1 / math.sqrt(k))
    w_up = rows((64 * tiles, k), BF16, cuda, g, 1 / math.sqrt(k))
    for m in (1, 20):
        x = rows((m, k), BF16, cuda, g)
        y, h = la.linear(x, w), la.gated_ffn(x, w[:64 * tiles], w_up, act="none")
        ref = x.double() @ w.double().T
        mag = x.double().abs() @ w.double().abs().T
        close(y, ref, U * ref.abs() + 64 * F32 * mag, "y")
        gate, up = ref[:, :64 * tiles], x.double() @ w_up.double().T
        mu = x.double().abs() @ w_up.double().abs().T
        close(h, gate * up, U * (gate * up).abs() + 64 * F32 * (mag[:, :64 * tiles] * up.abs() + gate.abs() * mu + mag[:, :64 * tiles] * mu * 64 * F32), "h")
        for _ in range(3):
            assert torch.equal(la.linear(x, w), y) and torch.equal(la.gated_ffn(x, w[:64 * tiles], w_up, act="none"), h)
    assert la.device_status() == 0
