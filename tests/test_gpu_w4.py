"""4-bit weights: the layout kernel against the rule it states (bit for bit), the products against a
plain form in 64 bits. A weight times a bf16 input is exact in 32 bits up to the scale's product; with
K terms in any order the sum is off by at most (K + 2) 2^-24 of the sum of magnitudes, and in practice
by its square root: the bound takes 32 + K / 64 roundings (a chain of K / 64 terms in each of the lanes
and tensor-core steps, then their joins), then half a bf16 step.
"""
import numpy as np
import pytest
import torch

import linear_attention_chunked_conv1d_gb300 as la
from tests.helpers import f64

pytestmark = pytest.mark.gpu


def unpack(q):
    """Weights 0..15 in order from the packed bytes."""
    n, half = q.shape
    word = q.astype(np.uint32).reshape(n, half // 4, 4)
    word = word[..., 0] | word[..., 1] << 8 | word[..., 2] << 16 | word[..., 3] << 24
    at = [4 * (e // 2) + 16 * (e % 2) for e in range(8)]
    return np.stack([word >> s & 15 for s in at], -1).reshape(n, half * 2)


def dense(q, scales):
    n, k = q.shape[0], q.shape[1] * 2
    w = unpack(q.cpu().numpy()).astype(np.float64) - 8
    return w * np.repeat(f64(scales), k // scales.shape[1], 1)


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N,K", [(1, 128), (37, 640), (300, 1152)])
def test_quantize_follows_its_rule(cuda, N, K, group):
    g = torch.Generator().manual_seed(N + group)
    w = torch.randn(N, K, generator=g).to(torch.bfloat16)
    w[0, :group] = 0  # a group of zeros
    w[-1, -group:] = torch.linspace(-7, 7, group).to(torch.bfloat16)  # ties among them
    wide = torch.full((N, K + 8), 3.0, dtype=torch.bfloat16, device=cuda)
    wide[:, :K] = w.to(cuda)
    q, scales = la.w4_quantize(wide[:, :K], group=group)
    torch.cuda.synchronize()
    top = w.float().view(N, K // group, group).abs().amax(-1)
    want_s = (top / 7.0).to(torch.bfloat16)
    assert torch.equal(scales.cpu(), want_s)
    sc = want_s.float()[..., None]
    r = torch.where(sc > 0, (w.float().view(N, K // group, group) / sc).clamp(-8, 7).round(), torch.zeros(()))
    assert np.array_equal(unpack(q.cpu().numpy()), (r.view(N, K) + 8).numpy().astype(np.uint32))


def product(cuda, M, N, K, group, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g).to(torch.bfloat16)
    q = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.int64).to(torch.uint8)
    s = (torch.rand(N, K // group, generator=g) + 0.1).to(torch.bfloat16)
    return x.to(cuda), q.to(cuda), s.to(cuda)


def check(y, x, q, s):
    w = dense(q, s)
    want, size = f64(x) @ w.T, abs(f64(x)) @ abs(w).T
    K = x.shape[1]
    err = (32 + K / 64) * 2.0 ** -24 * size
    assert np.all(abs(f64(y) - want) <= err + 2.0 ** -8 * (abs(want) + err))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 25, 32])
@pytest.mark.parametrize("N,K", [(1, 128), (15, 256), (17, 384), (128, 2048), (1001, 640)])
def test_matvec(cuda, M, N, K, group):
    x, q, s = product(cuda, M, N, K, group, seed=M + N)
    y = la.w4_matvec(x, q, s)
    torch.cuda.synchronize()
    check(y, x, q, s)


@pytest.mark.parametrize("K", [32, 64, 96, 160, 4096 + 32, 8192])
def test_matvec_inputs_of_odd_length(cuda, K):
    for M in (1, 5, 20):
        x, q, s = product(cuda, M, 70, K, 32, seed=K)
        y = la.w4_matvec(x, q, s)
        torch.cuda.synchronize()
        check(y, x, q, s)


def test_strides_and_neighbours(cuda):
    M, N, K = 11, 45, 512
    x, q, s = product(cuda, M, N, K, 64, seed=2)
    want = la.w4_matvec(x, q, s)
    wide = torch.full((M, K + 24), float("nan"), dtype=torch.bfloat16, device=cuda)
    wide[:, 8:K + 8] = x
    out = torch.full((M + 1, N + 6), 5.0, dtype=torch.bfloat16, device=cuda)
    la.w4_matvec(wide[:, 8:K + 8], q, s, out[:M, 3:N + 3])
    torch.cuda.synchronize()
    assert torch.equal(out[:M, 3:N + 3], want)
    out[:M, 3:N + 3] = 5.0
    assert torch.all(out == 5.0)


def test_a_row_does_not_depend_on_its_batch(cuda):
    x, q, s = product(cuda, 32, 300, 2048, 128, seed=3)
    whole = la.w4_matvec(x, q, s)
    for lo, hi in ((0, 1), (3, 4), (5, 13), (0, 17), (20, 32)):
        assert torch.equal(la.w4_matvec(x[lo:hi], q, s), whole[lo:hi]), (lo, hi)
    torch.cuda.synchronize()


def test_bad_rows_stay_by_themselves(cuda):
    x, q, s = product(cuda, 9, 64, 256, 32, seed=4)
    want = la.w4_matvec(x, q, s)
    x[4] = float("nan")
    x[7, 5] = float("inf")
    got = la.w4_matvec(x, q, s)
    torch.cuda.synchronize()
    keep = [0, 1, 2, 3, 5, 6, 8]
    assert torch.equal(got[keep], want[keep]) and torch.all(torch.isnan(got[4]))


def test_wide_weight_past_32_bits(cuda):
    """More than 2^32 weights: the last rows of q are read where they are."""
    N, K, group = 600000, 8192, 128
    q = torch.full((N, K // 2), 0x88, dtype=torch.uint8, device=cuda)  # zeros
    s = torch.ones(N, K // group, dtype=torch.bfloat16, device=cuda)
    q[-1] = 0x99  # ones
    x = torch.ones(1, K, dtype=torch.bfloat16, device=cuda)
    y = la.w4_matvec(x, q, s)
    torch.cuda.synchronize()
    assert torch.all(y[0, :-1] == 0) and float(y[0, -1]) == K


def test_quantized_weight_serves_the_product(cuda):
    """Laying out and multiplying: within the rounding of the weights of the bf16 product. Each weight is
    off by half a step, and by what the bf16 scale lost (7 * 2^-9 steps at the group's largest)."""
    N, K, M = 128, 1024, 4
    g = torch.Generator().manual_seed(5)
    w = torch.randn(N, K, generator=g).to(torch.bfloat16).to(cuda)
    x = torch.randn(M, K, generator=g).to(torch.bfloat16).to(cuda)
    q, s = la.w4_quantize(w, group=64)
    y = la.w4_matvec(x, q, s)
    torch.cuda.synchronize()
    step = np.repeat(f64(s), 64, 1)
    off = abs(dense(q, s) - f64(w))
    assert np.all(off <= step * (0.5 + 7 * 2.0 ** -8))
    want = f64(x) @ f64(w).T
    bound = abs(f64(x)) @ (step * (0.5 + 7 * 2.0 ** -8)).T
    assert np.all(abs(f64(y) - want) <= bound + 2.0 ** -7 * abs(want))


def test_graph_replay(cuda):
    x, q, s = product(cuda, 3, 500, 1024, 128, seed=6)
    y = torch.empty(3, 500, dtype=torch.bfloat16, device=cuda)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        la.w4_matvec(x, q, s, y)
    for seed in (7, 8):
        x.copy_(product(cuda, 3, 500, 1024, 128, seed=seed)[0])
        g.replay()
        torch.cuda.synchronize()
        check(y, x, q, s)


@pytest.mark.parametrize("N,K", [(16000, 512), (16000, 1024), (11450, 1536), (8000, 2016), (6900, 2560), (5700, 2816), (4850, 3584),
                                 (3001, 8096)])
def test_every_way_to_split_the_inputs(cuda, N, K):
    """One to eight blocks share an output's inputs, some of them fewer than the others and with a share of
    the outputs that does not divide the tile; a row's bits are the same in a batch of 32 and of 3."""
    x, q, s = product(cuda, 32, N, K, 32, seed=N)
    y = la.w4_matvec(x, q, s)
    few = la.w4_matvec(x[5:8], q, s)
    torch.cuda.synchronize()
    check(y, x, q, s)
    assert torch.equal(y[5:8], few)
