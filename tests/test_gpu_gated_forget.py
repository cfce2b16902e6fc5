"""The gated recurrence forgets: states, gradients and single inputs of 1e3 to 1e6 under gates that decay
within a few tokens leave nothing behind but what the running bound of test_gpu_gated_scan allows, which decays
with them. (What is left after n tokens is the product of their decays, to its own last places: a product held
as its difference from 1 keeps about 2^-24 of the state until the tile ends.)"""
import pytest
import torch

from tests.helpers import f64
from tests.test_gpu_gated_scan import backward, close, forward, gpu_pass, make

pytestmark = pytest.mark.gpu


def check(cuda, inp, lengths, dtype):
    C = inp["x"].shape[1]
    x, ab, dy = (f64(inp[n]) for n in ("x", "ab", "dy"))
    a, b = ab[:, :C], ab[:, C:]
    y_r, before, fin, err, err_b, fin_err = forward(x, a, b, f64(inp["h"]), lengths)
    dx_r, dab_r, dh0_r = backward(x, a, b, before, err_b, dy, f64(inp["dfinal"]), lengths)
    y, h, dx, dab, dh0 = gpu_pass(cuda, inp, lengths)
    close(y, y_r, err, dtype)
    close(h, fin, fin_err)
    close(dx, *dx_r, dtype)
    close(dab, *dab_r, dtype)
    close(dh0, *dh0_r)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths", [[100], [700], [64, 300, 0, 256, 37]], ids=["one tile", "chain", "packed"])
@pytest.mark.parametrize("size", [1e3, 1e4, 1e6])
def test_large_states_and_gradients_are_forgotten(cuda, size, lengths, dtype):
    inp = make(lengths, 72, dtype, seed=60)
    inp["h"] *= size
    inp["dfinal"] *= size
    check(cuda, inp, lengths, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("lengths", [[100], [700], [64, 300, 0, 256, 37]], ids=["one tile", "chain", "packed"])
def test_single_large_inputs_are_forgotten(cuda, lengths, dtype):
    """One x and one dy in about 50 is 1e4 to 1e6 times the others, at places that differ by channel."""
    inp = make(lengths, 72, dtype, seed=61)
    g = torch.Generator().manual_seed(62)
    for n in ("x", "dy"):
        v = inp[n]
        where = torch.rand(v.shape, generator=g) < 0.02
        v[where] = (v[where].float() * 10 ** (4 + 2 * torch.rand(int(where.sum()), generator=g))).to(v.dtype)
    check(cuda, inp, lengths, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_slow_and_fast_channels_side_by_side(cuda, dtype):
    """Gates of a channel are all alike: decays from 1 - 3e-4 (a = -8) to 3e-4 (a = 8) a token, and large states."""
    lengths, C = [900, 130], 72
    inp = make(lengths, C, dtype, seed=63)
    inp["ab"][:, :C] = torch.linspace(-8, 8, C).to(inp["ab"].dtype)
    inp["h"] *= 1e4
    inp["dfinal"] *= 1e4
    check(cuda, inp, lengths, dtype)
