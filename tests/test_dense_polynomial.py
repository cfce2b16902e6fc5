"""GELU's polynomial: the coefficients in csrc/dense.cuh against erfc, and against the error that is stated beside them."""
import os
import re

import torch

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "linear_attention_chunked_conv1d_gb300", "csrc", "dense.cuh")
# points closer than 10 / 2^20: between two of them an error of degree 6 in t does not pass what they show by a thousandth
X = torch.linspace(0, 10, 2 ** 20 + 1, dtype=torch.float64)


def source():
    text = open(SOURCE).read()
    body = text[text.index("uint64_t normal2("):]
    body = body[:body.index("\n}\n")]
    q = [float(c) for c in re.findall(r"both\(0\.5f \* (-?[\d.]+)f\)", body)]  # from t^6 down
    assert len(q) == 7
    stated = " ".join(text[:text.index("uint64_t normal2(")].replace("//", " ").split())
    said = re.search(r"largest relative error over that range is ([\d.]+e-\d+) .*?, ([\d.]+e-\d+) with t and Q in fp32", stated)
    return q, [float(v) for v in said.groups()]


def test_the_stated_error_holds():
    q, (said, _) = source()
    t = 1 / (1 + 0.375 * X)
    v = torch.zeros_like(X)
    for c in q:
        v = v * t + c
    off = ((v * t) / torch.special.erfcx(X) - 1).abs().max()
    assert 0.9 * said <= off <= said, float(off)


def test_the_stated_error_holds_in_fp32():
    """t and Q as the kernel computes them, fused multiply-adds among them, with a reciprocal that is rounded to the nearest."""
    q, (_, said) = source()
    f = lambda c: torch.tensor(c, dtype=torch.float64).float()  # noqa: E731
    z = (X * 2 ** 0.5).float()
    t = 1 / (1 + z * f(0.375 * 0.7071067811865476))
    v = torch.zeros_like(z)
    for c in q:
        v = (v.double() * t.double() + f(0.5 * c).double()).float()
    off = (2 * (v * t).double() / torch.special.erfcx(z.double() / 2 ** 0.5) - 1).abs().max()
    assert 0.8 * said <= off <= said, float(off)
