"""The dense half's gradients in 64 bits with the roundings that its calls state, and how near a result has to be to them.

The calls round on the way, each time to the nearest: z to bf16 where it is kept, gate and up to 24 bits (cut off), dz, dgate
and dup to bf16 where they become operands; in the whole block also n, h, dh and dn. Here these are rounded the same, so that
what is left of the difference is
  - the result's own rounding, at most U = 2^-8 of each value (half a step of bf16);
  - sums in fp32: (a few) 2^-24 of the absolute terms;
  - intermediate values whose sum in fp32 falls on the other side of a rounding's edge than the one in 64 bits. The sums are
    off by some 2^-22 of a value, a step is 2^-8 to 2^-7 of it: one in about 2^13 falls so, by a whole step (2 U) each, in no
    direction: sqrt(2^-13) 2 U = 0.022 U in norm for each rounding on the way, of which there are at most seven, with a gain
    of at most 4: 0.022 sqrt(7) 4 U < 0.25 U.
So results in bf16 are within 1.25 U in norm, those in fp32 within 0.25 U; a row's or a column's norm, of fewer values, within
twice that. One value of a product d w, where its d are what may have fallen so, is off by U of itself; by 2 U |d w| of its
largest term, if that is one of them (with eight terms to a sum it can be most of it: 1.007 of the bound was seen where the
largest term was taken for a usual one, in dgate, dup of 40000 rows of 8); and by the others' sum, in no direction: with 2^-13 of n terms
2 U sqrt(n 2^-13) of a usual term, that is 2 U / 90 of the matrix's root mean square, so for 90 such deviations 2 U of it."""
import math

import torch

U = torch.finfo(torch.bfloat16).eps / 2
BF16 = torch.bfloat16


def act64(z, act):
    return {"none": lambda: z, "relu": lambda: torch.relu(z), "silu": lambda: z * torch.sigmoid(z),
            "gelu": lambda: 0.5 * z * torch.erfc(-z / math.sqrt(2)),
            "gelu_tanh": lambda: z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))}[act]()


def slope64(z, act):
    z = z.detach().requires_grad_()
    with torch.enable_grad():
        return torch.autograd.grad(act64(z, act).sum(), z)[0]


def r16(t):
    return t.to(BF16).double()


def r24(t):
    return (t.float().contiguous().view(torch.int32) & -256).view(torch.float32).double()


def largest(d, w):
    """No less than the largest term of each value of d w."""
    return d.abs().amax(1)[:, None] * w.abs().amax(0)[None]


def linear_gradients(x, w, bias, dy, act):
    """dx, dw, dbias, the dz that the products take, and the largest terms of each."""
    x, w, dy = x.double(), w.double(), dy.double()
    z = x @ w.T + (0 if bias is None else bias.double())
    dz = dy if act == "none" else dy * slope64(r16(z), act)
    d = dz if act == "none" else r16(dz)
    # dbias is summed before dz is rounded: what may have fallen so is z, of which act' takes |z act''| <= 1.2
    return dict(dx=d @ w, dw=d.T @ x, dbias=dz.sum(0)), d, dict(dx=largest(d, w), dw=largest(d.T, x), dbias=1.2 * dy.abs().amax(0))


def gated_gradients(x, w_gate, w_up, dh, act):
    """dx, dw, dw_up, the dgate, dup that the products take, and the largest terms of each."""
    x, wg, wu, dh = x.double(), w_gate.double(), w_up.double(), dh.double()
    gate, up = r24(x @ wg.T), r24(x @ wu.T)
    dg, du = r16(dh * up * slope64(gate, act)), r16(dh * act64(gate, act))
    return (dict(dx=dg @ wg + du @ wu, dw=dg.T @ x, dw_up=du.T @ x), (dg, du),
            dict(dx=torch.maximum(largest(dg, wg), largest(du, wu)), dw=largest(dg.T, x), dw_up=largest(du.T, x)))


def norm_gradients(x, w, mean, rstd, dy, dskip):
    xh = (x - mean) * rstd
    u = dy * w
    return rstd * (u - u.mean(1, keepdim=True) - xh * (u * xh).mean(1, keepdim=True)) + dskip, (dy * xh).sum(0), dy.sum(0)


def block(x, norm_w, norm_b, w_gate, w_up, w_down, dy, act, eps=1e-5):
    """path.FeedForward: y and its gradients by name."""
    x, nw, nb, wg, wu, wd, dy = (t.double() for t in (x, norm_w, norm_b, w_gate, w_up, w_down, dy))
    var, mean = torch.var_mean(x, 1, unbiased=False, keepdim=True)
    rstd = 1 / torch.sqrt(var + eps)
    n = r16((x - mean) * rstd * nw + nb)
    h = r16(act64(n @ wg.T, act) * (n @ wu.T))
    dh = r16(dy @ wd)
    back, _, _ = gated_gradients(n, wg, wu, dh, act)
    dx, dnw, dnb = norm_gradients(x, nw, mean, rstd, r16(back["dx"]), dy)
    return dict(y=h @ wd.T + x, x=dx, norm_w=dnw, norm_b=dnb, w_gate=back["dw"], w_up=back["dw_up"], w_down=dy.T @ h)


def off(got, want, term=None):
    """By how much a result is further off than it may be: 1 or less is right. term: the largest term of each value, where each
    is to be looked at by itself."""
    e, want = got.double() - want, want.double()
    own = 1.0 if got.dtype == BF16 else 0.0
    norm = lambda t, **k: torch.linalg.vector_norm(t, **k)  # noqa: E731
    worst = [norm(e) / ((own + 0.25) * U * norm(want))]
    rms = norm(want) / math.sqrt(want.numel())
    if term is not None:
        worst.append((e.abs() / (U * (own * want.abs() + 2 * term + 2 * rms))).max())
    if want.dim() == 2 and min(want.shape) >= 8:
        for dim, n in ((0, want.shape[0]), (1, want.shape[1])):
            # a row of small values stands next to others whose terms it shares: a hundredth of a usual row's norm is added
            worst.append((norm(e, dim=dim) / (2 * (own + 0.25) * U * (norm(want, dim=dim) + 0.01 * rms * math.sqrt(n)))).max())
    worst = torch.stack(worst)
    return math.inf if bool(worst.isnan().any()) else float(worst.max())
