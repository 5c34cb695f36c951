"""The experts' products in 64 bits, and how far fp32 sums and one rounding may take a kernel from them.

A sum of K products in fp32, in any order and with K more roundings inside the matrix instructions, is off by at most
2 K 2^-24 times the sum of the products' magnitudes; the result's rounding adds half a step of its type. Activations: an
exponential with an error of (1 + |argument|) steps of 2^-23, the arguments' own roundings (a relative error of 2^-23 in an
argument of up to 2 x^2 or 1.6 (|x| + 0.045 |x|^3)), and a dozen elementary operations."""
import math

import torch

import all_reduce_reduction_ring_amd as ar

F64 = torch.float64
ACTS = (ar.AR_ACT_SILU, ar.AR_ACT_GELU, ar.AR_ACT_GELU_TANH)


def act(x, kind):
    if kind == ar.AR_ACT_SILU:
        return x * torch.sigmoid(x)
    if kind == ar.AR_ACT_GELU:
        return x * 0.5 * torch.special.erfc(-x * math.sqrt(0.5))
    return x * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3))


def slope(x, kind):
    with torch.enable_grad():
        y = x.detach().clone().requires_grad_()
        return torch.autograd.grad(act(y, kind).sum(), y)[0]


def act_error(x):
    """Of an activation next to its value, and of its slope next to 1."""
    a = x.abs()
    return (16 + 4 * a + 2 * a ** 2 + 0.2 * a ** 3) * 2.0 ** -23


def half_step(want, dtype):
    """Half a step of the type at `want` (and at twice its smallest number below that)."""
    f = torch.finfo(dtype)
    return want.abs() * (f.eps / 2) + f.smallest_normal * f.eps


def sum_error(k, magnitudes):
    return 2 * max(k, 1) * 2.0 ** -24 * magnitudes


def mm(a, b):
    """a b in 64 bits with the bound on an fp32 sum's error."""
    a, b = a.to(F64), b.to(F64)
    return a @ b, sum_error(a.shape[1], a.abs() @ b.abs())


def close(got, want, tol, what):
    got = got.to(F64)
    bad = ~((got - want).abs() <= tol)  # NaN is bad
    if bad.any():
        at = bad.nonzero()[0].tolist()
        g, w, t = (v[tuple(at)].item() for v in (got, want, tol))
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} off; first at {at}: got {g}, want {w} +- {t}")


def gated(x, wg, wu, kind, dtype):
    """((h, tolerance), (g, tolerance), (u, tolerance))"""
    g, eg = mm(x, wg.t())
    u, eu = mm(x, wu.t())
    h = act(g, kind) * u
    # |act'| <= 1.13
    eh = 1.13 * u.abs() * eg + act(g, kind).abs() * eu + 1.13 * eg * eu + h.abs() * act_error(g)
    return tuple((v, e * 1.01 + half_step(v, dtype) * 1.01) for v, e in ((h, eh), (g, eg), (u, eu)))


def slopes(dout, gate, up, kind, dtype):
    """((dgate, tolerance), (dup, tolerance))"""
    d, g, u = (t.to(F64) for t in (dout, gate, up))
    dg, du = d * u * slope(g, kind), d * act(g, kind)
    return ((dg, (d * u).abs() * act_error(g) + half_step(dg, dtype) * 1.01),
            (du, du.abs() * act_error(g) + half_step(du, dtype) * 1.01))


def rounded(value_and_error, dtype):
    v, e = value_and_error
    return v, e * 1.01 + half_step(v, dtype) * 1.01


def segments(counts, align, spare=0):
    """Starts of the experts' segments and the end, and rows of the buffers (spare ones behind the last segment)."""
    starts = [0]
    for c in counts:
        starts.append(starts[-1] + -(-c // align) * align)
    return starts, starts[-1] + spare
