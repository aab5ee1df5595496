"""64-bit plain forms of the products with an epilogue, and bounds on what fp32 sums
and one rounding may be off (not collected by pytest)."""
import math

import torch

ALPHA, LIMIT = 1.702, 7.0
GATED = ("silu_mul", "gelu_mul", "gelu_tanh_mul", "swiglu_clamp")
PLAIN = ("none", "silu", "gelu", "gelu_tanh", "relu2")
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a place, relative


def half(x, act):
    """Value and derivative of an activation without its up part, in 64 bits."""
    if act in ("silu", "swiglu_clamp"):
        a = ALPHA if act == "swiglu_clamp" else 1.0
        s = torch.special.expit(a * x)
        return x * s, s + a * x * s * (1 - s)
    if act == "gelu":
        c = 0.5 * torch.special.erfc(-x / math.sqrt(2))
        return x * c, c + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        s = torch.special.expit(2 * c * (x + 0.044715 * x ** 3))
        return x * s, s + x * s * (1 - s) * 2 * c * (1 + 3 * 0.044715 * x * x)
    if act == "relu2":
        return torch.relu(x) ** 2, 2 * torch.relu(x)
    return x, torch.ones_like(x)


def activation(p, act, alpha=ALPHA, limit=LIMIT):
    if act not in GATED:
        return half(p, act)[0]
    g, u = p.chunk(2, -1)
    if act == "swiglu_clamp":
        g, u = g.clamp(max=limit), u.clamp(-limit, limit)
        return g * torch.special.expit(alpha * g) * (u + 1)
    return half(g, act[:-4])[0] * u


def act_bound(p, dp, act, dtype):
    """What out = act(p) may be off where p is off by at most dp: the activation's
    steepness (|act'| <= 1.13 for the three smooth ones, 1.1 times that of its argument for
    the clamped gate, 2 |x| for the squared one), 2^-20 of its terms for exponential,
    reciprocal and polynomial (each a few 2^-23; the argument of the exponential is
    rounded, which costs |z| 2^-24 of a value that e^-|z| makes small), and half a place
    of the output's type."""
    if act == "none":
        y = p.abs()
        return dp + HALF[dtype] * (y + dp)
    if act == "relu2":
        d = 2 * torch.relu(p) * dp + dp * dp
        y = torch.relu(p) ** 2
        return d + 2.0 ** -23 * y + HALF[dtype] * (y + d)
    if act not in GATED:
        d = 1.13 * dp + 2.0 ** -20 * p.abs()
        return d + HALF[dtype] * (p.abs() + d)
    g, u = p.chunk(2, -1)
    dg, du = dp.chunk(2, -1)
    if act == "swiglu_clamp":
        g, u = g.clamp(max=LIMIT), u.clamp(-LIMIT, LIMIT)
        v, w = half(g, act)[0], u + 1
    else:
        v, w = half(g, act[:-4])[0], u
    d = (1.13 * dg + 2.0 ** -20 * g.abs()) * (w.abs() + du) + v.abs() * (du + 2.0 ** -23 * (1 + u.abs()))
    y = (v * w).abs()
    return d + HALF[dtype] * (y + d)


def product_bound(x, w, bias):
    """|fp32 sum - exact| of x w^T + bias: each of the K + 2 additions, in whatever order,
    is off by at most 2^-23 (a place: the matrix cores may cut) of the sum of the
    magnitudes; x and w in 64 bits."""
    s = x.abs() @ w.abs().t()
    if bias is not None:
        s = s + bias.abs()
    return (x.shape[1] + 2) * 2.0 ** -23 * s


def check(got, want, bound, what):
    got = got.double()
    bad = ~((got - want).abs() <= bound)
    assert not bad.any(), (what, int(bad.sum()), float((got - want).abs()[bad].max()), float(bound[bad].min()))
