"""The gradient of the epilogue where the kept product is not finite."""
import math

import numpy as np
import pytest
import torch

from scatter_grouped_gemm_amd import _lib as L
from epilogue_util import ALPHA, GATED, HALF, LIMIT, PLAIN, half
from gpu_util import DEV, announce, compact_layout, i32_dev

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
INF, NAN = math.inf, math.nan
SPECIAL = [NAN, INF, -INF, 0.5, -0.5, 1e30, -1e30]


def half_limits(x, act):
    """half(), with the values and derivatives at the infinities that the calls state: SiLU
    and both GELUs are NaN at -infinity (their formulas multiply it by 0), derivatives are
    the limits."""
    v, d = half(x.clamp(-1e3, 1e3) if act != "relu2" else x, act)      # NaN stays; past 1000 sigma and Phi are 0 or 1
    if act != "relu2" and act != "none":
        v = torch.where(x > 1e3, x, torch.where(x < -1e3, torch.zeros_like(x), v))
        v = torch.where(x == -INF, torch.full_like(x, NAN), v)
    return (x if act == "none" else v), d


def exact(p, d, act):
    if act not in GATED:
        return d * half_limits(p, act)[1]
    g, u = p.chunk(2, -1)
    if act != "swiglu_clamp":
        v, s = half_limits(g, act[:-4])
        return torch.cat([d * u * s, d * v], -1)
    v, s = half_limits(torch.where(g > LIMIT, torch.full_like(g, LIMIT), g), act)
    w = torch.where(u > LIMIT, torch.full_like(u, LIMIT), torch.where(u < -LIMIT, torch.full_like(u, -LIMIT), u)) + 1
    zero = torch.zeros_like(g)
    return torch.cat([torch.where(g > LIMIT, zero, d * w * s), torch.where(u.abs() > LIMIT, zero, d * v)], -1)


def same(got, want, bound, what):
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), (what, got, want)
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), (what, got, want)
    fin = torch.isfinite(want)
    assert torch.isfinite(got[fin]).all() and ((got - want).abs()[fin] <= bound[fin]).all(), (what, got, want)


@pytest.mark.parametrize("layout", ["dense", "compact", "masked"])
@pytest.mark.parametrize("counts", [[5, 0, 40], [700, 300, 1]])      # sums in one launch, and in two
@pytest.mark.parametrize("act", PLAIN + GATED)
def test_not_finite_products_kept(act, counts, layout):
    announce("not finite", act, counts, layout)
    n = len(SPECIAL)
    cols = 8 * ((n * n + 7) // 8)                # every special gate beside every special up part
    N = 2 * cols if act in GATED else cols
    if layout == "dense":
        counts = [sum(counts)]
    G, max_m, kw = len(counts), max(counts) + 3, {}
    if layout == "dense":
        rows = counts[0]
        first = [0]
    elif layout == "compact":
        m = compact_layout(counts)
        rows = len(m)
        first = np.concatenate([[0], np.cumsum([-(-c // 128) * 128 for c in counts])])[:-1].tolist()
        kw = dict(m_indices=i32_dev(m), expert_start_loc=i32_dev(np.array(first)), num_valid=i32_dev(np.array(counts)))
    else:
        rows, first = G * max_m, [g * max_m for g in range(G)]
        kw = dict(masked_m=i32_dev(np.array(counts)), max_m=max_m)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    pre = torch.randn(rows, N, generator=gen, device=DEV).to(BF)
    dout = (torch.randn(rows, cols, generator=gen, device=DEV).abs() + 0.5).to(BF)
    v = torch.tensor(SPECIAL, device=DEV).to(BF)
    hit = [first[g] + r for g in range(G) if counts[g] for r in {0, counts[g] - 1}]
    for r in hit:
        pre[r, :n * n] = v.repeat_interleave(n)
        if act in GATED:
            pre[r, cols:cols + n * n] = v.repeat(n)
    dpre, dbias = torch.empty(rows, N, dtype=BF, device=DEV), torch.empty(G, N, dtype=F32, device=DEV)
    L.moe_act_bwd(pre, dout, dpre, act, dbias=dbias, alpha=ALPHA, limit=LIMIT, **kw)
    torch.cuda.synchronize()
    for g in range(G):
        at = slice(first[g], first[g] + counts[g])
        p, d = pre[at].double(), dout[at].double()
        want = exact(p, d, act)
        # fp32: 2^-20 of each factor's terms (the slope's two add up to 2.2, 1.2 times that
        # with the clamped gate's alpha; |act| <= |p|), then one rounding
        if act in GATED:
            t = torch.cat([d * 2.7 * (p[:, cols:].abs() + 1), d * p[:, :cols].abs()], -1)
        else:
            t = d * (2 * p.abs() if act == "relu2" else 2.2)
        t = 2.0 ** -20 * torch.nan_to_num(t, nan=0.0, posinf=INF)      # a gradient beside a NaN is an exact 0
        same(dpre[at], want, t + HALF[BF] * (want.abs() + t), ("dpre", g))
        s = want.sum(0)
        bound = t.sum(0) + (counts[g] + 4) * 2.0 ** -24 * (want.abs() + t).sum(0)
        same(dbias[g], s, bound + HALF[F32] * (s.abs() + bound), ("dbias", g))


@pytest.mark.parametrize("T", [1, 33])
def test_the_tail_of_gelu(T):
    """x Phi(x) of negative x keeps a relative error of 4e-7 (Phi(-t) exp(t^2/2) as a polynomial,
    in fp32), t^2 / 2 times 2.75 places of 2^-24 (two products and a constant rounded in the
    exponential's argument), two of 2^-23 (exponential, reciprocal) and two of 2^-24 (the last
    products).  An identity weight passes x through."""
    x = torch.cat([torch.arange(-12.75, -1, 1 / 16), torch.arange(-1, 0, 1 / 128)]).to(BF)
    n = len(x) // 8 * 8
    x = x[:n].to(DEV)
    o = torch.empty(T, n, dtype=F32, device=DEV)
    L.moe_linear(x[None].expand(T, n).contiguous(), torch.eye(n, dtype=BF, device=DEV), o, act="gelu")
    t = -x.double()
    want = -t * 0.5 * torch.special.erfc(t / math.sqrt(2))
    bound = 4e-7 + 1.375 * t * t * 2.0 ** -24 + 2 * 2.0 ** -23 + 2 * 2.0 ** -24
    assert ((o.double() / want - 1).abs() <= bound).all(), float(((o.double() / want - 1).abs() / bound).max())
