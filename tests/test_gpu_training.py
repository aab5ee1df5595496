"""The training operators against plain implementations in 64 bits, with bounds
derived from their roundings: a bf16 result is off by at most 2^-8 of its value
from the last rounding, an fp32 operation by 2^-24, and a sum of n fp32 terms by
n * 2^-24 of the sum of their magnitudes (2^-23 a term through the matrix
instructions, whose inner additions need not round to nearest)."""
import numpy as np
import pytest
import torch

from scatter_grouped_gemm_amd import AdamW, MoELayer, inputs
from scatter_grouped_gemm_amd import _lib as L
from gpu_util import DEV, announce, compact_layout, distinct_ids, i32_dev, poison

pytestmark = pytest.mark.gpu

U16, U32 = 2.0 ** -8, 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator().manual_seed(seed)


def randn(seed, *shape, scale=1.0, dtype=BF):
    return (torch.randn(*shape, generator=gen(seed)) * scale).to(dtype)


def same_bits(a, b):
    return torch.equal(a.cpu().contiguous().view(torch.uint8), b.cpu().contiguous().view(torch.uint8))


def within(got, want, bound):
    got = got.cpu().double()
    assert got.shape == want.shape and got.numel() and torch.isfinite(got).all()
    over = (got - want).abs() - bound
    assert over.max().item() <= 0, f"off by {over.max().item():.3e} more than the bound {bound.max().item():.3e}"


def slots(seed, T, k, rows, held=0.7):
    """src2dst [T, k] of distinct rows, about a `held` part of the slots used."""
    rng = np.random.default_rng(seed)
    s = np.full(T * k, -1, np.int32)
    use = np.flatnonzero(rng.random(T * k) < (held if T * k > 2 else 1.0))[:rows]
    s[use] = rng.permutation(rows)[:len(use)]
    return s.reshape(T, k)


# ------------------------------------------------------------------------------
# combine, scatter, routing weights
# ------------------------------------------------------------------------------

TOKEN_CASES = [(1, 8, 1), (1, 256, 8), (7, 104, 3), (33, 256, 2), (64, 7168, 8), (5, 8200, 9), (3, 512, 32), (300, 1032, 6),
               (2, 8192, 4), (17, 64, 16)]


@pytest.mark.parametrize("T,H,k", TOKEN_CASES)
def test_combine_bwd(T, H, k):
    announce("combine_bwd", T, H, k)
    rows = T * k + 5
    s = slots(T + H + k, T, k, rows)
    if T > 1:
        s[0] = -1                       # a token without a held slot
    if k > 1:
        s[-1, 0], s[-1, 1] = rows, -7   # neither is a row
    Y, dout = randn(1, rows, H), randn(2, T, H, scale=0.1)
    w = torch.rand(T, k, generator=gen(3))
    st = torch.from_numpy(s).long()
    ok = (st >= 0) & (st < rows)
    named = torch.zeros(rows, dtype=torch.bool)
    named[st[ok]] = True
    Y[~named] = float("nan")            # rows that nothing names are not looked at
    dY, dw = poison((rows, H), BF), poison((T, k), F32)
    before = dY.clone()
    L.moe_combine_bwd(dout.to(DEV), Y.to(DEV), i32_dev(s), w.to(DEV), dY, dw)
    torch.cuda.synchronize()
    assert same_bits(dY[~named.to(DEV)], before[~named.to(DEV)])
    prod = w.double()[..., None] * dout.double()[:, None, :]
    want = torch.zeros(rows, H, dtype=torch.float64)
    want[st[ok]] = prod[ok]
    # one fp32 product, then one rounding to bf16
    within(dY[named.to(DEV)], want[named], want[named].abs() * (U16 * (1 + U16) + U32) + 1e-40)
    terms = torch.where(ok[..., None], Y.double()[st.clamp(0, rows - 1)] * dout.double()[:, None, :], 0.0)
    # chain of a thread, six steps across the lanes, at most 16 wavefronts
    nt = min(1024, -(-(H // 8) // 64) * 64)
    n = 8 * -(-H // (8 * nt)) + 6 + 16
    within(dw, terms.sum(-1), n * U32 * terms.abs().sum(-1))
    assert (dw.cpu()[~ok] == 0).all()


@pytest.mark.parametrize("T,H,k", TOKEN_CASES)
def test_scatter_bwd(T, H, k):
    announce("scatter_bwd", T, H, k)
    rows = T * k + 5
    s = slots(T + H + k, T, k, rows)
    if T > 1:
        s[0] = -1
    if k > 1:
        s[-1, 0], s[-1, 1] = rows, -7
    dX = randn(1, rows, H)
    st = torch.from_numpy(s).long()
    ok = (st >= 0) & (st < rows)
    named = torch.zeros(rows, dtype=torch.bool)
    named[st[ok]] = True
    dX[~named] = float("inf")
    dx = poison((T, H), BF)
    L.moe_scatter_bwd(dX.to(DEV), i32_dev(s), dx)
    terms = torch.where(ok[..., None], dX.double()[st.clamp(0, rows - 1)], 0.0)
    want = terms.sum(1)
    within(dx, want, want.abs() * U16 + k * U32 * (1 + U16) * terms.abs().sum(1))
    if T > 1:
        assert (dx[0] == 0).all()


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (5, 8, 2), (130, 64, 6), (9, 100, 8), (3, 256, 32), (2, 300, 8), (4, 1024, 8)])
def test_route_topk_bwd(T, E, k):
    announce("route_topk_bwd", T, E, k)
    ids = distinct_ids(np.random.default_rng(E), T, E, k)
    if T > 4 and k > 1:
        ids[1, 1] = ids[1, 0]           # one id twice: the sum of both
        ids[2, 0], ids[3, 0] = E, -1    # no expert
    w = torch.softmax(torch.randn(T, k, generator=gen(1)), 1)
    dw = torch.randn(T, k, generator=gen(2))
    out = poison((T, E), F32)
    L.moe_route_topk_bwd(i32_dev(ids), w.to(DEV), dw.to(DEV), out)
    wd, dd = w.double(), dw.double()
    term = wd * (dd - (wd * dd).sum(1, keepdim=True))
    # product, k additions, difference, product
    size = wd * (dd.abs() + (wd * dd.abs()).sum(1, keepdim=True)) * (k + 4) * U32
    want, bound = torch.zeros(T, E, dtype=torch.float64), torch.zeros(T, E, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            if 0 <= ids[t, j] < E:
                want[t, ids[t, j]] += term[t, j]
                bound[t, ids[t, j]] += 2 * size[t, j]
    within(out, want, bound)
    assert (out.cpu()[want == 0] == 0).all()


# ------------------------------------------------------------------------------
# SiLU-and-mul
# ------------------------------------------------------------------------------

def _silu_bwd_ref(gu, da):
    I = da.shape[1]
    g, u, da = gu.double()[:, :I], gu.double()[:, I:], da.double()
    s = torch.sigmoid(g)
    dg, du = da * u * s * (1 + g * (1 - s)), da * g * s
    # e^-g: its exponent is off by |g| 2^-24 and the value by 2^-23, the
    # reciprocal by 2^-23: s by (|g| + 6) 2^-23 of itself at most; 1 - s by that
    # and one more rounding; then six roundings of terms of size s (1 + |g|)
    b = 2.0 ** -23
    slope = s * b * (2 * g * g + 18 * g.abs() + 14)
    return dg, du, (da * u).abs() * slope + dg.abs() * U16, du.abs() * (U16 + (g.abs() + 10) * b)


@pytest.mark.parametrize("how", ["all", "compact", "masked"])
@pytest.mark.parametrize("M,I", [(1, 128), (6, 512), (130, 640), (9, 1408), (12, 2176)])
def test_silu_and_mul_bwd(M, I, how):
    announce("silu_and_mul_bwd", M, I, how)
    gu, da = randn(1, M, 2 * I, scale=2.0), randn(2, M, I)
    keep = torch.ones(M, dtype=torch.bool)
    kw = {}
    if how == "compact":
        keep = torch.rand(M, generator=gen(3)) < 0.6
        kw = dict(m_indices=i32_dev(np.where(keep.numpy(), 3, -1)))
    elif how == "masked":
        mx = 3 if M % 3 == 0 else M
        c = np.arange(M // mx) % (mx + 1)
        keep = torch.from_numpy((np.arange(M) % mx) < np.repeat(c, mx))
        kw = dict(masked_m=i32_dev(c), max_m=mx)
    gu[~keep], da[~keep] = float("nan"), float("nan")
    gu[:, 0] = torch.where(keep, torch.tensor(-120.0), torch.tensor(float("nan"))).to(BF)   # e^120 is past fp32
    gu[:, 1] = torch.where(keep, torch.tensor(200.0), torch.tensor(float("nan"))).to(BF)
    dgu, act = poison((M, 2 * I), BF), poison((M, I), BF)
    d0, a0 = dgu.clone(), act.clone()
    g_dev, da_dev = gu.to(DEV), da.to(DEV)
    L.silu_and_mul_bwd(g_dev, da_dev, dgu, act, **kw)
    torch.cuda.synchronize()
    kd = keep.to(DEV)
    assert same_bits(dgu[~kd], d0[~kd]) and same_bits(act[~kd], a0[~kd])
    if not keep.any():
        return
    dg, du, bg, bu = _silu_bwd_ref(gu[keep], da[keep])
    within(dgu[kd][:, :I], dg, bg + 1e-38)
    within(dgu[kd][:, I:], du, bu + 1e-38)
    fwd = poison((M, I), BF)
    L.silu_and_mul(g_dev, fwd, m_indices=kw.get("m_indices"), masked_m=kw.get("masked_m"), max_m=kw.get("max_m", 0))
    assert same_bits(act[kd], fwd[kd])
    L.silu_and_mul_bwd(g_dev, da_dev, g_dev, **kw)      # in place, without act
    assert same_bits(g_dev[kd], dgu[kd])


# ------------------------------------------------------------------------------
# products
# ------------------------------------------------------------------------------

COUNTS = [[1], [0], [128], [129, 0, 5], [0, 300, 64, 256, 0, 1], [17, 513, 128], [1030], [255, 257, 31, 2, 96, 64, 700]]
SHAPES = [(128, 128), (256, 384), (384, 256), (1408, 128), (128, 1408), (512, 640)]


def _operands(counts, N, K, seed, ints, extra=128):
    m = compact_layout(counts, extra_rows=extra)
    M = len(m)
    if ints:   # every partial sum is a whole number below 2^24
        draw = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=gen(seed)).to(BF)  # noqa: E731
        dC, A, B = draw(-3, 4, M, N), draw(-4, 5, M, K), draw(-2, 3, len(counts), N, K)
    else:
        dC, A, B = randn(seed, M, N), randn(seed + 1, M, K), randn(seed + 2, len(counts), N, K)
    keep = torch.from_numpy(m >= 0)
    dC[~keep], A[~keep] = float("nan"), float("inf")
    pad = [-(-c // 128) * 128 for c in counts]
    starts = np.concatenate([[0], np.cumsum(pad)[:-1]]).astype(np.int32)
    return m, keep, dC, A, B, starts, np.array(counts, np.int32)


def _round(x, dtype):
    return x.to(F32).to(dtype)      # exact in fp32 for whole numbers below 2^24


@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("counts", COUNTS, ids=str)
def test_dgrad(counts, N, K):
    announce("dgrad", counts, N, K)
    for ints in (True, False):
        m, keep, dC, _, B, _, _ = _operands(counts, N, K, 5, ints)
        dA = poison((len(m), K), BF)
        before = dA.clone()
        L.grouped_gemm_contig_dgrad(dC.to(DEV), B.to(DEV), dA, i32_dev(m))
        torch.cuda.synchronize()
        kd = keep.to(DEV)
        assert same_bits(dA[~kd], before[~kd])
        if not keep.any():
            continue
        e = torch.from_numpy(m[m >= 0]).long()
        want, size = torch.zeros(len(e), K, dtype=torch.float64), torch.zeros(len(e), K, dtype=torch.float64)
        for g in e.unique().tolist():
            rows = dC[keep][e == g].double()
            want[e == g], size[e == g] = rows @ B[g].double(), rows.abs() @ B[g].double().abs()
        if ints:
            assert torch.equal(dA[kd].cpu(), _round(want, BF))      # 0 and -0 are one value
        else:
            within(dA[kd], want, want.abs() * U16 + N * 2 * U32 * (1 + U16) * size)


@pytest.mark.parametrize("out,acc", [(BF, False), (BF, True), (F32, False), (F32, True)])
@pytest.mark.parametrize("N,K", SHAPES)
@pytest.mark.parametrize("counts", COUNTS, ids=str)
def test_wgrad(counts, N, K, out, acc):
    announce("wgrad", counts, N, K, out, acc)
    G = len(counts)
    for ints in (True, False):
        m, keep, dC, A, _, starts, nv = _operands(counts, N, K, 7, ints)
        old = torch.randint(-8, 9, (G, N, K), generator=gen(9)).to(out) if ints else randn(9, G, N, K, dtype=out)
        dB = old.to(DEV) if acc else poison((G, N, K), out)
        L.grouped_gemm_contig_wgrad(dC.to(DEV), A.to(DEV), i32_dev(starts), i32_dev(nv), dB, accumulate=acc)
        want, size = torch.zeros(G, N, K, dtype=torch.float64), torch.zeros(G, N, K, dtype=torch.float64)
        for g, (s, c) in enumerate(zip(starts, nv)):
            p, q = dC[s:s + c].double(), A[s:s + c].double()
            want[g], size[g] = p.t() @ q, p.abs().t() @ q.abs()
        if acc:
            want, size = want + old.double(), size + old.double().abs()
        if ints:
            assert torch.equal(dB.cpu(), _round(want, out))
        else:
            n = max(counts) + 2
            within(dB, want, want.abs() * (U16 if out is BF else U32) + n * 2 * U32 * (1 + U16) * size)


def test_wgrad_ranges_are_cut():
    """Ranges past M, negative counts and negative starts read nothing outside."""
    announce("wgrad ranges")
    M, N, K = 200, 128, 128
    dC, A = torch.ones(M, N, dtype=BF, device=DEV), torch.ones(M, K, dtype=BF, device=DEV)
    starts, nv = [0, 150, 500, -3, 10, 190], [1, 1000, 4, 4, -2, 10]
    dB = poison((6, N, K), F32)
    L.grouped_gemm_contig_wgrad(dC, A, i32_dev(np.array(starts)), i32_dev(np.array(nv)), dB)
    assert dB.amax((1, 2)).tolist() == [1.0, 50.0, 0.0, 0.0, 0.0, 10.0] == dB.amin((1, 2)).tolist()


def test_dgrad_row_does_not_depend_on_its_batch():
    announce("dgrad batch invariance")
    N, K = 512, 384
    dC, B = randn(1, 1024, N).to(DEV), randn(2, 1, N, K).to(DEV)
    whole = torch.empty(1024, K, dtype=BF, device=DEV)
    L.grouped_gemm_contig_dgrad(dC, B, whole, i32_dev(np.zeros(1024, np.int32)))
    for n in (1, 40, 129, 300):
        m = compact_layout([n], extra_rows=0)
        part = torch.zeros(len(m), K, dtype=BF, device=DEV)
        L.grouped_gemm_contig_dgrad(dC[:len(m)].contiguous(), B, part, i32_dev(m))
        assert same_bits(part[:n], whole[:n])


def test_products_with_more_rows_than_a_panel_of_32_bits():
    """Byte offsets past 2^32 in dC: a late expert's rows lie 4.4 GB in."""
    announce("large offsets")
    N, K = 16384, 128
    blocks = 1040
    M = blocks * 128
    dC = torch.zeros(M, N, dtype=BF, device=DEV)
    A = torch.zeros(M, K, dtype=BF, device=DEV)
    last = M - 128
    dC[last:last + 3] = 2.0
    A[last:last + 3] = 3.0
    m = np.full(M, -1, np.int32)
    m[last:last + 3] = 1
    B = torch.ones(2, N, K, dtype=BF, device=DEV)
    dA = torch.zeros(M, K, dtype=BF, device=DEV)
    L.grouped_gemm_contig_dgrad(dC, B, dA, i32_dev(m))
    assert (dA[last:last + 3] == 2.0 * N).all() and (dA[:last] == 0).all() and (dA[last + 3:] == 0).all()
    dB = poison((2, N, K), F32)
    L.grouped_gemm_contig_wgrad(dC, A, i32_dev(np.array([0, last])), i32_dev(np.array([0, 3])), dB)
    assert (dB[0] == 0).all() and (dB[1] == 18.0).all()


# ------------------------------------------------------------------------------
# AdamW
# ------------------------------------------------------------------------------

def _mix(x):
    x = x ^ (x >> 16)
    x = (x * 0x9E3779B1) & 0xffffffff
    x = x ^ (x >> 15)
    x = (x * 0x85EBCA77) & 0xffffffff
    return x ^ (x >> 16)


def _bits(seed, tensor, step, n):
    key = _mix((_mix((seed + 0x9E3779B9 * (tensor + 1)) & 0xffffffff) + step) & 0xffffffff)
    return _mix(_mix(torch.arange(n)) ^ key)


VALUES = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()


def _decoded(codes, scale, at, n):
    c = codes[at:at + n].cpu().view(torch.float8_e4m3fn).double()
    e = scale[at // 128: at // 128 + -(-n // 128)].cpu().double().repeat_interleave(128)[:n]
    return c * torch.exp2(e - 127)


def _check_codes(x, codes, scale, at, u, keep):
    """The codes of x: each the one that the random bits choose, except where the
    choice is within fp32's error of the border, and the scales of the groups."""
    n = x.numel()
    groups = -(-n // 128)
    size = torch.zeros(groups * 128, dtype=torch.float64)
    size[:n] = x.abs()
    top = size.view(-1, 128).amax(1)
    e = torch.where(top > 0, torch.ceil(torch.log2(top.clamp(min=1e-300) / 448)), torch.tensor(-126.0, dtype=torch.float64)).clamp(-126, 127)
    got_e = scale[at // 128: at // 128 + groups].cpu().double() - 127
    # a maximum within fp32's error of 448 * 2^e may take either exponent
    edge = torch.abs(torch.log2(top.clamp(min=1e-300) / 448) - e) < 1e-5
    assert ((got_e == e) | edge | (torch.abs(torch.log2(top.clamp(min=1e-300) / 448) - got_e) < 1e-5)).all()
    a = size[:n] / torch.exp2(got_e).repeat_interleave(128)[:n]
    got = codes[at:at + n].cpu().view(torch.float8_e4m3fn).double()
    assert (torch.sign(got) * torch.sign(x) >= 0).all()
    low = (torch.searchsorted(VALUES, a.clamp(max=448), right=True) - 1).clamp(0, 125)
    unit = VALUES[low + 1] - VALUES[low]
    part = (a - VALUES[low]) / unit + u / 65536
    want = VALUES[low + (part >= 1).long()]
    if keep:
        want = torch.where((a > 0) & (want == 0), VALUES[1], want)
    # a is off by a few 2^-23 of at most 16 units: 2^-17 of a unit around a border
    border = ((part - 1).abs() < 2.0 ** -17) | (part < 2.0 ** -17) | (part > 2 - 2.0 ** -17)
    assert ((got.abs() == want) | border).all()
    return (torch.copysign(got.abs(), x) - torch.copysign(a, x)) / unit


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("pdt,gdt", [(F32, F32), (F32, BF), (BF, F32), (BF, BF)])
def test_adamw_step(pdt, gdt, bits):
    announce("adamw", pdt, gdt, bits)
    sizes = [1, 7, 128, 129, 2048, 2055, 6000, 300, 40001]
    lr, b1, b2, eps, seed = 3e-3, 0.9, 0.99, 1e-8, 77
    wd = [0.0 if i % 2 else 0.1 for i in range(len(sizes))]
    P0 = [randn(i, n, scale=0.1, dtype=F32) for i, n in enumerate(sizes)]
    Gr = [randn(50 + i, n, scale=10.0 ** (i % 3 - 2), dtype=gdt) for i, n in enumerate(sizes)]
    for g in Gr:
        g[torch.rand(g.shape, generator=gen(4)) < 0.2] = 0       # rows that no token reached
    if sizes[3] > 20:
        Gr[3][:] = 0                                             # a whole group without gradient
    p = [x.to(pdt).to(DEV) for x in P0]
    gd = [g.to(DEV) for g in Gr]
    opt = AdamW(p, gd, lr=lr, betas=(b1, b2), eps=eps, weight_decay=wd, state_bits=bits, seed=seed)
    scale = torch.full((1,), 0.5, device=DEV)
    for step in (1, 2, 3):
        before = []
        for i, (n, at) in enumerate(zip(sizes, opt.offsets)):
            w = (opt.master[at:at + n] if pdt is BF else p[i]).cpu().double()
            if bits == 8:
                m, v = _decoded(opt.m, opt.m_scale, at, n), _decoded(opt.v, opt.v_scale, at, n) ** 2
            else:
                m, v = opt.m[at:at + n].cpu().double(), opt.v[at:at + n].cpu().double()
            before.append((w, m, v))
        opt.step(grad_scale=scale)
        torch.cuda.synchronize()
        assert opt.steps.item() == step and opt._counter[1].item() == 0
        for i, (n, at) in enumerate(zip(sizes, opt.offsets)):
            w, m, v = before[i]
            g = Gr[i].double() * 0.5
            msz, m = b1 * m.abs() + (1 - b1) * g.abs(), b1 * m + (1 - b1) * g
            v = b2 * v + (1 - b2) * g * g
            den = v.sqrt() / (1 - b2 ** step) ** 0.5 + eps
            up = lr / (1 - b1 ** step) / den
            want = w * (1 - lr * wd[i]) - up * m
            # m: the two constants, two products, a sum; then root, quotient and
            # products, each of the hardware's within 2^-23
            tol = 3 * U32 * w.abs() + up * msz * 24 * U32
            got = opt.master[at:at + n] if pdt is BF else p[i]
            within(got, want, tol + 1e-30)
            if pdt is BF:
                assert same_bits(p[i], got.to(BF))
            if bits == 32:
                within(opt.m[at:at + n], m, 5 * U32 * msz + 1e-38)
                within(opt.v[at:at + n], v, 7 * U32 * v + 1e-38)
            else:
                r = _bits(seed, i, step, n)
                _check_codes(m, opt.m, opt.m_scale, at, r & 0xffff, False)
                _check_codes(v.sqrt(), opt.v, opt.v_scale, at, r >> 16, True)


def test_adamw_8bit_rounding_has_no_bias():
    """One step from zero states: the mean error of the codes is within six
    standard deviations of zero (an error lies within one unit: sd at most 1/2)."""
    announce("adamw rounding")
    n = 1 << 20
    g = randn(3, n, dtype=F32)
    opt = AdamW([torch.zeros(n, device=DEV)], [g.to(DEV)], state_bits=8, seed=5, betas=(0.9, 0.999))
    opt.step()
    r = _bits(5, 0, 1, n)
    off = _check_codes(0.1 * g.double(), opt.m, opt.m_scale, 0, r & 0xffff, False)
    assert abs(off.mean().item()) < 6 * 0.5 / n ** 0.5
    x = (0.001 * g.double() ** 2).sqrt()
    off = _check_codes(x, opt.v, opt.v_scale, 0, r >> 16, True)
    inside = x > 1e-4 * x.max()       # away from the last code, where the root is kept above zero
    assert abs(off[inside].mean().item()) < 6 * 0.5 / inside.sum().item() ** 0.5


def test_adamw_many_tensors_and_an_empty_one():
    announce("adamw many tensors")
    sizes = [0] + [1 + (i * 37) % 500 for i in range(700)]
    ps = [torch.ones(n, device=DEV) for n in sizes]
    gs = [torch.full((n,), 2.0, device=DEV) for n in sizes]
    opt = AdamW(ps, gs, lr=0.25, eps=1e-12)
    opt.step()
    # first step: m / (1 - b1) = g, root of v / (1 - b2) = |g|: a step of lr
    for p in ps:
        if p.numel():
            assert (p - 0.75).abs().max().item() < 1e-6


# ------------------------------------------------------------------------------
# the whole layer
# ------------------------------------------------------------------------------

def _make(T, H, I, E, k, El=None, start=0, grad_dtype=BF, seed=11):
    x, logits, w13, w2 = inputs.small_case(seed, T, H, I, E, k, El=El)
    w13, w2 = (w13.float() * 4).to(BF), (w2.float() * 4).to(BF)
    layer = MoELayer(hidden=H, intermediate=I, num_experts=E, top_k=k, max_tokens=T, num_local_experts=El,
                     expert_start=start, train=True, grad_dtype=grad_dtype, device=DEV)
    layer.set_weights(w13.to(DEV), w2.to(DEV))
    return layer, x, logits, w13, w2


def _formula(x, logits, w13, w2, k, start):
    """The layer in 64 bits with autograd: (out, leaves)."""
    leaves = [t.double().requires_grad_() for t in (x, logits, w13, w2)]
    x, logits, w13, w2 = leaves
    El, I = w13.shape[0], w2.shape[2]
    top, ids = torch.topk(logits, k, dim=1)
    w = torch.softmax(top, 1)
    out = torch.zeros_like(x)
    for e in range(El):
        t, j = torch.nonzero(ids == e + start, as_tuple=True)
        if len(t):
            h = x[t] @ w13[e].t()
            a = torch.nn.functional.silu(h[:, :I]) * h[:, I:]
            out = out.index_add(0, t, w[t, j][:, None] * (a @ w2[e].t()))
    return out, leaves


LAYERS = [(64, 256, 512, 8, 2, None, 0), (1, 128, 128, 4, 2, None, 0), (200, 256, 384, 16, 4, 4, 8), (37, 384, 128, 6, 6, None, 0)]


@pytest.mark.parametrize("T,H,I,E,k,El,start", LAYERS)
def test_layer_gradients(T, H, I, E, k, El, start):
    announce("layer", T, H, I, E, k, El, start)
    layer, x, logits, w13, w2 = _make(T, H, I, E, k, El, start)
    dout = randn(21, T, H, scale=0.5)
    out = layer(x.to(DEV), logits.to(DEV))
    dx, dl = layer.backward(dout.to(DEV))
    ref, leaves = _formula(x, logits, w13, w2, k, start)
    ref.backward(dout.double())
    # at most eight values rounded to bf16 (each 2^-8 at most) lie on the way of any output
    for got, want in [(out, ref.detach())] + list(zip((dx, dl, layer.dw13, layer.dw2), (t.grad for t in leaves))):
        err = (got.cpu().double() - want).norm() / want.norm().clamp(min=1e-30)
        assert err < 8 * U16, err
    # against differences: along a random direction of each leaf the function's
    # change is what the gradient says (central differences, third-order error)
    for i, got in enumerate((dx, dl, layer.dw13, layer.dw2)):
        d = torch.randn(got.shape, generator=gen(31 + i), dtype=torch.float64)
        d = d + got.cpu().double() / got.cpu().double().abs().mean().clamp(min=1e-30)   # not orthogonal to it
        h = 1e-4 / d.abs().max()
        f = []
        for s in (1, -1):
            args = [x, logits, w13, w2]
            args[i] = args[i].double() + s * h * d
            f.append((_formula(*args, k, start)[0].detach() * dout.double()).sum())
        diff = ((f[0] - f[1]) / (2 * h)).item()
        assert abs((got.cpu().double() * d).sum().item() - diff) <= 8 * U16 * got.cpu().double().norm().item() * d.norm().item()


def test_layer_backward_once_and_accumulates():
    announce("layer accumulate")
    layer, x, logits, _, _ = _make(48, 256, 128, 8, 2, grad_dtype=F32)
    xd, ld = x.to(DEV), logits.to(DEV)
    dout = randn(5, 48, 256).to(DEV)
    layer(xd, ld)
    layer.backward(dout)
    one13, one2 = layer.dw13.clone(), layer.dw2.clone()
    with pytest.raises(ValueError):
        layer.backward(dout)
    layer(xd, ld)
    layer.backward(dout, accumulate=True)
    assert torch.equal(layer.dw13, one13 + one13) and torch.equal(layer.dw2, one2 + one2)
    layer(xd[:5], ld[:5])                               # a smaller batch after a larger one
    dx, dl = layer.backward(dout[:5])
    assert dx.shape == (5, 256) and dl.shape == (5, 8)
    live = torch.zeros(8, dtype=torch.bool)
    live[torch.topk(logits[:5], 2, 1)[1].reshape(-1)] = True
    assert (layer.dw2[~live.to(DEV)] == 0).all() and torch.isfinite(layer.dw2).all()


def test_layer_backward_of_given_routing_returns_weight_gradients():
    announce("layer given ids")
    layer, x, logits, _, _ = _make(33, 256, 128, 8, 2)
    top, ids = torch.topk(logits, 2, 1)
    w = torch.softmax(top, 1)
    dout = randn(5, 33, 256).to(DEV)
    layer(x.to(DEV), logits.to(DEV))
    dx, dl = (t.clone() for t in layer.backward(dout))
    layer(x.to(DEV), topk_ids=ids.int().to(DEV), topk_weights=w.to(DEV))
    dx2, dw = layer.backward(dout)
    assert dw.shape == (33, 2)
    out = torch.empty_like(dl)
    L.moe_route_topk_bwd(ids.int().to(DEV), w.to(DEV), dw, out)
    # the two softmaxes may differ by a few fp32 roundings
    assert (dx2.float() - dx.float()).abs().max() <= 2 * U16 * dx.float().abs().max()
    assert (out - dl).abs().max() <= 1e-4 * dl.abs().max()


@pytest.mark.parametrize("bits", [32, 8])
def test_captured_training_steps_match_eager_ones(bits):
    """Forward, backward and optimizer step as one captured graph, replayed with
    other work between, against the same steps run eagerly."""
    announce("captured step", bits)
    batches = [(randn(40 + i, 48, 256).to(DEV), torch.randn(48, 8, generator=gen(60 + i)).to(DEV)) for i in range(4)]
    dout = randn(5, 48, 256).to(DEV)

    def start():
        layer, _, _, _, _ = _make(48, 256, 128, 8, 2)
        return layer, layer.optimizer(lr=1e-2, weight_decay=0.1, state_bits=bits, seed=3)

    layer, opt = start()
    want = []
    for x, lg in batches:
        layer(x, lg)
        dx, dl = layer.backward(dout)
        opt.step()
        want.append([t.clone() for t in (dx, dl, layer.w13, layer.w2, opt.m, opt.v)])
    layer, opt = start()
    sx, sl = batches[0][0].clone(), batches[0][1].clone()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    layer.allocate_grads() if layer.dw13 is None else None
    with torch.cuda.graph(g, stream=side):
        layer(sx, sl)
        dx, dl = layer.backward(dout)
        opt.step()
    for (x, lg), ref in zip(batches, want):
        sx.copy_(x)
        sl.copy_(lg)
        g.replay()
        torch.randn(1000, device=DEV).sum()
        torch.cuda.synchronize()
        for a, b in zip((dx, dl, layer.w13, layer.w2, opt.m, opt.v), ref):
            assert same_bits(a, b)
    assert opt.steps.item() == len(batches)


def test_gradients_on_another_stream():
    announce("another stream")
    layer, x, logits, _, _ = _make(64, 256, 128, 8, 2)
    xd, ld, dout = x.to(DEV), logits.to(DEV), randn(5, 64, 256).to(DEV)
    layer(xd, ld)
    want = [t.clone() for t in layer.backward(dout)] + [layer.dw13.clone(), layer.dw2.clone()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        layer(xd, ld)
        got = layer.backward(dout)
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(list(got) + [layer.dw13, layer.dw2], want):
        assert same_bits(a, b)


def test_training_learns_a_copy():
    """Two layers, one imitating the other: a run of all operators together, for
    running (no bound on how far the error falls)."""
    announce("training run")
    T, H, I, E, k = 96, 256, 128, 8, 2
    teacher, x, logits, _, _ = _make(T, H, I, E, k, seed=1)
    pupil, _, _, _, _ = _make(T, H, I, E, k, seed=2)
    opt = pupil.optimizer(lr=3e-3, state_bits=8)
    xd, ld = x.to(DEV), logits.to(DEV)
    target = teacher(xd, ld).clone()
    for _ in range(5):
        out = pupil(xd, ld)
        pupil.backward((2 * (out.float() - target.float()) / H).to(BF))
        opt.step()
    assert all(torch.isfinite(t.float()).all() for t in (pupil.w13, pupil.w2, out))
