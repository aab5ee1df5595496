"""The products with bias, activation and residual in their epilogue, dense and grouped,
and the epilogue's gradient, against plain 64-bit forms at sizes and masks where they can
go wrong."""
import numpy as np
import pytest
import torch

from scatter_grouped_gemm_amd import _lib as L
from epilogue_util import ALPHA, GATED, HALF, LIMIT, PLAIN, act_bound, activation, check, half, product_bound
from gpu_util import DEV, announce, compact_layout, i32_dev

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
GUARD = 768.0      # an output element that no call may write keeps this


def rand(seed, *shape, scale=1.0, dtype=BF):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def linear_case(T, K, N, act, bias, residual, out, pre, pad, seed=0):
    """Inputs of one call, with rows a stride apart if pad."""
    wide = N // 2 if act in GATED else N
    x = rand(seed, T, K + pad)[:, :K]
    w = rand(seed + 1, N, K, scale=1.5 * K ** -0.5)
    b = None if bias is None else rand(seed + 2, N, dtype=bias)
    r = rand(seed + 3, T, wide + pad, dtype=out)[:, :wide] if residual else None
    o = torch.full((T + 1, wide + pad), GUARD, dtype=out, device=DEV)
    p = torch.full((T + 1, N), GUARD, dtype=BF, device=DEV) if pre else None
    return x, w, b, r, o, p


def run_linear(T, K, N, act="none", bias=None, residual=False, out=BF, pre=False, pad=0, seed=0):
    announce("linear", T, K, N, act, bias, residual, out, pre, pad)
    x, w, b, r, o, p = linear_case(T, K, N, act, bias, residual, out, pre, pad, seed)
    wide = N // 2 if act in GATED else N
    L.moe_linear(x, w, o[:T, :wide], bias=b, act=act, residual=r, pre=None if p is None else p[:T], alpha=ALPHA, limit=LIMIT)
    torch.cuda.synchronize()
    xd, wd, bd = x.double(), w.double(), None if b is None else b.double()
    want = xd @ wd.t() + (0 if b is None else bd)
    dp = product_bound(xd, wd, bd)
    y, e = activation(want, act), act_bound(want, dp, act, out)
    if r is not None:
        y = y + r.double()
        e = e + (HALF[out] + 2.0 ** -23) * (r.double().abs() + e)
    check(o[:T, :wide], y, e, "out")
    assert (o[T:] == GUARD).all() and (o[:, wide:] == GUARD).all()
    if p is not None:
        check(p[:T], want, dp + HALF[BF] * (want.abs() + dp), "pre")
        assert (p[T:] == GUARD).all()
    return o[:T, :wide].clone()


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 33, 64, 65, 127, 129, 300])
@pytest.mark.parametrize("K,N", [(8, 1), (24, 6), (64, 64), (72, 130), (136, 250), (1000, 256), (2056, 66)])
def test_linear_sizes(T, K, N):
    run_linear(T, K, N, out=F32, bias=F32, seed=T + K)


@pytest.mark.parametrize("act", PLAIN + GATED)
@pytest.mark.parametrize("bias,residual,out,pre,pad", [
    (None, False, BF, False, 0), (BF, True, BF, True, 8), (F32, True, F32, False, 0), (BF, False, F32, True, 24),
    (F32, False, BF, True, 0), (None, True, BF, True, 0)])
def test_linear_epilogues(act, bias, residual, out, pre, pad):
    for T, K, N in [(5, 128, 256), (70, 256, 128), (200, 384, 514), (517, 320, 1024)]:
        run_linear(T, K, N, act, bias, residual, out, pre, pad, seed=N)


@pytest.mark.parametrize("T,K,N,act,residual,pre", [
    (1, 7168, 4096, "silu_mul", False, False), (3, 2048, 7168, "none", True, False), (40, 4096, 4096, "gelu", False, True),
    (513, 1024, 4096, "swiglu_clamp", False, True), (1100, 2048, 2048, "none", True, False), (2050, 640, 4608, "gelu_tanh_mul", False, True),
    (4099, 1536, 2304, "relu2", True, True), (3000, 192, 5120, "silu_mul", True, False)])
def test_linear_large(T, K, N, act, residual, pre):
    run_linear(T, K, N, act, BF, residual, BF, pre, seed=T)


@pytest.mark.parametrize("T,K,N,act,residual,pre,pad", [
    (4100, 1032, 4104, "none", False, False, 0), (4099, 200, 4520, "gelu", True, False, 8), (2050, 328, 10016, "silu_mul", False, True, 0),
    (2309, 1096, 6416, "swiglu_clamp", False, False, 200), (3001, 72, 5192, "relu2", False, True, 0), (6000, 136, 2056, "none", True, False, 0),
    (2560, 704, 4168, "none", True, False, 0), (2600, 1000, 8208, "gelu_tanh_mul", False, True, 0)])
def test_linear_large_and_odd(T, K, N, act, residual, pre, pad):
    """Large tiles whose last step and last columns are part ones."""
    run_linear(T, K, N, act, BF, residual, BF, pre, pad, seed=T)


@pytest.mark.parametrize("T,K,N,act,pad", [(4100, 256, 4100, "none", 0), (3000, 200, 6152, "gelu", 12), (2600, 328, 8216, "silu_mul", 4),
                                           (2500, 448, 10248, "swiglu_clamp", 0)])
def test_linear_large_fp32(T, K, N, act, pad):
    """fp32 out of the large tiles, columns and rows of groups of four."""
    announce("large fp32", T, K, N, act, pad)
    x, w, b, _, o, _ = linear_case(T, K, N, act, F32, False, F32, False, 0)
    wide = N // 2 if act in GATED else N
    o = torch.full((T + 1, wide + pad), GUARD, device=DEV)
    L.moe_linear(x, w, o[:T, :wide], bias=b, act=act, alpha=ALPHA, limit=LIMIT)
    want = x.double() @ w.double().t() + b.double()
    dp = product_bound(x.double(), w.double(), b.double())
    check(o[:T, :wide], activation(want, act), act_bound(want, dp, act, F32), "out")
    assert (o[T:] == GUARD).all() and (o[:, wide:] == GUARD).all()
    small = torch.empty(40, wide, device=DEV)
    L.moe_linear(x[:40], w, small, bias=b, act=act, alpha=ALPHA, limit=LIMIT)
    assert torch.equal(small, o[:40, :wide])


@pytest.mark.parametrize("K,N", [(1000, 4360), (456, 5000)])
def test_linear_odd_rows_do_not_depend_on_each_other(K, N):
    w, x = rand(1, N, K, scale=K ** -0.5), rand(3, 4000, K)
    for act in ("none", "gelu_mul"):
        wide = N // 2 if act in GATED else N
        whole = torch.empty(4000, wide, dtype=BF, device=DEV)
        L.moe_linear(x, w, whole, act=act)
        for a, n in [(0, 1), (3999, 1), (100, 33), (1000, 130), (2000, 600), (0, 1500)]:
            o = torch.empty(n, wide, dtype=BF, device=DEV)
            L.moe_linear(x[a:a + n], w, o, act=act)
            assert torch.equal(o, whole[a:a + n]), (act, a, n)


def test_linear_rows_with_nan_behind_k():
    """What lies behind a row's K columns, in the gap to the next row, is never part of a sum."""
    for T, K, N in [(3, 72, 64), (200, 72, 256), (4000, 200, 4104), (4000, 712, 4104)]:
        wide = torch.full((T, K + 56), float("nan"), dtype=BF, device=DEV)
        wide[:, :K] = rand(1, T, K)
        w = rand(2, N, K, scale=K ** -0.5)
        o, ref = torch.empty(T, N, dtype=BF, device=DEV), torch.empty(T, N, dtype=BF, device=DEV)
        L.moe_linear(wide[:, :K], w, o)
        L.moe_linear(wide[:, :K].contiguous(), w, ref)
        assert torch.equal(o, ref) and not torch.isnan(o).any(), (T, K, N)


def test_linear_rows_do_not_depend_on_each_other():
    """A row has the same bits whatever the number of rows, so from every kernel that the sizes choose."""
    K, N = 1152, 2560
    w, b = rand(1, N, K, scale=K ** -0.5), rand(2, N)
    x = rand(3, 5000, K)
    for act in ("none", "swiglu_clamp", "gelu_mul"):
        wide = N // 2 if act in GATED else N
        whole = torch.empty(5000, wide, dtype=BF, device=DEV)
        pre = torch.empty(5000, N, dtype=BF, device=DEV)
        L.moe_linear(x, w, whole, bias=b, act=act, pre=pre)
        for a, n in [(0, 1), (77, 1), (4999, 1), (10, 7), (100, 16), (100, 33), (64, 64), (1000, 130), (2000, 600), (0, 1500)]:
            announce("rows", act, a, n)
            o, p = torch.empty(n, wide, dtype=BF, device=DEV), torch.empty(n, N, dtype=BF, device=DEV)
            L.moe_linear(x[a:a + n], w, o, bias=b, act=act, pre=p)
            assert torch.equal(o, whole[a:a + n]) and torch.equal(p, pre[a:a + n]), (act, a, n)
            o32 = torch.empty(n, wide, dtype=F32, device=DEV)
            L.moe_linear(x[a:a + n], w, o32, bias=b, act=act)
            assert torch.equal(o32.to(BF), o), (act, a, n)


def test_linear_in_place_residual_and_empty_batch():
    x, w = rand(1, 100, 256), rand(2, 384, 256, scale=1 / 16)
    for T in (100, 1):
        h = rand(3, T, 384)
        apart = torch.empty_like(h)
        L.moe_linear(x[:T], w, apart, residual=h)
        L.moe_linear(x[:T], w, h, residual=h)
        assert torch.equal(h, apart)
    L.moe_linear(x[:0], w, torch.empty(0, 384, dtype=BF, device=DEV))


def test_linear_not_finite():
    """Infinities and NaN stay in their row; an infinite sum goes through the activations as the formulas say."""
    x, w = rand(1, 40, 128), rand(2, 256, 128)
    ref = torch.empty(40, 256, dtype=BF, device=DEV)
    L.moe_linear(x, w, ref)
    x2 = x.clone()
    x2[3, 5], x2[20, 0] = float("nan"), float("inf")
    for act in PLAIN + GATED:
        wide = 128 if act in GATED else 256
        o, clean = torch.empty(40, wide, dtype=BF, device=DEV), torch.empty(40, wide, dtype=BF, device=DEV)
        L.moe_linear(x, w, clean, act=act)
        L.moe_linear(x2, w, o, act=act)
        keep = torch.ones(40, dtype=torch.bool, device=DEV)
        keep[3] = keep[20] = False
        assert torch.equal(o[keep], clean[keep]), act
        assert torch.isnan(o[3]).all(), act
        if act not in GATED:
            up = w[:, 0] > 0
            assert torch.isposinf(o[20][up]).all(), act
    # far out, where the sigmoid is 0 or 1 and x^3 leaves fp32
    big = torch.tensor([[1e20, -1e20, 3e38, -3e38, 50.0, -50.0, 1e4, -1e4]], dtype=F32, device=DEV)
    eye = torch.eye(8, dtype=BF, device=DEV)
    for act in PLAIN[:-1]:
        o = torch.empty(1, 8, dtype=F32, device=DEV)
        L.moe_linear(big.to(BF), eye, o, act=act)
        v = big.to(BF).double()
        want = v if act == "none" else torch.where(v > 0, v, torch.zeros_like(v))
        assert ((o.double() - want).abs() <= 2.0 ** -20 * want.abs() + 1e-15).all(), (act, o)


def test_linear_captured_and_on_another_stream():
    x, w, b = rand(1, 130, 512), rand(2, 512, 512, scale=1 / 22), rand(3, 512)
    o, p = torch.empty(130, 256, dtype=BF, device=DEV), torch.empty(130, 512, dtype=BF, device=DEV)
    d, dp, db = rand(4, 130, 256), torch.empty(130, 512, dtype=BF, device=DEV), torch.empty(512, dtype=F32, device=DEV)
    ws = torch.empty(L.moe_act_bwd_ws_bytes(130, 512, 1), dtype=torch.uint8, device=DEV)

    def step():
        L.moe_linear(x, w, o, bias=b, act="gelu_mul", pre=p)
        L.moe_act_bwd(p, d, dp, "gelu_mul", dbias=db, ws=ws)
    step()
    torch.cuda.synchronize()
    want = [t.clone() for t in (o, p, dp, db)]
    s = torch.cuda.Stream()
    for t in (o, p, dp, db):
        t.fill_(GUARD)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    assert all(torch.equal(a, t) for a, t in zip(want, (o, p, dp, db)))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(3):
        x.copy_(rand(10 + i, 130, 512))
        for t in (o, p, dp, db):
            t.fill_(GUARD)
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (o, p, dp, db)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, t) for a, t in zip(got, (o, p, dp, db))), i


# --- grouped ---------------------------------------------------------------------------

def quantised(fmt, x, w, masked):
    """(x, x_scale, w, w_scale, values of x, values of w) in a weight format; x [rows, K] or [G, max_m, K]."""
    K, (G, N, _) = x.shape[-1], w.shape
    if fmt == "bf16":
        return x, None, w, None, x.double(), w.double()
    flat = x.reshape(-1, K)
    q = torch.empty(flat.shape, dtype=torch.uint8, device=DEV)
    s = torch.empty(K // 128, len(flat), dtype=torch.uint8, device=DEV)
    L.moe_quant_fp8_ue8m0(flat, q, s)
    xv = q.view(torch.float8_e4m3fn).double() * torch.exp2(s.t().double() - 127).repeat_interleave(128, 1)
    if masked:
        s = s.view(K // 128, G, -1).transpose(0, 1).contiguous()
    if fmt == "fp8":
        wq, ws = torch.empty(w.shape, dtype=torch.uint8, device=DEV), torch.empty(G, N // 128, K // 128, dtype=torch.uint8, device=DEV)
        L.moe_quant_weight_fp8_ue8m0(w, wq, ws)
        wv = wq.view(torch.float8_e4m3fn).double() * torch.exp2(ws.double() - 127).repeat_interleave(128, 1).repeat_interleave(128, 2)
    else:
        four = fmt == "mxfp4"
        wq = torch.empty(G, N, K // 2 if four else K, dtype=torch.uint8, device=DEV)
        ws = torch.empty(G, N // 64, K // 128, 256, dtype=torch.uint8, device=DEV)
        L.moe_quant_weight_mx(w, "e2m1" if four else "e4m3", wq, ws)
        scale = torch.exp2(ws.view(G, N // 64, K // 128, 4, 16, 4).permute(0, 1, 5, 4, 2, 3).reshape(G, N, K // 32).double() - 127)
        if four:
            table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], dtype=torch.float64, device=DEV)
            v = table[torch.stack([wq & 15, wq >> 4], -1).long()].view(G, N, K)
        else:
            v = wq.view(torch.float8_e4m3fn).double()
        wv = (v.view(G, N, K // 32, 32) * scale[..., None]).view(G, N, K)
    return q.view(x.shape), s, wq, ws, xv.view(x.shape), wv


def e4m3_rows(y):
    """Rows [n, cols] in 64 bits as the values of their e4m3 codes, and the exponents."""
    n, c = y.shape
    top = y.abs().view(n, c // 128, 128).amax(2)
    e = torch.where(top > 0, torch.ceil(torch.log2(top / 448)), torch.full_like(top, -126.0)).clamp(-126, 127)
    return e


def grouped_inputs(counts, K, N, fmt, act, bias, layout, max_m=0, seed=0):
    G = len(counts)
    w = rand(seed + 1, G, N, K, scale=1.5 * K ** -0.5)
    b = None if bias is None else rand(seed + 2, G, N, dtype=bias)
    if layout == "compact":
        m = i32_dev(compact_layout(counts))
        x = rand(seed, len(m), K)
        x[m < 0] = float("nan")      # padding may hold anything
        idx = torch.nonzero(m >= 0).view(-1)
        return x, w, b, m, idx, m[idx].long()
    x = rand(seed, G, max_m, K)
    c = i32_dev(np.array(counts))
    x[torch.arange(max_m, device=DEV)[None] >= c[:, None]] = float("nan")      # so may these
    idx = torch.nonzero((torch.arange(max_m, device=DEV)[None] < c[:, None]).view(-1)).view(-1)
    return x, w, b, c, idx, idx // max_m


def run_grouped(counts, K, N, fmt, act, bias=BF, layout="compact", q8=False, pre=False, max_m=0, expected_m=0, seed=0):
    announce("grouped", list(counts)[:12], K, N, fmt, act, bias, layout, q8, pre, max_m, expected_m)
    masked = layout == "masked"
    x, w, b, info, idx, e = grouped_inputs(counts, K, N, fmt, act, bias, layout, max_m, seed)
    if fmt != "bf16":
        x = torch.nan_to_num(x)
    G, wide = len(counts), N // 2 if act in GATED else N
    xq, xs, wq, ws, xv, wv = quantised(fmt, x, w, masked)
    lead = tuple(x.shape[:-1])
    rows = int(np.prod(lead))
    out = torch.full(lead + (wide,), 0x5A, dtype=torch.uint8, device=DEV) if q8 else torch.full(lead + (wide,), GUARD, dtype=BF, device=DEV)
    os_ = torch.full((wide // 128 * rows,), 0x5A, dtype=torch.uint8, device=DEV) if q8 else None
    p = torch.full(lead + (N,), GUARD, dtype=BF, device=DEV) if pre else None
    wdt = {"bf16": False, "fp8": True}.get(fmt, fmt)
    if masked:
        L.grouped_gemm_masked_act(wdt, xq, xs, wq, ws, out, info, expected_m, bias=b, act=act, out_scale=os_, pre=p, alpha=ALPHA, limit=LIMIT)
    else:
        L.grouped_gemm_contig_act(wdt, xq, xs, wq, ws, out, info, bias=b, act=act, out_scale=os_, pre=p, alpha=ALPHA, limit=LIMIT)
    torch.cuda.synchronize()
    flat = out.view(rows, wide)
    free = torch.ones(rows, dtype=torch.bool, device=DEV)
    free[idx] = False
    assert (flat[free] == (0x5A if q8 else GUARD)).all(), "rows without an assignment were written"
    if pre:
        assert (p.view(rows, N)[free] == GUARD).all()
    xv = xv.view(rows, K)
    for g in range(G):
        r = idx[e == g]
        if not len(r):
            continue
        bd = None if b is None else b[g].double()
        want = xv[r] @ wv[g].t() + (0 if b is None else bd)
        dp = product_bound(xv[r], wv[g], bd)
        if pre:
            check(p.view(rows, N)[r], want, dp + HALF[BF] * (want.abs() + dp), "pre")
        y = activation(want, act)
        if not q8:
            check(flat[r], y, act_bound(want, dp, act, BF), ("out", g))
            continue
        d = act_bound(want, dp, act, F32)
        if masked:
            scale = os_.view(G, wide // 128, max_m)[g].t()[r - g * max_m]
        else:
            scale = os_.view(wide // 128, rows).t()[r]
        top, off = (t.view(len(r), wide // 128, 128).amax(2) for t in (y.abs(), d))
        exp = scale.double() - 127
        # the smallest exponent that holds the maximum, which is known up to off
        assert ((top - off <= 448 * torch.exp2(exp)) & ((top + off > 224 * torch.exp2(exp)) | (exp == -126))).all(), "scale"
        step = torch.exp2(exp).repeat_interleave(128, 1)
        # half a place of a code relative to the value, or of the subnormal codes' 2^-9
        check(flat[r].view(torch.float8_e4m3fn).double() * step, y, d + torch.maximum(2.0 ** -4 * (y.abs() + d), 2.0 ** -10 * step), ("codes", g))
    return out, p, os_


COUNTS = [[0, 1, 128, 17, 0, 300, 129, 64], [256, 0, 0], [1], [0, 0]]


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("act", ["none", "gelu", "relu2", "silu_mul", "swiglu_clamp", "gelu_mul"])
def test_contig(fmt, act):
    for counts in COUNTS:
        for K, N in [(128, 256), (384, 512), (256, 128)]:
            if N % 256 and act in GATED:
                continue
            run_grouped(counts, K, N, fmt, act, bias=BF if K != 384 else F32, pre=fmt == "bf16" and K != 128, seed=K)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("act", ["none", "gelu_tanh", "silu_mul", "swiglu_clamp"])
@pytest.mark.parametrize("expected_m", [0, 8, 32, 64])
def test_masked(fmt, act, expected_m):
    for counts, max_m in [([0, 5, 33, 17, 70, 1], 70), ([200, 0, 16], 200), ([0, 0], 40)]:
        for K, N in [(256, 512), (128, 128)]:
            if N % 256 and act in GATED:
                continue
            run_grouped(counts, K, N, fmt, act, bias=BF if N == 512 else None, layout="masked", pre=fmt == "bf16" and N == 512,
                        max_m=max_m, expected_m=expected_m, seed=K)


@pytest.mark.parametrize("fmt", ["fp8", "mxfp8", "mxfp4", "bf16"])
@pytest.mark.parametrize("layout", ["compact", "masked"])
def test_quantised_output(fmt, layout):
    for act in ("silu_mul", "swiglu_clamp"):
        run_grouped([0, 1, 128, 17, 40], 256, 768, fmt, act, layout=layout, q8=True, max_m=150, expected_m=16 if act == "silu_mul" else 0)


@pytest.mark.parametrize("counts,K,N,act", [
    ([1500, 0, 700, 1025, 3, 256, 257, 512], 512, 3584, "swiglu_clamp"), ([3000, 2100], 1024, 4096, "gelu_mul"),
    ([40] * 64, 640, 1408 * 2, "silu_mul"), ([900, 1, 2000], 1536, 4096, "none"), ([0] * 30 + [600] + [0] * 30, 256, 1280, "relu2")])
def test_contig_large(counts, K, N, act):
    run_grouped(counts, K, N, "bf16", act, pre=True)
    run_grouped(counts, K, N, "bf16", act, bias=None)


def test_grouped_layouts_and_dense_agree():
    """A row has the same bits from the compact and the masked layout and from the dense product."""
    K, N, G = 768, 1536, 3
    counts = [300, 5, 129]
    for act in ("none", "swiglu_clamp", "gelu"):
        wide = N // 2 if act in GATED else N
        x, w, b, m, idx, e = grouped_inputs(counts, K, N, "bf16", act, F32, "compact", seed=5)
        out, pre = torch.empty(len(m), wide, dtype=BF, device=DEV), torch.empty(len(m), N, dtype=BF, device=DEV)
        L.grouped_gemm_contig_act(False, x, None, w, None, out, m, bias=b, act=act, pre=pre)
        xm = torch.zeros(G, 300, K, dtype=BF, device=DEV)
        for g in range(G):
            r = idx[e == g]
            xm[g, :len(r)] = x[r]
            o, p = torch.empty(len(r), wide, dtype=BF, device=DEV), torch.empty(len(r), N, dtype=BF, device=DEV)
            L.moe_linear(x[r], w[g], o, bias=b[g], act=act, pre=p)
            assert torch.equal(o, out[r]) and torch.equal(p, pre[r]), (act, g)
        for em in (0, 16, 32, 64):
            om, pm = torch.empty(G, 300, wide, dtype=BF, device=DEV), torch.empty(G, 300, N, dtype=BF, device=DEV)
            L.grouped_gemm_masked_act(False, xm, None, w, None, om, i32_dev(np.array(counts)), em, bias=b, act=act, pre=pm)
            for g in range(G):
                r = idx[e == g]
                assert torch.equal(om[g, :len(r)], out[r]) and torch.equal(pm[g, :len(r)], pre[r]), (act, em, g)


def test_grouped_without_epilogue_is_the_plain_product():
    x, w, b, m, idx, e = grouped_inputs([130, 0, 260, 7], 512, 768, "bf16", "none", None, "compact", seed=9)
    x = torch.nan_to_num(x)
    a, c = torch.empty(len(m), 768, dtype=BF, device=DEV), torch.empty(len(m), 768, dtype=BF, device=DEV)
    L.grouped_gemm_contig_act(False, x, None, w, None, a, m)
    L.grouped_gemm_contig(False, x, None, w, None, c, m)
    assert torch.equal(a[idx], c[idx])


# --- gradient --------------------------------------------------------------------------

def exact_bwd(p, d, act):
    if act not in GATED:
        return d * half(p, act)[1]
    g, u = p.chunk(2, -1)
    if act == "swiglu_clamp":
        v, s = half(g.clamp(max=LIMIT), act)
        return torch.cat([d * s * (u.clamp(-LIMIT, LIMIT) + 1) * (g <= LIMIT), d * v * (u.abs() <= LIMIT)], -1)
    v, s = half(g, act[:-4])
    return torch.cat([d * s * u, d * v], -1)


def bwd_terms(p, d, act):
    """Magnitudes that exponential, reciprocal and polynomial are off by 2^-20 of: the
    derivative's terms are at most 1 + |x| max(s (1 - s) |z'|) <= 2.2 (1.2 times the
    clamped gate's alpha), and 2 |x| for the squared ReLU."""
    if act == "none":
        return torch.zeros_like(p)
    if act not in GATED:
        return d.abs() * (2 * p.abs() if act == "relu2" else 2.2)
    g, u = p.chunk(2, -1)
    w = u.abs() + 1 if act == "swiglu_clamp" else u.abs()
    return torch.cat([2.2 * 1.2 * d.abs() * w, d.abs() * g.abs()], -1)


@pytest.mark.parametrize("act", PLAIN + GATED)
@pytest.mark.parametrize("layout", ["dense", "compact", "masked"])
@pytest.mark.parametrize("db,acc", [(F32, False), (BF, True), (F32, True), (None, False)])
def test_act_bwd(act, layout, db, acc):
    for counts, N, max_m in [([0, 1, 128, 17, 300, 0, 129], 256, 300), ([5, 33], 2560, 40), ([700], 16, 700), ([64, 0, 65], 1040, 70)]:
        announce("act_bwd", act, layout, db, acc, counts, N)
        counts = counts if layout != "dense" else [sum(counts)]
        G, wide = len(counts), N // 2 if act in GATED else N
        kw = {}
        if layout == "dense":
            rows = counts[0]
            idx, e = torch.arange(rows, device=DEV), torch.zeros(rows, dtype=torch.long, device=DEV)
        elif layout == "compact":
            m = i32_dev(compact_layout(counts))
            rows = len(m)
            idx = torch.nonzero(m >= 0).view(-1)
            e = m[idx].long()
            starts = np.concatenate([[0], np.cumsum([-(-c // 128) * 128 for c in counts])])[:-1]
            kw = dict(m_indices=m, expert_start_loc=i32_dev(starts), num_valid=i32_dev(np.array(counts)))
        else:
            rows = G * max_m
            c = i32_dev(np.array(counts))
            idx = torch.nonzero((torch.arange(max_m, device=DEV)[None] < c[:, None]).view(-1)).view(-1)
            e = idx // max_m
            kw = dict(masked_m=c, max_m=max_m)
        pre, dout = rand(N, rows, N, scale=4.0), rand(N + 1, rows, wide)
        free = torch.ones(rows, dtype=torch.bool, device=DEV)
        free[idx] = False
        pre[free], dout[free] = float("nan"), float("nan")
        if act == "swiglu_clamp" and len(idx):   # on the limits, past them, and just inside
            pre[idx[0], :6] = torch.tensor([7.0, 7.03125, 6.96875, -100.0, 100.0, -7.0], device=DEV)
            pre[idx[0], wide:wide + 6] = torch.tensor([7.0, -7.0, 7.03125, -7.03125, 1.0, -1.0], device=DEV)
        dpre = torch.full((rows, N), GUARD, dtype=BF, device=DEV)
        dbias = None if db is None else rand(7, G, N, dtype=db)
        old = None if db is None else dbias.double()
        L.moe_act_bwd(pre, dout, dpre, act, dbias=dbias, accumulate=acc, alpha=ALPHA, limit=LIMIT, **kw)
        inplace = pre.clone()
        L.moe_act_bwd(inplace, dout, inplace, act, alpha=ALPHA, limit=LIMIT, **{k: v for k, v in kw.items() if k in ("m_indices", "masked_m", "max_m")})
        torch.cuda.synchronize()
        assert (dpre[free] == GUARD).all()
        assert torch.equal(inplace[idx], dpre[idx])
        p, d = pre[idx].double(), dout[idx].double()
        want, t = exact_bwd(p, d, act), 2.0 ** -20 * bwd_terms(p, d, act)
        check(dpre[idx], want, t + HALF[BF] * (want.abs() + t), "dpre")
        if db is None:
            continue
        for g in range(G):
            r = e == g
            n = int(r.sum())
            s, mag = want[r].sum(0), want[r].abs().sum(0)
            bound = t[r].sum(0) + (n + 4) * 2.0 ** -24 * (mag + t[r].sum(0))
            if acc:
                s = s + old[g]
                bound = bound + 2.0 ** -24 * (s.abs() + bound)
            check(dbias[g], s, bound + HALF[db] * (s.abs() + bound), ("dbias", g))


@pytest.mark.parametrize("act", ["none", "gelu", "swiglu_clamp"])
@pytest.mark.parametrize("M,N", [(5, 16), (300, 272), (1500, 1024)])
def test_act_bwd_of_an_fp32_output(act, M, N):
    """dout in fp32, as moe_linear's fp32 output has it; act none rounds it to bf16."""
    announce("fp32 dout", act, M, N)
    wide = N // 2 if act in GATED else N
    pre, dout = rand(1, M, N, scale=3.0), rand(2, M, wide, dtype=F32)
    dpre, db = torch.empty(M, N, dtype=BF, device=DEV), torch.empty(N, dtype=F32, device=DEV)
    L.moe_act_bwd(None if act == "none" else pre, dout, dpre, act, dbias=db, alpha=ALPHA, limit=LIMIT)
    want, t = exact_bwd(pre.double(), dout.double(), act), 2.0 ** -20 * bwd_terms(pre.double(), dout.double(), act)
    check(dpre, want, t + HALF[BF] * (want.abs() + t), "dpre")
    check(db, want.sum(0), t.sum(0) + (M + 4) * 2.0 ** -24 * (want.abs() + t).sum(0) + HALF[F32] * want.sum(0).abs(), "dbias")


def test_bias_gradient_alone():
    d = rand(1, 1000, 264)
    db = torch.empty(264, dtype=F32, device=DEV)
    L.moe_act_bwd(None, d, None, "none", dbias=db)
    s = d.double()
    check(db, s.sum(0), 1004 * 2.0 ** -24 * s.abs().sum(0), "dbias")
    empty = torch.full((264,), 3.0, device=DEV)
    L.moe_act_bwd(None, d[:0], None, "none", dbias=empty, accumulate=True)
    assert (empty == 3.0).all()
    L.moe_act_bwd(None, d[:0], None, "none", dbias=empty)
    assert (empty == 0.0).all()


@pytest.mark.parametrize("act", PLAIN[1:] + GATED)
def test_act_bwd_against_differences(act):
    """The gradient's definition against differences of the forward kernel's outputs (an
    identity weight passes the values through).  Central differences with step 2h are off
    by at most h^2/6 of the third derivative (below 3 here; 0 at kinks, which are kept
    away), the outputs by 2^-20 of their magnitudes over h."""
    n, h = 64, 2.0 ** -5
    wide = n // 2 if act in GATED else n
    p = (rand(3, 50, n, scale=2.0).float() * 16).round() / 16    # p, p + h and p - h are bf16 values: |p| < 8 has steps of 2^-5
    p = p.clamp(-6, 6)
    if act == "relu2":
        p = torch.where(p.abs() < 0.25, torch.full_like(p, 0.25), p)
    eye = torch.eye(n, dtype=BF, device=DEV)
    d = rand(4, 50, wide)
    dp = torch.empty(50, n, dtype=BF, device=DEV)
    L.moe_act_bwd(p.to(BF), d, dp, act, alpha=ALPHA, limit=LIMIT)
    assert torch.equal(p.to(BF).float(), p)
    for part in range(2 if act in GATED else 1):
        vals = []
        for sgn in (1, -1):
            q = p.clone()
            cols = slice(part * wide, (part + 1) * wide) if act in GATED else slice(0, n)
            q[:, cols] += sgn * h
            assert torch.equal(q.to(BF).float(), q)
            o = torch.empty(50, wide, dtype=F32, device=DEV)
            L.moe_linear(q.to(BF), eye, o, act=act, alpha=ALPHA, limit=LIMIT)
            vals.append(o.double())
        up = p[:, wide:].abs() + 1 if act in GATED and part == 0 else torch.ones(50, wide, device=DEV)
        diff = (vals[0] - vals[1]) / (2 * h) * d.double()
        bound = d.double().abs() * up.double() * (h * h / 2 * 3) + d.double().abs() * (vals[0].abs() + vals[1].abs()) * 2.0 ** -20 / h + 1e-6
        check(dp[:, cols], diff, bound + HALF[BF] * (diff.abs() + bound), (act, part))


# --- offsets past 32 bits -----------------------------------------------------------------

def spot_check(x, w, bias, out, pre, act, rows, idx_w=None):
    """Rows of a large product against 64 bits."""
    xd = x[rows].double()
    wd, bd = w.double(), None if bias is None else bias.double()
    want = xd @ wd.t() + (0 if bd is None else bd)
    dp = product_bound(xd, wd, bd)
    check(out[rows], activation(want, act), act_bound(want, dp, act, out.dtype), "out")
    if pre is not None:
        check(pre[rows], want, dp + HALF[BF] * (want.abs() + dp), "pre")


@pytest.mark.parametrize("T,K,N,act,pre", [(70001, 72, 32768, "gelu", True), (70001, 128, 32768, "swiglu_clamp", True),
                                           (70001, 32776, 64, "none", False), (70001, 32768, 24, "silu", False),
                                           (24, 16392, 140000, "relu2", False), (600, 16384, 140032, "none", False)])
def test_linear_past_32_bits(T, K, N, act, pre):
    announce("past 32 bits", T, K, N, act)
    x, w, b = rand(1, T, K), rand(2, N, K, scale=K ** -0.5), rand(3, N)
    wide = N // 2 if act in GATED else N
    o = torch.empty(T, wide, dtype=BF, device=DEV)
    p = torch.empty(T, N, dtype=BF, device=DEV) if pre else None
    L.moe_linear(x, w, o, bias=b, act=act, pre=p, alpha=ALPHA, limit=LIMIT)
    rows = torch.tensor(sorted({0, 1, T // 2, T - 2, T - 1} & set(range(T))), device=DEV)
    spot_check(x, w, b, o, p, act, rows)


def test_grouped_and_gradient_past_32_bits():
    G, K, N = 40, 8192, 8192          # 5.4 GB of weights
    counts = [0] * 10 + [300] + [0] * 20 + [7] + [0] * 7 + [129]
    x, w, b, m, idx, e = grouped_inputs(counts, K, N, "bf16", "silu_mul", BF, "compact")
    out, pre = torch.empty(len(m), N // 2, dtype=BF, device=DEV), torch.empty(len(m), N, dtype=BF, device=DEV)
    L.grouped_gemm_contig_act(False, x, None, w, None, out, m, bias=b, act="silu_mul", pre=pre)
    for g in (10, 31, 39):
        r = idx[e == g]
        spot_check(x, w[g], b[g], out, pre, "silu_mul", r[:: max(1, len(r) // 5)])
    xm = torch.zeros(G, 300, K, dtype=BF, device=DEV)
    om = torch.empty(G, 300, N // 2, dtype=BF, device=DEV)
    for g in (10, 31, 39):
        xm[g, :counts[g]] = x[idx[e == g]]
    L.grouped_gemm_masked_act(False, xm, None, w, None, om, i32_dev(np.array(counts)), 0, bias=b, act="silu_mul")
    for g in (10, 31, 39):
        assert torch.equal(om[g, :counts[g]], out[idx[e == g]]), g
    del x, w, xm, om
    M, N = 70001, 32768
    pre, dout = rand(1, M, N), rand(2, M, N // 2)
    dpre, db = torch.empty_like(pre), torch.empty(N, dtype=F32, device=DEV)
    L.moe_act_bwd(pre, dout, dpre, "silu_mul", dbias=db)
    rows = torch.tensor([0, M // 2, M - 1], device=DEV)
    p, d = pre[rows].double(), dout[rows].double()
    want, t = exact_bwd(p, d, "silu_mul"), 2.0 ** -20 * bwd_terms(p, d, "silu_mul")
    check(dpre[rows], want, t + HALF[BF] * (want.abs() + t), "dpre")
    total = torch.zeros(N, dtype=torch.float64, device=DEV)
    mag = torch.zeros(N, dtype=torch.float64, device=DEV)
    for a in range(0, M, 4096):
        g = exact_bwd(pre[a:a + 4096].double(), dout[a:a + 4096].double(), "silu_mul")
        total += g.sum(0)
        mag += g.abs().sum(0) + bwd_terms(pre[a:a + 4096].double(), dout[a:a + 4096].double(), "silu_mul").sum(0) * 2.0 ** -20 * 2.0 ** 24 / M
    # a sum of M terms in blocks of at most 128 rows and 16 stretches of them: no chain of
    # additions is longer than 128 + 16 + M / 16 / 16, far below M
    check(db, total, (M + 4) * 2.0 ** -24 * mag, "dbias")
