"""Products and gradients of sizes that reach each kernel of the few-rows product and of the
bias gradient's sums, against 64 bits and against larger calls."""
import numpy as np
import pytest
import torch

from scatter_grouped_gemm_amd import _lib as L
from epilogue_util import ALPHA, GATED, HALF, LIMIT, act_bound, activation, check, half, product_bound
from gpu_util import DEV, announce, compact_layout, i32_dev

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
GUARD = 768.0


def rand(seed, *shape, scale=1.0, dtype=BF):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


# (K, N): twice the columns a wavefront from N 8192 on, whole groups and odd ones, up to the
# last N; and one below it
@pytest.mark.parametrize("K,N", [(8, 8200), (72, 12290), (200, 16384), (456, 8194), (136, 8192), (1000, 4102)])
@pytest.mark.parametrize("act,pre,residual,out", [("none", False, False, F32), ("gelu", True, True, BF), ("silu_mul", True, False, BF),
                                                  ("swiglu_clamp", False, True, F32), ("gelu_mul", True, True, BF)])
def test_few_rows_and_many_columns(K, N, act, pre, residual, out):
    wide, most = N // 2 if act in GATED else N, 70
    w, b = rand(2, N, K, scale=1.5 * K ** -0.5), rand(3, N, dtype=F32)
    x, r = rand(1, most, K), rand(4, most, wide, dtype=out) if residual else None
    ref, ref_p = torch.empty(most, wide, dtype=out, device=DEV), torch.empty(most, N, dtype=BF, device=DEV)
    L.moe_linear(x, w, ref, bias=b, act=act, residual=r, pre=ref_p if pre else None, alpha=ALPHA, limit=LIMIT)
    want = x.double() @ w.double().t() + b.double()
    dp = product_bound(x.double(), w.double(), b.double())
    y, bound = activation(want, act), act_bound(want, dp, act, F32 if residual else out)
    if residual:        # added in fp32 before the one rounding
        y = y + r.double()
        bound = bound + 2.0 ** -24 * y.abs() + HALF[out] * (y.abs() + bound)
    for T in (1, 8, 9, 16, 17, 32):
        announce("few rows", T, K, N, act, pre, residual, out)
        o = torch.full((T + 1, wide), GUARD, dtype=out, device=DEV)
        p = torch.full((T + 1, N), GUARD, dtype=BF, device=DEV)
        L.moe_linear(x[:T], w, o[:T], bias=b, act=act, residual=None if r is None else r[:T], pre=p[:T] if pre else None, alpha=ALPHA, limit=LIMIT)
        torch.cuda.synchronize()
        assert (o[T] == GUARD).all() and (p[T] == GUARD).all()
        assert torch.equal(o[:T], ref[:T])
        check(o[:T], y[:T], bound[:T], "out")
        if pre:
            assert torch.equal(p[:T], ref_p[:T])
            check(p[:T], want[:T], dp[:T] + HALF[BF] * (want[:T].abs() + dp[:T]), "pre")


# sums of many columns and experts: 64 of them a workgroup from N G 65536 on
@pytest.mark.parametrize("layout,counts,N", [
    ("dense", [1500], 65552), ("dense", [130], 131088), ("compact", [300, 0, 129, 700, 1, 64, 0, 20], 8208),
    ("compact", [200, 1, 0, 65] * 16, 1040), ("masked", [40, 0, 137, 1, 64, 137, 9, 100] * 2, 4112),
])
@pytest.mark.parametrize("act,db,acc", [("gelu", F32, False), ("swiglu_clamp", BF, True), ("none", F32, True)])
def test_bias_gradients_of_many_columns(layout, counts, N, act, db, acc):
    announce("bias gradient", layout, counts, N, act, db, acc)
    G, kw = len(counts), {}
    wide = N // 2 if act in GATED else N
    assert N * G > 65536
    if layout == "masked":
        max_m = max(counts)
        rows, first = G * max_m, [g * max_m for g in range(G)]
        kw = dict(masked_m=i32_dev(np.array(counts)), max_m=max_m)
    elif layout == "compact":
        m = compact_layout(counts)
        rows, first = len(m), np.concatenate([[0], np.cumsum([-(-c // 128) * 128 for c in counts])])[:-1].tolist()
        kw = dict(m_indices=i32_dev(m), expert_start_loc=i32_dev(np.array(first)), num_valid=i32_dev(np.array(counts)))
    else:
        rows, first = counts[0], [0]
    assert rows > 1024 or rows > 128 * G          # sums in a launch of their own
    pre, dout = rand(1, rows, N, scale=3.0), rand(2, rows, wide)
    free = torch.ones(rows, dtype=torch.bool, device=DEV)
    for g in range(G):
        free[first[g]:first[g] + counts[g]] = False
    pre[free], dout[free] = float("nan"), float("nan")
    dpre, dbias = torch.full((rows, N), GUARD, dtype=BF, device=DEV), rand(3, G, N, dtype=db)
    old = dbias.double()
    L.moe_act_bwd(None if act == "none" else pre, dout, dpre, act, dbias=dbias, accumulate=acc, alpha=ALPHA, limit=LIMIT, **kw)
    torch.cuda.synchronize()
    assert (dpre[free] == GUARD).all()
    for g in range(G):
        at = slice(first[g], first[g] + counts[g])
        p, d = pre[at].double(), dout[at].double()
        if act == "swiglu_clamp":
            q, u = p.chunk(2, 1)
            v, s = half(q.clamp(max=LIMIT), act)
            want = torch.cat([d * (u.clamp(-LIMIT, LIMIT) + 1) * s * (q <= LIMIT), d * v * (u.abs() <= LIMIT)], 1)
            t = torch.cat([2.64 * d.abs() * (u.abs() + 1), d.abs() * q.abs()], 1)
        else:
            want = d * half(p, act)[1]
            t = torch.zeros_like(d) if act == "none" else 2.2 * d.abs()
        t = 2.0 ** -20 * t
        check(dpre[at], want, t + HALF[BF] * (want.abs() + t), ("dpre", g))
        total = want.sum(0)
        bound = t.sum(0) + (counts[g] + 4) * 2.0 ** -24 * (want.abs() + t).sum(0)
        if acc:
            total = total + old[g]
            bound = bound + 2.0 ** -24 * (total.abs() + bound)
        check(dbias[g], total, bound + HALF[db] * (total.abs() + bound), ("dbias", g))


@pytest.mark.parametrize("fmt", ["fp8", "mxfp8", "mxfp4"])
@pytest.mark.parametrize("layout", ["compact", "masked"])
@pytest.mark.parametrize("act,q8", [("none", False), ("swiglu_clamp", False), ("silu_mul", True)])
def test_quantised_rows_without_an_assignment_hold_anything(fmt, layout, act, q8):
    """NaN codes and NaN scales in rows that hold no assignment: the others' outputs keep their bits."""
    announce("padding", fmt, layout, act, q8)
    counts, K, N = [0, 1, 128, 17, 200], 384, 512
    G, wide, max_m = len(counts), N // 2 if act in GATED else N, 205
    if layout == "compact":
        m = compact_layout(counts)
        rows, valid = len(m), torch.from_numpy(m).to(DEV) >= 0
    else:
        rows = G * max_m
        valid = (torch.arange(max_m, device=DEV)[None] < i32_dev(np.array(counts))[:, None]).view(-1)
    x, w, b = rand(1, rows, K), rand(2, G, N, K, scale=1.5 * K ** -0.5), rand(3, G, N)
    q, s = torch.empty(rows, K, dtype=torch.uint8, device=DEV), torch.empty(K // 128, rows, dtype=torch.uint8, device=DEV)
    L.moe_quant_fp8_ue8m0(x, q, s)
    if fmt == "fp8":
        wq, ws = torch.empty(w.shape, dtype=torch.uint8, device=DEV), torch.empty(G, N // 128, K // 128, dtype=torch.uint8, device=DEV)
        L.moe_quant_weight_fp8_ue8m0(w, wq, ws)
    else:
        wq = torch.empty(G, N, K // (2 if fmt == "mxfp4" else 1), dtype=torch.uint8, device=DEV)
        ws = torch.empty(G, N // 64, K // 128, 256, dtype=torch.uint8, device=DEV)
        L.moe_quant_weight_mx(w, "e2m1" if fmt == "mxfp4" else "e4m3", wq, ws)
    found = []
    for spoilt in (False, True):
        if spoilt:
            q[~valid], s[:, ~valid] = 0x7F, 0xFF
        out = torch.full((rows, wide), 0x5A, dtype=torch.uint8, device=DEV) if q8 else torch.full((rows, wide), GUARD, dtype=BF, device=DEV)
        os_ = torch.full((wide // 128 * rows,), 0x5A, dtype=torch.uint8, device=DEV) if q8 else None
        kw = dict(bias=b, act=act, out_scale=os_, alpha=ALPHA, limit=LIMIT)
        if layout == "compact":
            L.grouped_gemm_contig_act(fmt if fmt != "fp8" else True, q, s, wq, ws, out, i32_dev(m), **kw)
        else:
            L.grouped_gemm_masked_act(fmt if fmt != "fp8" else True, q.view(G, max_m, K), s.view(K // 128, G, max_m).transpose(0, 1).contiguous(),
                                      wq, ws, out.view(G, max_m, wide), i32_dev(np.array(counts)), 0, **kw)
        torch.cuda.synchronize()
        assert (out[~valid] == (0x5A if q8 else GUARD)).all()
        found.append((out, os_))
    assert torch.equal(found[0][0], found[1][0]) and (not q8 or torch.equal(found[0][1], found[1][1]))
    assert q8 or not torch.isnan(found[0][0].float()).any()
