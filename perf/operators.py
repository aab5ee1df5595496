"""The training operators of the expert path: cases, plain forms and 64-bit values.

The gradients of the weighted combine (down to the router's logits), of the
scatter, of SiLU-and-mul and of the grouped products, and the AdamW step.  Each
case is one operator at one size; ``run`` computes it in plain torch operations
(``own`` false) or through the library (``own`` true) on the same state.

Layouts are those of include/moe.h: ``src2dst`` [T][k] holds the row of each
assignment (-1 where its expert is not held), the compact layout pads every
expert to 128 rows tagged -1 in ``m_indices``, the masked one gives each expert
``max_m`` rows.  Rows that hold no assignment keep what the output buffer held
(zeros here).
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128       # rows an expert is padded to in the compact layout
GROUP = 128       # elements that share a scale in the 8-bit optimizer states
BETA1, BETA2, EPS, DECAY, LR, SEED = 0.9, 0.95, 1e-8, 0.1, 3e-4, 1234
STEPS = 100       # optimizer steps taken before the one that is run


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one step of the tiny model: the call itself is what costs
        dict(name="combine_bwd_tiny", op="combine_bwd", T=64, H=256, E=8, El=8, k=2, skew=False, layout="compact"),
        # a full prefill-sized batch over 256 experts
        dict(name="combine_bwd_prefill", op="combine_bwd", T=8192, H=7168, E=256, El=256, k=8, skew=False, layout="compact"),
        # one share of 32 experts out of 256, an odd batch in the masked layout: most slots live elsewhere
        dict(name="scatter_bwd_share_masked", op="scatter_bwd", T=1021, H=7168, E=256, El=32, k=8, skew=False, layout="masked"),
        # long batch, popular and dead experts
        dict(name="scatter_bwd_skewed", op="scatter_bwd", T=16384, H=4096, E=128, El=128, k=8, skew=True, layout="compact"),
        # a few tokens, mostly padding rows
        dict(name="silu_bwd_tiny", op="silu_bwd", T=33, I=512, E=8, El=8, k=2, skew=False, layout="compact"),
        # the wide activations of eight large experts
        dict(name="silu_bwd_wide", op="silu_bwd", T=4096, I=14336, E=8, El=8, k=2, skew=False, layout="compact"),
        # many small experts with ragged rows: gradient of w13's input
        dict(name="dgrad_ragged", op="dgrad", T=777, N=2816, K=2048, E=64, El=64, k=6, skew=True),
        # eight large experts, gradient of w13's input
        dict(name="dgrad_large", op="dgrad", T=4096, N=28672, K=4096, E=8, El=8, k=2, skew=False),
        # w2's gradient added to an fp32 buffer over micro-batches; some experts see no token
        dict(name="wgrad_accumulate", op="wgrad", T=8192, N=2048, K=1408, E=64, El=64, k=6, skew=True, out="fp32", accumulate=True),
        # eight large experts, w13's gradient in bf16
        dict(name="wgrad_large", op="wgrad", T=4096, N=28672, K=4096, E=8, El=8, k=2, skew=False, out="bf16", accumulate=False),
        # a router and a few small fp32 tensors
        dict(name="adamw_small", op="adamw", count=5, mean=40000, bits=32, param="fp32", grad="fp32"),
        # both matrices of 64 experts, each a tensor of its own, states in 8 bits
        dict(name="adamw_experts_8bit", op="adamw", count=128, mean=4325376, bits=8, param="bf16", grad="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of lo .. hi."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["combine_bwd", "scatter_bwd", "silu_bwd", "dgrad", "wgrad", "adamw"])
    if op == "adamw":
        count = _log(rng, 1, 200)
        return dict(op=op, count=count, mean=_log(rng, 30, min(30000000, 280000000 // count)), bits=rng.choice([8, 32]),
                    param=rng.choice(["bf16", "fp32"]), grad=rng.choice(["bf16", "fp32"]))
    E = rng.choice([4, 8, 16, 60, 64, 128, 256])
    k = rng.choice([1, 2, 4, 6, 8])
    k = min(k, E)
    El = rng.choice([E, E, max(1, E // 8)])
    skew = rng.random() < 0.4
    if op in ("dgrad", "wgrad"):
        N, K = 128 * _log(rng, 1, 64), 128 * _log(rng, 1, 40)
        El = min(El, max(1, 600000000 // (N * K)))
        E = max(El, k) if El < E and rng.random() < 0.5 else E
        T = _log(rng, 1, max(2, min(16384, 700000000000 // (N * K * k))))
        case = dict(op=op, T=T, N=N, K=K, E=E, El=El, k=k, skew=skew)
        if op == "wgrad":
            case.update(out=rng.choice(["bf16", "fp32"]), accumulate=rng.random() < 0.5)
        return case
    T = _log(rng, 1, 12288)
    layout = "masked" if El * T <= 32768 and rng.random() < 0.4 else "compact"
    if op == "silu_bwd":
        I = 128 * _log(rng, 1, min(112, max(1, 900000 // (T * k))))
        return dict(op=op, T=T, I=I, E=E, El=El, k=k, skew=skew, layout=layout)
    H = 128 * _log(rng, 1, 64) if rng.random() < 0.8 else 8 * _log(rng, 1, 900)
    return dict(op=op, T=T, H=H, E=E, El=El, k=k, skew=skew, layout=layout)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _routing(case, g):
    """Router output and the expert layout of it, as the forward leaves them."""
    T, E, El, k = case["T"], case["E"], case["El"], case["k"]
    logits = torch.randn(T, E, generator=g, device="cuda")
    if case["skew"]:  # Zipf-like popularity, and experts that no token takes
        rank = torch.randperm(E, generator=g, device="cuda") + 1
        dead = min(E // 8, E - k)
        logits = logits - 1.2 * torch.log(rank.float()) - 1e4 * (rank > E - dead)
    top, ids = torch.sort(logits, dim=1, descending=True, stable=True)
    ids, weights = ids[:, :k].contiguous(), torch.softmax(top[:, :k], dim=1)
    flat = ids.reshape(-1)
    local = flat < El
    counts = torch.bincount(flat[local], minlength=El)
    order = torch.sort(torch.where(local, flat, El), stable=True)[1][: int(counts.sum())]
    first = torch.cumsum(counts, 0) - counts
    within = torch.arange(len(order), device="cuda") - first[flat[order]]
    A = T * k
    if case.get("layout") == "masked":
        rows, starts = El * T, torch.arange(El, device="cuda") * T
    else:
        rows = BLOCK * (min(A, El) + (A - min(A, El)) // BLOCK)
        padded = (counts + BLOCK - 1) // BLOCK * BLOCK
        starts = torch.cumsum(padded, 0) - padded
    src2dst = torch.full((A,), -1, device="cuda")
    src2dst[order] = starts[flat[order]] + within
    m_indices = torch.full((rows,), -1, device="cuda")
    m_indices[src2dst[order]] = flat[order]
    i32 = lambda t: t.to(torch.int32).contiguous()  # noqa: E731
    return dict(ids=i32(ids), weights=weights.contiguous(), rows=rows, src2dst=i32(src2dst.view(T, k)), m_indices=i32(m_indices),
                starts=i32(starts), counts=i32(counts), runs=list(zip(starts.tolist(), counts.tolist())), logits=logits)


def _sizes(case):
    """Elements of each tensor: between 0.4 and 1.6 of the mean, odd ones among them."""
    return [max(1, int(case["mean"] * (0.4 + 1.2 * ((i * 5 + 3) % 8) / 7)) - i % 3) for i in range(case["count"])]


def _spans(case):
    """(start, size) of each tensor in the flat buffers: tensors begin at whole groups."""
    at, spans = 0, []
    for n in _sizes(case):
        spans.append((at, n))
        at += (n + GROUP - 1) // GROUP * GROUP
    return spans, at


def _exponent(amax):
    """The smallest e in [-126, 127] with amax <= 448 * 2^e."""
    frac, e = torch.frexp(amax)  # amax = frac * 2^e, frac in [0.5, 1); 448 = 0.875 * 2^9
    e = e - 9 + (frac > 0.875).to(e.dtype)
    return torch.where(amax > 0, e, -126).clamp(-126, 127)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case=case)
    if op == "adamw":
        spans, total = _spans(case)
        bf16 = case["param"] == "bf16"
        master = _randn(g, total, scale=0.02, dtype=torch.float32)
        grad = _randn(g, total, scale=1e-3, dtype=torch.bfloat16 if case["grad"] == "bf16" else torch.float32)
        m = _randn(g, total, scale=3e-4, dtype=torch.float32)
        v = _randn(g, total, scale=1e-3, dtype=torch.float32).square_()
        hole = torch.ones(total, dtype=torch.bool, device="cuda")
        for a, n in spans:
            hole[a:a + n] = False
        for t in (master, grad, m, v):  # nothing between the tensors
            t.masked_fill_(hole, 0)
        s.update(spans=spans, steps=STEPS, grad=grad, param=master.to(torch.bfloat16) if bf16 else master, master=master if bf16 else None)
        if case["bits"] == 8:
            for name, t in (("m", m), ("v", v.sqrt_())):
                e = _exponent(t.view(-1, GROUP).abs().amax(1))
                s[name] = torch.ldexp(t.view(-1, GROUP), -e[:, None]).to(torch.float8_e4m3fn).view(-1).view(torch.uint8)
                s[name + "_scale"] = (e + 127).to(torch.uint8)
        else:
            s.update(m=m, v=v)
        if own:
            from scatter_grouped_gemm_amd import AdamW
            cut = lambda t: [t[a:a + n] for a, n in spans]  # noqa: E731
            opt = AdamW(cut(s["param"]), cut(grad), lr=LR, betas=(BETA1, BETA2), eps=EPS, weight_decay=DECAY, state_bits=case["bits"], seed=SEED)
            opt.steps.fill_(STEPS)
            for name in ("master", "m", "v", "m_scale", "v_scale"):
                if s.get(name) is not None:
                    s[name] = getattr(opt, name).copy_(s[name])
            s["opt"] = opt
        return s
    r = _routing(case, g)
    s.update({n: r[n] for n in ("ids", "weights", "src2dst", "m_indices", "starts", "counts", "runs", "rows")})
    zeros = lambda *shape, dtype=torch.bfloat16: torch.zeros(*shape, dtype=dtype, device="cuda")  # noqa: E731
    rows, T = r["rows"], case["T"]
    if op == "combine_bwd":
        H = case["H"]
        s.update(dout=_randn(g, T, H, scale=0.02), y=_randn(g, rows, H), dy=zeros(rows, H),
                 dweights=zeros(T, case["k"], dtype=torch.float32), dlogits=zeros(T, case["E"], dtype=torch.float32))
    elif op == "scatter_bwd":
        s.update(drows=_randn(g, rows, case["H"], scale=0.02), dx=zeros(T, case["H"]))
    elif op == "silu_bwd":
        I = case["I"]
        s.update(gateup=_randn(g, rows, 2 * I), dact=_randn(g, rows, I, scale=0.02), dgateup=zeros(rows, 2 * I), act=zeros(rows, I))
    elif op == "dgrad":
        s.update(dc=_randn(g, rows, case["N"], scale=0.02), b=_randn(g, case["El"], case["N"], case["K"], scale=0.02), da=zeros(rows, case["K"]))
    else:
        dt = torch.float32 if case["out"] == "fp32" else torch.bfloat16
        shape = (case["El"], case["N"], case["K"])
        s.update(dc=_randn(g, rows, case["N"], scale=0.02), a=_randn(g, rows, case["K"]),
                 db=_randn(g, *shape, scale=0.5, dtype=dt) if case["accumulate"] else zeros(*shape, dtype=dt))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    from scatter_grouped_gemm_amd import _lib as L
    case = s["case"]
    op, masked = case["op"], case.get("layout") == "masked"
    if op == "combine_bwd":
        L.moe_combine_bwd(s["dout"], s["y"], s["src2dst"], s["weights"], s["dy"], s["dweights"])
        L.moe_route_topk_bwd(s["ids"], s["weights"], s["dweights"], s["dlogits"])
        return dict(dy=s["dy"], dweights=s["dweights"], dlogits=s["dlogits"])
    if op == "scatter_bwd":
        L.moe_scatter_bwd(s["drows"], s["src2dst"], s["dx"])
        return dict(dx=s["dx"])
    if op == "silu_bwd":
        if masked:
            L.silu_and_mul_bwd(s["gateup"], s["dact"], s["dgateup"], s["act"], masked_m=s["counts"], max_m=case["T"])
        else:
            L.silu_and_mul_bwd(s["gateup"], s["dact"], s["dgateup"], s["act"], m_indices=s["m_indices"])
        return dict(dgateup=s["dgateup"], act=s["act"])
    if op == "dgrad":
        L.grouped_gemm_contig_dgrad(s["dc"], s["b"], s["da"], s["m_indices"])
        return dict(da=s["da"])
    if op == "wgrad":
        L.grouped_gemm_contig_wgrad(s["dc"], s["a"], s["starts"], s["counts"], s["db"], accumulate=case["accumulate"])
        return dict(db=s["db"])
    s["opt"].step()
    return _adamw_outputs(s)


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "combine_bwd":
        w, T = s["weights"], case["T"]
        held = s["src2dst"] >= 0
        row = s["src2dst"].clamp(min=0).long()
        dout = s["dout"].float()
        dweights = (s["y"][row].float() * dout[:, None, :]).sum(-1).masked_fill(~held, 0)
        dy = torch.zeros(s["rows"] + 1, case["H"], dtype=torch.bfloat16, device="cuda")  # the last row takes the slots held elsewhere
        dy[torch.where(held, row, s["rows"]).view(-1)] = (w[..., None] * dout[:, None, :]).to(torch.bfloat16).view(-1, case["H"])
        inner = w * (dweights - (w * dweights).sum(1, keepdim=True))
        dlogits = torch.zeros(T, case["E"], device="cuda").scatter_(1, s["ids"].long(), inner)
        return dict(dy=dy[:-1], dweights=dweights, dlogits=dlogits)
    if op == "scatter_bwd":
        held = s["src2dst"] >= 0
        rows = s["drows"][s["src2dst"].clamp(min=0).long()].float()
        return dict(dx=rows.masked_fill(~held[..., None], 0).sum(1).to(torch.bfloat16))
    if op == "silu_bwd":
        I = case["I"]
        gate, up, da = s["gateup"][:, :I].float(), s["gateup"][:, I:].float(), s["dact"].float()
        sig = 1 / (1 + torch.exp(-gate))
        skip = (s["m_indices"] < 0)[:, None]
        dgateup = torch.cat([da * up * sig * (1 + gate * (1 - sig)), da * gate * sig], 1).masked_fill(skip, 0)
        return dict(dgateup=dgateup.to(torch.bfloat16), act=(gate * sig * up).masked_fill(skip, 0).to(torch.bfloat16))
    if op == "dgrad":
        da = torch.zeros(s["rows"], case["K"], dtype=torch.bfloat16, device="cuda")
        for e, (at, n) in enumerate(s["runs"]):
            if n:
                da[at:at + n] = (s["dc"][at:at + n].float() @ s["b"][e].float()).to(torch.bfloat16)
        return dict(da=da)
    if op == "wgrad":
        db = s["db"]
        for e, (at, n) in enumerate(s["runs"]):
            if n:
                p = s["dc"][at:at + n].float().t() @ s["a"][at:at + n].float()
                db[e] = ((db[e].float() + p) if case["accumulate"] else p).to(db.dtype)
            elif not case["accumulate"]:
                db[e] = 0
        return dict(db=db)
    s["steps"] += 1
    t = s["steps"]
    c1, c2 = 1 - BETA1 ** t, math.sqrt(1 - BETA2 ** t)
    w = s["param"] if s["master"] is None else s["master"]
    for i, (a, n) in enumerate(s["spans"]):
        b = a + (n + GROUP - 1) // GROUP * GROUP  # whole groups: what is behind the tensor's end stays zero
        grad = s["grad"][a:b].float()
        if case["bits"] == 8:
            m = torch.ldexp(s["m"][a:b].view(torch.float8_e4m3fn).float().view(-1, GROUP), s["m_scale"][a // GROUP:b // GROUP, None].int() - 127).view(-1)
            v = torch.ldexp(s["v"][a:b].view(torch.float8_e4m3fn).float().view(-1, GROUP), s["v_scale"][a // GROUP:b // GROUP, None].int() - 127).view(-1).square()
        else:
            m, v = s["m"][a:b], s["v"][a:b]
        m = BETA1 * m + (1 - BETA1) * grad
        v = BETA2 * v + (1 - BETA2) * grad * grad
        root = torch.sqrt(v)
        w[a:b] = w[a:b] * (1 - LR * DECAY) - (LR / c1) * m / (root / c2 + EPS)
        if s["master"] is not None:
            s["param"][a:b] = w[a:b].to(torch.bfloat16)
        if case["bits"] == 8:
            r = _random(b - a, i, t)
            s["m"][a:b], s["m_scale"][a // GROUP:b // GROUP] = _rounded(m, r & 0xffff)
            s["v"][a:b], s["v_scale"][a // GROUP:b // GROUP] = _rounded(root, r >> 16, keep=True)
        else:
            s["m"][a:b], s["v"][a:b] = m, v
    return _adamw_outputs(s)


def _adamw_outputs(s):
    out = dict(param=s["param"], m=s["m"], v=s["v"])
    if s["master"] is not None:
        out["master"] = s["master"]
    if s["case"]["bits"] == 8:  # the values that codes and scales stand for
        out.update(m=s["m"].view(torch.float8_e4m3fn), v=s["v"].view(torch.float8_e4m3fn),
                   m_scale=s["m_scale"].view(torch.float8_e8m0fnu), v_scale=s["v_scale"].view(torch.float8_e8m0fnu))
    return out


def _mix(x):
    x = x ^ (x >> 16)
    x = (x * 0x9E3779B1) & 0xffffffff
    x = x ^ (x >> 15)
    x = (x * 0x85EBCA77) & 0xffffffff
    return x ^ (x >> 16)


def _random(n, tensor, step):
    """The 32 random bits of each element of one tensor at one step (element numbers here stay below 2^32)."""
    key = _mix((_mix((SEED + 0x9E3779B9 * (tensor + 1)) & 0xffffffff) + step) & 0xffffffff)
    return _mix(_mix(torch.arange(n, device="cuda")) ^ key)


def _rounded(x, bits, keep=False):
    """x in groups of 128 as e4m3 codes and scale bytes, rounded up with the probability of the
    remainder: the remainder in units of the code's last place plus 16 random bits, cut off.
    keep: a positive value never becomes zero."""
    x = x.view(-1, GROUP)
    e = _exponent(x.abs().amax(1))
    a = torch.ldexp(x.abs(), -e[:, None])
    unit = (torch.frexp(a)[1] - 1).clamp(min=-6) - 3
    q = torch.floor(torch.ldexp(a, -unit) + bits.view(-1, GROUP).float() / 65536)
    if keep:
        q = torch.where((a > 0) & (q == 0), 1.0, q)
    codes = torch.copysign(torch.ldexp(q, unit), x).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8).view(-1), (e + 127).to(torch.uint8)


# ---------------------------------------------------------------------------
# work and exact values
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "adamw":
        n = sum(_sizes(case))
        state = 4 + 4 / GROUP if case["bits"] == 8 else 16
        each = (10 if case["param"] == "bf16" else 8) + (2 if case["grad"] == "bf16" else 4) + state
        return {"bytes": n * each, "flops": 14 * n}
    T, k, El = case["T"], case["k"], case["El"]
    A = max(1, T * k * El // case["E"])  # assignments held here, with even routing
    if op == "combine_bwd":
        H = case["H"]
        return {"bytes": 2 * T * H + 4 * A * H + 16 * T * k + 4 * T * case["E"], "flops": 3 * A * H}
    if op == "scatter_bwd":
        return {"bytes": 2 * case["H"] * (A + T) + 4 * T * k, "flops": A * case["H"]}
    if op == "silu_bwd":
        return {"bytes": 12 * A * case["I"], "flops": 16 * A * case["I"]}
    N, K = case["N"], case["K"]
    used = min(El, A)  # experts whose weights are read
    if op == "dgrad":
        return {"bytes": 2 * (A * (N + K) + used * N * K), "flops": 2 * A * N * K}
    each = (4 if case["out"] == "fp32" else 2) * (2 if case["accumulate"] else 1)
    return {"bytes": 2 * A * (N + K) + each * (used if case["accumulate"] else El) * N * K, "flops": 2 * A * N * K}


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    d = lambda t: t.double()  # noqa: E731
    if op == "adamw":
        return _exact_adamw(s)
    T, k, rows = case["T"], case["k"], s["rows"]
    where = torch.nonzero(s["src2dst"].view(-1) >= 0).view(-1)   # held assignments
    row, token = s["src2dst"].view(-1)[where].long(), where // k
    if op == "combine_bwd":
        dy = torch.zeros(rows, case["H"], dtype=torch.float64, device="cuda")
        dy[row] = d(s["weights"]).view(-1)[where, None] * d(s["dout"])[token]
        dw = torch.zeros(T * k, dtype=torch.float64, device="cuda")
        dw[where] = torch.linalg.vecdot(d(s["y"][row]), d(s["dout"][token]))
        dw = dw.view(T, k)
        w = d(s["weights"])  # the softmax over the kept slots: its Jacobian as a matrix
        jac = torch.diag_embed(w) - w[:, :, None] * w[:, None, :]
        dl = torch.zeros(T, case["E"], dtype=torch.float64, device="cuda")
        dl.scatter_add_(1, s["ids"].long(), (jac * dw[:, None, :]).sum(-1))
        return dict(dy=dy, dweights=dw, dlogits=dl)
    if op == "scatter_bwd":
        dx = torch.zeros(T, case["H"], dtype=torch.float64, device="cuda")
        return dict(dx=dx.index_add_(0, token, d(s["drows"][row])))
    if op == "silu_bwd":
        I = case["I"]
        gate, up, da = d(s["gateup"][row, :I]), d(s["gateup"][row, I:]), d(s["dact"][row])
        half = torch.tanh(gate / 2)                              # sigma(g) = (1 + tanh(g/2)) / 2
        silu, slope = gate * (1 + half) / 2, (1 + half) / 2 + gate * (1 - half * half) / 4
        dgateup, act = (torch.zeros(rows, n, dtype=torch.float64, device="cuda") for n in (2 * I, I))
        dgateup[row, :I], dgateup[row, I:], act[row] = da * up * slope, da * silu, silu * up
        return dict(dgateup=dgateup, act=act)
    at, n = (np.array([r[i] for r in s["runs"]]) for i in (0, 1))
    if op == "dgrad":
        out = torch.zeros(rows, case["K"], dtype=torch.float64, device="cuda")
        for e in np.flatnonzero(n):
            out[at[e]:at[e] + n[e]] = torch.matmul(d(s["dc"][at[e]:at[e] + n[e]]), d(s["b"][e]))
        return dict(da=out)
    out = d(s["db"])
    if not case["accumulate"]:
        out.zero_()
    for e in np.flatnonzero(n):
        out[e] += torch.matmul(d(s["a"][at[e]:at[e] + n[e]].t()), d(s["dc"][at[e]:at[e] + n[e]])).t()
    return dict(db=out)


def _exact_adamw(s):
    case, t = s["case"], STEPS + 1
    d = lambda x: x.double()  # noqa: E731
    q = case["bits"] == 8
    out = {name: torch.zeros(s["grad"].numel(), dtype=torch.float64, device="cuda") for name in ("param", "m", "v")}
    if q:
        out.update({name: torch.full((s["m_scale"].numel(),), 2.0 ** -126, dtype=torch.float64, device="cuda") for name in ("m_scale", "v_scale")})
        value = torch.arange(127, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()  # 0 .. 448, rising
    start = d(s["param"] if s["master"] is None else s["master"])
    for i, (a, n) in enumerate(s["spans"]):
        groups = (n + GROUP - 1) // GROUP
        g0 = a // GROUP
        grad, m, v = d(s["grad"][a:a + n]), s["m"][a:a + n], s["v"][a:a + n]
        if q:
            each = lambda name: torch.exp2(d(s[name][g0:g0 + groups]) - 127).repeat_interleave(GROUP)[:n]  # noqa: E731
            m, v = d(m.view(torch.float8_e4m3fn)) * each("m_scale"), (d(v.view(torch.float8_e4m3fn)) * each("v_scale")) ** 2
        m, v = torch.lerp(grad, d(m), BETA1), torch.lerp(grad ** 2, d(v), BETA2)
        move = (m / (1 - BETA1 ** t)) / ((v / (1 - BETA2 ** t)) ** 0.5 + EPS) + DECAY * start[a:a + n]
        out["param"][a:a + n] = start[a:a + n] - LR * move
        if not q:
            out["m"][a:a + n], out["v"][a:a + n] = m, v
            continue
        bits = _random(n, i, t)
        for name, x, u in (("m", m, bits % 65536), ("v", v ** 0.5, bits // 65536)):
            size = torch.zeros(groups * GROUP, dtype=torch.float64, device="cuda")
            size[:n] = x.abs()
            top = size.view(-1, GROUP).amax(1)
            e = torch.where(top > 0, torch.ceil(torch.log2(top / 448)), -126.0).clamp(-126, 127)
            scale = torch.exp2(e)
            size = size[:n] / scale.repeat_interleave(GROUP)[:n]
            low = torch.searchsorted(value, size, right=True) - 1   # the code at or below
            low = low.clamp(max=125)
            part = (size - value[low]) / (value[low + 1] - value[low])
            code = value[low + (part + u / 65536 >= 1).long()]
            if name == "v":
                code = torch.where((size > 0) & (code == 0), value[1], code)
            out[name][a:a + n] = torch.sign(x) * code
            out[name + "_scale"][g0:g0 + groups] = scale
    if s["master"] is not None:
        out["master"] = out["param"]
    return out
