"""Products with an epilogue and the epilogue's gradient: cases, plain forms and 64-bit values.

``linear`` is a dense product with bias, activation and residual (the router's
logits, a shared expert beside the routed ones), ``grouped`` the expert products
with a bias and an activation for each expert's rows, ``act_bwd`` the gradient of
the activation with the bias gradients.  Each case is one operator at one size;
``run`` computes it in plain torch operations (``own`` false) or through the
library (``own`` true) on the same state.

Layouts are those of include/moe.h: the compact layout pads every expert to 128
rows tagged -1 in ``m_indices``, the masked one gives each expert ``max_m`` rows.
Rows that hold no assignment keep what the output buffer held (zeros here).
Gated activations take a row's first half as the gate and the second as the up part.
"""
import math

import torch

own = False

BLOCK = 128                # rows an expert is padded to in the compact layout; channels that share an FP8 scale
ALPHA, LIMIT = 1.702, 7.0  # of the clamped activation
GATED = ("silu_mul", "gelu_mul", "gelu_tanh_mul", "swiglu_clamp")
PLAIN = ("none", "silu", "gelu", "gelu_tanh", "relu2")


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # the router's logits for a handful of tokens while serving
        dict(name="linear_router_tokens", op="linear", T=7, K=7168, N=256, act="none", bias="fp32", residual=False, out="fp32", pre=False, pad=0),
        # the same for a full prefill
        dict(name="linear_router_prefill", op="linear", T=8192, K=7168, N=256, act="none", bias="fp32", residual=False, out="fp32", pre=False, pad=0),
        # a shared expert's gate and up for a single token
        dict(name="linear_up_token", op="linear", T=1, K=7168, N=4096, act="silu_mul", bias="none", residual=False, out="bf16", pre=False, pad=0),
        # its way down for an odd prefill, added to what the routed experts gave
        dict(name="linear_down_prefill", op="linear", T=8191, K=2048, N=7168, act="none", bias="none", residual=True, out="bf16", pre=False, pad=0),
        # a wide gated layer in training: what the gradient needs is kept
        dict(name="linear_wide_training", op="linear", T=4096, K=4096, N=28672, act="gelu_tanh_mul", bias="bf16", residual=False, out="bf16", pre=True, pad=0),
        # one step of the tiny model: the call itself is what costs
        dict(name="grouped_tiny", op="grouped", T=64, K=256, N=1024, E=8, El=8, k=2, skew=False, layout="compact", fmt="bf16", act="swiglu_clamp", pre=False),
        # eight large experts in training
        dict(name="grouped_up_training", op="grouped", T=4096, K=4096, N=28672, E=8, El=8, k=2, skew=False, layout="compact", fmt="bf16", act="swiglu_clamp", pre=True),
        # the way down with biases: long batch, popular and dead experts
        dict(name="grouped_down_skewed", op="grouped", T=16384, K=1536, N=4096, E=128, El=128, k=8, skew=True, layout="compact", fmt="bf16", act="none", pre=False),
        # decoding on one share of 32 experts out of 256, 4-bit weights
        dict(name="grouped_up_decode_mxfp4", op="grouped", T=256, K=7168, N=4096, E=256, El=32, k=8, skew=False, layout="masked", fmt="mxfp4", act="swiglu_clamp", pre=False),
        # a few tokens, mostly padding rows
        dict(name="act_bwd_tiny", op="act_bwd", T=33, N=1024, E=8, El=8, k=2, skew=False, layout="compact", act="gelu_mul"),
        # the wide activations of eight large experts
        dict(name="act_bwd_wide", op="act_bwd", T=4096, N=28672, E=8, El=8, k=2, skew=False, layout="compact", act="swiglu_clamp"),
        # a dense layer of an odd batch
        dict(name="act_bwd_dense", op="act_bwd", T=8191, N=4096, E=1, El=1, k=1, skew=False, layout="dense", act="gelu"),
    ]


def _log(rng, lo, hi):
    """A whole number spread evenly over the logarithm of lo .. hi."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "linear", "grouped", "grouped", "act_bwd"])
    act = rng.choice(GATED) if rng.random() < 0.5 else rng.choice(PLAIN)
    if op == "linear":
        K = 8 * _log(rng, 1, 1792)
        N = rng.choice([_log(rng, 1, 512), 8 * _log(rng, 16, 3584)])
        N += N % 2 if act in GATED else 0
        T = _log(rng, 1, max(2, min(16384, 900000000000 // (N * K))))
        return dict(op=op, T=T, K=K, N=N, act=act, bias=rng.choice(["none", "bf16", "fp32"]), residual=rng.random() < 0.4,
                    out=rng.choice(["bf16", "bf16", "fp32"]), pre=rng.random() < 0.3, pad=rng.choice([0, 0, 8, 200]))
    E = rng.choice([4, 8, 16, 60, 64, 128, 256])
    k = min(E, rng.choice([1, 2, 4, 6, 8]))
    El = rng.choice([E, E, max(1, E // 8)])
    skew = rng.random() < 0.4
    layout = rng.choice(["compact", "masked"])
    if op == "grouped":
        K, N = 128 * _log(rng, 1, 56), 256 * _log(rng, 1, 56)
        El = min(El, max(1, 600000000 // (N * K)))
        E = max(El, k) if El < E and rng.random() < 0.5 else E
        T = _log(rng, 1, max(2, min(16384, 900000000000 // (N * K * k))))
        layout = layout if El * T <= 32768 else "compact"
        fmt = rng.choice(["bf16", "bf16", "fp8", "mxfp8", "mxfp4"])
        act = rng.choice(GATED + ("none", "none", "gelu", "relu2"))
        return dict(op=op, T=T, K=K, N=N, E=E, El=El, k=k, skew=skew, layout=layout, fmt=fmt, act=act, pre=fmt == "bf16" and rng.random() < 0.4)
    T = _log(rng, 1, 12288)
    layout = rng.choice(["dense", layout]) if El * T <= 32768 else rng.choice(["dense", "compact"])
    if layout == "dense":
        E = El = k = 1
        skew = False
    rows = T if layout == "dense" else El * T if layout == "masked" else BLOCK * min(T * k, El) + T * k
    return dict(op=op, T=T, N=256 * _log(rng, 1, min(112, max(1, 900000 // rows))), E=E, El=El, k=k, skew=skew, layout=layout, act=act)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, scale=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _zeros(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def _routing(case, g):
    """The rows of the experts, as the scatter leaves them, and (start, rows) of each for the plain form."""
    T, E, El, k = case["T"], case["E"], case["El"], case["k"]
    logits = torch.randn(T, E, generator=g, device="cuda")
    if case["skew"]:  # Zipf-like popularity, and experts that no token takes
        rank = torch.randperm(E, generator=g, device="cuda") + 1
        dead = min(E // 8, E - k)
        logits = logits - 1.2 * torch.log(rank.float()) - 1e4 * (rank > E - dead)
    ids = torch.topk(logits, k, dim=1).indices
    counts = torch.bincount(ids.view(-1), minlength=E)[:El]
    if case["layout"] == "masked":
        rows, starts = El * T, torch.arange(El, device="cuda") * T
    else:
        A = T * k
        rows = BLOCK * (min(A, El) + (A - min(A, El)) // BLOCK)
        padded = (counts + BLOCK - 1) // BLOCK * BLOCK
        starts = torch.cumsum(padded, 0) - padded
    expert = torch.repeat_interleave(torch.arange(El, device="cuda"), counts)
    held = starts[expert] + torch.arange(len(expert), device="cuda") - (torch.cumsum(counts, 0) - counts)[expert]
    m_indices = torch.full((rows,), -1, device="cuda")
    m_indices[held] = expert
    i32 = lambda t: t.to(torch.int32).contiguous()  # noqa: E731
    return dict(rows=rows, m_indices=i32(m_indices), starts=i32(starts), counts=i32(counts), runs=list(zip(starts.tolist(), counts.tolist())))


def _exponent(amax, top):
    """The smallest e in [-126, 127] with amax <= top * 2^e."""
    e = torch.ceil(torch.log2(amax.double() / top)).clamp(-126, 127)
    return torch.where(amax > 0, e, -126.0).to(torch.int32)


def _fp8_rows(x):
    """Rows as e4m3 with one exponent for 128 channels: codes [M, K], scale bytes [K/128, M]."""
    M, K = x.shape
    e = _exponent(x.view(M, K // BLOCK, BLOCK).abs().amax(2), 448)
    q = torch.ldexp(x.float().view(M, K // BLOCK, BLOCK), -e[..., None]).to(torch.float8_e4m3fn).view(M, K)
    return q.view(torch.uint8), (e + 127).to(torch.uint8).t().contiguous()


def _fp8_blocks(w):
    """Weights as e4m3 with one exponent for 128 x 128 values: codes and scale bytes [G, N/128, K/128]."""
    G, N, K = w.shape
    b = w.view(G, N // BLOCK, BLOCK, K // BLOCK, BLOCK)
    e = _exponent(b.abs().amax(4).amax(2), 448)
    q = torch.ldexp(b.float(), -e[:, :, None, :, None]).to(torch.float8_e4m3fn).view(G, N, K)
    return q.view(torch.uint8), (e + 127).to(torch.uint8)


def _mx(w, fmt):
    """Weights with one exponent for 32 values of a row: codes, and scale bytes in the products' tiles
    (those of the 4 x 64 blocks of 64 rows and 128 values lie together: value block, row % 16, row / 16)."""
    G, N, K = w.shape
    b = w.view(G, N, K // 32, 32)
    e = _exponent(b.abs().amax(3), 448 if fmt == "mxfp8" else 6)
    v = torch.ldexp(b.float(), -e[..., None])
    if fmt == "mxfp8":
        q = v.to(torch.float8_e4m3fn).view(G, N, K).view(torch.uint8)
    else:  # 0, 1/2, 1, 3/2, 2, 3, 4, 6: to the nearest, ties to the even code
        edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
        low, high = torch.bucketize(v.abs(), edges), torch.bucketize(v.abs(), edges, right=True)
        code = torch.where(low % 2 == 0, low, high)  # they differ at a tie only
        code = (code + 8 * torch.signbit(v)).to(torch.uint8).view(G, N, K // 2, 2)
        q = code[..., 0] | (code[..., 1] << 4)
    tiles = (e + 127).to(torch.uint8).view(G, N // 64, 4, 16, K // BLOCK, 4).permute(0, 1, 4, 5, 3, 2)
    return q.contiguous(), tiles.reshape(G, N // 64, K // BLOCK, 256).contiguous()


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case=case)
    N = case["N"]
    wide = N // 2 if case["act"] in GATED else N   # columns of the activation
    if op == "linear":
        T, K = case["T"], case["K"]
        s.update(x=_randn(g, T, K + case["pad"])[:, :K], w=_randn(g, N, K, scale=K ** -0.5),
                 out=_zeros(T, wide, dtype=torch.float32 if case["out"] == "fp32" else torch.bfloat16),
                 bias=None, residual=None, pre=_zeros(T, N) if case["pre"] else None)
        if case["bias"] != "none":
            s["bias"] = _randn(g, N, scale=0.5, dtype=torch.float32 if case["bias"] == "fp32" else torch.bfloat16)
        if case["residual"]:
            s["residual"] = _randn(g, T, wide + case["pad"], dtype=s["out"].dtype)[:, :wide]
        return s
    if case["layout"] == "dense":
        s.update(rows=case["T"], runs=[(0, case["T"])], m_indices=None, starts=None, counts=None)
    else:
        s.update(_routing(case, g))
    rows, El = s["rows"], case["El"]
    if op == "act_bwd":
        s.update(pre=_randn(g, rows, N, scale=3.0), dout=_randn(g, rows, wide, scale=0.02), dpre=_zeros(rows, N),
                 dbias=_zeros(El, N, dtype=torch.float32))
        return s
    K, fmt = case["K"], case["fmt"]
    x = _randn(g, rows, K)
    w = _randn(g, El, N, K, scale=3 * K ** -0.5)
    s.update(x=x, x_scale=None, w=w, w_scale=None, bias=_randn(g, El, N, scale=0.5), out=_zeros(rows, wide),
             pre=_zeros(rows, N) if case["pre"] else None)
    if fmt != "bf16":
        s["x"], scale = _fp8_rows(x)
        if case["layout"] == "masked":  # [K/128][rows] of each expert
            scale = scale.view(K // BLOCK, El, case["T"]).transpose(0, 1).contiguous()
        s["x_scale"] = scale
        s["w"], s["w_scale"] = _fp8_blocks(w) if fmt == "fp8" else _mx(w, fmt)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    return (_run_own if own else _run_plain)(state)


def _outputs(s, *names):
    return {n: s[n] for n in names if s[n] is not None}


def _run_own(s):
    from scatter_grouped_gemm_amd import _lib as L
    case = s["case"]
    op, act, masked = case["op"], case["act"], case.get("layout") == "masked"
    if op == "linear":
        L.moe_linear(s["x"], s["w"], s["out"], bias=s["bias"], act=act, residual=s["residual"], pre=s["pre"], alpha=ALPHA, limit=LIMIT)
        return _outputs(s, "out", "pre")
    if op == "act_bwd":
        if masked:
            L.moe_act_bwd(s["pre"], s["dout"], s["dpre"], act, dbias=s["dbias"], masked_m=s["counts"], max_m=case["T"], alpha=ALPHA, limit=LIMIT)
        elif s["m_indices"] is None:
            L.moe_act_bwd(s["pre"], s["dout"], s["dpre"], act, dbias=s["dbias"], alpha=ALPHA, limit=LIMIT)
        else:
            L.moe_act_bwd(s["pre"], s["dout"], s["dpre"], act, dbias=s["dbias"], m_indices=s["m_indices"], expert_start_loc=s["starts"],
                          num_valid=s["counts"], alpha=ALPHA, limit=LIMIT)
        return _outputs(s, "dpre", "dbias")
    wdt = {"bf16": False, "fp8": True}.get(case["fmt"], case["fmt"])
    if masked:
        El, T = case["El"], case["T"]
        rows3 = lambda t: None if t is None else t.view(El, T, -1)  # noqa: E731
        L.grouped_gemm_masked_act(wdt, rows3(s["x"]), s["x_scale"], s["w"], s["w_scale"], rows3(s["out"]), s["counts"], min(T, max(1, T * case["k"] // case["E"])),
                                  bias=s["bias"], act=act, pre=rows3(s["pre"]), alpha=ALPHA, limit=LIMIT)
    else:
        L.grouped_gemm_contig_act(wdt, s["x"], s["x_scale"], s["w"], s["w_scale"], s["out"], s["m_indices"],
                                  bias=s["bias"], act=act, pre=s["pre"], alpha=ALPHA, limit=LIMIT)
    return _outputs(s, "out", "pre")


def _act(pre, act):
    """The activation of a product in fp32."""
    if act in GATED:
        g, u = pre.chunk(2, 1)
        if act == "swiglu_clamp":
            g, u = g.clamp(max=LIMIT), u.clamp(-LIMIT, LIMIT)
            return g / (1 + torch.exp(-ALPHA * g)) * (u + 1)
        return _act(g, act[:-4]) * u
    if act == "silu":
        return pre / (1 + torch.exp(-pre))
    if act == "gelu":
        return pre * 0.5 * torch.special.erfc(pre * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return pre / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (pre + 0.044715 * pre ** 3)))
    if act == "relu2":
        return torch.relu(pre) ** 2
    return pre


def _slope(x, act):
    """Value and derivative of an activation without its up part, in fp32."""
    if act in ("silu", "swiglu_clamp"):
        a = ALPHA if act == "swiglu_clamp" else 1.0
        s = 1 / (1 + torch.exp(-a * x))
        return x * s, s * (1 + a * x * (1 - s))
    if act == "gelu":
        c = 0.5 * torch.special.erfc(x * -math.sqrt(0.5))
        return x * c, c + x * torch.exp(-0.5 * x * x) * (1 / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        b = 2 * math.sqrt(2 / math.pi)
        s = 1 / (1 + torch.exp(-b * (x + 0.044715 * x ** 3)))
        return x * s, s + x * s * (1 - s) * b * (1 + 3 * 0.044715 * x * x)
    if act == "relu2":
        return torch.relu(x) ** 2, 2 * torch.relu(x)
    return x, torch.ones_like(x)


def _weight(s, e):
    """Expert e's weights in fp32."""
    fmt, w = s["case"]["fmt"], s["w"][e]
    if fmt == "bf16":
        return w.float()
    if fmt == "fp8":
        scale = torch.exp2(s["w_scale"][e].float() - 127).repeat_interleave(BLOCK, 0).repeat_interleave(BLOCK, 1)
        return w.view(torch.float8_e4m3fn).float() * scale
    N, K = s["case"]["N"], s["case"]["K"]
    scale = torch.exp2(s["w_scale"][e].view(N // 64, K // BLOCK, 4, 16, 4).permute(0, 4, 3, 1, 2).reshape(N, K // 32).float() - 127)
    if fmt == "mxfp8":
        v = w.view(torch.float8_e4m3fn).float()
    else:
        value = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], device=w.device)
        v = value[torch.stack([w & 15, w >> 4], -1).long()]
    return (v.view(N, K // 32, 32) * scale[..., None]).view(N, K)


def _rows(s, at, n, e):
    """Rows at .. at + n (all of expert e) of the product's input in fp32."""
    x = s["x"][at:at + n]
    if s["case"]["fmt"] == "bf16":
        return x.float()
    if s["case"]["layout"] == "masked":
        scale = s["x_scale"][e, :, at - e * s["case"]["T"]:][:, :n]
    else:
        scale = s["x_scale"][:, at:at + n]
    return x.view(torch.float8_e4m3fn).float() * torch.exp2(scale.t().float() - 127).repeat_interleave(BLOCK, 1)


def _run_plain(s):
    case = s["case"]
    op, act = case["op"], case["act"]
    if op == "linear":
        pre = s["x"].float() @ s["w"].float().t()
        if s["bias"] is not None:
            pre += s["bias"].float()
        out = _act(pre, act)
        if s["residual"] is not None:
            out = out + s["residual"].float()
        s["out"].copy_(out)
        if s["pre"] is not None:
            s["pre"].copy_(pre)
        return _outputs(s, "out", "pre")
    if op == "act_bwd":
        d = s["dout"].float()
        if act in GATED:
            g, u = s["pre"].float().chunk(2, 1)
            if act == "swiglu_clamp":
                v, slope = _slope(g.clamp(max=LIMIT), act)
                dg = d * (u.clamp(-LIMIT, LIMIT) + 1) * slope * (g <= LIMIT)
                du = d * v * (u.abs() <= LIMIT)
            else:
                v, slope = _slope(g, act[:-4])
                dg, du = d * u * slope, d * v
            d = torch.cat([dg, du], 1)
        else:
            d = d * _slope(s["pre"].float(), act)[1]
        if case["layout"] == "dense":
            s["dpre"].copy_(d)
            s["dbias"].copy_(d.sum(0, keepdim=True))
            return _outputs(s, "dpre", "dbias")
        valid = s["m_indices"] >= 0
        s["dpre"].copy_(d.masked_fill(~valid[:, None], 0))
        for e, (at, n) in enumerate(s["runs"]):
            s["dbias"][e] = d[at:at + n].sum(0)
        return _outputs(s, "dpre", "dbias")
    for e, (at, n) in enumerate(s["runs"]):  # expert by expert, as a torch program has it
        if n:
            pre = _rows(s, at, n, e) @ _weight(s, e).t() + s["bias"][e].float()
            s["out"][at:at + n] = _act(pre, act)
            if s["pre"] is not None:
                s["pre"][at:at + n] = pre
    return _outputs(s, "out", "pre")


# ---------------------------------------------------------------------------
# work and exact values
# ---------------------------------------------------------------------------

def work(case):
    op, T, N = case["op"], case["T"], case["N"]
    wide = N // 2 if case["act"] in GATED else N
    if op == "linear":
        K, each = case["K"], 4 if case["out"] == "fp32" else 2
        moved = 2 * (T * K + N * K) + each * T * wide * (2 if case["residual"] else 1) + {"none": 0, "bf16": 2, "fp32": 4}[case["bias"]] * N
        return {"bytes": moved + (2 * T * N if case["pre"] else 0), "flops": 2 * T * N * K}
    El = case["El"]
    A = max(1, T * case["k"] * El // case["E"])  # assignments held here, with even routing
    if op == "act_bwd":
        return {"bytes": 2 * A * (2 * N + wide) + 4 * El * N, "flops": 16 * A * N}
    K, fmt = case["K"], case["fmt"]
    used = min(El, A)  # experts whose weights are read
    weight = {"bf16": 2, "fp8": 1 + 1 / BLOCK ** 2, "mxfp8": 1 + 1 / 32, "mxfp4": 0.5 + 1 / 32}[fmt]
    moved = A * K * (2 if fmt == "bf16" else 1 + 1 / BLOCK) + used * N * (K * weight + 2) + 2 * A * (wide + (N if case["pre"] else 0))
    return {"bytes": moved, "flops": 2 * A * N * K}


def _exact_half(x, act):
    """Value and derivative in 64 bits, from the definitions: x Phi(x) by the error function, the others by tanh."""
    if act in ("silu", "swiglu_clamp"):
        a = ALPHA if act == "swiglu_clamp" else 1.0
        t = torch.tanh(a * x / 2)
        return x * (1 + t) / 2, (1 + t) / 2 + x * a * (1 - t * t) / 4
    if act == "gelu":
        return x * (1 + torch.erf(x / 2 ** 0.5)) / 2, (1 + torch.erf(x / 2 ** 0.5)) / 2 + x * torch.exp(-x * x / 2) / (2 * math.pi) ** 0.5
    if act == "gelu_tanh":
        c = (2 / math.pi) ** 0.5
        t = torch.tanh(c * (x + 0.044715 * x ** 3))
        return x * (1 + t) / 2, (1 + t) / 2 + x * (1 - t * t) * c * (1 + 0.134145 * x * x) / 2
    if act == "relu2":
        return torch.where(x > 0, x * x, 0.0), torch.where(x > 0, 2 * x, 0.0)
    return x, torch.ones_like(x)


def _exact_act(pre, act):
    if act not in GATED:
        return _exact_half(pre, act)[0]
    half = pre.shape[1] // 2
    gate, up = pre[:, :half], pre[:, half:]
    if act == "swiglu_clamp":
        return _exact_half(torch.minimum(gate, torch.full_like(gate, LIMIT)), act)[0] * (1 + torch.where(up.abs() > LIMIT, torch.sign(up) * LIMIT, up))
    return _exact_half(gate, act[: -len("_mul")])[0] * up


def exact(case, seed):
    s, op, act = prepare(case, seed), case["op"], case["act"]
    d = lambda t: t.double()  # noqa: E731
    if op == "linear":
        pre = torch.matmul(d(s["x"]), d(s["w"]).t())
        if s["bias"] is not None:
            pre = pre + d(s["bias"])
        out = _exact_act(pre, act)
        found = dict(out=out if s["residual"] is None else out + d(s["residual"]))
        return dict(found, pre=pre) if s["pre"] is not None else found
    full = lambda t: torch.zeros(t.shape, dtype=torch.float64, device="cuda")  # noqa: E731
    if op == "act_bwd":
        found = dict(dpre=full(s["dpre"]), dbias=full(s["dbias"]))
        for e, (at, n) in enumerate(s["runs"]):
            pre, da = d(s["pre"][at:at + n]), d(s["dout"][at:at + n])
            if act not in GATED:
                grad = da * _exact_half(pre, act)[1]
            else:
                half = pre.shape[1] // 2
                gate, up = pre[:, :half], pre[:, half:]
                if act == "swiglu_clamp":
                    value, slope = _exact_half(torch.minimum(gate, torch.full_like(gate, LIMIT)), act)
                    inside = up.abs() <= LIMIT
                    grad = torch.cat([da * torch.where(gate > LIMIT, 0.0, slope) * torch.where(inside, up + 1, torch.sign(up) * LIMIT + 1),
                                      da * torch.where(inside, value, 0.0)], 1)
                else:
                    value, slope = _exact_half(gate, act[: -len("_mul")])
                    grad = torch.cat([da * slope * up, da * value], 1)
            found["dpre"][at:at + n] = grad
            found["dbias"][e] = torch.einsum("rn->n", grad)
        return found
    found = {n: full(s[n]) for n in ("out", "pre") if s[n] is not None}
    fmt, K, N = case["fmt"], case["K"], case["N"]
    power = lambda b: torch.exp2(d(b) - 127)  # noqa: E731
    for e, (at, n) in enumerate(s["runs"]):
        if not n:
            continue
        x, w = s["x"][at:at + n], s["w"][e]
        if fmt == "bf16":
            x, w = d(x), d(w)
        else:
            xs = s["x_scale"][e][:, :n] if case["layout"] == "masked" else s["x_scale"][:, at:at + n]
            x = (d(x.view(torch.float8_e4m3fn)).view(n, K // BLOCK, BLOCK) * power(xs).t()[:, :, None]).view(n, K)
            if fmt == "fp8":
                w = (d(w.view(torch.float8_e4m3fn)).view(N // BLOCK, BLOCK, K // BLOCK, BLOCK) * power(s["w_scale"][e])[:, None, :, None]).view(N, K)
            else:
                row, blk = torch.arange(N, device="cuda")[:, None], torch.arange(K // 32, device="cuda")[None]
                place = ((row // 64) * (K // BLOCK) + blk // 4) * 256 + (blk % 4) * 64 + (row % 16) * 4 + (row % 64) // 16
                ws = power(s["w_scale"][e].view(-1)[place])
                if fmt == "mxfp8":
                    w = d(w.view(torch.float8_e4m3fn))
                else:
                    code = torch.empty(N, K, dtype=torch.uint8, device="cuda")
                    code[:, 0::2], code[:, 1::2] = w % 16, w // 16
                    size, sign = d(code % 8), 1 - 2 * d(code // 8)
                    # exponent and one mantissa bit: below 2 halves, then (2 + m) * 2^(exponent - 2)
                    w = sign * torch.where(size < 4, size / 2, (2 + size % 2) * torch.exp2(torch.floor(size / 2) - 2))
                w = (w.view(N, K // 32, 32) * ws[..., None]).view(N, K)
        pre = torch.matmul(x, w.t()) + d(s["bias"][e])
        found["out"][at:at + n] = _exact_act(pre, act)
        if "pre" in found:
            found["pre"][at:at + n] = pre
    return found
