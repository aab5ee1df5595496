"""The layer with a router, a shared expert, expert biases and other activations: its
forward and backward as a whole against the same computation in 64 bits."""
import pytest
import torch

from scatter_grouped_gemm_amd import MoELayer
from epilogue_util import ALPHA, GATED, LIMIT, activation
from gpu_util import DEV, announce

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def rand(g, *shape, scale=1.0, dtype=BF):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


class Case:
    """A layer with everything, and its weights."""

    def __init__(self, seed=0, T=200, H=256, I=384, E=16, k=4, S=256, act="swiglu_clamp", bias=True, router=True, El=None,
                 start=0, **kw):
        g = torch.Generator(device=DEV)
        g.manual_seed(seed)
        self.k, self.E, self.El, self.start, self.act, self.S = k, E, El or E, start, act, S
        self.layer = MoELayer(hidden=H, intermediate=I, num_experts=E, top_k=k, max_tokens=T, num_local_experts=El,
                              expert_start=start, router=router, router_bias=router, shared_intermediate=S, expert_bias=bias,
                              activation=act, alpha=ALPHA, limit=LIMIT, device=DEV, **kw)
        self.x = rand(g, T, H)
        self.w13, self.w2 = rand(g, self.El, 2 * I, H, scale=1.5 * H ** -0.5), rand(g, self.El, H, I, scale=I ** -0.5)
        self.b13, self.b2 = (rand(g, self.El, 2 * I), rand(g, self.El, H)) if bias else (None, None)
        self.gate, self.gate_bias = (rand(g, E, H, scale=2 * H ** -0.5), rand(g, E, dtype=F32)) if router else (None, None)
        self.s13, self.s2 = (rand(g, 2 * S, H, scale=1.5 * H ** -0.5), rand(g, H, S, scale=S ** -0.5)) if S else (None, None)
        self.layer.set_weights(self.w13, self.w2)
        if bias:
            self.layer.set_bias(self.b13, self.b2)
        if router:
            self.layer.set_router(self.gate, self.gate_bias)
        if S:
            self.layer.set_shared(self.s13, self.s2)
        self.dout = rand(g, T, H, scale=0.1)

    def leaves(self):
        return {n: t.double().requires_grad_() for n in ("x", "w13", "w2", "b13", "b2", "gate", "gate_bias", "s13", "s2")
                if (t := getattr(self, n)) is not None}

    def exact(self, p, ids):
        """The layer in 64 bits, for the experts that the layer chose."""
        logits = p["x"] @ p["gate"].t() + p["gate_bias"]
        top = torch.softmax(torch.gather(logits, 1, ids.long()), 1)
        out = torch.zeros_like(p["x"])
        for e in range(self.El):
            t, j = torch.nonzero(ids == e + self.start, as_tuple=True)
            pre = p["x"][t] @ p["w13"][e].t() + (p["b13"][e] if "b13" in p else 0)
            y = activation(pre, self.act) @ p["w2"][e].t() + (p["b2"][e] if "b2" in p else 0)
            out = out.index_add(0, t, top[t, j][:, None] * y)
        if "s13" in p:
            out = out + activation(p["x"] @ p["s13"].t(), self.act) @ p["s2"].t()
        return out


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


def check_routing(c, ids):
    """The chosen experts are the most probable ones in 64 bits, up to logits that fp32 cannot tell apart."""
    logits = c.x.double() @ c.gate.double().t() + c.gate_bias.double()
    best = logits.topk(c.k, 1).values
    assert (torch.gather(logits, 1, ids.long()) - best).abs().max() < 1e-4


@pytest.mark.parametrize("act", GATED)
@pytest.mark.parametrize("fmt,layout", [("bf16", "compact"), ("bf16", "masked"), ("fp8", "compact"), ("mxfp8", "masked"),
                                        ("mxfp4", "compact"), ("mxfp4", "masked")])
def test_forward(act, fmt, layout):
    announce("layer", act, fmt, layout)
    kw = dict(fp8=fmt != "bf16", layout=layout, weight_format=None if fmt in ("bf16", "fp8") else fmt)
    c = Case(act=act, **kw)
    for name in ("x_buf", "act", "y", "out", "logits", "shared_act", "src2dst"):
        getattr(c.layer, name).view(torch.uint8).fill_(0xFF)
    out = c.layer(c.x)
    torch.cuda.synchronize()
    ids = c.layer.topk_ids
    check_routing(c, ids)
    want = c.exact(c.leaves(), ids).detach()
    # roundings to bf16 of activation, product, combine and residual sum: each 2^-9 of the
    # value on average, and less than one of the output's in norm each.  FP8: activations
    # and weights within 2^-4 each, 2.6% on average, twice; 4-bit weights 2^-2, 12% on
    # average, twice, of the routed part
    assert off(out, want) < {"bf16": 4 * 2 ** -9, "fp8": 0.08, "mxfp8": 0.08, "mxfp4": 0.25}[fmt]
    # FP8 or not, the shared expert and the router are BF16
    if layout == "compact" and fmt == "bf16":
        apart = c.layer(c.x, c.layer.router_logits(c.x).clone())
        assert torch.equal(apart, out)


@pytest.mark.parametrize("layout", ["compact", "masked"])
def test_a_token_does_not_depend_on_its_batch(layout):
    whole = Case(T=300, layout=layout)
    ref = whole.layer(whole.x).clone()
    for T in (1, 7, 33, 64, 129):
        part = Case(T=T, layout=layout)
        for n in ("w13", "w2"):
            getattr(part.layer, n).copy_(getattr(whole.layer, n))
        part.layer.set_bias(whole.b13, whole.b2)
        part.layer.set_router(whole.gate, whole.gate_bias)
        part.layer.set_shared(whole.s13, whole.s2)
        assert torch.equal(part.layer(whole.x[:T].contiguous()), ref[:T]), T


def test_the_layer_without_extras_is_as_before():
    a = Case(act="silu_mul", bias=False, router=False, S=0, layout="compact")
    logits = torch.randn(200, 16, device=DEV)
    out = a.layer(a.x, logits).clone()
    assert a.layer.plain and a.layer.b13 is None and not hasattr(a.layer, "shared_act")
    from scatter_grouped_gemm_amd import _lib as L
    y, act = torch.empty_like(a.layer.y), torch.empty_like(a.layer.act)
    L.grouped_gemm_contig_silu(False, a.layer.x_buf, None, a.layer.w13, None, act, a.layer.m_indices)
    L.grouped_gemm_contig(False, act, None, a.layer.w2, None, y, a.layer.m_indices)
    again = torch.empty_like(out)
    L.moe_combine(y, a.layer.src2dst, a.layer.topk_weights, again)
    assert torch.equal(out, again)


GRADS = dict(w13="dw13", w2="dw2", b13="db13", b2="db2", gate="dgate", gate_bias="dgate_bias", s13="dshared_w13", s2="dshared_w2")


def check_grads(c, dx, p):
    for n, leaf in p.items():
        got = dx if n == "x" else getattr(c.layer, GRADS[n])
        if n in ("gate", "gate_bias"):
            assert (got[c.E:] == 0).all()
            got = got[:c.E]
        # roundings to bf16 of the activations, the gradients on the way and the result: up
        # to five of 2^-9 on average in each chain; the router's passes through differences
        # of weighted sums (softmax), which cancel by up to a few times
        assert off(got, leaf.grad) < (0.04 if n in ("gate", "gate_bias") else 0.012), (n, off(got, leaf.grad))


@pytest.mark.parametrize("act", GATED)
@pytest.mark.parametrize("grad_dtype", [BF, F32])
def test_backward(act, grad_dtype):
    announce("layer backward", act, grad_dtype)
    c = Case(act=act, train=True, grad_dtype=grad_dtype)
    c.layer(c.x)
    dx, dlogits = c.layer.backward(c.dout)
    torch.cuda.synchronize()
    p = c.leaves()
    c.exact(p, c.layer.topk_ids).backward(c.dout.double())
    check_grads(c, dx, p)
    assert dlogits.shape == (200, 16)
    first = [g.clone() for g in c.layer.gradients()]
    c.layer(c.x)
    c.layer.backward(c.dout, accumulate=True)
    for a, b in zip(first, c.layer.gradients()):
        # doubled exactly, but for the sum's own rounding
        assert ((b.double() - 2 * a.double()).abs() <= 2.0 ** -7 * a.double().abs() + 1e-30).all() if grad_dtype is BF else \
            torch.allclose(b, 2 * a, rtol=1e-6, atol=0)


@pytest.mark.parametrize("kw", [dict(S=0), dict(router=False), dict(bias=False), dict(bias=False, act="silu_mul"),
                                dict(router=False, S=0)])
def test_backward_of_parts(kw):
    announce("layer backward", kw)
    c = Case(train=True, **kw)
    gate = c.gate
    if gate is None:          # routing from outside
        c.gate, c.gate_bias = torch.randn(16, 256, device=DEV), torch.zeros(16, device=DEV)
        logits = (c.x.double() @ c.gate.double().t()).float()
        c.layer(c.x, logits)
        p = {n: t for n, t in c.leaves().items() if not n.startswith("gate")}
        fixed = c.leaves()
        q = dict(p, gate=fixed["gate"].detach(), gate_bias=fixed["gate_bias"].detach())
        # the logits are an input of their own
        lg = logits.double().requires_grad_()
        dx, dlogits = c.layer.backward(c.dout)
        ids = c.layer.topk_ids.long()
        top = torch.softmax(torch.gather(lg, 1, ids), 1)
        out = torch.zeros_like(p["x"])
        for e in range(16):
            t, j = torch.nonzero(ids == e, as_tuple=True)
            pre = p["x"][t] @ p["w13"][e].t() + p["b13"][e]
            out = out.index_add(0, t, top[t, j][:, None] * (activation(pre, c.act) @ p["w2"][e].t() + p["b2"][e]))
        if "s13" in p:
            out = out + activation(p["x"] @ p["s13"].t(), c.act) @ p["s2"].t()
        out.backward(c.dout.double())
        check_grads(c, dx, p)
        assert off(dlogits, lg.grad) < 0.04
        return
    c.layer(c.x)
    dx, _ = c.layer.backward(c.dout)
    p = c.leaves()
    c.exact(p, c.layer.topk_ids).backward(c.dout.double())
    check_grads(c, dx, p)


def test_backward_of_a_share_and_of_given_ids():
    c = Case(train=True, E=16, El=5, start=6)
    c.layer(c.x)
    dx, _ = c.layer.backward(c.dout)
    p = c.leaves()
    c.exact(p, c.layer.topk_ids).backward(c.dout.double())
    check_grads(c, dx, p)
    before = c.layer.dgate.clone()
    ids, tw = c.layer.topk_ids.clone(), c.layer.topk_weights.clone()
    c.layer(c.x, topk_ids=ids, topk_weights=tw)
    dx2, dtw = c.layer.backward(c.dout)
    assert dtw.shape == (200, 4) and torch.equal(c.layer.dgate, before)


def test_logits_given_to_a_layer_with_a_router():
    """The router's gradients stay, dlogits come in rows of E, as without a router."""
    a, b = Case(train=True, S=0), Case(train=True, S=0, router=False)
    logits = torch.randn(200, 16, device=DEV)
    for n in ("w13", "w2"):
        getattr(b.layer, n).copy_(getattr(a.layer, n))
    b.layer.set_bias(a.b13, a.b2)
    assert torch.equal(a.layer(a.x, logits), b.layer(a.x, logits))
    (dx, dl), (dx2, dl2) = a.layer.backward(a.dout), b.layer.backward(a.dout)
    assert dl.is_contiguous() and torch.equal(dx, dx2) and torch.equal(dl, dl2)
    assert (a.layer.dgate == 0).all()


def test_training_steps_captured():
    """Forward, backward and AdamW step of the whole layer in a graph, against the same steps run eagerly."""
    def make():
        c = Case(train=True, T=130, seed=3)
        return c, c.layer.optimizer(lr=1e-2, weight_decay=0.1)
    a, oa = make()
    b, ob = make()
    assert len(b.layer.parameters()) == len(b.layer.gradients()) == 8

    def step(c, o, x):
        out = c.layer(x)
        c.layer.backward(c.dout)
        o.step()
        return out
    x = b.x.clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b.layer(x)                       # warm, without a step
        b.layer.backward(b.dout)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step(b, ob, x)
    for i in range(4):
        new = torch.randn(130, 256, generator=torch.Generator().manual_seed(i)).to(BF).to(DEV)
        x.copy_(new)
        g.replay()
        torch.cuda.synchronize()
        want = step(a, oa, new)
        assert torch.equal(out, want), i
        for p, q in zip(a.layer.parameters(), b.layer.parameters()):
            assert torch.equal(p, q), i
    assert (b.layer.gate[16:] == 0).all()


def test_two_layers_on_two_streams():
    a, b = Case(seed=1, train=True), Case(seed=2, train=True)
    want = []
    for c in (a, b):
        out = c.layer(c.x).clone()
        dx = c.layer.backward(c.dout)[0].clone()
        want.append((out, dx, [g.clone() for g in c.layer.gradients()]))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for c, s in zip((a, b), streams):
        with torch.cuda.stream(s):
            out = c.layer(c.x)
            got.append((out, c.layer.backward(c.dout)[0], c.layer.gradients()))
    torch.cuda.synchronize()
    for (o, d, gs), (o2, d2, gs2) in zip(want, got):
        assert torch.equal(o, o2) and torch.equal(d, d2) and all(torch.equal(p, q) for p, q in zip(gs, gs2))


def test_refusals():
    kw = dict(hidden=256, intermediate=256, num_experts=8, top_k=2, max_tokens=16, device=DEV)
    for bad in (dict(activation="gelu"), dict(activation="none"), dict(router_bias=True), dict(shared_intermediate=100)):
        with pytest.raises(ValueError):
            MoELayer(**kw, **bad)
    x = torch.zeros(16, 256, dtype=BF, device=DEV)
    layer = MoELayer(**kw, router=True, shared_intermediate=128, expert_bias=True, train=True)
    layer.set_weights(torch.zeros(8, 512, 256, dtype=BF, device=DEV), torch.zeros(8, 256, 256, dtype=BF, device=DEV))
    with pytest.raises(ValueError, match="set_bias"):
        layer(x)
    layer.set_bias(torch.zeros(8, 512), torch.zeros(8, 256))
    with pytest.raises(ValueError, match="set_router"):
        layer.optimizer()
    with pytest.raises(ValueError, match="another router"):
        layer.set_router(torch.zeros(8, 256), torch.zeros(8))
    layer.set_router(torch.zeros(8, 256))
    with pytest.raises(ValueError, match="set_shared"):
        layer(x)
    plain = MoELayer(**kw)
    for call in (lambda: plain.set_bias(None, None), lambda: plain.set_router(None), lambda: plain.set_shared(None, None),
                 lambda: plain(x)):
        with pytest.raises(ValueError):
            call()
