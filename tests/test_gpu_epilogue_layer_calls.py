"""Calls of the layer with a router, a shared expert and biases that a program makes
around it: on its own output, in shares, with batches of other sizes."""
import pytest
import torch

from scatter_grouped_gemm_amd import _lib as L
from epilogue_util import activation
from gpu_util import DEV, announce
from test_gpu_epilogue_layer import Case, check_grads, off

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("layout", ["compact", "masked"])
def test_a_layer_on_its_own_output(layout):
    """x may be what the last forward returned: the same weights one after the other."""
    announce("own output", layout)
    c = Case(layout=layout)
    want = c.layer(c.layer(c.x).clone()).clone()
    got = c.layer(c.layer(c.x))
    assert torch.equal(got, want)


@pytest.mark.parametrize("kw", [dict(), dict(S=0), dict(router=False)])
def test_training_on_its_own_output_is_refused_where_backward_reads_x(kw):
    c = Case(train=True, **kw)
    give = () if c.gate is not None else (torch.randn(200, 16, device=DEV),)
    out = c.layer(c.x, *give)
    with pytest.raises(ValueError, match="own output"):
        c.layer(out, *give)
    with pytest.raises(ValueError, match="forward"):       # nothing is left for backward
        c.layer.backward(c.dout)
    c.layer(out.clone(), *give)
    c.layer.backward(c.dout)


def test_training_on_its_own_output_without_extras():
    c = Case(train=True, S=0, router=False, bias=False, act="silu_mul")
    logits = torch.randn(200, 16, device=DEV)
    first = c.layer(c.x, logits).clone()
    want = c.layer(first, logits).clone()
    dx = c.layer.backward(c.dout)[0].clone()
    c.layer(c.x, logits)
    assert torch.equal(c.layer(c.layer.out, logits), want)
    assert torch.equal(c.layer.backward(c.dout)[0], dx)


def test_shares_add_up_to_the_whole():
    """Two layers with a part of the experts each and the same router, one of them with the
    shared expert: outputs, dx, dlogits and the router's gradients are parts of the whole's."""
    whole = Case(train=True, grad_dtype=F32)
    shares = []
    for start, El, S in ((0, 5, 256), (5, 11, 0)):
        c = Case(train=True, grad_dtype=F32, El=El, start=start, S=S)
        c.layer.set_weights(whole.w13[start:start + El], whole.w2[start:start + El])
        c.layer.set_bias(whole.b13[start:start + El], whole.b2[start:start + El])
        c.layer.set_router(whole.gate, whole.gate_bias)
        if S:
            c.layer.set_shared(whole.s13, whole.s2)
        shares.append(c)
    got = []
    for c in shares:
        out = c.layer(whole.x)
        dx, dlogits = c.layer.backward(whole.dout)
        got.append(dict(out=out, dx=dx, dlogits=dlogits, dgate=c.layer.dgate[:16], dgate_bias=c.layer.dgate_bias[:16]))
    ids = shares[0].layer.topk_ids
    assert torch.equal(ids, shares[1].layer.topk_ids)
    p = whole.leaves()
    out = whole.exact(p, ids)
    out.backward(whole.dout.double())
    want = dict(out=out.detach(), dx=p["x"].grad, dgate=p["gate"].grad, dgate_bias=p["gate_bias"].grad)
    # dlogits: those of the same weights in one layer
    whole.layer(whole.x)
    want["dlogits"] = whole.layer.backward(whole.dout)[1].double()
    for n, w in want.items():
        a, b = (g[n].double() for g in got)
        # the whole's bounds (4 roundings forward, 5 on dx's way, the router's differences), each
        # relative to the part that was rounded; two layers' dlogits are compared with each other
        tol = {"out": 4 * 2 ** -9, "dx": 0.012}.get(n, 0.04) * (2 if n == "dlogits" else 1)
        assert (a + b - w).norm() <= tol * (a.norm() + b.norm()), n
        assert a.norm() > 0.1 * w.norm() and b.norm() > 0.1 * w.norm(), n


def left(c, back):
    """Copies of what a step returned and left in the layer."""
    return [t.clone() for t in (c.layer.out[:len(back[0])], *back, *c.layer.gradients())]


@pytest.mark.parametrize("own", ["router", "logits", "ids"])
@pytest.mark.parametrize("T", [77, 33, 129])
def test_a_batch_after_a_longer_one(own, T):
    """Nothing of a longer batch before, or of what the buffers held, is in a shorter one's
    output and gradients."""
    announce("shorter batch", own, T)
    c, fresh = Case(train=True), Case(train=True)
    for n in ("x_buf", "gateup", "act", "y", "out", "logits", "shared_act", "shared_pre", "shared_dact", "dy", "dx", "dx_parts",
              "dlogits", "dlogits16", "dtopk_weights", "src2dst"):
        getattr(fresh.layer, n).view(torch.uint8).fill_(0xFF)
    c.layer(c.x)
    c.layer.backward(c.dout)
    found = []
    for case in (c, fresh):
        case.x, case.dout = case.x[:T].contiguous(), case.dout[:T].contiguous()
        logits = (case.x.double() @ case.gate.double().t() + case.gate_bias.double()).float()
        if own == "ids":
            weights, ids = torch.topk(torch.softmax(logits, 1), case.k)
            ids, weights = ids.int(), (weights / weights.sum(1, keepdim=True)).contiguous()
            case.layer.topk_ids[:T] = ids
            case.layer(case.x, topk_ids=ids, topk_weights=weights)
        else:
            case.layer(case.x, *(() if own == "router" else (logits,)))
        if own != "router":                         # what a backward of given logits leaves alone
            case.layer.allocate_grads()
        found.append(left(case, case.layer.backward(case.dout)))
    assert all(torch.equal(a, b) for a, b in zip(*found))
    p = c.leaves()
    out = c.exact(p, c.layer.topk_ids[:T])
    out.backward(c.dout.double())
    assert off(c.layer.out[:T], out.detach()) < 4 * 2 ** -9
    if own == "router":
        check_grads(c, c.layer.dx[:T], p)
    else:                                           # the router's part of dx is not in it
        q = {n: t for n, t in c.leaves().items() if not n.startswith("gate")}
        check_grads(c, c.layer.dx[:T], experts_alone(c, q))
        assert (c.layer.dgate == 0).all() and (c.layer.dgate_bias == 0).all()


def experts_alone(c, q):
    """c's leaves without the router's, with the gradients of a routing that does not depend on x."""
    fixed = Case.leaves(c)
    ids = c.layer.topk_ids[:len(c.x)]
    full = dict(q, gate=fixed["gate"].detach(), gate_bias=fixed["gate_bias"].detach())
    frozen = q["x"].detach() @ full["gate"].t() + full["gate_bias"]
    top = torch.softmax(torch.gather(frozen, 1, ids.long()), 1)
    out = torch.zeros_like(q["x"])
    for e in range(c.E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        pre = q["x"][t] @ q["w13"][e].t() + q["b13"][e]
        out = out.index_add(0, t, top[t, j][:, None] * (activation(pre, c.act) @ q["w2"][e].t() + q["b2"][e]))
    out = out + activation(q["x"] @ q["s13"].t(), c.act) @ q["s2"].t()
    out.backward(c.dout.double())
    return q


@pytest.mark.parametrize("kw", [dict(), dict(router=False), dict(S=0), dict(bias=False), dict(router=False, S=0)])
def test_training_on_a_batch_without_tokens(kw):
    """A share of a batch may be empty: no gradient then, or (accumulate) the one before."""
    announce("no tokens", kw)
    c = Case(train=True, **kw)
    give = () if c.gate is not None else (torch.randn(200, 16, device=DEV),)
    c.layer(c.x, *give)
    c.layer.backward(c.dout)
    before = [g.clone() for g in c.layer.gradients()]
    for accumulate in (True, False):
        out = c.layer(c.x[:0], *(t[:0] for t in give))
        dx, dlogits = c.layer.backward(c.dout[:0], accumulate=accumulate)
        assert out.shape == dx.shape == (0, 256) and dlogits.shape == (0, 16)
        for g, b in zip(c.layer.gradients(), before):
            assert torch.equal(g, b) if accumulate else (g == 0).all()


@pytest.mark.parametrize("act", ["none", "gelu", "swiglu_clamp"])
@pytest.mark.parametrize("G", [1, 3])
def test_bias_gradients_of_no_rows(act, G):
    """Compact and dense layouts of no rows: 0, or what is there."""
    N = 256
    none = lambda n: torch.empty(0, n, dtype=BF, device=DEV)  # noqa: E731
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device=DEV)  # noqa: E731
    kw = {} if G == 1 else dict(m_indices=i32(0), expert_start_loc=i32(G), num_valid=i32(G))
    for dtype in (F32, BF):
        db = torch.full((G, N), 3.0, dtype=dtype, device=DEV)
        for accumulate, want in ((True, 3.0), (False, 0.0)):
            L.moe_act_bwd(none(N), none(N // 2 if act == "swiglu_clamp" else N), none(N), act, dbias=db, accumulate=accumulate, **kw)
            assert (db == want).all()
    L.moe_act_bwd(none(N), none(N // 2 if act == "swiglu_clamp" else N), none(N), act, m_indices=kw.get("m_indices"))
