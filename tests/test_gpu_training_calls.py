"""Calls that the training operators' documentation allows and their single tests
do not make."""
import pytest
import torch

from scatter_grouped_gemm_amd import AdamW
from scatter_grouped_gemm_amd import _lib as L
from gpu_util import DEV, announce
from test_gpu_training import BF, F32, U32, _make, gen, randn, same_bits, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
def test_a_plan_cut_short_updates_nothing(bits):
    announce("adamw plan cut", bits)
    p = randn(1, 5000, dtype=F32).to(DEV)
    before = p.clone()
    o = AdamW([p], [torch.ones_like(p)], state_bits=bits)
    for cut in (8, 16, 80):
        L.moe_adamw_step(o._plan[:-cut].contiguous(), o.lr, o._counter, 0.9, 0.95, 1e-8)
    torch.cuda.synchronize()
    assert same_bits(p, before) and not o.m.any() and not o.v.any()
    o.step()
    assert not same_bits(p, before)


def test_adamw_with_parameters_that_require_gradients():
    announce("adamw parameters")
    a = randn(1, 700).to(DEV)
    b = torch.nn.Parameter(a.clone())
    g = randn(2, 700).to(DEV)
    x, y = AdamW([a], [g], state_bits=8), AdamW([b], [g], state_bits=8)
    for o in (x, y, x, y):
        o.step()
    assert same_bits(a, b.detach()) and same_bits(x.m, y.m) and not y.master.requires_grad


def test_a_captured_backward_needs_its_gradients():
    announce("captured backward")
    layer, x, logits, _, _ = _make(32, 256, 128, 8, 2)
    xd, ld, dout = x.to(DEV), logits.to(DEV), randn(5, 32, 256).to(DEV)
    layer(xd, ld)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        torch.zeros(8, device=DEV)
        with pytest.raises(ValueError, match="allocate_grads"):
            layer.backward(dout)
    assert layer.dw13 is None
    layer.backward(dout)                                     # the forward is still there


def test_accumulating_over_replays_and_small_batches():
    """Forward and an accumulating fp32 backward captured once, replayed over
    batches: the sum of the batches' gradients, the same as eager calls."""
    announce("accumulate replays")
    T = 40
    batches = [(randn(40 + i, T, 256).to(DEV), torch.randn(T, 8, generator=gen(60 + i)).to(DEV)) for i in range(3)]
    dout = randn(5, T, 256).to(DEV)
    eager = _make(T, 256, 128, 8, 2, grad_dtype=F32)[0]
    for x, lg in batches:
        eager(x, lg)
        eager.backward(dout, accumulate=True)
    layer = _make(T, 256, 128, 8, 2, grad_dtype=F32)[0]
    layer.allocate_grads()
    sx, sl = batches[0][0].clone(), batches[0][1].clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer(sx, sl)
        layer.backward(dout, accumulate=True)
    layer.allocate_grads()
    for x, lg in batches:
        sx.copy_(x)
        sl.copy_(lg)
        graph.replay()
        torch.cuda.synchronize()
    assert layer.dw13.any() and same_bits(layer.dw13, eager.dw13) and same_bits(layer.dw2, eager.dw2)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-45, 1e-40, 1.5e-38, 1e-37])
def test_adamw_with_the_smallest_eps(eps, bits):
    """Weights without a gradient stay as they were, the others move by lr: the first
    step's m / (1 - b1) is the gradient and its root of v / (1 - b2) its magnitude."""
    announce("adamw eps", eps, bits)
    lr = 0.01
    w, g = randn(1, 6000, dtype=F32), randn(2, 6000, dtype=F32)
    g[::3] = 0
    g[2048:4096] = 0                                         # whole groups too
    p = w.to(DEV)
    AdamW([p], [g.to(DEV)], lr=lr, betas=(0.9, 0.99), eps=eps, state_bits=bits).step()
    assert same_bits(p.cpu()[g == 0], w[g == 0])
    # constants, products, root and quotient of a step as in the bound of the plain step's test
    within(p, w.double() - lr * torch.sign(g.double()), 3 * U32 * w.double().abs() + 24 * U32 * lr)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_plan_cut_short_counts_no_step(bits):
    """The step behind such calls is the first one: its bias corrections and random
    bits are those of a fresh optimizer."""
    announce("adamw plan cut counts", bits)
    p = randn(1, 5000, dtype=F32).to(DEV)
    q, g = p.clone(), randn(2, 5000, dtype=F32).to(DEV)
    o, fresh = AdamW([p], [g], state_bits=bits, seed=3), AdamW([q], [g], state_bits=bits, seed=3)
    whole = o._plan
    for cut in (8, 16, 80):
        L.moe_adamw_step(whole[:-cut].contiguous(), o.lr, o._counter, 0.9, 0.95, 1e-8)
    other = whole.clone()
    other[0] += 1                                            # not a plan
    L.moe_adamw_step(other, o.lr, o._counter, 0.9, 0.95, 1e-8)
    assert o._counter.tolist() == [0, 0]
    o.step(), fresh.step()
    assert o._counter.tolist() == [1, 0]
    assert same_bits(p, q) and same_bits(o.m, fresh.m) and same_bits(o.v, fresh.v)


def test_backward_behind_a_forward_that_failed_is_refused():
    announce("layer forward that fails")
    layer, x, logits, _, _ = _make(16, 256, 128, 4, 2)
    xd, dout = x.to(DEV), randn(1, 16, 256).to(DEV)
    layer(xd, logits.to(DEV))
    ids = torch.zeros(8, 2, dtype=torch.int32, device=DEV)
    with pytest.raises(AssertionError):                      # the weights are not on the device: fails in the combine
        layer(xd[:8], topk_ids=ids, topk_weights=torch.ones(8, 2))
    with pytest.raises(ValueError, match="forward"):
        layer.backward(dout)
    layer(xd, logits.to(DEV))
    layer.backward(dout)


def test_an_empty_batch_through_the_layer():
    """No rows behind a batch with rows: its gradients are zero, or what they were."""
    announce("layer empty batch")
    layer, x, logits, _, _ = _make(16, 256, 128, 4, 2)
    xd, ld, dout = x.to(DEV), logits.to(DEV), randn(1, 16, 256).to(DEV)
    layer(xd, ld)
    layer.backward(dout)
    had = layer.dw13.clone()
    layer(xd[:0], ld[:0])
    layer.backward(dout[:0], accumulate=True)
    assert had.any() and same_bits(layer.dw13, had)
    out = layer(xd[:0], ld[:0])
    dx, dl = layer.backward(dout[:0])
    assert out.shape == dx.shape == (0, 256) and dl.shape == (0, 4)
    assert not layer.dw13.any() and not layer.dw2.any()


def test_adamw_resumed_in_an_optimizer_of_another_seed():
    announce("adamw resume seed")
    g = randn(1, 5000).to(DEV)
    a = randn(2, 5000).to(DEV)
    b = torch.zeros_like(a)
    o, n = (AdamW([p], [g], lr=1e-2, state_bits=8, seed=seed) for p, seed in ((a, 4), (b, 9)))
    o.step(), o.step()
    n.load_state_dict({k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in o.state_dict().items()})
    o.step(), n.step()
    assert same_bits(a, b) and same_bits(o.m, n.m) and same_bits(o.v, n.v)


@pytest.mark.parametrize("beta2,steps", [(0.95, 150), (0.999, 400)])
def test_adamw_8bit_second_moment_over_many_steps(beta2, steps):
    """The kernel's v against the formula in 64 bits: above it by what the root's variance
    adds at each step, and by nothing else."""
    announce("adamw many steps", beta2, steps)
    n = 1 << 20
    g = torch.ones(n, device=DEV)
    o = AdamW([torch.zeros(n, device=DEV)], [g], betas=(0.9, beta2), state_bits=8, seed=2)
    scale_of = lambda: torch.exp2(o.v_scale.double() - 127).repeat_interleave(128)  # noqa: E731
    dg = torch.Generator(device=DEV)
    dg.manual_seed(4)
    v, mean = torch.zeros(n, dtype=torch.float64, device=DEV), torch.zeros(n, dtype=torch.float64, device=DEV)
    gained = noise = 0.0
    for _ in range(steps):
        g.normal_(generator=dg)
        o.step()
        g2 = g.double() ** 2
        want = beta2 * v + (1 - beta2) * g2
        root, scale = want.sqrt(), scale_of()
        unit = torch.exp2(torch.floor(torch.log2(root / scale)).clamp(min=-6) - 3) * scale
        f = root / unit - torch.floor(root / unit)
        spread = f * (1 - f) * unit ** 2
        gained = beta2 * gained + spread.mean().item()
        noise = beta2 ** 2 * noise + ((2 * root + unit) ** 2 * spread).mean().item() / n
        v, mean = (o.v.view(torch.float8_e4m3fn).double() * scale) ** 2, beta2 * mean + (1 - beta2) * g2
    over = (v.mean() - mean.mean()).item()
    # six standard deviations; 16 random bits carry up to 2^-16 too seldom, which takes
    # 2 r u 2^-16 <= v 2^-18 at a step, fp32 some v 2^-22; the mean of v is below 1.25
    assert 0 < gained and abs(over - gained) <= 6 * noise ** 0.5 + steps * 1.25 * (2.0 ** -18 + 2.0 ** -22)
