"""Calls of the training operators that their documentation allows or that have to
be refused: parameters that require gradients, tensors named twice, sizes past what
a launch can hold (no GPU needed)."""
import ctypes

import pytest
import torch

from scatter_grouped_gemm_amd import AdamW, MoELayer
from scatter_grouped_gemm_amd import _lib as L

P = 4096  # non-null, 16-byte aligned, never dereferenced


def test_adamw_takes_parameters_that_require_gradients():
    p = torch.nn.Parameter(torch.randn(130).bfloat16())
    o = AdamW([p], [torch.zeros(130).bfloat16()], state_bits=8)
    assert not o.master.requires_grad and o.master.grad_fn is None
    assert torch.equal(o.master[:130], p.detach().float())
    o.reset_master()
    saved = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in o.state_dict().items()}
    saved["master"] += 1
    o.load_state_dict(saved)
    assert torch.equal(p.detach(), saved["master"][:130].bfloat16()) and p.is_leaf and p.requires_grad


def test_adamw_refuses_parameters_that_share_memory():
    a, g = torch.zeros(256), torch.zeros(256)
    for params in ([a, a], [a, a[:64]], [a[128:], a[:132]]):
        with pytest.raises(ValueError, match="share"):
            AdamW(params, [torch.zeros_like(p) for p in params])
    AdamW([a[:128], a[128:]], [g[:128], g[:128]])            # neighbours; gradients may be shared
    AdamW([a[:0], a[:0], a], [g[:0], g[:0], g])              # nothing to share


def test_adamw_state_of_another_kind_is_a_value_error():
    o = AdamW([torch.zeros(130)], [torch.zeros(130)])
    with pytest.raises(ValueError):
        o.load_state_dict({})
    with pytest.raises(ValueError):
        o.load_state_dict({k: v for k, v in o.state_dict().items() if k != "offsets"})


def test_sizes_past_a_launch_are_refused():
    lib = L.lib()
    c = lambda T=4, k=2, H=256: lib.moe_combine_bwd(P, P, 10, P, P, T, k, H, P, P, None)  # noqa: E731
    s = lambda T=4, k=2, H=256: lib.moe_scatter_bwd(P, 10, P, T, k, H, P, None)  # noqa: E731
    for f in (c, s):
        for kw in (dict(H=(1 << 30) + 8), dict(H=2147483640), dict(T=1 << 26, H=512), dict(T=1 << 22, H=8192)):
            assert f(**kw) == L.MOE_EUNSUPPORTED, (f, kw)
    assert lib.moe_route_topk_bwd(P, P, P, 1 << 26, 8, 2, P, None) == L.MOE_EUNSUPPORTED
    assert lib.silu_and_mul_bwd(P, P, 1 << 26, 128, None, None, 0, P, P, None) == L.MOE_EUNSUPPORTED


def test_gradients_are_allocated_once():
    """An optimizer that holds them would go on reading the old ones."""
    layer = MoELayer(num_experts=4, top_k=2, hidden=128, intermediate=128, max_tokens=8, train=True, device="cpu")
    layer.allocate_grads()
    a, b = layer.dw13, layer.dw2
    a.fill_(1)
    b.fill_(1)
    layer.allocate_grads()
    assert layer.dw13 is a and layer.dw2 is b and not a.any() and not b.any()


def test_adamw_refuses_an_eps_that_is_zero_in_fp32():
    for eps in (1e-46, 1e-300, float("nan"), -1e-8):
        with pytest.raises(ValueError, match="eps"):
            AdamW([torch.zeros(8)], [torch.zeros(8)], eps=eps)
    AdamW([torch.zeros(8)], [torch.zeros(8)], eps=1e-45)     # the smallest fp32 number


def test_a_forward_that_fails_leaves_nothing_for_backward():
    """Its first calls have overwritten what the forward before it had left."""
    layer = MoELayer(num_experts=4, top_k=2, hidden=128, intermediate=128, max_tokens=8, train=True, device="cpu")
    before = layer._saved = (8, layer.topk_ids, layer.topk_weights, True)
    with pytest.raises(ValueError, match="capacity"):         # refused before anything is written
        layer(torch.zeros(9, 128, dtype=torch.bfloat16), torch.zeros(9, 4))
    assert layer._saved is before
    with pytest.raises(AssertionError):                       # not on the device
        layer(torch.zeros(8, 128, dtype=torch.bfloat16), torch.zeros(8, 4))
    with pytest.raises(ValueError, match="forward"):
        layer.backward(torch.zeros(8, 128, dtype=torch.bfloat16))


def test_a_layer_that_backward_could_not_serve_is_refused():
    """Past 8160 blocks of 128 rows forward still runs, the gradient products do not;
    nor do they with other sizes past their limits."""
    make = lambda train=True, **kw: MoELayer(**{**dict(num_experts=4, top_k=2, hidden=128, intermediate=128,  # noqa: E731
                                                       max_tokens=8, train=train, device="meta"), **kw})
    most = 8160 * 128
    rows = lambda T: L.moe_compact_rows_bound(2 * T, 4, 128)  # noqa: E731
    T = max(t for t in range(most // 2 - 400, most // 2) if rows(t) <= most)
    assert rows(T + 64) > most
    assert make(max_tokens=T).rows <= most
    for kw in (dict(max_tokens=T + 64), dict(hidden=4194304 + 128), dict(intermediate=4194304), dict(hidden=192),
               dict(num_experts=1025)):
        with pytest.raises(ValueError, match="gradient products"):
            make(**kw)
    assert make(train=False, layout="compact", max_tokens=T + 64).rows > most
    for sizes, want in [((0, 128, 128, 1), True), ((most, 128, 128, 1024), True), ((most + 1, 128, 128, 1), False),
                        ((128, 64, 128, 1), False), ((128, 128, 128, 0), False), ((1 << 40, 128, 128, 1), False),
                        ((-1, 128, 128, 1), False)]:
        assert L.grouped_gemm_grads_supported(*sizes) is want, sizes


def test_adamw_state_holds_the_seed():
    make = lambda seed: AdamW([torch.zeros(130)], [torch.zeros(130)], state_bits=8, seed=seed)  # noqa: E731
    saved = make(5).state_dict()
    assert saved["seed"] == 5
    o = make(7)
    with pytest.raises(ValueError):
        o.load_state_dict({**saved, "state_bits": 32})
    with pytest.raises(ValueError, match="seed"):
        o.load_state_dict({**saved, "seed": None})
    assert o.seed == 7                                        # nothing was taken over
    o.load_state_dict(saved)
    assert o.seed == 5
    o = make(7)
    o.load_state_dict({k: v for k, v in saved.items() if k != "seed"})   # saved without one
    assert o.seed == 7


@pytest.mark.parametrize("numel", [(1 << 63) - 1, (1 << 63) - 2047, 1 << 62, (1 << 31) * 2048, ((1 << 31) - 1) * 2048 + 1])
def test_adamw_plan_refuses_tensors_past_its_pieces(numel):
    """Also where rounding such a size up would pass 64 bits."""
    t = dict(param=P, grad=P, m=P, v=P, param_dtype=L.MOE_DTYPE_FP32, grad_dtype=L.MOE_DTYPE_FP32, state_bits=32)
    for arr in ([dict(numel=numel)], [dict(numel=5000), dict(numel=numel)], [dict(numel=((1 << 31) - 1) * 2048), dict(numel=1)]):
        ts = (L.AdamwTensor * len(arr))(*[L.AdamwTensor(**t, **a) for a in arr])
        assert L.lib().moe_adamw_plan_bytes(ts, len(arr)) == 0
        assert L.lib().moe_adamw_plan(ts, len(arr), None, 1 << 40) == L.MOE_EUNSUPPORTED


def test_weights_of_a_training_layer_are_allocated_once():
    """An optimizer that holds them would go on updating the old ones."""
    make = lambda train: MoELayer(num_experts=4, top_k=2, hidden=128, intermediate=128, max_tokens=8, train=train, device="cpu")  # noqa: E731
    layer = make(True)
    layer.set_weights(torch.ones(4, 256, 128), torch.ones(4, 128, 128))
    opt = layer.optimizer()
    layer.allocate_weights()
    assert opt.params[0] is layer.w13 and opt.params[1] is layer.w2 and (layer.w13 == 1).all()
    other = make(False)
    other.allocate_weights()
    w13 = other.w13
    other.allocate_weights()
    assert other.w13 is not w13


def test_adamw_refuses_gradients_in_a_parameters_memory():
    """One workgroup would read what another writes."""
    a, b = torch.zeros(512), torch.zeros(512)
    for params, grads in [([a], [a.view(torch.bfloat16)[:512]]), ([a[:256]], [a[128:384]]), ([a[:256], b[:256]], [b[:256], b[256:]]),
                          ([a[:4], b, a[256:]], [a[64:68], b.clone(), a[128:384]]), ([a[:256]], [a[252:508]])]:
        with pytest.raises(ValueError, match="share"):
            AdamW(params, grads)
    AdamW([a[:256]], [a[256:]])                               # beside it
    AdamW([a[:4], b, a[256:]], [a[64:68], b.clone(), b[:256].clone()])
    AdamW([a[:0], a], [a[:0], b])
    AdamW([a], [a])                                           # read and written by the same lanes


@pytest.mark.parametrize("beta2,steps", [(0.95, 300), (0.999, 2000)])
def test_the_8bit_second_moment_over_many_steps(beta2, steps):
    """The decoded v against the formula in 64 bits, with the format's rounding in plain
    torch: the root's expectation is kept, so v gains the root's variance f (1 - f) u^2 at
    each step.  With d = |v' - v| / (r' + r) the way that a step moves the root, r being a
    code, f (1 - f) u <= d, and u <= r' / 8: all in all at most an eighth of |g^2 - v|."""
    from perf.operators import GROUP, _rounded
    gen = torch.Generator().manual_seed(3)
    n = 64 * GROUP

    def held(v):
        bits = torch.randint(0, 65536, (n,), generator=gen)
        codes, e = _rounded(v.sqrt().float(), bits, keep=True)
        unit = torch.exp2(e.double() - 127).repeat_interleave(GROUP)
        return codes.view(torch.float8_e4m3fn).double() * unit, unit

    v, mean = held(torch.ones(n, dtype=torch.float64))[0] ** 2, torch.ones(n, dtype=torch.float64)
    gained = noise = 0.0                  # of the mean over the elements: expectation and variance
    most = 0.0
    for _ in range(steps):
        g2 = torch.randn(n, generator=gen, dtype=torch.float64) ** 2
        most = max(most, (g2 - v).abs().mean().item())
        want = beta2 * v + (1 - beta2) * g2
        root = want.sqrt()
        got, scale = held(want)
        unit = torch.exp2(torch.floor(torch.log2(root / scale)).clamp(min=-6) - 3) * scale
        f = root / unit - torch.floor(root / unit)
        spread = f * (1 - f) * unit ** 2
        gained = beta2 * gained + spread.mean().item()
        noise = beta2 ** 2 * noise + ((2 * root + unit) ** 2 * spread).mean().item() / n
        v, mean = got ** 2, beta2 * mean + (1 - beta2) * g2
    over = (v.mean() - mean.mean()).item()
    # six standard deviations; 16 random bits carry up to 2^-16 too seldom, which takes
    # 2 r u 2^-16 <= v 2^-18 at a step, fp32 some v 2^-22; the mean of v is below 1.25
    assert abs(over - gained) <= 6 * noise ** 0.5 + steps * 1.25 * (2.0 ** -18 + 2.0 ** -22)
    assert 0 < gained <= most / 8
