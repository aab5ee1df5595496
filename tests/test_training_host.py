"""The training calls on the host: arguments that must be refused before any
device work, the optimizer's plan, and the layer's refusals (no GPU needed)."""
import ctypes

import numpy as np
import pytest
import torch

from scatter_grouped_gemm_amd import AdamW, MoELayer
from scatter_grouped_gemm_amd import _lib as L

P = 4096  # non-null, 16-byte aligned, never dereferenced: every call here is refused or empty


def test_combine_and_scatter_gradients_refuse():
    lib = L.lib()
    c = lambda dout=P, Y=P, rows=10, s=P, w=P, T=4, k=2, H=256, dY=P, dw=P: lib.moe_combine_bwd(  # noqa: E731
        dout, Y, rows, s, w, T, k, H, dY, dw, None)
    for kw, want in [(dict(T=-1), 1), (dict(k=0), 1), (dict(k=33), 1), (dict(H=0), 1), (dict(rows=-1), 1),
                     (dict(H=100), 2), (dict(dout=None), 1), (dict(Y=None), 1), (dict(s=None), 1),
                     (dict(w=None), 1), (dict(dY=None), 1), (dict(dw=None), 1), (dict(dout=P + 8), 2),
                     (dict(Y=P + 2), 2), (dict(dY=P + 4), 2), (dict(T=0, dout=None, s=None), 0)]:
        assert c(**kw) == want, kw
    s = lambda dX=P, rows=10, sd=P, T=4, k=2, H=256, dx=P: lib.moe_scatter_bwd(dX, rows, sd, T, k, H, dx, None)  # noqa: E731
    for kw, want in [(dict(T=-1), 1), (dict(k=33), 1), (dict(H=12), 2), (dict(dX=None), 1), (dict(sd=None), 1),
                     (dict(dx=None), 1), (dict(dx=P + 2), 2), (dict(dX=P + 8), 2), (dict(rows=-2), 1), (dict(T=0), 0)]:
        assert s(**kw) == want, kw
    r = lambda i=P, w=P, d=P, T=4, E=8, k=2, o=P: lib.moe_route_topk_bwd(i, w, d, T, E, k, o, None)  # noqa: E731
    for kw, want in [(dict(E=0), 1), (dict(E=1025), 1), (dict(k=9), 1), (dict(i=None), 1), (dict(w=None), 1),
                     (dict(d=None), 1), (dict(o=None), 1), (dict(T=-1), 1), (dict(T=0, o=None), 0)]:
        assert r(**kw) == want, kw


def test_silu_gradient_refuses():
    lib = L.lib()
    c = lambda gu=P, da=P, M=16, I=128, mi=None, mm=None, mx=0, dg=P, a=P: lib.silu_and_mul_bwd(  # noqa: E731
        gu, da, M, I, mi, mm, mx, dg, a, None)
    for kw, want in [(dict(M=-1), 1), (dict(I=0), 1), (dict(I=100), 2), (dict(mi=P, mm=P, mx=8), 1),
                     (dict(mm=P, mx=0), 1), (dict(mm=P, mx=5), 1), (dict(gu=None), 1), (dict(da=None), 1),
                     (dict(dg=None), 1), (dict(a=P + 2), 2), (dict(dg=P + 8), 2), (dict(I=1 << 27), 2), (dict(M=0), 0)]:
        assert c(**kw) == want, kw


def test_product_gradients_refuse():
    lib = L.lib()
    d = lambda c=P, b=P, a=P, m=P, M=256, N=256, K=256, G=2: lib.grouped_gemm_contig_dgrad(  # noqa: E731
        c, b, a, m, M, N, K, G, None)
    w = lambda c=P, a=P, s=P, n=P, dt=0, acc=0, b=P, M=256, N=256, K=256, G=2: lib.grouped_gemm_contig_wgrad(  # noqa: E731
        c, a, s, n, dt, acc, b, M, N, K, G, None)
    for f in (d, w):
        for kw, want in [(dict(M=-1), 1), (dict(N=0), 1), (dict(K=-128), 1), (dict(G=-1), 1), (dict(N=200), 2),
                         (dict(K=64), 2), (dict(N=8388608), 2), (dict(K=8388608), 2), (dict(M=8160 * 128 + 1), 2),
                         (dict(N=1 << 22, K=1 << 22, G=1024), 2),
                         (dict(G=1025), 2), (dict(c=None), 1), (dict(a=None), 1), (dict(b=None), 1),
                         (dict(a=P + 8), 2), (dict(b=P + 2), 2), (dict(c=P + 4), 2), (dict(G=0), 0)]:
            assert f(**kw) == want, (f, kw)
    assert d(M=0) == 0 and d(m=None) == 1
    for kw, want in [(dict(s=None), 1), (dict(n=None), 1), (dict(dt=1), 2), (dict(dt=2), 2), (dict(M=0, b=None), 1)]:
        assert w(**kw) == want, kw


def _tensor(**kw):
    f = dict(param=P, master=P, grad=P, m=P, v=P, m_scale=P, v_scale=P, numel=5000, weight_decay=0.1,
             param_dtype=L.MOE_DTYPE_BF16, grad_dtype=L.MOE_DTYPE_FP32, state_bits=8)
    f.update(kw)
    return L.AdamwTensor(**f)


def test_adamw_plan_lists_every_chunk_once():
    sizes = [5000, 0, 1, 2048, 2049]
    ts = [_tensor(numel=n) for n in sizes]
    plan = L.moe_adamw_plan(ts).numpy()
    chunks = plan[16 + 80 * len(ts):].view(np.int32).reshape(-1, 2)
    want = [(i, c) for i, n in enumerate(sizes) for c in range(-(-n // 2048))]
    assert [tuple(r) for r in chunks.tolist()] == want
    assert plan[8:16].view(np.int32).tolist() == [len(ts), len(want)]
    arr = (L.AdamwTensor * len(ts))(*ts)
    n = L.lib().moe_adamw_plan_bytes(arr, len(ts))
    assert n == len(plan)
    buf = (ctypes.c_uint8 * n)()
    assert L.lib().moe_adamw_plan(arr, len(ts), buf, n - 1) == L.MOE_ECAPACITY
    assert L.lib().moe_adamw_plan(arr, len(ts), None, n) == L.MOE_EINVAL


@pytest.mark.parametrize("bad,want", [
    (dict(numel=-1), 1), (dict(param=None), 1), (dict(grad=None), 1), (dict(m=None), 1), (dict(v=None), 1),
    (dict(master=None), 1), (dict(m_scale=None), 1), (dict(v_scale=None), 1), (dict(param_dtype=1), 2),
    (dict(grad_dtype=3), 2), (dict(state_bits=4), 2), (dict(param=P + 8), 2), (dict(grad=P + 2), 2),
    (dict(m=P + 4), 2), (dict(v=P + 4), 2), (dict(master=P + 4), 2)])
def test_adamw_plan_refuses(bad, want):
    arr = (L.AdamwTensor * 2)(_tensor(), _tensor(**bad))
    buf = (ctypes.c_uint8 * 65536)()
    assert L.lib().moe_adamw_plan_bytes(arr, 2) == 0
    assert L.lib().moe_adamw_plan(arr, 2, buf, 65536) == want
    assert L.lib().moe_adamw_plan(None, 2, buf, 65536) == L.MOE_EINVAL
    assert L.lib().moe_adamw_plan(arr, -1, buf, 65536) == L.MOE_EINVAL


def test_adamw_step_refuses():
    f = lambda plan=P, n=64, lr=P, g=None, c=P, b1=0.9, b2=0.95, eps=1e-8: L.lib().moe_adamw_step(  # noqa: E731
        plan, n, lr, g, c, b1, b2, eps, 0, None)
    for kw, want in [(dict(plan=None), 1), (dict(lr=None), 1), (dict(c=None), 1), (dict(n=8), 1), (dict(b1=1.0), 1),
                     (dict(b2=-0.1), 1), (dict(eps=0.0), 1), (dict(b1=float("nan")), 1), (dict(plan=P + 8), 2),
                     (dict(c=P + 4), 2)]:
        assert f(**kw) == want, kw


def test_adamw_class_refuses():
    p, g = torch.zeros(64), torch.zeros(64)
    for args, kw in [(([], []), {}), (([p], [g, g]), {}), (([p], [g[:32]]), {}), (([p.double()], [g.double()]), {}),
                     (([p[::2]], [g[::2]]), {}), (([p[1:]], [g[1:]]), {}), (([p], [g]), dict(state_bits=16)),
                     (([p], [g]), dict(betas=(1.0, 0.9))), (([p], [g]), dict(eps=0.0)),
                     (([p], [g]), dict(weight_decay=[0.1, 0.1]))]:
        with pytest.raises(ValueError):
            AdamW(*args, **kw)
    # masters are the parameters' values, tensors start at whole groups of 128
    a, b = torch.randn(130).bfloat16(), torch.randn(7)
    o = AdamW([a, b], [torch.zeros(130), torch.zeros(7).bfloat16()], state_bits=8)
    assert o.offsets == [0, 256] and o.m.dtype == torch.uint8 and o.m_scale.shape == (3,)
    assert torch.equal(o.master[:130], a.float())


def test_adamw_state_round_trip_on_host():
    a, b = torch.randn(130).bfloat16(), torch.randn(7)
    make = lambda p, q, bits=8: AdamW([p, q], [torch.zeros_like(p), torch.zeros_like(q)], state_bits=bits)  # noqa: E731
    o = make(a, b)
    for t in (o.master, o.m, o.v, o.m_scale, o.v_scale, o.steps, o.lr):
        t.copy_(torch.arange(t.numel()).to(t.dtype))
    saved = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in o.state_dict().items()}
    c = torch.zeros(130).bfloat16()
    n = make(c, b)
    n.load_state_dict(saved)
    for k, v in saved.items():
        assert torch.equal(v, n.state_dict()[k]) if isinstance(v, torch.Tensor) else v == n.state_dict()[k]
    assert torch.equal(c, torch.arange(130).float().bfloat16()) and n._counter[1] == 0
    for other in (make(a, b, 32), make(b, a)):
        with pytest.raises(ValueError):
            other.load_state_dict(saved)
    with pytest.raises(ValueError):
        n.load_state_dict({**saved, "m": saved["m"][:128]})


def test_wrappers_refuse_host_tensors_types_and_shapes():
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    for call in [
        lambda: L.moe_combine_bwd(bf(4, 256), bf(8, 256), i32(4, 2), torch.zeros(4, 2), bf(8, 256), torch.zeros(4, 2)),
        lambda: L.moe_combine_bwd(bf(4, 256), bf(8, 128), i32(4, 2), torch.zeros(4, 2), bf(8, 256), torch.zeros(4, 2)),
        lambda: L.moe_scatter_bwd(bf(8, 256), i32(4, 2), torch.zeros(4, 256)),
        lambda: L.moe_route_topk_bwd(i32(4, 2), torch.zeros(4, 2), torch.zeros(4, 3), torch.zeros(4, 8)),
        lambda: L.silu_and_mul_bwd(bf(8, 256), bf(8, 128), bf(8, 256), masked_m=i32(3), max_m=2),
        lambda: L.grouped_gemm_contig_dgrad(bf(128, 128), bf(2, 128, 256), bf(128, 128), i32(128)),
        lambda: L.grouped_gemm_contig_wgrad(bf(128, 128), bf(128, 256), i32(2), i32(2), bf(2, 128, 256).half()),
    ]:
        with pytest.raises(ValueError):
            call()


def test_layer_training_refusals():
    def layer(**kw):
        return MoELayer(hidden=128, intermediate=128, num_experts=8, top_k=2, max_tokens=16, device="cpu", **kw)

    for kw in [dict(fp8=True, train=True), dict(layout="masked", train=True), dict(train=True, grad_dtype=torch.float16)]:
        with pytest.raises(ValueError):
            layer(**kw)
    lay = layer(train=True)
    assert lay.layout == "compact" and lay.gateup is not None
    with pytest.raises(ValueError):
        lay.backward(torch.zeros(16, 128, dtype=torch.bfloat16))    # no forward yet
    with pytest.raises(ValueError):
        lay.optimizer()                                             # no weights yet
    for f in (lambda: layer().backward(None), lambda: layer().optimizer(), lambda: layer().allocate_grads()):
        with pytest.raises(ValueError):
            f()
