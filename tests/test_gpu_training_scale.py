"""The training operators where sizes change what they do: many experts and
uneven ones (how the weight gradient's tiles are dealt), offsets past 32 bits,
shares of the experts, empty batches, non-finite values."""
import numpy as np
import pytest
import torch

from scatter_grouped_gemm_amd import AdamW, MoELayer, inputs
from scatter_grouped_gemm_amd import _lib as L
from gpu_util import DEV, announce, compact_layout, i32_dev, poison
from test_gpu_training import BF, F32, U16, U32, VALUES, _bits, _make, gen, randn, same_bits, within

pytestmark = pytest.mark.gpu


def _ints(lo, hi, *shape):
    """Whole numbers lo .. hi - 1, drawn on the device from the shape."""
    g = torch.Generator(device=DEV)
    g.manual_seed(sum(shape))
    return torch.randint(lo, hi, shape, generator=g, device=DEV).to(BF)


def _case(kind, G, rng):
    if kind == "zipf":
        c = [int(4000 / (i + 1) ** 1.2) + 1 for i in range(G)]
    elif kind == "one":
        c = [0] * G
        c[G // 2] = 3000
    elif kind == "even":
        c = [97] * G
    elif kind == "few":
        c = rng.integers(0, 4, G).tolist()
    else:
        c = rng.integers(0, 500, G).tolist()
    c = [0 if rng.random() < 0.2 else x for x in c]
    rng.shuffle(c)
    return c


# (rows of the experts, experts, N, K): tiles of an XCD's share below and above its
# workgroups, odd numbers of tiles, half tiles on either side
DEALT = [("zipf", 64, 512, 384), ("zipf", 7, 2048, 2176), ("zipf", 200, 128, 128), ("one", 33, 768, 256), ("even", 40, 640, 512),
         ("few", 1024, 128, 128), ("few", 300, 384, 128), ("any", 16, 4096, 4224), ("any", 90, 256, 640), ("any", 3, 128, 8192),
         ("even", 2, 8320, 2048)]


@pytest.mark.parametrize("out,acc", [(BF, False), (F32, True), (BF, True)])
@pytest.mark.parametrize("kind,G,N,K", DEALT)
def test_every_tile_of_the_weight_gradient_once(kind, G, N, K, out, acc):
    """Whole numbers, so that a tile left out or added twice shows exactly."""
    announce("wgrad dealt", kind, G, N, K, out, acc)
    counts = _case(kind, G, np.random.default_rng(G + N))
    m = compact_layout(counts, extra_rows=128)
    pad = np.array([-(-c // 128) * 128 for c in counts])
    starts = np.concatenate([[0], np.cumsum(pad)[:-1]])
    dC, A = _ints(-1, 2, len(m), N), _ints(-1, 3, len(m), K)
    old = _ints(-3, 4, G, N, K).to(out) if acc else None
    dB = old.clone() if acc else poison((G, N, K), out)
    L.grouped_gemm_contig_wgrad(dC, A, i32_dev(starts), i32_dev(np.array(counts)), dB, accumulate=acc)
    for g, (s, c) in enumerate(zip(starts.tolist(), counts)):
        want = dC[s:s + c].float().t() @ A[s:s + c].float()   # whole numbers below 2^24: exact in fp32
        if acc:
            want = want + old[g].float()
        assert torch.equal(dB[g], want.to(out)), (g, c)


@pytest.mark.parametrize("G,N,K", [(300, 256, 128), (1024, 128, 256), (40, 512, 640), (5, 1408, 4096)])
def test_input_gradient_of_many_runs(G, N, K):
    announce("dgrad runs", G, N, K)
    rng = np.random.default_rng(G)
    counts = _case("any" if G < 100 else "few", G, rng)
    m = compact_layout(counts, extra_rows=256)
    dC, B = _ints(-1, 2, len(m), N), _ints(-1, 3, G, N, K)
    dA = poison((len(m), K), BF)
    before = dA.clone()
    L.grouped_gemm_contig_dgrad(dC, B, dA, i32_dev(m))
    at = 0
    for g, c in enumerate(counts):
        assert torch.equal(dA[at:at + c].float(), (dC[at:at + c].float() @ B[g].float()).to(BF).float()), g
        at += -(-c // 128) * 128
    pad = torch.from_numpy(m < 0).to(DEV)
    assert same_bits(dA[pad], before[pad])


def test_input_gradient_rows_are_the_same_in_either_kernel():
    """Few rows take the narrow kernel, many the wide one: a row's bits agree."""
    announce("dgrad narrow and wide")
    N, K = 640, 1408
    dC, B = randn(1, 6000, N).to(DEV), randn(2, 1, N, K).to(DEV)
    wide = torch.zeros(6000, K, dtype=BF, device=DEV)      # 47 * 6 tiles
    L.grouped_gemm_contig_dgrad(dC, B, wide, torch.zeros(6000, dtype=torch.int32, device=DEV))
    for n in (1, 63, 64, 65, 130, 1000):                   # at most 8 * 6
        part = torch.zeros(n, K, dtype=BF, device=DEV)
        L.grouped_gemm_contig_dgrad(dC[:n].contiguous(), B, part, torch.zeros(n, dtype=torch.int32, device=DEV))
        assert same_bits(part, wide[:n]), n


def test_a_product_longer_than_the_waits_count():
    """One expert, one tile, a long reduction, against 64 bits."""
    announce("long reduction")
    n = 20011
    dC, A = randn(1, n, 128, scale=0.1).to(DEV), randn(2, n, 256).to(DEV)
    dB = poison((1, 128, 256), F32)
    L.grouped_gemm_contig_wgrad(dC, A, i32_dev(np.array([0])), i32_dev(np.array([n])), dB)
    want, size = dC.double().t() @ A.double(), dC.double().abs().t() @ A.double().abs()
    within(dB[0], want.cpu(), (n * 2 * U32 * size).cpu())


def test_rows_past_32_bits():
    """Rows whose byte offsets pass 2^32, in the token and activation gradients."""
    announce("offsets")
    rows, H, T = 340_000, 8192, 3                       # 5.6 GB
    Y = torch.zeros(rows, H, dtype=BF, device=DEV)
    s = np.array([[rows - 1, 5], [-1, rows - 2], [7, rows - 3]])
    for r in s[s >= 0]:
        Y[r] = float(r % 7 + 1)
    dout = torch.full((T, H), 0.5, dtype=BF, device=DEV)
    w = torch.tensor([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]], device=DEV)
    dY, dw = torch.zeros(rows, H, dtype=BF, device=DEV), poison((T, 2), F32)
    L.moe_combine_bwd(dout, Y, i32_dev(s), w, dY, dw)
    want = torch.tensor([[0.0 if r < 0 else 0.5 * H * (r % 7 + 1) for r in row] for row in s.tolist()])
    assert torch.equal(dw.cpu(), want)
    for t in range(T):
        for j in range(2):
            if s[t, j] >= 0:
                assert (dY[s[t, j]] == 0.5 * w[t, j]).all()
    dx = poison((T, H), BF)
    L.moe_scatter_bwd(Y, i32_dev(s), dx)
    assert torch.equal(dx[:, 0].float().cpu(), torch.tensor([sum(r % 7 + 1 for r in row if r >= 0) for row in s.tolist()]).float())
    del Y, dY
    M, I = 160_000, 14336                               # 9.2 GB of halves
    gu, da = torch.zeros(M, 2 * I, dtype=BF, device=DEV), torch.zeros(M, I, dtype=BF, device=DEV)
    gu[-1, :I], gu[-1, I:], da[-1] = 0.0, 3.0, 2.0
    m = np.full(M, -1, np.int32)
    m[-1] = 0
    L.silu_and_mul_bwd(gu, da, gu, m_indices=i32_dev(m))
    assert (gu[-1, :I] == 3.0).all() and (gu[-1, I:] == 0.0).all()   # 2 * 3 * s(0), and 2 * 0 * s(0)


def test_adamw_past_32_bits():
    """A tensor of more than 2^32 elements: its end against the formula and the
    random bits of its elements' numbers."""
    announce("adamw 2^32")
    n = (1 << 32) + 300
    p = torch.zeros(n, device=DEV)
    g = torch.zeros(n, dtype=BF, device=DEV)
    tail = randn(3, 300, scale=1e-3)
    g[-300:] = tail.to(DEV)
    opt = AdamW([p], [g], lr=0.5, betas=(0.9, 0.99), state_bits=8, seed=9)
    opt.step()
    x = tail.double()
    want = -0.5 * torch.sign(x) * (x.abs() / (x.abs() + 1e-8))
    within(p[-300:], want, want.abs() * 40 * U32)
    assert (p[:: 1 << 20][:-1] == 0).all()
    # the group that begins at 2^32, its codes by the definition
    key = _mixed_key(9, 0, 1) ^ 1
    bits = _mix_all(torch.arange(128), key)
    m = (0.1 * x[:128]).abs()
    e = torch.ceil(torch.log2(m.max() / 448))
    assert opt.m_scale[(1 << 32) // 128].item() == e.item() + 127
    a = m / torch.exp2(e)
    low = torch.searchsorted(VALUES, a, right=True) - 1
    part = (a - VALUES[low]) / (VALUES[low + 1] - VALUES[low]) + (bits & 0xffff) / 65536
    code = VALUES[low + (part >= 1).long()]
    got = opt.m[1 << 32: (1 << 32) + 128].cpu().view(torch.float8_e4m3fn).double().abs()
    assert ((got == code) | ((part - 1).abs() < 2.0 ** -17)).all()


def _mixed_key(seed, tensor, step):
    from test_gpu_training import _mix
    return _mix((_mix((seed + 0x9E3779B9 * (tensor + 1)) & 0xffffffff) + step) & 0xffffffff)


def _mix_all(i, key):
    from test_gpu_training import _mix
    return _mix(_mix(i) ^ key)


def test_adamw_non_finite_gradients_stay_where_they_are():
    announce("adamw nan")
    for bits in (8, 32):
        ps = [torch.ones(1000, device=DEV), torch.ones(1000, device=DEV)]
        gs = [torch.ones(1000, device=DEV), torch.ones(1000, device=DEV)]
        gs[0][5], gs[0][700] = float("nan"), float("inf")
        opt = AdamW(ps, gs, lr=0.1, state_bits=bits)
        opt.step()
        bad = ~torch.isfinite(ps[0])
        assert bad.nonzero().view(-1).tolist() == [5, 700]
        assert torch.isfinite(ps[1]).all() and torch.equal(ps[1], ps[1][:1].expand(1000))
        assert torch.equal(ps[0][:5], ps[1][:5])


def test_adamw_resumes_from_its_state():
    announce("adamw state")
    for bits in (8, 32):
        def make(p):
            return AdamW([p], [g], lr=1e-2, weight_decay=0.1, state_bits=bits, seed=4)
        g = randn(1, 5000).to(DEV)
        a = randn(2, 5000).to(DEV)
        o = make(a)
        o.step(), o.step()
        b = torch.zeros_like(a)
        n = make(b)
        n.load_state_dict({k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in o.state_dict().items()})
        o.step(), n.step()
        assert same_bits(a, b) and same_bits(o.m, n.m) and same_bits(o.v, n.v) and n.steps.item() == 3


def test_shares_of_the_experts_add_up():
    """Two layers with half of the experts each: their dx, dlogits and outputs add
    up to the whole layer's."""
    announce("shares")
    T, H, I, E, k = 70, 256, 256, 8, 3
    whole, x, logits, w13, w2 = _make(T, H, I, E, k)
    dout = randn(5, T, H, scale=0.5).to(DEV)
    xd, ld = x.to(DEV), logits.to(DEV)
    out = whole(xd, ld).float().clone()
    dx, dl = (t.float().clone() for t in whole.backward(dout))
    sums = [torch.zeros_like(t) for t in (out, dx, dl)]
    for start in (0, 4):
        part = MoELayer(hidden=H, intermediate=I, num_experts=E, top_k=k, max_tokens=T, num_local_experts=4,
                        expert_start=start, train=True, device=DEV)
        part.set_weights(w13[start:start + 4].to(DEV), w2[start:start + 4].to(DEV))
        got = [part(xd, ld).float()]
        got += [t.float() for t in part.backward(dout)]
        for s, t in zip(sums, got):
            s += t
        assert same_bits(part.dw13, whole.dw13[start:start + 4]) and same_bits(part.dw2, whole.dw2[start:start + 4])
    # each share rounds its sum to bf16 once more, in out and dx
    for s, t, u in zip(sums, (out, dx, dl), (U16, U16, 16 * U32)):
        assert (s - t).abs().max() <= 3 * u * max(t.abs().max(), s.abs().max())


def test_empty_and_single_batches():
    announce("empty batch")
    layer, x, logits, _, _ = _make(16, 256, 128, 4, 2)
    layer(x.to(DEV), logits.to(DEV))
    layer.backward(randn(1, 16, 256).to(DEV))
    e = torch.empty(0, 256, dtype=BF, device=DEV)
    z = [torch.zeros(0, 2, device=DEV), torch.zeros(0, 2, dtype=torch.int32, device=DEV)]
    L.moe_combine_bwd(e, layer.y, z[1], z[0], layer.dy, z[0])
    L.moe_scatter_bwd(layer.y, z[1], e)
    L.moe_route_topk_bwd(z[1], z[0], z[0], torch.empty(0, 4, device=DEV))
    L.silu_and_mul_bwd(torch.empty(0, 256, dtype=BF, device=DEV), torch.empty(0, 128, dtype=BF, device=DEV),
                       torch.empty(0, 256, dtype=BF, device=DEV))
    none = torch.empty(0, 256, dtype=BF, device=DEV)
    B = randn(2, 3, 128, 256).to(DEV)
    L.grouped_gemm_contig_dgrad(torch.empty(0, 128, dtype=BF, device=DEV), B, none, torch.empty(0, dtype=torch.int32, device=DEV))
    dB = poison((3, 128, 256), BF)
    c = torch.tensor([5, 0, 1], dtype=torch.int32, device=DEV)       # cut at M = 0 rows
    L.grouped_gemm_contig_wgrad(torch.empty(0, 128, dtype=BF, device=DEV), none, torch.zeros_like(c), c, dB)
    assert (dB == 0).all()
    # every slot elsewhere: nothing is held here
    part = MoELayer(hidden=256, intermediate=128, num_experts=8, top_k=2, max_tokens=9, num_local_experts=2,
                    expert_start=6, train=True, device=DEV)
    part.set_weights(randn(1, 2, 256, 256).to(DEV), randn(2, 2, 256, 128).to(DEV))
    lg = torch.zeros(9, 8)
    lg[:, :2] = 5.0
    out = part(x[:9].to(DEV), lg.to(DEV))
    dx, dl = part.backward(randn(3, 9, 256).to(DEV))
    for t in (out, dx, dl, part.dw13, part.dw2):
        assert (t == 0).all()


def test_products_on_two_streams_at_once():
    """Calls that overlap share nothing: each gives what it gives alone."""
    announce("two streams")
    cases = []
    for seed, counts in ((1, [300, 5, 700]), (2, [64] * 9)):
        m = compact_layout(counts)
        pad = np.array([-(-c // 128) * 128 for c in counts])
        st = np.concatenate([[0], np.cumsum(pad)[:-1]])
        cases.append((randn(seed, len(m), 1024).to(DEV), randn(seed + 5, len(m), 640).to(DEV),
                      randn(seed + 9, len(counts), 1024, 640).to(DEV), i32_dev(m), i32_dev(st), i32_dev(np.array(counts))))

    def run(c):
        dA = torch.zeros(c[0].shape[0], 640, dtype=BF, device=DEV)
        dB = torch.zeros(c[2].shape, dtype=BF, device=DEV)
        L.grouped_gemm_contig_dgrad(c[0], c[2], dA, c[3])
        L.grouped_gemm_contig_wgrad(c[0], c[1], c[4], c[5], dB)
        return dA, dB

    alone = [run(c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for _ in range(3):
        for s, c in zip(streams, cases):
            with torch.cuda.stream(s):
                got.append(run(c))
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        for a, b in zip(g, alone[i % 2]):
            assert same_bits(a, b)


def test_calls_refuse_another_device_and_order():
    announce("refusals on the device")
    bf = lambda *s: torch.zeros(*s, dtype=BF, device=DEV)  # noqa: E731
    m = torch.zeros(256, dtype=torch.int32, device=DEV)
    for call in [
        lambda: L.grouped_gemm_contig_dgrad(bf(128, 256).t(), bf(2, 128, 256), bf(256, 256), m),      # not contiguous
        lambda: L.grouped_gemm_contig_dgrad(bf(256, 128), bf(2, 128, 256), bf(256, 256), m.cpu()),
        lambda: L.grouped_gemm_contig_dgrad(bf(256, 128), bf(2, 128, 256), bf(256, 256).float(), m),
        lambda: L.moe_scatter_bwd(bf(8, 256), torch.zeros(4, 2, dtype=torch.int64, device=DEV), bf(4, 256)),
    ]:
        with pytest.raises(ValueError):
            call()
    with pytest.raises(L.MoeError):                                   # a view that begins inside 16 bytes
        flat = torch.zeros(8 * 256 + 1, dtype=BF, device=DEV)
        L.moe_scatter_bwd(flat[1:].view(8, 256), torch.zeros(4, 2, dtype=torch.int32, device=DEV), bf(4, 256))
