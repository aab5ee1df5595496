"""Refusals of the products with an epilogue and of its gradient on the host (no GPU:
every call here fails validation, so nothing is launched)."""
import ctypes

import pytest
import torch

from scatter_grouped_gemm_amd import _lib as L

P = 4096        # a non-null, aligned address that is never dereferenced
BAD = 4104      # not 16-byte aligned
INF = float("inf")


def linear(A=P, lda=256, B=2 * P, bias=None, bdt=0, act=0, alpha=1.702, limit=7.0, res=None, ldr=0, odt=0, out=3 * P, ldo=64,
           pre=None, M=4, N=64, K=256):
    return L.lib().moe_linear(A, lda, B, bias, bdt, act, alpha, limit, res, ldr, odt, out, ldo, pre, M, N, K, None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), L.MOE_EINVAL), (dict(N=0), L.MOE_EINVAL), (dict(K=0), L.MOE_EINVAL), (dict(A=None), L.MOE_EINVAL),
    (dict(B=None), L.MOE_EINVAL), (dict(out=None), L.MOE_EINVAL), (dict(act=5), L.MOE_EINVAL), (dict(act=8), L.MOE_EINVAL),
    (dict(act=13), L.MOE_EINVAL), (dict(act=-1), L.MOE_EINVAL), (dict(act=12, limit=0.0), L.MOE_EINVAL),
    (dict(act=12, limit=float("nan")), L.MOE_EINVAL), (dict(act=12, alpha=0.0), L.MOE_EINVAL),
    (dict(act=12, alpha=float("nan")), L.MOE_EINVAL), (dict(act=9, N=63), L.MOE_EINVAL), (dict(lda=248), L.MOE_EINVAL),
    (dict(ldo=63), L.MOE_EINVAL), (dict(res=P, ldr=63), L.MOE_EINVAL), (dict(K=252, lda=256), L.MOE_EUNSUPPORTED),
    (dict(lda=260), L.MOE_EUNSUPPORTED), (dict(odt=1), L.MOE_EUNSUPPORTED), (dict(bias=P, bdt=1), L.MOE_EUNSUPPORTED),
    (dict(A=BAD), L.MOE_EUNSUPPORTED), (dict(B=BAD), L.MOE_EUNSUPPORTED), (dict(out=4097), L.MOE_EUNSUPPORTED),
    (dict(odt=16, out=4098), L.MOE_EUNSUPPORTED), (dict(bias=4098, bdt=16), L.MOE_EUNSUPPORTED),
    (dict(pre=4097), L.MOE_EUNSUPPORTED), (dict(lda=1 << 22), L.MOE_EUNSUPPORTED),
    (dict(act=9, N=1 << 20, K=4096, lda=4096, ldo=1 << 20), L.MOE_EUNSUPPORTED),
    (dict(M=(1 << 30), N=1 << 20, ldo=1 << 20), L.MOE_EUNSUPPORTED),
    (dict(out=P), L.MOE_EINVAL), (dict(out=2 * P), L.MOE_EINVAL), (dict(pre=P), L.MOE_EINVAL), (dict(pre=3 * P), L.MOE_EINVAL),
    (dict(res=3 * P, ldr=72), L.MOE_EINVAL),              # in place, but with other rows
    (dict(M=0, A=None, B=None, out=None), L.MOE_OK),
])
def test_linear_refusals(kw, want):
    assert linear(**kw) == want


def contig(dtype=0, A=P, As=None, B=2 * P, Bs=None, bias=None, bdt=0, act=0, alpha=1.702, limit=7.0, odt=0, out=3 * P, os=None,
           pre=None, m=P, M=256, N=256, K=256, G=2):
    return L.lib().grouped_gemm_contig_act(dtype, A, As, B, Bs, bias, bdt, act, alpha, limit, odt, out, os, pre, m, M, N, K, G, None)


def masked(dtype=0, A=P, As=None, B=2 * P, Bs=None, bias=None, bdt=0, act=0, alpha=1.702, limit=7.0, odt=0, out=3 * P, os=None,
           pre=None, m=P, em=0, max_m=64, N=256, K=256, G=2):
    return L.lib().grouped_gemm_masked_act(dtype, A, As, B, Bs, bias, bdt, act, alpha, limit, odt, out, os, pre, m, em, max_m, N, K, G, None)


@pytest.mark.parametrize("call", [contig, masked])
@pytest.mark.parametrize("kw,want", [
    (dict(N=0), L.MOE_EINVAL), (dict(K=0), L.MOE_EINVAL), (dict(G=0), L.MOE_EINVAL), (dict(A=None), L.MOE_EINVAL),
    (dict(B=None), L.MOE_EINVAL), (dict(out=None), L.MOE_EINVAL), (dict(m=None), L.MOE_EINVAL), (dict(act=6), L.MOE_EINVAL),
    (dict(act=12, limit=-1.0), L.MOE_EINVAL), (dict(act=12, alpha=INF), L.MOE_EINVAL),
    (dict(N=64), L.MOE_EUNSUPPORTED), (dict(K=64), L.MOE_EUNSUPPORTED), (dict(act=9, N=128), L.MOE_EUNSUPPORTED),
    (dict(dtype=7), L.MOE_EUNSUPPORTED), (dict(dtype=1), L.MOE_EUNSUPPORTED),        # FP8 without scales
    (dict(odt=1, os=P), L.MOE_EUNSUPPORTED),                                            # e4m3 output is a gated one's
    (dict(act=9, odt=1), L.MOE_EINVAL), (dict(act=9, odt=16), L.MOE_EUNSUPPORTED), (dict(bias=P, bdt=2), L.MOE_EUNSUPPORTED),
    (dict(dtype=1, As=P, Bs=P, pre=P), L.MOE_EUNSUPPORTED),                             # pre needs bf16 weights
    (dict(A=BAD), L.MOE_EUNSUPPORTED), (dict(B=BAD), L.MOE_EUNSUPPORTED), (dict(bias=BAD), L.MOE_EUNSUPPORTED),
    (dict(out=BAD), L.MOE_EUNSUPPORTED), (dict(pre=BAD), L.MOE_EUNSUPPORTED),
    (dict(act=9, N=1 << 20, K=4096), L.MOE_EUNSUPPORTED), (dict(out=P), L.MOE_EINVAL), (dict(pre=3 * P), L.MOE_EINVAL),
])
def test_grouped_refusals(call, kw, want):
    assert call(**kw) == want


def test_grouped_refusals_of_one_layout():
    assert contig(M=-1) == L.MOE_EINVAL and contig(M=0, m=None) == L.MOE_OK
    assert masked(max_m=0) == L.MOE_EINVAL and masked(em=-1) == L.MOE_EINVAL and masked(G=1025) == L.MOE_EUNSUPPORTED
    assert contig(M=8177 * 128) == L.MOE_EUNSUPPORTED


def bwd(pre=P, dout=P, M=2560, N=256, act=9, alpha=1.702, limit=7.0, m=None, mm=None, max_m=0, st=None, nv=None, G=1,
        dpre=P, ddt=16, acc=0, db=None, ws=P, nws=1 << 30, odt=0):
    return L.lib().moe_act_bwd(pre, odt, dout, M, N, act, alpha, limit, m, mm, max_m, st, nv, G, dpre, ddt, acc, db, ws, nws, None)


@pytest.mark.parametrize("kw,want", [
    (dict(M=-1), L.MOE_EINVAL), (dict(N=0), L.MOE_EINVAL), (dict(G=0), L.MOE_EINVAL), (dict(act=7), L.MOE_EINVAL),
    (dict(pre=None), L.MOE_EINVAL), (dict(dout=None), L.MOE_EINVAL), (dict(dpre=None, db=P), L.MOE_EINVAL),
    (dict(act=0, dpre=None), L.MOE_EINVAL), (dict(m=P, mm=P, max_m=64), L.MOE_EINVAL), (dict(mm=P), L.MOE_EINVAL),
    (dict(mm=P, max_m=100), L.MOE_EINVAL), (dict(mm=P, max_m=64, G=3, db=P), L.MOE_EINVAL), (dict(G=2), L.MOE_EINVAL),
    (dict(m=P, db=P, G=2), L.MOE_EINVAL), (dict(m=P, db=P, G=2, st=P), L.MOE_EINVAL), (dict(db=P, ws=None), L.MOE_EINVAL),
    (dict(db=P, nws=16), L.MOE_ECAPACITY), (dict(db=P, ddt=1), L.MOE_EUNSUPPORTED), (dict(odt=1), L.MOE_EUNSUPPORTED), (dict(N=8), L.MOE_EUNSUPPORTED),
    (dict(act=1, N=4), L.MOE_EUNSUPPORTED), (dict(M=1 << 26), L.MOE_EUNSUPPORTED), (dict(N=(1 << 27) + 16), L.MOE_EUNSUPPORTED),
    (dict(pre=BAD), L.MOE_EUNSUPPORTED), (dict(dout=BAD), L.MOE_EUNSUPPORTED), (dict(dpre=BAD), L.MOE_EUNSUPPORTED),
    (dict(db=BAD), L.MOE_EUNSUPPORTED), (dict(db=P, ws=BAD), L.MOE_EUNSUPPORTED), (dict(M=0, pre=None, dout=None), L.MOE_OK),
])
def test_act_bwd_refusals(kw, want):
    assert bwd(**kw) == want


def test_act_bwd_ws_bytes():
    for M, N, G in [(129, 16, 1), (8191, 4096, 1), (131072, 28672, 256)]:
        n = L.moe_act_bwd_ws_bytes(M, N, G)
        assert n >= -(-M // 16) * N * 4 and n % 4 == 0
    for bad in [(0, 16, 1), (160, 0, 1), (160, 16, 0), (-1, 16, 1), (128, 16, 1), (1024, 4096, 8)]:   # the last two need none
        assert L.moe_act_bwd_ws_bytes(*bad) == 0


def test_binding_refuses_wrong_tensors():
    """The Python layer names what is wrong before any call: types, shapes, activations, devices."""
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError, match="unknown activation"):
        L.moe_linear(bf(4, 64), bf(32, 64), bf(4, 32), act="swish")
    with pytest.raises(ValueError, match="even number"):
        L.moe_linear(bf(4, 64), bf(31, 64), bf(4, 15), act="silu_mul")
    with pytest.raises(ValueError, match="bf16 or fp32"):
        L.moe_linear(bf(4, 64), bf(32, 64), torch.zeros(4, 32, dtype=torch.float16))
    with pytest.raises(ValueError, match="x: is on cpu"):
        L.moe_linear(bf(4, 64), bf(32, 64), bf(4, 32))
    with pytest.raises(ValueError, match="differ in their reduction"):
        L.grouped_gemm_contig_act(False, bf(128, 128), None, bf(2, 128, 256), None, bf(128, 128), torch.zeros(128, dtype=torch.int32))
    with pytest.raises(ValueError, match="differ in their experts"):
        L.grouped_gemm_masked_act(False, bf(3, 8, 128), None, bf(2, 128, 128), None, bf(3, 8, 128), torch.zeros(3, dtype=torch.int32), 0)
    with pytest.raises(ValueError, match="do not make up"):
        L.moe_act_bwd(bf(10, 32), bf(10, 32), bf(10, 32), "silu", masked_m=torch.zeros(3, dtype=torch.int32), max_m=4)
    with pytest.raises(ValueError, match="pre and dpre are needed"):
        L.moe_act_bwd(None, bf(10, 32), None, "silu")
    with pytest.raises(ValueError, match="expert_start_loc and num_valid"):
        L.moe_act_bwd(bf(10, 32), bf(10, 32), bf(10, 32), "silu", dbias=torch.zeros(2, 32), m_indices=torch.zeros(10, dtype=torch.int32))


def test_activation_names_match_the_header():
    import os
    import re
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe.h")).read()
    defined = {m[0].lower(): int(m[1]) for m in re.findall(r"#define MOE_ACT_(\w+) (\d+)", src)}
    assert defined == L.ACTIVATIONS
    assert all((L.ACTIVATIONS[a] >= 8) == (a in L.GATED_ACTIVATIONS) for a in L.ACTIVATIONS)
