"""Refusals on the host of products with an epilogue whose outputs are their inputs (no
GPU: every call here fails validation, so nothing is launched)."""
import pytest

from scatter_grouped_gemm_amd import _lib as L
from test_epilogue_host import P, bwd, contig, linear, masked


@pytest.mark.parametrize("kw", [
    dict(pre=5 * P, res=5 * P, ldr=64),            # the kept product in the residual's place: written before that is read
    dict(pre=5 * P, bias=5 * P), dict(bias=3 * P),
])
def test_linear_refuses_outputs_that_are_inputs(kw):
    assert linear(**kw) == L.MOE_EINVAL


@pytest.mark.parametrize("call", [contig, masked])
@pytest.mark.parametrize("kw", [dict(bias=3 * P), dict(pre=5 * P, bias=5 * P)])
def test_grouped_refuses_outputs_that_are_inputs(call, kw):
    assert call(**kw) == L.MOE_EINVAL


@pytest.mark.parametrize("kw", [
    dict(act=9, dpre=2 * P), dict(act=1, odt=16, dpre=2 * P),      # dpre in dout's place, where an element has another one
    dict(act=1, db=P, dpre=3 * P), dict(act=1, db=2 * P, dpre=3 * P), dict(act=1, db=3 * P, dpre=3 * P),
])
def test_act_bwd_refuses_outputs_that_are_inputs(kw):
    assert bwd(pre=P, dout=2 * P, **kw) == L.MOE_EINVAL


@pytest.mark.parametrize("kw", [
    dict(act=1), dict(act=9), dict(act=0), dict(act=9, G=8),        # a batch without tokens: none of its tensors has an address
    dict(act=9, G=8, db=P, acc=1, st=P, nv=P, ws=None, nws=0), dict(act=0, db=P, acc=1, ws=None, nws=0),
])
def test_act_bwd_of_no_rows(kw):
    assert bwd(M=0, pre=None, dout=None, dpre=None, **kw) == L.MOE_OK


@pytest.mark.parametrize("kw,want", [
    (dict(), L.MOE_OK), (dict(act=9), L.MOE_OK), (dict(dtype=1, Bs=P), L.MOE_OK), (dict(dtype=3, Bs=P, act=9, odt=1), L.MOE_OK),
    (dict(B=None), L.MOE_EINVAL), (dict(N=64), L.MOE_EUNSUPPORTED), (dict(dtype=1), L.MOE_EUNSUPPORTED), (dict(act=6), L.MOE_EINVAL),
])
def test_contig_of_no_rows(kw, want):
    assert contig(M=0, A=None, out=None, m=None, **kw) == want
