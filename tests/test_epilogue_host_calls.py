"""Refusals on the host of products with an epilogue whose outputs are their inputs (no
GPU: every call here fails validation, so nothing is launched)."""
import pytest

from scatter_grouped_gemm_amd import _lib as L
from test_epilogue_host import P, contig, linear, masked


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
