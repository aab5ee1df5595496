"""Calls of the layer with a router, a shared expert and biases that a program makes
around it: on its own output, in shares, with batches of other sizes."""
import pytest
import torch

from scatter_grouped_gemm_amd import MoELayer
from gpu_util import DEV, announce
from test_gpu_epilogue_layer import Case

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
