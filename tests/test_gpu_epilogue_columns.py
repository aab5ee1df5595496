"""The gradient of the epilogue with more columns than a launch's second dimension counts."""
import pytest
import torch

from scatter_grouped_gemm_amd import _lib as L
from gpu_util import DEV, announce

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
ONE, TWO = 65535 * 128, 65535 * 512      # columns in one such dimension: sums in one launch, and else


def integers(seed, M, n):
    """-3 .. 3: their products and sums are exact."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randint(0, 7, (M, n), generator=g, device=DEV, dtype=torch.int8) - 3).to(BF)


@pytest.mark.parametrize("cols,M,db", [(ONE, 2, True), (ONE + 8, 3, True), (TWO, 2, False), (TWO + 8, 2, False), (1 << 27, 1, True),
                                       (1 << 27, 1, False), (TWO + 512, 130, True)])
def test_many_columns(cols, M, db):
    announce("columns", cols, M, db)
    p, d = integers(1, M, cols), integers(2, M, cols)
    dp, dbias = torch.full((M, cols), 77.0, dtype=BF, device=DEV), torch.full((cols,), 77.0, device=DEV) if db else None
    L.moe_act_bwd(p, d, dp, "relu2", dbias=dbias)
    torch.cuda.synchronize()
    total = torch.zeros(cols, device=DEV)
    for r in range(M):
        want = 2 * torch.relu(p[r].float()) * d[r].float()
        assert torch.equal(dp[r].float(), want), r
        total += want
    assert not db or torch.equal(dbias, total)


@pytest.mark.parametrize("cols,M,db", [(ONE + 16, 2, True), (TWO + 16, 2, False), (1 << 26, 1, True)])
def test_many_columns_gated(cols, M, db):
    """The clamped activation far out, where it is g (u + 1) and all is exact: gates of 64 .. 70 uncut."""
    announce("columns, gated", cols, M, db)
    p, d = torch.cat([integers(1, M, cols) + 67, integers(2, M, cols)], 1), integers(3, M, cols)
    dp, dbias = torch.full((M, 2 * cols), 77.0, dtype=BF, device=DEV), torch.full((2 * cols,), 77.0, device=DEV) if db else None
    L.moe_act_bwd(p, d, dp, "swiglu_clamp", dbias=dbias, limit=float("inf"))
    torch.cuda.synchronize()
    total = torch.zeros(2 * cols, device=DEV)
    for r in range(M):
        want = torch.cat([d[r].float() * (p[r, cols:].float() + 1), d[r].float() * p[r, :cols].float()])
        assert torch.equal(dp[r].float(), want), r
        total += want
    assert not db or torch.equal(dbias, total)
