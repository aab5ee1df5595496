"""The input gradient's three kernels: 64 x 64 tiles as long as each has a compute
unit, 128 x 128 up to three for two units, 256 x 256 beyond."""
import numpy as np
import pytest
import torch

from scatter_grouped_gemm_amd import _lib as L
from gpu_util import DEV, announce, compact_layout, i32_dev, poison
from test_gpu_training import BF, randn, same_bits
from test_gpu_training_scale import _ints

pytestmark = pytest.mark.gpu


def _units():
    return torch.cuda.get_device_properties(0).multi_processor_count


def _kernel(M, K):
    if -(-M // 64) * (K // 64) <= _units():
        return "64"
    return "128" if 2 * -(-M // 128) * (K // 128) <= 3 * _units() else "256"


@pytest.mark.parametrize("counts,N,K,extra", [
    ([1], 128, 2048, 896), ([1024], 128, 2048, 0), ([127, 0, 65, 64, 129, 1], 256, 1664, 128),
    ([130, 500, 0, 0, 63], 384, 1408, 72), ([3, 0, 1, 128, 64, 2, 9, 200], 1152, 3200, 0),
    ([40] * 24, 256, 1024, 256), ([900, 70], 4224, 4096, 0)])
def test_tiles_of_128(counts, N, K, extra):
    """Whole numbers, so that the sums are exact; rows without an expert hold NaN and
    stay as they were; a last block that is not whole."""
    announce("dgrad 128", counts, N, K, extra)
    m = compact_layout(counts, extra_rows=extra)
    assert _kernel(len(m), K) == "128"
    named = torch.from_numpy(m >= 0).to(DEV)
    dC, B = _ints(-1, 2, len(m), N), _ints(-1, 3, len(counts), N, K)
    dC[~named] = float("nan")
    dA = poison((len(m), K), BF)
    before = dA.clone()
    L.grouped_gemm_contig_dgrad(dC, B, dA, i32_dev(m))
    at = 0
    for g, c in enumerate(counts):
        want = (dC[at:at + c].float() @ B[g].float()).to(BF)
        assert torch.equal(dA[at:at + c].float(), want.float()), g
        at += -(-c // 128) * 128
    assert same_bits(dA[~named], before[~named])


def test_a_block_cut_by_the_last_row():
    announce("dgrad cut")
    M, N, K = 128 * 5 + 77, 256, 2048
    assert _kernel(M, K) == "128"
    dC, B = _ints(-1, 2, M, N), _ints(-1, 3, 2, N, K)
    room = poison((M + 128, K), BF)
    before = room.clone()
    m = np.zeros(M, np.int32)
    m[640:] = 1
    L.grouped_gemm_contig_dgrad(dC, B, room[:M], i32_dev(m))
    assert torch.equal(room[:640].float(), (dC[:640].float() @ B[0].float()).to(BF).float())
    assert torch.equal(room[640:M].float(), (dC[640:].float() @ B[1].float()).to(BF).float())
    assert same_bits(room[M:], before[M:])


def test_128_columns_of_the_widest_weights():
    """64 rows of a B with 2^22 columns are 2^29 bytes, 128 rows of such a dC 2^30."""
    announce("dgrad widest")
    M, N, K = 128 * 300, 4194304 // 32, 128                  # 300 tiles of 128 x 128; dC 10 GB
    assert _kernel(M, K) == "128"
    dC, B = torch.zeros(M, N, dtype=BF, device=DEV), _ints(-1, 2, 1, N, K)
    for r in (0, 127, 128, 20000, M - 1):
        dC[r] = _ints(-1, 3, N)
    dA = torch.empty(M, K, dtype=BF, device=DEV)
    L.grouped_gemm_contig_dgrad(dC, B, dA, i32_dev(np.zeros(M, np.int32)))
    rows = torch.tensor([0, 1, 127, 128, 20000, M - 1], device=DEV)
    assert torch.equal(dA[rows].float(), (dC[rows].float() @ B[0].float()).to(BF).float())


def test_all_three_kernels_give_the_same_bits():
    announce("dgrad same bits")
    N, K, blocks = 1152, 2560, 24
    dC, B = randn(1, blocks * 128, N).to(DEV), randn(2, 2, N, K).to(DEV)
    m = np.repeat(np.arange(blocks) % 2, 128).astype(np.int32)
    m[5 * 128 + 3:6 * 128] = -1

    def run(lo, hi):
        out = torch.zeros((hi - lo) * 128, K, dtype=BF, device=DEV)
        L.grouped_gemm_contig_dgrad(dC[lo * 128:hi * 128], B, out, i32_dev(m[lo * 128:hi * 128]))
        return out
    assert _kernel(blocks * 128, K) == "256" and _kernel(8 * 128, K) == "128" and _kernel(128, K) == "64"
    whole = run(0, blocks)
    for lo in range(0, blocks, 8):
        assert same_bits(run(lo, lo + 8), whole[lo * 128:(lo + 8) * 128]), lo
    for b in range(0, blocks, 5):
        assert same_bits(run(b, b + 1), whole[b * 128:(b + 1) * 128]), b


# valid rows of consecutive 128-row blocks and their experts: blocks that are not full
# in the middle of an expert's, half blocks, empty ones
_ROWS = [3, 128, 128, 64, 0, 127, 128, 1, 128, 128, 65, 128, 0, 128, 100, 77]
_IDS = [0, 0, 0, 0, 0, 1, 1, 1, 1, 0, 0, 2, 2, 2, 2, 2]


@pytest.mark.parametrize("times,K,cut,tile", [(1, 4096, 0, "256"), (1, 4096, 30, "256"), (40, 512, 51, "256"),
                                              (1, 1408, 0, "128"), (1, 1408, 51, "128"), (1, 256, 0, "64"), (1, 256, 51, "64")])
def test_blocks_that_are_not_full(times, K, cut, tile):
    """Padding rows inside an expert's blocks hold NaN and are neither read into a row
    nor written, whichever kernel takes the call; the last block may be cut."""
    announce("dgrad partial blocks", times, K, cut)
    N = 256
    m = np.full(16 * times * 128, -1, np.int32)
    for b in range(16 * times):
        m[b * 128:b * 128 + _ROWS[b % 16]] = _IDS[b % 16]
    m = m[:len(m) - cut]
    assert _kernel(len(m), K) == tile
    dC, B = _ints(-1, 2, len(m), N), _ints(-1, 3, 3, N, K)
    named = torch.from_numpy(m >= 0).to(DEV)
    dC[~named] = float("nan")
    dA = poison((len(m), K), BF)
    before = dA.clone()
    L.grouped_gemm_contig_dgrad(dC, B, dA, i32_dev(m))
    for e in range(3):
        at = torch.from_numpy(m == e).to(DEV)
        assert torch.equal(dA[at].float(), (dC[at].float() @ B[e].float()).to(BF).float()), e
    assert same_bits(dA[~named], before[~named])


def test_as_many_runs_as_blocks():
    """8160 blocks of one row each: every XCD's share of the run table is full."""
    announce("dgrad 8160 runs")
    N, K, blocks = 128, 256, 8160
    m = np.full(blocks * 128, -1, np.int32)
    m[::128] = np.arange(blocks) // 4000
    rows = torch.arange(0, blocks * 128, 128, device=DEV)
    dC, B = torch.full((blocks * 128, N), float("nan"), dtype=BF, device=DEV), _ints(-1, 3, 3, N, K)
    dC[rows] = _ints(-1, 2, blocks, N)
    dA = poison((blocks * 128, K), BF)
    L.grouped_gemm_contig_dgrad(dC, B, dA, i32_dev(m))
    want = torch.bmm(dC[rows].float()[:, None], B.float()[rows // 128 // 4000])[:, 0]
    assert torch.equal(dA[rows].float(), want.to(BF).float())
    dA[rows] = poison((1, K), BF)
    assert torch.equal(dA.view(torch.int16), poison((blocks * 128, K), BF).view(torch.int16))
