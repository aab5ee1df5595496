"""The weight gradient's two kernels: 256 x 256 tiles, and 128 x 128 tiles where
there are few tiles (at most two for each compute unit, or six with at most 1024
rows an expert) or few rows (at most 256 an expert, added to fp32)."""
import numpy as np
import pytest
import torch

from scatter_grouped_gemm_amd import _lib as L
from gpu_util import DEV, announce, compact_layout, i32_dev, poison
from test_gpu_training import BF, F32, randn, same_bits
from test_gpu_training_scale import _ints

pytestmark = pytest.mark.gpu

KINDS = [(BF, False), (F32, False), (F32, True), (BF, True)]


def _layout(counts):
    m = compact_layout(counts, extra_rows=128)
    pad = np.array([-(-c // 128) * 128 for c in counts])
    return np.concatenate([[0], np.cumsum(pad)[:-1]]), m


def _exact(counts, N, K, out, acc):
    """Whole numbers: a tile or row left out or added twice shows exactly.  Rows
    outside the experts' ranges hold NaN."""
    starts, m = _layout(counts)
    outside = torch.from_numpy(np.asarray(m) < 0).to(DEV)
    dC, A = _ints(-1, 2, len(m), N), _ints(-1, 3, len(m), K)
    dC[outside] = float("nan")
    A[outside] = float("nan")
    G = len(counts)
    old = _ints(-3, 4, G, N, K).to(out) if acc else None
    dB = old.clone() if acc else poison((G, N, K), out)
    L.grouped_gemm_contig_wgrad(dC, A, i32_dev(starts), i32_dev(np.array(counts)), dB, accumulate=acc)
    for g, (s, c) in enumerate(zip(starts.tolist(), counts)):
        want = dC[s:s + c].float().t().contiguous() @ A[s:s + c].float()   # whole numbers below 2^24: exact
        if acc:
            want += old[g].float()
        assert torch.equal(dB[g].float(), want.to(out).float()), g


@pytest.mark.parametrize("out,acc", KINDS)
@pytest.mark.parametrize("G,N,K,lo,hi", [
    (800, 128, 256, 0, 5), (600, 384, 128, 0, 200), (64, 640, 640, 0, 900), (64, 640, 640, 300, 301), (100, 512, 640, 257, 500)])
def test_wide_tiles_at_odd_sizes(G, N, K, lo, hi, out, acc):
    """More than six 128 x 128 tiles a compute unit, halves of 256 x 256 tiles on either side."""
    announce("wgrad wide", G, N, K, lo, hi, out, acc)
    counts = np.random.default_rng(G + N).integers(lo, hi, G)
    if lo == 0:
        counts[::7] = 0
    _exact(counts.tolist(), N, K, out, acc)


@pytest.mark.parametrize("out,acc", KINDS)
@pytest.mark.parametrize("counts,N,K", [
    ([0], 128, 128), ([1], 128, 128), ([63], 128, 256), ([65], 256, 128), ([128], 384, 640), ([129], 128, 128),
    ([20003], 256, 384), ([0, 7000, 0, 1, 64, 130], 384, 384), ([5, 0, 9000], 1152, 1280), ([900, 1023, 0, 1025, 1], 1664, 2048)])
def test_few_tiles(counts, N, K, out, acc):
    announce("wgrad few tiles", counts, N, K, out, acc)
    _exact(counts, N, K, out, acc)


@pytest.mark.parametrize("counts", [[64] * 8, [0, 700, 3, 0, 128, 1, 64, 200], [0] * 7 + [1]])
def test_few_rows_added_to_fp32(counts):
    announce("wgrad few rows", counts)
    _exact(counts, 4096, 2176, F32, True)


@pytest.mark.parametrize("N,K", [(128, 4194304), (4194304, 128)])
def test_few_rows_at_the_widest_matrices(N, K):
    """64 rows of K fp32 are 2^30 bytes, 64 rows of dC or A 2^29."""
    announce("wgrad widest", N, K)
    counts = [67]
    dC, A = _ints(-1, 2, 128, N), _ints(-1, 3, 128, K)
    dB = torch.ones(1, N, K, dtype=F32, device=DEV)
    L.grouped_gemm_contig_wgrad(dC, A, i32_dev(np.array([30])), i32_dev(np.array(counts)), dB, accumulate=True)
    p, q = dC[30:97].float().t().contiguous(), A[30:97].float()
    step = 1 << 18
    for n in range(0, N, step):
        for k in range(0, K, step):
            want = p[n:n + step] @ q[:, k:k + step].contiguous() + 1
            assert torch.equal(dB[0, n:n + step, k:k + step], want), (n, k)


@pytest.mark.parametrize("out,acc", KINDS)
def test_both_kernels_give_the_same_bits(out, acc):
    """An expert's gradient depends on its own rows alone: alone it has few tiles,
    among 64 it has wide ones."""
    announce("wgrad same bits", out, acc)
    counts = np.random.default_rng(5).integers(200, 700, 64)
    counts[[3, 9, 20, 40]] = [0, 1, 64, 65]
    starts, m = _layout(counts.tolist())
    assert len(m) > 256 * 64
    dC, A = randn(1, len(m), 640).to(DEV), randn(2, len(m), 640).to(DEV)
    old = randn(3, 64, 640, 640, dtype=out).to(DEV)
    dB = old.clone()
    L.grouped_gemm_contig_wgrad(dC, A, i32_dev(starts), i32_dev(counts), dB, accumulate=acc)
    for g in [3, 9, 20, 40, 0, 63, int(np.argmax(counts))]:
        one = old[g:g + 1].clone()
        L.grouped_gemm_contig_wgrad(dC, A, i32_dev(starts[g:g + 1]), i32_dev(counts[g:g + 1]), one, accumulate=acc)
        assert same_bits(one[0], dB[g]), g


@pytest.mark.parametrize("G", [6, 80])
def test_ranges_are_cut_in_both_kernels(G):
    """Ranges past M, negative counts and negative starts read nothing outside."""
    announce("wgrad ranges", G)
    M, N, K = 200, 640, 512
    dC, A = torch.ones(M, N, dtype=BF, device=DEV), torch.ones(M, K, dtype=BF, device=DEV)
    starts, nv = np.zeros(G, np.int32), np.zeros(G, np.int32)
    starts[-6:], nv[-6:] = [0, 150, 500, -3, 10, 190], [1, 1000, 4, 4, -2, 10]
    dB = poison((G, N, K), F32)
    L.grouped_gemm_contig_wgrad(dC, A, i32_dev(starts), i32_dev(nv), dB)
    want = [0.0] * (G - 6) + [1.0, 50.0, 0.0, 0.0, 0.0, 10.0]
    assert dB.amax((1, 2)).tolist() == want == dB.amin((1, 2)).tolist()
