"""Static checks of the gfx950 assembly of the products with an epilogue (no GPU needed:
the sources are compiled to assembly here).

The wide kernel's waits for loads to LDS count the vector memory instructions issued
behind them, so the number and place of these instructions is part of its correctness:
a step issues 2, 4 and 2 loads in the load parts of its phases 1, 2 and 3, an epilogue
8 stores (gated) or 16, 16 more with the kept product, and one load of the bias."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "scatter_grouped_gemm_amd", "csrc")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"


def _assembly(tmp_path_factory, name, kernel):
    """{template arguments: lines of the kernel}, and the text."""
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    from scatter_grouped_gemm_amd import build
    out = tmp_path_factory.mktemp("isa") / (name + ".s")
    subprocess.run([HIPCC, *build.FLAGS, "--cuda-device-only", "-S", os.path.join(CSRC, name + ".hip"), "-o", str(out)],
                   check=True, capture_output=True)
    text = out.read_text()
    found, key = {}, None
    for line in text.splitlines():
        m = re.match(r"_ZN3moe\S*?" + kernel + r"I((?:L[bi]\d+E)+)E\S*:", line)
        if m:
            key = tuple(int(x) for x in re.findall(r"L[bi](\d+)E", m.group(1)))
            found[key] = []
        elif line.startswith(".Lfunc_end"):
            key = None
        elif key is not None:
            found[key].append(line.split(";")[0].strip())
    return found, text


@pytest.fixture(scope="module")
def wide(tmp_path_factory):
    return _assembly(tmp_path_factory, "linear_wide", "linear_wide_kernel")


@pytest.fixture(scope="module")
def thin(tmp_path_factory):
    return _assembly(tmp_path_factory, "linear_thin", "linear_thin_kernel")


@pytest.fixture(scope="module")
def tile(tmp_path_factory):
    return _assembly(tmp_path_factory, "linear", "linear_tile_kernel")


def _no_spills(found, text, n):
    assert len(found) == n
    assert not re.search(r"\bscratch_(load|store)", text)
    sizes = [int(x) for x in re.findall(r"\.private_segment_fixed_size:\s+(\d+)", text)]
    assert len(sizes) == n and not any(sizes)


def test_no_register_is_spilled(wide, thin, tile):
    _no_spills(*wide, 18)    # (grouped, gated, pre, residual, fp32, tail)
    _no_spills(*thin, 12)    # (loads of A, blocks of 16 rows of B, gated)
    _no_spills(*tile, 8)     # (BM, BN, stages, gated)


def _to_lds(line, width="dwordx4"):
    return line.startswith("buffer_load_" + width + " ") and line.endswith(" lds")


def test_loads_of_a_wide_step_are_where_its_waits_count_them(wide):
    for key, lines in wide[0].items():
        parts, now = [], [0, 0]          # (loads to LDS, MFMAs) between barriers
        for line in lines:
            if line.startswith("s_barrier"):
                parts.append(tuple(now))
                now = [0, 0]
            elif _to_lds(line):
                now[0] += 1
            elif line.startswith("v_mfma"):
                now[1] += 1
        mfma = [i for i, p in enumerate(parts) if p[1]]
        assert all(parts[i] == (0, 16) for i in mfma) and 15 <= len(mfma) <= 18, (key, parts)
        loads = [sum(p[0] for p in parts[a + 1:b]) for a, b in zip(mfma, mfma[1:])]
        loads.append(now[0] + sum(p[0] for p in parts[mfma[-1] + 1:]))
        assert [x for x in loads if x] == [2, 4, 2] * 4, (key, loads)


def test_stores_of_a_wide_epilogue(wide):
    for key, lines in wide[0].items():
        grouped, gated, pre, res, f32, tail = key
        n = sum(line.startswith("buffer_store_dwordx4") for line in lines)
        assert n == (8 if gated else 16) * (2 if f32 else 1) + (16 if pre else 0), (key, n)
        others = [line for line in lines if re.match(r"(global|flat)_store|buffer_store(?!_dwordx4)|global_atomic", line)]
        assert not others, (key, others[:3])
        bias = sum(_to_lds(line, "dword") for line in lines)
        assert bias == 2, (key, bias)            # of the first tile, and behind an epilogue
        old = sum(line.startswith("buffer_load_dwordx4") and not line.endswith(" lds") for line in lines)
        assert old == (16 if res else 0), (key, old)


def test_loads_of_a_thin_group(thin):
    """Groups of U L loads, each by one of two ways, at the start (rolled up or not) and in
    the loop, whose one wait leaves all but the oldest group in flight."""
    for (al, nb, gated), lines in thin[0].items():
        per = al + 2 * nb
        u = 4 if per == 3 else 2
        groups = 63 // (per * u) + 1
        waits = [line for line in lines if re.match(r"s_waitcnt vmcnt\(%d\)" % (per * u * (groups - 2)), line)]
        assert len(waits) == 1, (al, nb, gated)
        n = sum(map(_to_lds, lines))
        assert n % (2 * per * u) == 0 and n >= 4 * per * u, (al, nb, gated, n)
        # the reads carry their own wait
        at = [i for i, line in enumerate(lines) if line.startswith("ds_read_b128")]
        assert len(at) == 2 * u * ((al + 1) // 2 + nb)
        assert any(lines[i].startswith("s_waitcnt lgkmcnt(0)") for i in range(at[-1] + 1, at[-1] + 4)), (al, nb, gated)


def test_loads_of_a_tile_step(tile):
    """Behind each step's wait and barrier its stage is filled again, by one of two ways."""
    for (bm, bn, stages, gated), lines in tile[0].items():
        per = (bm + bn) // 32
        at = [i for i, line in enumerate(lines) if line.startswith("s_barrier")]
        assert len(at) == stages + 1, (bm, bn)
        for a, b in zip(at[1:], at[2:]):
            assert sum(map(_to_lds, lines[a:b])) == 2 * per, (bm, bn, gated)
