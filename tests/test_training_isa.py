"""Static checks of the gradient products' gfx950 assembly (no GPU needed: the
source is compiled to assembly here).

Their waits for loads to LDS count the vector memory instructions issued behind
them, so the number and place of these instructions is part of their correctness:
a step issues 2, 4 and 2 loads in the load parts of its phases 1, 2 and 3, and an
epilogue 16 stores (bf16) or 32 (fp32), whatever the compiler makes of the rest.
"""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "scatter_grouped_gemm_amd", "csrc")
HIPCC = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{(wgrad, fp32, accumulate) or "thin": lines of the kernel}, and the text."""
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    from scatter_grouped_gemm_amd import build
    out = tmp_path_factory.mktemp("isa") / "gemm_grad.s"
    subprocess.run([HIPCC, *build.FLAGS, "--cuda-device-only", "-S", os.path.join(CSRC, "gemm_grad.hip"), "-o", str(out)],
                   check=True, capture_output=True)
    text = out.read_text()
    found, name = {}, None
    for line in text.splitlines():
        m = re.match(r"_ZN3moe\S*?(gemm_grad_kernelILb(\d)ELb(\d)ELb(\d)E|dgrad_thin_kernel)\S*:", line)
        if m:
            name = "thin" if m.group(2) is None else tuple(int(m.group(i)) for i in (2, 3, 4))
            found[name] = []
        elif line.startswith(".Lfunc_end"):
            name = None
        elif name is not None:
            found[name].append(line.split(";")[0].strip())
    return found, text


def test_no_register_is_spilled(kernels):
    found, text = kernels
    assert sorted(k for k in found if k != "thin") == [(0, 0, 0), (1, 0, 0), (1, 0, 1), (1, 1, 0), (1, 1, 1)]
    assert not re.search(r"\bscratch_(load|store)", text)
    sizes = [int(x) for x in re.findall(r"\.private_segment_fixed_size:\s+(\d+)", text)]
    assert len(sizes) == 6 and not any(sizes)


def test_loads_of_a_step_are_where_its_waits_count_them(kernels):
    found, _ = kernels
    for key, lines in found.items():
        if key == "thin":
            continue
        # (loads to LDS, MFMAs) between barriers, from the first MFMA part on
        parts, now = [], [0, 0]
        for line in lines:
            if line.startswith("s_barrier"):
                parts.append(tuple(now))
                now = [0, 0]
            elif line.startswith("buffer_load") and line.endswith(" lds"):
                now[0] += 1
            elif line.startswith("v_mfma"):
                now[1] += 1
        mfma = [i for i, p in enumerate(parts) if p[1]]
        # four steps of four phases; a pair's last part may be there twice, for the two
        # ways out of its loads, and may stand before them
        assert all(parts[i] == (0, 16) for i in mfma) and 15 <= len(mfma) <= 18, key
        loads = [sum(p[0] for p in parts[a + 1:b]) for a, b in zip(mfma, mfma[1:])]
        if key[2]:                                           # accumulating: a barrier ends the last loads
            loads.append(parts[mfma[-1] + 1][0])
        else:
            loads.append(now[0] + sum(p[0] for p in parts[mfma[-1] + 1:]))
        assert [x for x in loads if x] == [2, 4, 2] * 4, (key, loads)


def test_stores_of_an_epilogue(kernels):
    found, _ = kernels
    for key, lines in found.items():
        if key == "thin":
            continue
        n = sum(line.startswith("buffer_store_dwordx4") for line in lines)
        assert n == (32 if key[1] else 16), (key, n)
        others = [line for line in lines if re.match(r"(global|flat)_store|buffer_store(?!_dwordx4)|global_atomic", line)]
        assert not others, (key, others[:3])


def test_the_narrow_kernel_issues_four_loads_a_step(kernels):
    lines = kernels[0]["thin"]
    at = [i for i, line in enumerate(lines) if line.startswith("s_barrier")]
    assert len(at) == 1                                       # one barrier: the step's
    behind = [line for line in lines[at[0]:] if line.startswith("buffer_load") and line.endswith(" lds")]
    assert len(behind) == 4
    assert any(re.match(r"s_waitcnt vmcnt\(24\)", line) for line in lines)
