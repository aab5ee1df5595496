"""Static checks of the gfx950 assembly of the weight gradient's kernel for few
tiles or few rows (no GPU needed: the source is compiled to assembly here).

Its waits for loads to LDS leave the eight loads of the next stage in flight, so a
step issues eight, after everyone has read the stage and before the next wait."""
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
    """{(fp32, accumulate): lines of the kernel}, and the text."""
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    from scatter_grouped_gemm_amd import build
    out = tmp_path_factory.mktemp("isa") / "wgrad_short.s"
    subprocess.run([HIPCC, *build.FLAGS, "--cuda-device-only", "-S", os.path.join(CSRC, "wgrad_short.hip"), "-o", str(out)],
                   check=True, capture_output=True)
    text = out.read_text()
    found, name = {}, None
    for line in text.splitlines():
        m = re.match(r"_ZN3moe\S*?wgrad_short_kernelILb(\d)ELb(\d)E\S*:", line)
        if m:
            name = (int(m.group(1)), int(m.group(2)))
            found[name] = []
        elif line.startswith(".Lfunc_end"):
            name = None
        elif name is not None:
            found[name].append(line.split(";")[0].strip())
    return found, text


def test_no_register_is_spilled(kernels):
    found, text = kernels
    assert sorted(found) == [(0, 0), (0, 1), (1, 0), (1, 1)]
    assert not re.search(r"\bscratch_(load|store)", text)
    assert not any(int(x) for x in re.findall(r"\.private_segment_fixed_size:\s+(\d+)", text))


def _is_load(line):
    return line.startswith("buffer_load") and line.endswith(" lds")


def test_eight_loads_a_step_and_what_waits_for_them(kernels):
    for key, lines in kernels[0].items():
        at = [i for i, line in enumerate(lines) if line.startswith("s_barrier")]
        assert len(at) == 4, key                              # a pair of steps, two barriers a step
        first, read, second, again = at
        parts = [lines[:first], lines[first:read], lines[read:second], lines[second:again], lines[again:]]
        assert [sum(map(_is_load, p)) for p in parts] == [16, 0, 8, 0, 8], key
        assert [sum(x.startswith("v_mfma") for x in p) for p in parts] == [0, 32, 0, 32, 0], key
        assert [sum(x.startswith("ds_read") for x in p) for p in parts] == [0, 32, 0, 32, 0], key
        for p in (parts[0], parts[2]):                        # this stage's loads have arrived before the barrier
            waits = [x for x in p if "vmcnt" in x]
            assert len(waits) == 1 and re.match(r"s_waitcnt vmcnt\(8\)", waits[0]), (key, waits)
            assert not any(_is_load(x) for x in p[p.index(waits[0]):]), key
        assert not any("vmcnt" in x for p in (parts[1], parts[3]) for x in p), key
        for p in (parts[1], parts[3]):                        # and its reads before it is loaded again
            last = max(i for i, x in enumerate(p) if x.startswith("ds_read"))
            assert any("lgkmcnt(0)" in x for x in p[last:]), key
        ended = [x for x in parts[4] if x.startswith("s_waitcnt vmcnt")]
        assert re.match(r"s_waitcnt vmcnt\(0\)", ended[0]), (key, ended)


def test_stores_of_a_tile(kernels):
    for key, lines in kernels[0].items():
        assert sum(line.startswith("buffer_store_dwordx4") for line in lines) == (16 if key[0] else 8), key
        assert not [x for x in lines if re.match(r"(global|flat)_store|buffer_store(?!_dwordx4)|global_atomic", x)], key


def test_the_input_gradient_of_few_tiles(tmp_path):
    """The same for its 128 x 128 tiles: eight loads a step, no wait between a step's
    barriers, eight stores, nothing spilled."""
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    from scatter_grouped_gemm_amd import build
    out = tmp_path / "dgrad_short.s"
    subprocess.run([HIPCC, *build.FLAGS, "--cuda-device-only", "-S", os.path.join(CSRC, "dgrad_short.hip"), "-o", str(out)],
                   check=True, capture_output=True)
    text = out.read_text()
    assert not re.search(r"\bscratch_(load|store)", text)
    lines = [x.split(";")[0].strip() for x in text[:text.index(".Lfunc_end")].splitlines()]
    at = [i for i, line in enumerate(lines) if line.startswith("s_barrier")]
    assert len(at) == 4
    first, read, second, again = at
    parts = [lines[:first], lines[first:read], lines[read:second], lines[second:again], lines[again:]]
    assert [sum(map(_is_load, p)) for p in parts] == [16, 0, 8, 0, 8]
    assert [sum(x.startswith("v_mfma") for x in p) for p in parts] == [0, 32, 0, 32, 0]
    assert [sum(x.startswith("ds_read") for x in p) for p in parts] == [0, 24, 0, 24, 0]
    start = next(i for i, x in enumerate(parts[0]) if _is_load(x))
    for p in (parts[0][start:], parts[2]):
        waits = [x for x in p if "vmcnt" in x]
        assert len(waits) == 1 and re.match(r"s_waitcnt vmcnt\(8\)", waits[0]), waits
        assert not any(_is_load(x) for x in p[p.index(waits[0]):])
    for p in (parts[1], parts[3]):
        assert not any("vmcnt" in x for x in p)
        last = max(i for i, x in enumerate(p) if x.startswith("ds_read"))
        assert any("lgkmcnt(0)" in x for x in p[last:])
    ended = [x for x in parts[4] if x.startswith("s_waitcnt vmcnt")]
    assert re.match(r"s_waitcnt vmcnt\(0\)", ended[0])
    assert sum(line.startswith("buffer_store_dwordx4") for line in lines) == 8
    assert not [x for x in lines if re.match(r"(global|flat)_store|buffer_store(?!_dwordx4)|global_atomic", x)]
