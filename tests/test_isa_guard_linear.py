"""CPU check of the generated gfx950 code of the linear's tile kernel.

Its direct-to-LDS loads are inline assembly, with M0 set in the same statement
(followed by the one wait state a DMA that reads a freshly written M0 needs) and
completion tracked by in-order vmcnt waits.  That is sound only while the
compiler's own code uses neither M0 nor vector memory between the first DMA and
the drain after the last step (a load or a spill of its own would be counted by
those waits), and while nothing spills.  The source is compiled to assembly with
the build's flags (cross-compiling; no GPU needed)."""
import os
import re
import subprocess

import pytest

from tests.test_isa_guard import CSRC, ROOT, _hipcc, _split_asm


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    hipcc = _hipcc()
    if hipcc is None:
        pytest.skip("hipcc not available")
    out = tmp_path_factory.mktemp("isa") / "linear_tile.s"
    cmd = [hipcc, "-O3", "-std=c++17", "-I", os.path.join(ROOT, "include"), "--offload-arch=gfx950",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-mllvm", "-amdgpu-mfma-vgpr-form",
           "--cuda-device-only", "-S", "-o", str(out), os.path.join(CSRC, "linear_tile.hip")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    text = out.read_text()
    found = {}
    for m in re.finditer(r"^(_ZN3moe\w*linear_tile_kernel\w*):(?:\s*;.*)?$", text, re.M):
        found[m.group(1)] = text[m.end():text.find("s_endpgm", m.end())]
    scratch = dict(re.findall(r"\.name:\s+(_ZN3moe\w*linear_tile_kernel\w*)\n(?:.*\n)*?\s+\.private_segment_fixed_size:\s+(\d+)",
                              text))
    assert found, "no tile kernels in the assembly"
    return found, scratch


def test_the_flags_are_the_builds():
    text = open(os.path.join(ROOT, "block_scaled_fp4_pre_amd", "build.py")).read()
    assert '"linear_tile.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"]' in text


def test_m0_only_in_dma_statements(kernels):
    for name, body in kernels[0].items():
        compiler, blocks, _ = _split_asm(body)
        assert not [t for t in compiler if re.search(r"\bm0\b", t)], name
        dmas = [b for b in blocks if any(re.search(r"\bm0\b", t) for t in b)]
        assert dmas, name
        for b in dmas:
            assert len(b) == 3 and b[0].startswith("s_mov_b32 m0,") and b[1].startswith("s_nop"), (name, b)
            assert b[2].startswith("global_load_lds_dword"), (name, b)


def test_no_other_vector_memory_while_the_ring_runs(kernels):
    """Between the first DMA and the drain (the last inline wait of vmcnt(0)) the
    compiler issues no vector memory and no vmcnt wait of its own."""
    for name, body in kernels[0].items():
        lines = body.splitlines()
        first = next(i for i, t in enumerate(lines) if "global_load_lds" in t)
        drain = max(i for i, t in enumerate(lines) if re.search(r"s_waitcnt vmcnt\(0\) lgkmcnt\(0\)\s*$", t)
                    and "ASMSTART" in lines[i - 1])
        asm = True                                  # the first DMA is inside its statement
        for t in (t.strip() for t in lines[first:drain]):
            asm = True if t.startswith(";;#ASMSTART") else False if t.startswith(";;#ASMEND") else asm
            if not asm and not t.startswith(";"):
                assert not re.match(r"(global|flat|buffer|scratch)_", t), (name, t)
                assert not (t.startswith("s_waitcnt") and "vmcnt" in t), (name, t)


def test_no_scratch(kernels):
    found, scratch = kernels
    for name in found:
        assert scratch.get(name) == "0", (name, scratch.get(name))
