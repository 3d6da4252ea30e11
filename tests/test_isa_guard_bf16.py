"""CPU check of the generated gfx950 code of the bfloat16 products' kernels, as
tests/test_isa_guard_linear.py's for the linear's: their direct-to-LDS copies are inline assembly
counted by vmcnt waits, sound only while the compiler uses neither M0 nor vector
memory of its own between the first copy and the drain, and while nothing spills."""
import os
import re
import subprocess

import pytest

from tests.test_isa_guard import CSRC, ROOT, _hipcc, _split_asm


FLAGS = {"bf16_tile": ["-mllvm", "-amdgpu-mfma-vgpr-form"], "bf16_split": []}


@pytest.fixture(scope="module", params=FLAGS)
def kernels(request, tmp_path_factory):
    hipcc = _hipcc()
    if hipcc is None:
        pytest.skip("hipcc not available")
    name = request.param
    out = tmp_path_factory.mktemp("isa") / f"{name}.s"
    cmd = [hipcc, "-O3", "-std=c++17", "-I", os.path.join(ROOT, "include"), "--offload-arch=gfx950",
           "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", *FLAGS[name],
           "--cuda-device-only", "-S", "-o", str(out), os.path.join(CSRC, f"{name}.hip")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    text = out.read_text()
    found = {}
    for m in re.finditer(rf"^(_ZN3moe\w*{name}_kernel\w*):(?:\s*;.*)?$", text, re.M):
        found[m.group(1)] = text[m.end():text.find(".section", m.end())]
    scratch = dict(re.findall(rf"\.name:\s+(_ZN3moe\w*{name}_kernel\w*)\n(?:.*\n)*?\s+\.private_segment_fixed_size:\s+(\d+)",
                              text))
    assert found, "no kernels in the assembly"
    return found, scratch


def test_the_flags_are_the_builds():
    text = open(os.path.join(ROOT, "block_scaled_fp4_pre_amd", "build.py")).read()
    assert '"bf16_tile.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form"]' in text


def test_m0_only_in_copy_statements(kernels):
    for name, body in kernels[0].items():
        compiler, blocks, _ = _split_asm(body)
        assert not [t for t in compiler if re.search(r"\bm0\b", t)], name
        copies = [b for b in blocks if any(re.search(r"\bm0\b", t) for t in b)]
        assert copies, name
        for b in copies:
            assert len(b) == 3 and b[0].startswith("s_mov_b32 m0,") and b[1].startswith("s_nop"), (name, b)
            assert b[2].startswith("global_load_lds_dword"), (name, b)


def test_no_other_vector_memory_while_copies_are_in_flight(kernels):
    for name, body in kernels[0].items():
        lines = body.splitlines()
        first = next(i for i, t in enumerate(lines) if "global_load_lds" in t)
        drain = max(i for i, t in enumerate(lines) if re.search(r"s_waitcnt vmcnt\(0\) lgkmcnt\(0\)\s*$", t)
                    and "ASMSTART" in lines[i - 1])
        asm = True                                  # the first copy is inside its statement
        for t in (t.strip() for t in lines[first:drain]):
            asm = True if t.startswith(";;#ASMSTART") else False if t.startswith(";;#ASMEND") else asm
            if not asm and not t.startswith(";"):
                assert not re.match(r"(global|flat|buffer|scratch)_", t), (name, t)
                assert not (t.startswith("s_waitcnt") and "vmcnt" in t), (name, t)


def test_no_scratch(kernels):
    found, scratch = kernels
    for name in found:
        assert scratch.get(name) == "0", (name, scratch.get(name))
