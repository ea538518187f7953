"""The 4-bit tile kernels, as compiled for gfx950: their waits leave no copy of the step at hand in flight.

A step's copies into LDS are complete at `s_waitcnt vmcnt(N)` if the steps after it have issued at least N
loads since.  The compiler may make one load of two (a lane's scales of two groups), so N is compared with the loads in
the code that it made, on the host (no GPU).
"""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gemm_f32_amd", "csrc")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    """{mangled name: assembly} of the kernels of w4_tile.hip."""
    clang = next((c for c in ("/opt/rocm/lib/llvm/bin/clang++", shutil.which("amdclang++") or "") if c and os.path.exists(c)),
                 None)
    if clang is None:
        pytest.skip("no ROCm clang++ to compile gfx950 assembly")
    out = str(tmp_path_factory.mktemp("asm") / "w4_tile.s")
    subprocess.run([clang, "-mllvm", "-amdgpu-mfma-vgpr-form=1", "--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang",
                    "-target-feature", "-Xclang", "-packed-fp32-ops", "-I" + os.path.join(ROOT, "include"), "-I" + CSRC,
                    "--cuda-device-only", "-S", "-x", "hip", os.path.join(CSRC, "w4_tile.hip"), "-o", out],
                   check=True, capture_output=True)
    asm = open(out).read()
    return {m.group(1): asm[m.end():asm.index("s_endpgm", m.end())] for m in re.finditer(r"^(_Z\S*k_w4_tile\S*): ;", asm, re.M)}


def steps(body):
    """(N, loads) of every explicit partial wait: loads issued from it to the next explicit wait."""
    parts = body.split("#ASMSTART")
    waits = [(i, int(m.group(1))) for i, p in enumerate(parts) if (m := re.match(r"\s*s_waitcnt vmcnt\((\d+)\) lgkmcnt", p))]
    for (i, n), (j, _) in zip(waits, waits[1:]):
        if n > 0:
            code = "".join(parts[i:j])
            yield n, len(re.findall(r"^\s*(?:global|buffer)_load_", code, re.M)), "lds" in code


# kernels per step of a ring of three (one later step in flight) and of four (two)
@pytest.mark.parametrize("kernel,later", [("k_w4_tileI", 1), ("k_w4_tile_tI", 2)])
def test_waits_cover_the_copies_of_a_step(kernels, kernel, later):
    seen = 0
    for name, body in kernels.items():
        if kernel not in name:
            continue
        for n, loads, copies in steps(body):
            assert copies and n <= later * loads, f"{name}: vmcnt({n}) after {later} step(s) of {loads} loads"
            seen += 1
    assert seen >= 3 * 12, "the kernels' waits were not found"


def test_no_scratch_memory(kernels):
    for name, body in kernels.items():
        assert "scratch_" not in body, name
