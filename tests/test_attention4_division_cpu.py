"""The division of the work over a 4-bit cache, which has weights of its own, compiled for the host."""
import os
import shutil
import subprocess

import pytest

from test_attention_division_cpu import CSRC, HERE, INCLUDE, constant


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
@pytest.mark.parametrize("kernel", ["kn11_attend.cu", "kn12_attend_tc.cu"])
def test_every_tile_falls_to_one_cta(kernel, tmp_path):
    with open(os.path.join(CSRC, "dt_attend.cuh")) as f:
        s = f.read()

    def piece(first, last):  # what needs no GPU
        return s[s.index(first):s.index(last)]
    body = piece("constexpr int AT_TILE", "// One warp: the share of CTA") + piece("// Walks a CTA's segments", "// Factor from a product")
    (tmp_path / "division_body.h").write_text(body)
    with open(os.path.join(HERE, "attention_division.cpp")) as f:
        program = f.read()
    for form in ("AtPlan<K_ROWS", "AtWalk<K_ROWS, K_ATOM"):
        assert form + ">" in program
        program = program.replace(form + ">", form + ", 4>")
    (tmp_path / "division.cpp").write_text(program)
    exe = str(tmp_path / "division")
    flags = ["-DK_%s=%s" % (n, constant(kernel, c)) for n, c in (("ROWS", "ROWS"), ("ATOM", "ATOM"), ("MIN_SHARE", "MIN_SHARE4"))]
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", str(tmp_path), "-I", INCLUDE, *flags, str(tmp_path / "division.cpp"),
                    "-o", exe], check=True)
    r = subprocess.run([exe, "4000"], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout
