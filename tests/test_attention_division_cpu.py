"""Tree attention's division of the work, compiled for the host from the kernels' header."""
import os
import re
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "speculative_decoding_draft_bf16_gb300", "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")


def constant(source, name):
    with open(os.path.join(CSRC, source)) as f:
        return re.search(r"constexpr \w+ (?:\w+ = \w+, )*%s = (\d+)" % name, f.read()).group(1)


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
@pytest.mark.parametrize("kernel", ["kn11_attend.cu", "kn12_attend_tc.cu"])
def test_every_tile_falls_to_one_cta(kernel, tmp_path):
    with open(os.path.join(CSRC, "dt_attend.cuh")) as f:
        s = f.read()

    def piece(first, last):  # what needs no GPU
        return s[s.index(first):s.index(last)]
    body = piece("constexpr int AT_TILE", "// One warp: the share of CTA") + piece("// Walks a CTA's segments", "// Factor from a product")
    (tmp_path / "division_body.h").write_text(body)
    exe = str(tmp_path / "division")
    flags = ["-DK_%s=%s" % (n, constant(kernel, n)) for n in ("ROWS", "ATOM", "MIN_SHARE")]
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", str(tmp_path), "-I", INCLUDE, *flags,
                    os.path.join(HERE, "attention_division.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe, "4000"], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout
