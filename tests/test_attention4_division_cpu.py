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
    forms = [("AtPlan<K_ROWS>", "AtPlan<K_ROWS, 4>"), ("AtWalk<K_ROWS, K_ATOM>", "AtWalk<K_ROWS, K_ATOM, 4>")]
    if kernel == "kn11_attend.cu":
        # the larger head, and shares of two sizes, in every second batch
        forms += [("AtShare s;", "AtShareLead<%s> s; s.head = head, s.half = lead ? grid / 2 : 0;" % constant(kernel, "LEAD")),
                  ("long long total = 0;", "const bool full = it % 2; const uint32_t head = full ? Plan::HEAD_FULL : Plan::HEAD;"
                   " const uint32_t least = K_MIN_SHARE + head - Plan::HEAD; long long total = 0;"),
                  ("Plan::req(a, b));", "Plan::req(a, b), head);"), ("Plan::cost(a, r)", "Plan::cost(a, r, head)"),
                  ("total / K_MIN_SHARE", "total / least"),
                  ("std::map<std::tuple", "const bool lead = full && ctas == grid && grid % 2 == 0; std::map<std::tuple")]
    for old, new in forms:
        assert old in program, old
        program = program.replace(old, new)
    (tmp_path / "division.cpp").write_text(program)
    exe = str(tmp_path / "division")
    flags = ["-DK_%s=%s" % (n, constant(kernel, c)) for n, c in (("ROWS", "ROWS"), ("ATOM", "ATOM"), ("MIN_SHARE", "MIN_SHARE4"))]
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", str(tmp_path), "-I", INCLUDE, *flags, str(tmp_path / "division.cpp"),
                    "-o", exe], check=True)
    r = subprocess.run([exe, "4000"], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout == "ok\n", r.stdout
