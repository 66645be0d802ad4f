"""The choice between the kernels of the FP4 x FP4 products (csrc/fp4_ways.h), on the host: the sizes of fp4_ways.py take the
ways that it says, so that an estimate fitted anew does not leave a kernel without a test."""
from __future__ import annotations

import os
import re
import shutil
import subprocess

import pytest

from fp4_ways import CONTIGUOUS, DENSE, MASKED, PAIRS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "fp8_gemm_nt_gb300", "csrc")
FORMS = {"dense": DENSE, "contiguous": CONTIGUOUS, "masked": MASKED}


@pytest.fixture(scope="module")
def ways(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    exe = tmp_path_factory.mktemp("ways") / "fp4_ways_check"
    build = subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, os.path.join(ROOT, "tests", "fp4_ways_check.cpp"), "-o", str(exe)],
                           capture_output=True, text=True)
    assert build.returncode == 0, build.stderr

    def of(form, sizes, sms=152):
        args = [f"{form}:{','.join(map(str, s))}" for s in sizes]
        out = subprocess.run([str(exe), str(sms), *args], capture_output=True, text=True, timeout=60)
        assert out.returncode == 0, out.stderr
        return [tuple(map(int, line.split())) for line in out.stdout.splitlines()]
    return of


@pytest.mark.parametrize("form", FORMS)
def test_sizes_take_the_ways_they_stand_for(ways, form):
    assert dict(zip([s for s, _ in FORMS[form]], ways(form, [s for s, _ in FORMS[form]]))) == dict(FORMS[form])
    assert dict(zip(PAIRS[form], (w[0] for w in ways(form, PAIRS[form].values())))) == {bn: bn for bn in PAIRS[form]}
    assert all(w[1] == 0 for w in ways(form, PAIRS[form].values()))


def test_every_kernel_is_among_them():
    splits = re.search(r"kSplits\[\] = \{(.*?)\};", open(os.path.join(CSRC, "fp4_ways.h")).read()).group(1)
    splits = {tuple(map(int, p)) for p in re.findall(r"\{(\d+), (\d+)\}", splits)}
    pairs = {(128, 0), (256, 0), (384, 0)}
    assert {w for _, w in DENSE} == splits | pairs
    assert {w for _, w in CONTIGUOUS} == pairs and {w for _, w in MASKED} == pairs


def test_any_size_takes_a_way(ways):
    sizes = [(m, n, k) for m in (1, 100, 129, 5000, 1 << 30) for n in (16, 1040, 1 << 30) for k in (128, 16384, 1 << 30)]
    for sms in (1, 2, 20, 152):
        for bn, w in ways("dense", sizes, sms):
            assert (bn, w) in {(128, 0), (256, 0), (384, 0), (64, 1), (64, 2), (64, 4), (96, 2), (128, 1), (128, 2), (192, 1)}
    # on few SMs a cluster of four is more than there is room for
    assert all(w != 4 for _, w in ways("dense", sizes, 8))
