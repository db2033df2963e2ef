"""The form that a call of the microscaled product takes: the shapes that the
GPU tests multiply take the forms that they are listed under, and no form is
missing.  The library's own choice (csrc/mx_plan.h), compiled for the host."""
import itertools
import os
import shutil
import subprocess

import pytest

from tests import mx_shapes

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SMS = 148
LISTS = {0: mx_shapes.WIDE_K, 1: mx_shapes.NARROW_K}  # by whether both are of 4 bits


@pytest.fixture(scope="module")
def forms(tmp_path_factory):
    """Forms of (T, N, K, 4 bits both, rows of y on 16-byte boundaries)."""
    if shutil.which("g++") is None:
        pytest.skip("needs g++")
    exe = tmp_path_factory.mktemp("plan") / "plan"
    subprocess.run(["g++", "-std=c++17", "-O2", "-I", os.path.join(ROOT, "expert_ffn_execution_b200", "csrc"),
                    os.path.join(ROOT, "tests", "native", "mx_plan_check.cpp"), "-o", str(exe)], check=True)

    def ask(calls):
        r = subprocess.run([str(exe)], input="\n".join(f"{T} {N} {K} {f4} {al} {SMS}" for T, N, K, f4, al in calls),
                           capture_output=True, text=True, check=True)
        out = []
        for (T, N, K, _, _), line in zip(calls, r.stdout.splitlines(), strict=True):
            nt, ranks, wide = map(int, line.split())
            if nt:
                ctas = -(-N // 128) * -(-T // nt) * ranks
                out.append((nt, ranks, 1 if ranks <= 2 and ctas <= SMS else 2))
            else:
                out.append((0, bool(wide)))
        return out
    return ask


@pytest.mark.parametrize("f4", [0, 1])
def test_listed_shapes_take_their_forms(forms, f4):
    listed = [(form, s) for form, shapes in LISTS[f4].items() for s in shapes]
    got = forms([(*s, f4, int(form != (0, False))) for form, s in listed])
    assert [(g, s) for g, (_, s) in zip(got, listed)] == listed


@pytest.mark.parametrize("f4", [0, 1])
def test_every_form_is_listed(forms, f4):
    calls = [(T, N, K, f4, al)
             for T, N, K in itertools.product((1, 5, 16, 20, 32, 33, 64, 65, 90, 128, 150, 256, 300, 512, 1000, 4096),
                                              (1, 129, 700, 1300, 2563, 4100, 5001, 8200, 10240, 16000, 25000, 40000),
                                              (128, 384, 640, 896, 1152, 1664, 2176, 2688, 4224, 5504, 8192, 16384))
             for al in (0, 1)]
    assert set(forms(calls)) == set(LISTS[f4])
