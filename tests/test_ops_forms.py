"""The choice of a product's form goes by the tiles that its launch makes: csrc/forms.h, on the host."""

import os
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "deterministic_shot_all_gb300", "csrc")


def _run(tmp_path, *first):
    from deterministic_shot_all_gb300 import _build
    exe = str(tmp_path / "forms_check")
    dirs = [*first, CSRC, os.path.join(ROOT, "include")]
    subprocess.run([_build.nvcc(), "-std=c++17", "-O1", os.path.join(ROOT, "tests", "c_abi", "forms_check.cpp"),
                    *(f"-I{d}" for d in dirs), "-o", exe], check=True)
    return subprocess.run([exe], capture_output=True, text=True)


def test_estimates_count_the_tiles_of_the_launch(tmp_path):
    r = _run(tmp_path)
    assert r.returncode == 0, r.stdout
    assert int(r.stdout.split()[0]) > 10000


@pytest.mark.parametrize("right,wrong", [
    ("products * ceil_div(c.rows, wide ? 2 * kLanes : bn)", "ceil_div(products * c.rows, wide ? 2 * kLanes : bn)"),
    ("tiles = tiles_of(c, false, bn, 1).all();", "tiles = ceil_div(c.cols, kLanes) * ceil_div((c.p2 ? 2 : 1) * c.rows, bn);"),
    ("tiles = tiles_of(c, true, bn, 1).all();", "tiles = ceil_div((c.p2 ? 2 : 1) * c.rows, 256) * ceil_div(c.cols, bn);")])
def test_the_check_sees_a_miscount(tmp_path, right, wrong):
    with open(os.path.join(CSRC, "forms.h")) as f:
        text = f.read()
    assert text.count(right) == 1
    (tmp_path / "forms.h").write_text(text.replace(right, wrong))
    assert _run(tmp_path, str(tmp_path)).returncode == 1
