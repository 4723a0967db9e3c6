"""Reads of rows off 16 bytes stay inside their matrices: the kernels' own address arithmetic, on the host."""

import os
import shutil
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "deterministic_shot_all_gb300", "csrc")


def _run(tmp_path, headers, *flags):
    cxx = shutil.which(os.environ.get("CXX", "g++"))
    assert cxx, "a C++ compiler is needed"
    exe = str(tmp_path / "spans_check")
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", os.path.join(ROOT, "tests", "c_abi", "spans_check.cpp"), "-I",
                    headers, "-o", exe, *flags], check=True)
    return subprocess.run([exe], capture_output=True, text=True)


def test_reads_stay_inside(tmp_path):
    r = _run(tmp_path, CSRC)
    assert r.returncode == 0, r.stdout
    assert int(r.stdout.split()[0]) > 1000000


@pytest.mark.parametrize("right,wrong", [
    ("return uint32_t((row + bytes - first_unit(row) + 15) >> 4);",
     "return uint32_t((row + bytes - first_unit(row) + 31) >> 4);"),                # a unit too many
    ("at + 16 <= hi ? 16 : uint32_t(hi - at)", "16"),                              # past the matrix's end
    ("at + 16 <= hi ? 16 : uint32_t(hi - at)", "at + 16 <= hi ? 16 : uint32_t(hi - at) - 1"),
    ("return row & ~uintptr_t(15);", "return row & ~uintptr_t(31);"),              # before its begin
    ("c.fast = o.mn ? col + 8 <= o.ncols : true;", "c.fast = true;"),
    ("row < o.nrows ? int(o.ncols)", "row <= o.nrows ? int(o.ncols)"),
    ("cols - c0 >= int64_t(kRealignChunk) + odd", "cols - c0 >= int64_t(kRealignChunk)"),
    ("c + c0 >= 0 && c + 1 < rest", "c + c0 >= 0 && c < rest")])
def test_the_check_sees_a_read_outside(tmp_path, right, wrong):
    with open(os.path.join(CSRC, "spans.h")) as f:
        text = f.read()
    assert text.count(right) == 1
    (tmp_path / "spans.h").write_text(text.replace(right, wrong))
    assert _run(tmp_path, str(tmp_path)).returncode == 1
