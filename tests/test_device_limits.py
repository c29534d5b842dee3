"""Kernels' shared-memory limits hold for one device each: the record of what was
set (csrc/nys_device.h), compiled with the host compiler around a fake of the call
that sets them."""
import os
import shutil
import subprocess

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "streaming_nystr_landmark_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include "nys_device.h"

int main() {
  static nys::PerDevice limits;
  int calls = 0, answer = 0;
  auto ask = [&](int device, size_t bytes) {
    const int before = calls;
    const int rc = limits.raise(device, bytes, 100, [&] { ++calls; return answer; });
    std::printf("%d %d\n", calls - before, rc);
  };
  ask(0, 100);              // within what every device has
  ask(0, 200); ask(0, 200); ask(0, 150);
  ask(1, 200); ask(1, 200); // another device has a limit of its own
  ask(0, 300); ask(1, 250);
  answer = 7;
  ask(2, 200);              // refused
  answer = 0;
  ask(2, 200); ask(2, 200); // and asked for again
  ask(1000, 200); ask(1000, 200); ask(-1, 200);
}
"""


def test_limits_are_set_once_for_each_device(tmp_path):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "limits.cpp", tmp_path / "limits"
    src.write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-Wall", "-Werror", f"-I{CSRC}", str(src), "-o", str(exe)],
                   check=True)
    got = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout.split("\n")
    assert got[:-1] == ["0 0", "1 0", "0 0", "0 0", "1 0", "0 0", "1 0", "1 0", "1 7", "1 0", "0 0",
                        "1 0", "1 0", "1 0"]


def test_no_kernel_keeps_a_record_of_its_own():
    """Every shared-memory limit is set through that record."""
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as fh:
            text = fh.read()
        assert ("cudaFuncSetAttribute" in text) == (name == "nys_device.h"), name
