"""Set-up that every device of a process needs for itself (a kernel's
shared-memory limit holds on the device it was set on), on the host."""
import glob
import os
import re
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gemm_deterministic_bf16_gb300", "csrc")

PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "per_device.h"
int main() {
  static detffn::PerDevice ready;
  std::vector<int> set;
  int fail = 0;
  auto call = [&](int device) { return ready.once(device, [&] { set.push_back(device); return fail; }); };
  // A device's first call sets it up and later ones do not; a second device's does again.
  if (call(0) || call(0) || call(1) || call(0) || call(1) || call(63) || call(63)) return 1;
  if (set != std::vector<int>{0, 1, 63}) return 2;
  // A failure is reported, and tried again.
  fail = 7;
  if (call(2) != 7 || call(2) != 7 || call(1) != 0) return 3;
  fail = 0;
  if (call(2) || call(2)) return 4;
  if (set != std::vector<int>{0, 1, 63, 2, 2, 2}) return 5;
  // Devices beyond those kept are set up at every call.
  if (call(64) || call(64) || call(1000)) return 6;
  return set.size() == 9 ? 0 : 7;
}
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs a host compiler")
def test_each_device_is_set_up(tmp_path):
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(PROGRAM)
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_no_kernel_is_set_up_for_one_device_alone():
    """Every cudaFuncSetAttribute stands inside a once_per_device."""
    seen = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"\bcudaFuncSetAttribute\s*\(", text):
            before = text[:m.start()]
            at = before.rfind("once_per_device(")
            assert at >= 0 and "call_once" not in before[at:], path
            depth = 0
            for c in before[at + len("once_per_device"):]:
                depth += (c == "(") - (c == ")")
            assert depth > 0, (path, before.count("\n") + 1)
            seen += 1
    assert seen >= 5
