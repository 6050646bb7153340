"""Numbers that belong to a device (the resident clusters by which the paged attention chooses its launch) are kept
by device: a C++ program over the header that the library uses, with a fake for the CUDA query."""
import os
import subprocess

from conftest import ROOT

PROGRAM = r"""
#include <cstdio>
#include <initializer_list>
#include "per_device.h"

enum Rc { kOk = 0, kBad = 2 };
int asked = 0;

int main() {
  static ntx::PerDevice<9> fit;
  int v = -1;
  auto ask = [](int dev, int size) {
    return [=](int* n) { ++asked; *n = 1000 * dev + size; return kOk; };
  };
  for (int round = 0; round < 3; ++round)
    for (int dev : {0, 1, 63})
      for (int size = 1; size < 9; ++size)
        if (fit.get(dev, size, &v, ask(dev, size)) != kOk || v != 1000 * dev + size) return 1;
  if (asked != 3 * 8) return 2;  // once for each
  for (int round = 0; round < 2; ++round)
    for (int dev : {64, 200, -1})  // not kept, right all the same
      if (fit.get(dev, 3, &v, ask(dev, 3)) != kOk || v != 1000 * dev + 3) return 3;
  if (asked != 3 * 8 + 6) return 4;
  // a query that fails is not kept; a count of zero is
  if (fit.get(5, 1, &v, [](int*) { return kBad; }) != kBad) return 5;
  if (fit.get(5, 1, &v, [](int* n) { *n = 0; return kOk; }) != kOk || v != 0) return 6;
  if (fit.get(5, 1, &v, [](int* n) { *n = 7; return kOk; }) != kOk || v != 0) return 7;
  std::puts("kept by device");
}
"""


def test_numbers_are_kept_by_device(tmp_path):
    src = tmp_path / "t.cpp"
    src.write_text(PROGRAM)
    exe = str(tmp_path / "t")
    inc = os.path.join(ROOT, "quantized_weight_gemv_dequant_b200", "csrc")
    subprocess.run(["g++", "-std=c++17", "-Wall", "-Werror", "-I", inc, str(src), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and "kept by device" in r.stdout, r.returncode

