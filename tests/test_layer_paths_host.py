"""Host logic of the layer operators that needs no GPU, beside the refusals of
tests/test_layer_host.py."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_sparse_top_mean_b200", "csrc")


def test_a_device_is_recorded_for_itself_alone(tmp_path):
    """Kernels' shared memory limits are raised once a device: device 64 must not stand for
    device 0, whose launches would then fail."""
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src = tmp_path / "once.cc"
    src.write_text("""#include "device_once.cuh"
int main() {
  for (int a = 0; a < 200; ++a) {
    msa::DeviceOnce once;
    once.mark(a);
    for (int b = -1; b < 200; ++b)
      if (once.done(b) != (a == b && a < 64)) return 1;
  }
  return 0;
}
""")
    exe = str(tmp_path / "once")
    subprocess.run([cxx, "-std=c++17", "-x", "c++", "-I", CSRC, str(src), "-o", exe], check=True)
    assert subprocess.run([exe]).returncode == 0
