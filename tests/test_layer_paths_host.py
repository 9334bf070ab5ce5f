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


def test_append_refuses_an_eps_that_fp32_rounds_to_zero():
    """0 stands for no norm in the C entry: a smaller eps would leave the norm out silently."""
    from block_sparse_top_mean_b200.layer import _append_eps
    assert _append_eps(None, None, None) == 0.0
    assert _append_eps(2.0 ** -126, None, None) == 2.0 ** -126
    for eps in (0.0, -1e-6, 1e-46, 1e-300, float("nan")):
        with pytest.raises(ValueError, match="eps"):
            _append_eps(eps, None, None)
    with pytest.raises(ValueError, match="need eps"):
        _append_eps(None, None, object())


@pytest.mark.gpu
def test_append_with_a_tiny_eps_normalises_or_refuses():
    import torch

    import block_sparse_top_mean_b200 as msa
    k = torch.full((1, 1, 64), 3.0, device="cuda")
    pool, other = torch.zeros(1, 1, 16, 64, device="cuda"), torch.zeros(1, 1, 16, 64, device="cuda")
    one, cu = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([1], [0, 1]))
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="eps"):
        msa.paged_append(k, k, pool, other, table, one, cu, eps=1e-46)
    msa.paged_append(k, k, pool, other, table, one, cu, eps=2.0 ** -126)
    assert (pool[0, 0, 0] == 1).all() and (other[0, 0, 0] == 3).all()
