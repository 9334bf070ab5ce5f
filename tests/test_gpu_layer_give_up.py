"""How the attention over a paged cache gives up: one copy of every CTA's stream is lost, so that
its waits run out (after about a millisecond in this build, two seconds in the library's).  The
kernels must end, with their own copies and products waited for, and report it; the GPU stays
usable and a call of the library itself is right afterwards."""
import ctypes
import glob
import os
import subprocess

import pytest
import torch

from block_sparse_top_mean_b200 import _lib, build
from test_gpu_layer import Step
from test_gpu_layer import msa  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lossy(tmp_path_factory):
    """lossy(n): msa_paged_attn_fwd of a library without copy n of any CTA's stream."""
    made = {}

    def fn(n):
        if n in made:
            return made[n]
        out = str(tmp_path_factory.mktemp("lossy") / f"libmsa_lossy{n}.so")
        csrc = os.path.join(build.PKG, "csrc")
        sources = [os.path.join(csrc, f) for f in ("layer_api.cu", "host_util.cu",
                                                   "qk_norm_rope.cu", "paged_append.cu")]
        sources += sorted(glob.glob(os.path.join(csrc, "paged_attn*.cu")))
        subprocess.run([build._nvcc(), *build.ARCH, "-O1", "-std=c++17", "-shared", "-t", "0",
                        "-Xcompiler", "-fPIC", f"-DMSA_LOSE_COPY={n}",
                        "-DMSA_WAIT_CLOCKS=2000000LL", "-I", os.path.join(build.ROOT, "include"),
                        "-o", out, *sources, "-lcuda"], check=True, capture_output=True, text=True)
        made[n] = ctypes.CDLL(out).msa_paged_attn_fwd
        made[n].restype, made[n].argtypes = _lib.SIGNATURES["msa_paged_attn_fwd"]
        return made[n]
    return fn


SEQS = {   # runs that end before a ring is full, and runs that go round it
    "short": [(90, 390), (1, 300), (30, 500)],
    "long": [(40, 9000), (1, 20000), (7, 12000)],
}


@pytest.mark.parametrize("seqs", SEQS)
@pytest.mark.parametrize("d", [64, 128])
def test_chunk_kernel_gives_up(msa, lossy, monkeypatch, d, seqs):  # noqa: F811
    """The first values are lost: products of the first keys are under way."""
    _give_up(msa, lossy(1), monkeypatch, Step(torch.bfloat16, d, 8, 2, 64, SEQS[seqs]), None)


@pytest.mark.parametrize("seqs", SEQS)
@pytest.mark.parametrize("dtype,d,max_new", [
    (torch.bfloat16, 128, 1), (torch.bfloat16, 128, 4), (torch.bfloat16, 64, 1),
    (torch.float32, 128, 1), (torch.float32, 64, 2), (torch.float32, 128, None),
    (torch.float32, 64, None)])
def test_ring_kernels_give_up(msa, lossy, monkeypatch, dtype, d, max_new, seqs):  # noqa: F811
    """The first tile is lost (the only one of some CTAs: 240 tiles of 32 keys on 296 of them)."""
    _give_up(msa, lossy(0), monkeypatch, Step(dtype, d, 8, 2, 64, SEQS[seqs]), max_new)


def _give_up(msa, lossy, monkeypatch, st, max_new):  # noqa: F811
    from block_sparse_top_mean_b200 import layer
    ws = msa.paged_workspace(st.q, st.kp, st.dev[1])
    with monkeypatch.context() as m:
        m.setitem(layer._fns, "msa_paged_attn_fwd", lossy)
        for _ in range(2):
            st.attn(msa, ws=ws, max_new=max_new)
            assert msa.read_device_error(ws) == msa.DEVERR_TIMEOUT
    msa.clear_device_error(ws)
    o, lse = st.attn(msa, ws=ws, max_new=max_new)
    assert msa.read_device_error(ws) == 0
    st.check(o, lse)
