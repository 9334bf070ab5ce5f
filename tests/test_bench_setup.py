"""bench.py's process group set-up on the CPU: no rank is through before every rank has connected."""
import os
import sys
import time

import torch.multiprocessing as mp

from test_multirank_cpu import _free_port

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _setup(rank, port, out):
    sys.path.insert(0, ROOT)
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port), RANK=str(rank),
                      LOCAL_RANK=str(rank), WORLD_SIZE="2", CUDA_VISIBLE_DEVICES="")
    import torch.distributed as dist

    import bench
    connect = dist.init_process_group

    def late(*args, **kw):
        connect(*args, **kw)
        time.sleep(1.5)
        out["connected"] = time.monotonic()

    if rank == 0:
        dist.init_process_group = late
    assert bench.dist_setup() == (2, rank, rank)
    out[rank] = time.monotonic()
    dist.destroy_process_group()


def test_no_rank_leaves_before_all_are_connected():
    manager = mp.get_context("spawn").Manager()
    out = manager.dict()
    mp.spawn(_setup, args=(_free_port(), out), nprocs=2, join=True)
    assert out[1] >= out["connected"]
