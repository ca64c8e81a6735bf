"""The benchmark's multi-rank aggregation (replicas: the slowest rank sets the step
time) on two gloo ranks on the CPU."""
import os
import socket

import torch.multiprocessing as mp


def _free_port():
    s = socket.socket()
    s.bind(("127.0.0.1", 0))
    p = s.getsockname()[1]
    s.close()
    return p


def _worker(rank, world, port, out):
    import torch.distributed as dist
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port), RANK=str(rank), WORLD_SIZE=str(world))
    dist.init_process_group("gloo", rank=rank, world_size=world)
    import bench
    r, w, _ = bench.dist_env()
    bench.barrier(w)
    out[rank] = bench.max_over_ranks(10.0 + 5.0 * r, w)
    dist.destroy_process_group()


def test_max_over_two_gloo_ranks():
    ctx = mp.get_context("spawn")
    mgr = ctx.Manager()
    out = mgr.dict()
    port = _free_port()
    ps = [ctx.Process(target=_worker, args=(r, 2, port, out)) for r in range(2)]
    for p in ps:
        p.start()
    for p in ps:
        p.join(60)
        assert p.exitcode == 0
    assert dict(out) == {0: 15.0, 1: 15.0}


def test_single_rank_is_identity():
    import bench
    assert bench.max_over_ranks(3.5, 1) == 3.5
    assert bench.dist_env()[1] >= 1


def test_the_traffic_figure_is_void_after_any_edit_that_can_change_it(tmp_path, monkeypatch):
    """The layer kernel, its packing and the host code that chooses its grid and splits."""
    import shutil
    import bench
    src = os.path.join("moe_decode_megakernel_warp_gb300", "csrc")
    shutil.copytree(os.path.join(bench.ROOT, src), str(tmp_path / src))
    whole = bench.kernel_sha256()
    monkeypatch.setattr(bench, "ROOT", str(tmp_path))
    assert bench.kernel_sha256() == whole
    for name in ("msm_kernel.cu", "msm_device.cuh", "msm_internal.h", "msm_pack.cu", "msm_api.cu"):
        p = tmp_path / src / name
        old = p.read_bytes()
        p.write_bytes(old + b"\n")
        assert bench.kernel_sha256() != whole, name
        p.write_bytes(old)
