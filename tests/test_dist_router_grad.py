"""Data parallelism of the router's gradient on CPU (gloo ranks): the centroids'
gradient is summed over the ranks with the experts'."""
import os
import socket

import numpy as np
import torch
import torch.distributed as dist
import torch.multiprocessing as mp


def _grads(rank):
    rng = np.random.default_rng(400 + rank)
    new = lambda *s: torch.from_numpy(rng.normal(0, 1, s).astype(np.float32))
    return {"dW1": new(3, 8, 4), "dW2": new(3, 4, 8), "dcentroids": new(16, 128), "dlogits": new(5, 16)}


def _worker(rank, world, port, q):
    os.environ["MASTER_ADDR"] = "127.0.0.1"
    os.environ["MASTER_PORT"] = str(port)
    dist.init_process_group("gloo", rank=rank, world_size=world)
    from fp8_block_scaled_sigmoid_b200.layer import reduce_weight_grads
    q.put((rank, {k: v.numpy() for k, v in reduce_weight_grads(_grads(rank), dist.group.WORLD).items()}))
    dist.barrier()
    dist.destroy_process_group()


def test_the_centroids_gradient_sums_over_the_ranks():
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    procs = [ctx.Process(target=_worker, args=(r, 2, port, q)) for r in range(2)]
    for p in procs:
        p.start()
    res = dict(q.get(timeout=120) for _ in procs)
    for p in procs:
        p.join(timeout=60)
        assert p.exitcode == 0
    a, b = _grads(0), _grads(1)
    for rank, own in ((0, a), (1, b)):
        for k in ("dW1", "dW2", "dcentroids"):
            assert np.array_equal(res[rank][k], (a[k] + b[k]).numpy()), k
        assert np.array_equal(res[rank]["dlogits"], own["dlogits"].numpy())   # a token's own: not summed
