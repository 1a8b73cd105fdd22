"""Layer-wise distributed Muon with a gradient multiplier on CPU ranks: every
rank's local step receives its own multiplier, and the ranks end with the
parameters of a single-process step on the scaled gradients."""

import os

import numpy as np
import pytest
import torch
import torch.multiprocessing as mp

from test_distributed_cpu import SHAPES, _free_port, _inputs, _oracle_step

SCALE = 0.375


def _scaled_step(params, grads, momenta, grad_scale, **kw):
    s = float(grad_scale)
    _oracle_step(params, [None if g is None else g * s for g in grads], momenta, **kw)


def _worker(rank, world, port, out):
    import torch.distributed as dist
    from muon_newton_schulz_03_b200.distributed import LayerwiseMuon
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port))
    dist.init_process_group("gloo", rank=rank, world_size=world)
    try:
        P, G, M = ([torch.tensor(x) for x in xs] for xs in _inputs())
        lw = LayerwiseMuon(group=None, local_step=_scaled_step, rounds=3)
        lw.step(P, G, M, lr=0.01, beta=0.9, wd=0.1, grad_scale=torch.tensor([SCALE]))
        out[rank] = [p.numpy() for p in P]
    finally:
        dist.destroy_process_group()


@pytest.mark.parametrize("world", [1, 2])
def test_layerwise_step_with_grad_scale(world):
    out = mp.Manager().dict()
    mp.spawn(_worker, args=(world, _free_port(), out), nprocs=world, join=True)
    P, G, M = ([torch.tensor(x) for x in xs] for xs in _inputs())
    _oracle_step(P, [g * SCALE for g in G], M, lr=0.01, beta=0.9, wd=0.1)
    for r in range(world):
        assert all(np.array_equal(out[r][i], P[i].numpy()) for i in range(len(SHAPES)))
