"""Clipping over a process group, on the CPU with two gloo ranks: the partial sums
of squares of the ranks are added word by word, whatever each rank holds.  The GPU
entry points are replaced by their definitions on the CPU."""
import math
import os
import socket

import torch
import torch.distributed as dist
import torch.multiprocessing as mp

import bit_microscaled_numerics_amd as nv


def _sumsq(grads):
    """nv.grad_sumsq's contract: words that add up to the sum of squares."""
    words = torch.zeros(nv.NVFP4_SUMSQ_WORDS, dtype=torch.float64)
    for i, g in enumerate(grads):
        words[i % words.numel()] += g.double().square().sum()
    return words


def _clip(grads, max_norm, partials=None, out=None):
    norm = partials.sum().sqrt()
    for g in grads:
        g.mul_(min(1.0, max_norm / (norm.item() + 1e-6)))
    return norm.float().reshape(1)


def _rank(rank, port, results):
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port))
    dist.init_process_group("gloo", rank=rank, world_size=2)
    from bit_microscaled_numerics_amd import lm
    lm.grad_sumsq, lm.clip_grads = _sumsq, _clip
    zeros = torch.zeros
    lm.torch.zeros = lambda *a, **kw: zeros(*a, **{k: v for k, v in kw.items() if k != "device"})
    shards = [[torch.full((5,), 2.0), torch.full((3,), -1.0)], [torch.full((7,), 4.0)]]
    for case, mine in (("both", shards[rank]), ("one", shards[0] if rank == 0 else [])):
        ps = [torch.nn.Parameter(torch.zeros_like(g)) for g in mine]
        for p, g in zip(ps, mine):
            p.grad = g.clone()
        norm = lm.clip_grad_norm(ps, 1.0, group=dist.group.WORLD)
        results[(rank, case)] = (norm.item(), [p.grad.tolist() for p in ps])
    dist.destroy_process_group()


def test_norm_counts_every_rank():
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    results = mp.Manager().dict()
    mp.spawn(_rank, (port, results), nprocs=2)
    both, one = math.sqrt(5 * 4 + 3 + 7 * 16), math.sqrt(5 * 4 + 3)
    for rank in (0, 1):
        assert abs(results[(rank, "both")][0] - both) < 1e-5
        assert abs(results[(rank, "one")][0] - one) < 1e-5
    assert abs(results[(0, "both")][1][0][0] - 2.0 / both) < 1e-5
    assert abs(results[(1, "both")][1][0][0] - 4.0 / both) < 1e-5
    assert results[(1, "one")][1] == []
