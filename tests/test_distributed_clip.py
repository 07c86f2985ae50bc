"""Clipping over ranks (CPU, gloo): every rank scales by the same total, bit for bit, and takes part
in the all-reduce whatever it holds."""
import os

import pytest
import torch
import torch.distributed as dist
import torch.multiprocessing as mp

from mixture_experts_layer_65_b200 import parallel
from tests.test_distributed import _free_port


def _run(fn, world):
    ctx = mp.get_context("spawn")
    q = ctx.Queue()
    port = _free_port()
    procs = [ctx.Process(target=_enter, args=(fn, r, world, port, q)) for r in range(world)]
    for p in procs:
        p.start()
    got = dict(q.get(timeout=120) for _ in procs)
    for p in procs:
        p.join(60)
        assert p.exitcode == 0
    return got


def _enter(fn, rank, world, port, q):
    os.environ["MASTER_ADDR"] = "127.0.0.1"
    os.environ["MASTER_PORT"] = str(port)
    dist.init_process_group("gloo", rank=rank, world_size=world)
    try:
        q.put((rank, fn(rank)))
    finally:
        dist.destroy_process_group()


def _totals(rank):
    """The ranks' sums of the same replicated gradients differ in their last bits."""
    seen = []

    def sumsq(ts):
        s = sum(t.double().square().sum() for t in ts).reshape(1)
        return s * (1 + rank * 2.0 ** -52)

    def scale(ts, total, max_norm):
        seen.append(total.clone())
        return total.sqrt().float()

    shared, own = [torch.arange(1.0, 6.0) / 3], [torch.full((2, 2), 0.7 + rank)]
    parallel.clip_grad_norm(shared, own, 1.0, sumsq_fn=sumsq, scale_fn=scale)
    parallel.clip_grad_norm([], own, 1.0, sumsq_fn=sumsq, scale_fn=scale)
    parallel.clip_grad_norm(shared if rank != 1 else [], own, 1.0, sumsq_fn=sumsq, scale_fn=scale)
    return [float(t) for t in seen]


@pytest.mark.parametrize("world", [2, 3])
def test_every_rank_scales_by_the_same_total(world):
    got = _run(_totals, world)
    assert all(got[r] == got[0] for r in range(world))
    own = sum(4 * (torch.full((1,), 0.7 + r).double().item()) ** 2 for r in range(world))
    shared = float((torch.arange(1.0, 6.0) / 3).double().square().sum())
    for total, want in zip(got[0], (own + shared, own, own + shared)):
        assert total == pytest.approx(want, rel=1e-14)


def _one_without(rank):
    def sumsq(ts):
        return sum(t.double().square().sum() for t in ts).reshape(1)

    def scale(ts, total, max_norm):
        return total.sqrt().float()

    own = [torch.full((3,), 2.0)] if rank == 0 else []
    first = parallel.clip_grad_norm([], own, 1.0, sumsq_fn=sumsq, scale_fn=scale)
    nobody = parallel.clip_grad_norm([], [], 1.0, sumsq_fn=sumsq, scale_fn=scale)
    after = torch.ones(1)
    dist.all_reduce(after)      # the ranks' collectives still belong together
    return float(first), first.dtype == torch.float32, float(nobody), float(after)


def test_a_rank_without_gradients_takes_part():
    got = _run(_one_without, 2)
    assert got[0] == got[1] == (pytest.approx(12.0 ** 0.5, rel=1e-7), True, 0.0, 2.0)


def _one_refused(rank):
    scaled = []

    def sumsq(ts):
        if any(t.dtype == torch.int32 for t in ts):
            raise ValueError("not a gradient")
        return sum(t.double().square().sum() for t in ts).reshape(1)

    def scale(ts, total, max_norm):
        scaled.append(float(total))
        return total.sqrt().float()

    got = []
    for own in ([torch.ones(3, dtype=torch.int32 if rank else torch.float32)], [None if rank else torch.ones(3)]):
        try:
            norm = parallel.clip_grad_norm([], own, 1.0, sumsq_fn=sumsq, scale_fn=scale)
            got.append(str(float(norm)))
        except (ValueError, AttributeError) as e:
            got.append(type(e).__name__)
    after = torch.ones(1)
    dist.all_reduce(after)
    return got, len(scaled), float(after)


def test_a_rank_whose_gradients_are_refused_takes_part():
    got = _run(_one_refused, 2)
    assert got[0] == (["nan", "nan"], 2, 2.0)
    assert got[1] == (["ValueError", "AttributeError"], 0, 2.0)
