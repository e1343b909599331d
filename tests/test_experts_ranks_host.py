"""Clipping over gloo ranks where something is not finite or not alike, without a GPU:
the kernels are replaced by torch."""
import os

import pytest
import torch
import torch.distributed as dist
import torch.multiprocessing as mp

from combine_moe_topk_gb300 import autograd as A
from combine_moe_topk_gb300 import binding as B
from combine_moe_topk_gb300 import ep as EP


class _List(list):
    tensors = property(lambda self: list(self))


def _norm(g, norm=None, device_status=None):
    n = torch.stack([t.double().square().sum() for t in g]).sum().sqrt().float().view(1) if len(g) else torch.zeros(1)
    if device_status is not None and not torch.isfinite(n).all():
        device_status |= B.MOE_DEV_NONFINITE
    return n


def _clip(g, norm, max_norm, out=None):
    if torch.isfinite(norm).all():
        for t in g:
            t.mul_(min(1.0, max_norm / (float(norm) + 1e-6)))


def _rank(rank, R, port, q, case):
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port))
    dist.init_process_group("gloo", rank=rank, world_size=R)
    try:
        word = torch.zeros(1, dtype=torch.int32)
        A._status = lambda t: word
        B.GradList = _List
        B.moe_grad_norm = _norm
        B.moe_grad_clip = _clip
        own, common = [torch.arange(1.0, 6.0) * (rank + 1)], [torch.arange(4.0)]
        if case == "nan" and rank == 1:
            own[0][2] = float("nan")
        if case == "large":  # each part is in fp32's range, the norm of all is not
            own[0].fill_(1.5e38)
        if case == "unlike":  # another order of the sum on one rank
            common[0][3] += 1e-3 * rank
        if case == "none" and rank == 0:
            own = []
        before = [t.clone() for t in own + common]
        norm = EP.clip_grad_norm(own, common, 0.5)
        q.put((rank, float(norm), int(word), [b.tolist() for b in before], [t.tolist() for t in own + common]))
    finally:
        dist.destroy_process_group()


def _run(case):
    R, ctx = 2, mp.get_context("spawn")
    q = ctx.Queue()
    port = 31800 + os.getpid() % 1000
    procs = [ctx.Process(target=_rank, args=(r, R, port, q, case)) for r in range(R)]
    for p in procs:
        p.start()
    got = sorted((q.get(timeout=300) for _ in procs), key=lambda r: r[0])
    for p in procs:
        p.join(timeout=120)
        assert p.exitcode == 0
    return got


@pytest.mark.parametrize("case", ["nan", "large"])
def test_a_norm_that_is_not_finite_reaches_every_ranks_status(case):
    for _, norm, word, before, after in _run(case):
        assert not torch.isfinite(torch.tensor(norm)) and word == B.MOE_DEV_NONFINITE
        assert str(before) == str(after)


@pytest.mark.parametrize("case", ["unlike", "none"])
def test_every_rank_clips_to_the_same_norm(case):
    got = _run(case)
    assert got[0][1] == got[1][1] and all(word == 0 for _, _, word, _, _ in got)
    own = [sum(v * v for t in before[:-1] for v in t) for _, _, _, before, _ in got]
    want = (sum(own) + sum(v * v for v in got[0][3][-1])) ** 0.5  # the replicated part of the first rank
    assert abs(got[0][1] - want) <= 1e-5 * want
    for _, norm, _, before, after in got:
        for b, a in zip(before, after):
            assert all(abs(y - x * (0.5 / (norm + 1e-6))) <= 1e-6 * abs(x) for x, y in zip(b, a))


# ---- the calls of the ranks' clipping where a rank holds only one kind of gradients -------

class _Far:
    """A gradient on a device that is not the current one."""
    device = torch.device("cuda", 1)


@pytest.fixture
def one_rank(monkeypatch):
    """A group of one rank; the devices that are made current, and under which device each kernel is called."""
    at, log = [0], []

    class device:
        def __init__(self, d):
            self.to = torch.device(d).index

        def __enter__(self):
            at.append(self.to)

        def __exit__(self, *exc):
            at.pop()

    class grad_list(list):
        def __init__(self, tensors):
            super().__init__(tensors)
            self.at = self[0].device.index if self else at[-1]  # without tensors: the current device

    def norm(g, norm=None, device_status=None):
        log.append(("norm", g.at))
        return torch.ones(1)

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(B, "GradList", grad_list)
    monkeypatch.setattr(B, "moe_grad_norm", norm)
    monkeypatch.setattr(B, "moe_grad_clip", lambda g, norm, max_norm, out=None: log.append(("clip", g.at)))
    monkeypatch.setattr(A, "_status", lambda t: None)
    dist.init_process_group("gloo", init_method=f"tcp://127.0.0.1:{32900 + os.getpid() % 1000}", rank=0, world_size=1)
    yield log
    dist.destroy_process_group()


@pytest.mark.parametrize("sharded,replicated", [([], [_Far()]), ([_Far()], []), ([_Far()], (t for t in [_Far()]))])
def test_all_kernels_run_on_the_gradients_device(one_rank, sharded, replicated):
    EP.clip_grad_norm(sharded, replicated, 1.0)
    assert one_rank == [("norm", 1), ("norm", 1), ("clip", 1), ("clip", 1)]
