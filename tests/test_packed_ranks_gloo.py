"""A packed step over ranks whose rows have different numbers of targets: every rank weighs
its targets by (ranks / targets of all ranks), and the average over ranks is the gradient of the
one mean over all targets, as a single rank with all rows has it.  Two gloo ranks on the CPU, the
oracle's loss; the library does the same with its communicator (one integer summed)."""
import os
import re
import socket

import numpy as np
import pytest
import torch
import torch.multiprocessing as mp

T, D, V, WORLD = 12, 5, 7, 2


def _row(rank):
    g = np.random.default_rng(10 + rank)
    return g.standard_normal((T, D)), g.integers(0, V, T)


def _targets(rank, masks):
    from oracle import packed as op
    return op.targets(_row(rank)[1], op.documents([5, 7]), masks[rank])


def _worker(rank, port, masks, out):
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port), RANK=str(rank),
                      WORLD_SIZE=str(WORLD), LOCAL_RANK=str(rank))
    from layer_streamed_qlora_nf4_b200 import dp
    from oracle import packed as op
    dp.init("gloo", timeout_s=60)
    w = np.random.default_rng(1).standard_normal((D, V))
    x, _ = _row(rank)
    y = _targets(rank, masks)
    count = torch.tensor([int((y >= 0).sum())])
    torch.distributed.all_reduce(count)
    _, loss, dl = op.cross_entropy(x @ w, y, np.full(T, float(WORLD)), int(count))
    grad = dp.average_(torch.from_numpy(x.T @ dl))
    out[rank] = grad.numpy().copy(), float(dp.average_(torch.tensor([loss], dtype=torch.float64)))
    dp.barrier()
    torch.distributed.destroy_process_group()


@pytest.mark.parametrize("marked", [(12, 2), (9, 0), (0, 0)])
def test_the_mean_is_over_the_targets_of_all_ranks(marked):
    from oracle import packed as op
    masks = [(np.arange(T) >= T - n).astype(np.uint8) for n in marked]
    with socket.socket() as s:
        s.bind(("127.0.0.1", 0))
        port = s.getsockname()[1]
    ctx = mp.get_context("spawn")
    out = ctx.Manager().dict()
    procs = [ctx.Process(target=_worker, args=(r, port, masks, out)) for r in range(WORLD)]
    for p in procs:
        p.start()
    for p in procs:
        p.join(120)
        assert p.exitcode == 0
    x = np.concatenate([_row(r)[0] for r in range(WORLD)])
    y = np.concatenate([_targets(r, masks) for r in range(WORLD)])
    w = np.random.default_rng(1).standard_normal((D, V))
    _, loss, dl = op.cross_entropy(x @ w, y, None, int((y >= 0).sum()))
    for rank in range(WORLD):
        grad, mean = out[rank]
        # fp64 sums of two dozen terms of size 1
        assert np.abs(grad - x.T @ dl).max() <= 1e-14 and abs(mean - loss) <= 1e-14


def test_the_step_sums_its_targets_before_the_first_loss():
    """The order in the library's step: count, sum over ranks, losses divided by it."""
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                        "layer_streamed_qlora_nf4_b200", "csrc", "stack.cu")
    text = open(path).read()
    at = [text.index(s) for s in ("prepare_row(mb, true)", "all_reduce(w.count, w.count, 1, ncclInt32, "
                                  "ncclSum", "launch_packed_ce(", "launch_packed_loss(")]
    assert at == sorted(at)
    assert re.search(r"ranks = sum_counts \? h->grad_world : 1;", text)
    assert len(re.findall(r"cs, ranks\)\)", text)) == 2
