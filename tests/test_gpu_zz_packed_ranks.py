"""Packed steps with gradients averaged over ranks, on the one GPU of a test box: a one-rank
NCCL communicator drives the sum of the targets and the all-reduces (several ranks that wait on
one another are never run on one GPU; the arithmetic of several ranks is checked on the CPU,
test_packed_ranks_gloo.py).  In a fresh process, bounded by a timeout."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def test_one_rank_equals_none():
    env = dict(os.environ)
    env.setdefault("NCCL_SOCKET_IFNAME", "lo")
    r = subprocess.run([sys.executable, os.path.join(HERE, "packed_ranks_child.py")], env=env,
                       cwd=os.path.dirname(HERE), capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "packed ranks ok" in r.stdout, r.stdout[-3000:] + r.stderr[-3000:]
