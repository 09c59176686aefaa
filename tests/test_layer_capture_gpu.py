"""The layer operators captured into a graph by the first calls of a process,
and graphs that replay at the same time."""
import os
import subprocess
import sys

import pytest
import torch

import nonlinear_rnn_paragru_b200 as pr

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
import torch
import nonlinear_rnn_paragru_b200 as pr
g = torch.Generator().manual_seed(0)
r = lambda *s: torch.randn(s, generator=g).cuda()
u, lam, w, d = r(2, 700, 3, 264).bfloat16(), r(264) - 4, r(264), r(2, 700, 264)

def layer():
    h = pr.linrec_solve(pr.PARARNN_LIN_DECAY, u, lam)
    s, x = pr.block_norm(h, gate=u[:, :, 0], w_post=w, res=u[:, :, 1], w_pre=w)
    n = pr.block_norm_adjoint(h, x, s, gate=u[:, :, 0], w_post=w, res=u[:, :, 1], w_pre=w)
    a = pr.linrec_adjoint(pr.PARARNN_LIN_DECAY, u, lam, None, None, h, n["dh"])
    return [h, s, x, *n.values(), *a.values(), pr.linrec_step(pr.PARARNN_LIN_DECAY, u[:, 0], lam)]

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = layer()
u.mul_(0.5)
graph.replay()
want = layer()
assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip(got, want))
print("equal")
"""


def test_first_calls_of_a_process_are_captured(cuda_ok):
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "equal" in r.stdout, r.stderr[-2000:]


def test_graphs_that_replay_at_the_same_time(cuda_ok):
    # each graph has its scratch to itself
    made = []
    for k in range(3):
        g = torch.Generator().manual_seed(k)
        r = lambda *s: torch.randn(s, generator=g).cuda()  # noqa: E731
        u, lam, w, d = r(2, 2000, 3, 264).bfloat16(), r(264) - 4, r(264), r(2, 2000, 264)

        def layer(u=u, lam=lam, w=w, d=d):
            h = pr.linrec_solve(pr.PARARNN_LIN_DECAY, u, lam)
            n = pr.block_norm_adjoint(h, d, d, w_post=w, w_pre=w, res=u[:, :, 1])
            return [h, *n.values(), *pr.linrec_adjoint(pr.PARARNN_LIN_DECAY, u, lam, None, None, h, n["dh"]).values()]

        want, graph, stream = layer(), torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            got = layer()
        made.append((graph, stream, got, want, layer))     # with the inputs, which the graph reads
    torch.cuda.synchronize()
    for _ in range(20):
        for graph, stream, *_ in made:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, got, want, _ in made:
        assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip(got, want))
