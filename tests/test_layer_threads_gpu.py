"""The layer operators called from two host threads at once, their first calls
among them."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROGRAM = r"""
import threading, torch
import nonlinear_rnn_paragru_b200 as pr
pr.load_library()

def inputs(D, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g).cuda()
    N = 300
    b = lambda: r(N, D).bfloat16()
    return dict(h=r(N, D), ds=b(), dx=b(), gate=b(), res=b(), w_post=r(D), scale=r(D), w_pre=r(D))

def scan(T, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn((2, T, 2, 128), generator=g).bfloat16().cuda()

# one kernel, two widths: rings of 192 and of 48 KB
work = [(inputs(4096, 1), scan(700, 2)), (inputs(1024, 3), scan(300, 4))]
torch.cuda.synchronize()
out, err, start = [[], []], [], threading.Barrier(2)

def run(k):
    try:
        s = torch.cuda.Stream()
        start.wait()
        for _ in range(20):
            out[k].append((pr.block_norm_adjoint(**work[k][0], stream=s),
                           pr.linrec_solve(pr.PARARNN_LIN_GRU, work[k][1], stream=s)))
        s.synchronize()
    except Exception as e:
        err.append(e)

threads = [threading.Thread(target=run, args=(k,)) for k in (0, 1)]
[t.start() for t in threads]
[t.join() for t in threads]
assert not err, err
for k in (0, 1):
    want = pr.block_norm_adjoint(**work[k][0]), pr.linrec_solve(pr.PARARNN_LIN_GRU, work[k][1])
    for g, h in out[k]:
        assert all(torch.equal(g[n], want[0][n]) for n in g) and torch.equal(h, want[1])
print("equal")
"""


def test_first_calls_of_two_threads(cuda_ok):
    r = subprocess.run([sys.executable, "-c", PROGRAM], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "equal" in r.stdout, r.stderr[-2000:]
