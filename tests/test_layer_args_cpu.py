"""Argument checks of the layer operators' entry points that need no GPU: the
calls that carry options and a status word, and sizes at the ends of the ranges.
They pass made-up addresses, so they run in a process that sees no GPU."""
import json
import os
import subprocess
import sys

import pytest

import nonlinear_rnn_paragru_b200 as pr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _cases():
    bf16, gru, dec = pr.PARARNN_BF16, pr.PARARNN_LIN_GRU, pr.PARARNN_LIN_DECAY
    C = {}

    def solve(name, want, **o):
        a = dict(cell=gru, u=0x1000, dt=bf16, sb=128, st=64, sg=32, lam=None, bias=None, h0=None, reset=None,
                 h=0x3000, B=1, T=2, D=32, kappa=8.0, status=None, opts=None, stream=None)
        a.update(o)
        C["solve_" + name] = ("pararnn_linrec_solve_ex", list(a.values()), want)
    solve("status_misaligned", -5, status=0x2002)
    solve("no_h", -1, h=None)
    # sizes whose products or sums pass 31, 32 or 64 bits on the way
    solve("D_too_large", -6, T=1, D=(1 << 31) - 8)
    solve("D_and_T_too_large", -6, T=2, D=(1 << 30) + 8)
    solve("product_of_2_64", -6, B=1 << 30, T=1 << 30, D=16)
    solve("B_too_large", -6, B=(1 << 31) - 1, T=1, D=8)

    def adj(name, want, **o):
        a = dict(cell=dec, u=0x1000, dt=bf16, sb=128, st=64, sg=32, lam=0x2000, bias=None, h0=None, reset=None,
                 h=0x3000, g=0x4000, du=0x5000, ddt=bf16, dlam=None, dbias=None, dh0=None, B=1, T=2, D=32,
                 kappa=8.0, status=None, ws=0x10000, wsb=1 << 20, opts=None, stream=None)
        a.update(o)
        C["adjoint_" + name] = ("pararnn_linrec_adjoint_ex", list(a.values()), want)
    adj("status_misaligned", -5, status=0x2001)
    adj("ws_too_small", -3, wsb=64)
    adj("D_too_large", -6, T=1, D=(1 << 31) - 8, wsb=1 << 62)
    adj("product_of_2_64", -6, B=1 << 30, T=1 << 30, D=16, wsb=1 << 62)

    def size(name, want, *a):
        C["size_" + name] = ("pararnn_linrec_workspace_size", list(a), want)
    size("D_too_large", 0, gru, 1, 1, (1 << 31) - 8)
    size("product_of_2_64", 0, dec, 1 << 30, 1 << 30, 16)
    size("B_too_large", 0, dec, (1 << 31) - 1, 1, 8)

    def nadj(name, want, **o):
        a = dict(h=0x1000, hd=pr.PARARNN_F32, lh=64, g=None, gd=0, lg=0, act=0, wpost=None, r=None, rd=0, lr=0,
                 sc=None, wpre=0x2000, ds=0x3000, dsd=bf16, lds=64, dx=0x4000, dxd=bf16, ldx=64, dh=0x5000,
                 dg=None, dres=None, dwpost=None, dsc=None, dwpre=None, eps=1e-6, N=2, D=64, status=None,
                 ws=0x10000, wsb=1 << 22, opts=None, stream=None)
        a.update(o)
        C["norm_adjoint_" + name] = ("pararnn_block_norm_adjoint_ex", list(a.values()), want)
    nadj("status_misaligned", -5, status=0x2001)
    nadj("ws_too_small", -3, wsb=16)
    return C


def _main():
    if os.environ.get("CUDA_VISIBLE_DEVICES", None) != "":
        print("refusing: these calls pass made-up device addresses", file=sys.stderr)
        return 2
    lib = pr.load_library()
    print(json.dumps({k: int(getattr(lib, fn)(*a)) for k, (fn, a, _) in _cases().items()}))
    return 0


@pytest.fixture(scope="module")
def host_rcs():
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="", PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, os.path.abspath(__file__)], env=env, capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    return json.loads(r.stdout.strip().splitlines()[-1])


@pytest.mark.parametrize("case", sorted(_cases()))
def test_entry_points_reject_bad_arguments_on_host(host_rcs, case):
    assert host_rcs[case] == _cases()[case][2]


if __name__ == "__main__":
    sys.exit(_main())
