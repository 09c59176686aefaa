"""Pins of the fp64 restatement of the gated linear recurrence and the block
norm (torch autograd in float64, central differences, closed forms), and the
argument checks of their entry points that need no GPU."""
import json
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle
import nonlinear_rnn_paragru_b200 as pr
from oracle import layer as ol

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CELLS = {"lin_gru": (ol.LIN_GRU, 2), "lin_decay": (ol.LIN_DECAY, 3)}


def _draw(cell, B, T, D, seed=0, resets=0.2):
    g = torch.Generator().manual_seed(seed)
    c, G = CELLS[cell]
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    return dict(cell=c, u=r(B, T, G, D), lam=r(D) - 1 if c == ol.LIN_DECAY else None, bias=0.3 * r(G, D),
                h0=r(B, D), reset=torch.rand((B, T), generator=g) < resets), r(B, T, D)


def _torch_seq(x):
    """The recurrence in torch float64, for autograd."""
    p = x["u"] + x["bias"]
    if x["cell"] == ol.LIN_GRU:
        z = torch.sigmoid(p[..., 0, :])
        a, b = 1 - z, z * torch.tanh(p[..., 1, :])
    else:
        la = -8.0 * torch.nn.functional.softplus(x["lam"]) * torch.sigmoid(p[..., 0, :])
        a, b = la.exp(), torch.sqrt(1 - (2 * la).exp()) * torch.sigmoid(p[..., 1, :]) * p[..., 2, :]
    h, out = x["h0"], []
    for t in range(p.shape[1]):
        h = a[:, t] * (h * (~x["reset"][:, t, None])) + b[:, t]
        out.append(h)
    return torch.stack(out, 1)


@pytest.mark.parametrize("cell", CELLS)
def test_linrec_oracle_equals_autograd(cell):
    x, g = _draw(cell, 2, 9, 5)
    names = [k for k in ("u", "lam", "bias", "h0") if x[k] is not None]
    for k in names:
        x[k].requires_grad_(True)
    h = _torch_seq(x)
    H, _ = ol.lin_seq(**x)
    assert np.abs(H - h.detach().numpy()).max() < 1e-13
    want = dict(zip(names, torch.autograd.grad((h * g).sum(), [x[k] for k in names])))
    got = ol.lin_adjoint(x["cell"], x["u"], x["lam"], x["bias"], x["h0"], H, g, x["reset"])
    for k in names:
        assert np.abs(got["d" + k][0] - want[k].numpy()).max() < 1e-11, k


@pytest.mark.parametrize("cell", CELLS)
def test_linrec_oracle_equals_differences(cell):
    x, g = _draw(cell, 1, 6, 3, seed=4)
    H, _ = ol.lin_seq(**x)
    got = ol.lin_adjoint(x["cell"], x["u"], x["lam"], x["bias"], x["h0"], H, g, x["reset"])
    eps = 1e-5
    for k in ("u", "lam", "bias", "h0"):
        if x[k] is None:
            continue
        flat = x[k].view(-1)
        for i in range(flat.numel()):
            v = flat[i].item()
            up, dn = [], []
            for s, to in ((1, up), (-1, dn)):
                flat[i] = v + s * eps
                to.append((ol.lin_seq(**x)[0] * g.numpy()).sum())
            flat[i] = v
            num = (up[0] - dn[0]) / (2 * eps)
            assert abs(got["d" + k][0].reshape(-1)[i] - num) < 1e-7 * (1 + abs(num)), (k, i)


def test_lin_gru_is_paragru_without_recurrent_weights():
    x, _ = _draw("lin_gru", 2, 12, 8, resets=0.0)
    u3 = np.stack([x["u"][:, :, 0], np.random.RandomState(0).randn(2, 12, 8), x["u"][:, :, 1]], 2)
    b3 = np.stack([x["bias"][0], np.zeros(8), x["bias"][1]])
    ref = oracle.gru_seq(u3, np.zeros((3, 8)), b3, x["h0"].numpy())
    assert np.abs(ol.lin_seq(**x)[0] - ref).max() < 1e-14


def test_linrec_oracle_closed_forms():
    T, D = 40, 4
    u = np.zeros((1, T, 2, D))
    u[:, :, 1] = 50.0                         # z = 1/2, c = 1: h_t = 1 - 2^-t (1 - h0)
    H, _ = ol.lin_seq(ol.LIN_GRU, u, h0=np.full((1, D), -3.0))
    assert np.allclose(H[0, :, 0], 1 - 0.5 ** np.arange(1, T + 1) * 4, atol=1e-15)
    u[:, :, 0] = -np.inf                      # z = 0: the state stays
    H, _ = ol.lin_seq(ol.LIN_GRU, u, h0=np.full((1, D), -3.0))
    assert (H == -3.0).all()
    every = np.ones((1, T), bool)             # a reset at every step: h_t = b_t
    u[:, :, 0] = 0.0
    H, _ = ol.lin_seq(ol.LIN_GRU, u, h0=np.full((1, D), -3.0), reset=every)
    assert np.allclose(H, 0.5, atol=1e-15)


PARTS = [dict(), dict(post=1), dict(gate=1), dict(pre=1), dict(res=1, pre=1), dict(post=1, gate=1),
         dict(post=1, gate=1, res=1, scale=1, pre=1), dict(scale=1, res=1), dict(gate=1, scale=1, pre=1)]


def _parts(p, N, D, seed=1):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    return dict(h=r(N, D), gate=r(N, D) if p.get("gate") else None, w_post=r(D) if p.get("post") else None,
                res=r(N, D) if p.get("res") else None, scale=r(D) if p.get("scale") else None,
                w_pre=r(D) if p.get("pre") else None), r(N, D), r(N, D)


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("p", PARTS, ids=lambda p: "_".join(p) or "none")
def test_block_norm_oracle_equals_autograd(p, act):
    x, ds, dx = _parts(p, 3, 10)
    eps = 1e-3
    leaves = {k: v.requires_grad_(True) for k, v in x.items() if v is not None}
    rms = lambda v: v / torch.sqrt(v.pow(2).mean(-1, keepdim=True) + eps)  # noqa: E731
    y = x["h"] if x["w_post"] is None else rms(x["h"]) * x["w_post"]
    if x["gate"] is not None:
        y = y * (torch.nn.functional.silu(x["gate"]) if act == "silu" else torch.sigmoid(x["gate"]))
    if x["scale"] is not None:
        y = y * x["scale"]
    s = y if x["res"] is None else y + x["res"]
    loss = (s * ds).sum()
    got = ol.block_norm(**x, act=act, eps=eps)
    assert np.abs(got["s"][0] - s.detach().numpy()).max() < 1e-13
    if x["w_pre"] is not None:
        xo = rms(s) * x["w_pre"]
        loss = loss + (xo * dx).sum()
        assert np.abs(got["x"][0] - xo.detach().numpy()).max() < 1e-12
    want = dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))
    adj = ol.block_norm_adjoint(ds=ds, dx=dx if x["w_pre"] is not None else None, act=act, eps=eps, **x)
    name = dict(h="dh", gate="dgate", w_post="dw_post", res="dres", scale="dscale", w_pre="dw_pre")
    assert set(adj) == {name[k] for k in leaves}
    for k in leaves:
        assert np.abs(adj[name[k]][0] - want[k].numpy()).max() < 1e-11, k


# -------------------------------------------- argument checks without a GPU
# The calls pass made-up addresses, so they run in a process that sees no GPU.
def _host_cases():
    f32, bf16, gru, dec = pr.PARARNN_F32, pr.PARARNN_BF16, pr.PARARNN_LIN_GRU, pr.PARARNN_LIN_DECAY
    C = {}

    def solve(name, want, **o):
        a = dict(cell=gru, u=0x1000, dt=bf16, sb=128, st=64, sg=32, lam=None, bias=None, h0=None, reset=None,
                 h=0x3000, B=1, T=2, D=32, kappa=8.0, stream=None)
        a.update(o)
        C["solve_" + name] = ("pararnn_linrec_solve", list(a.values()), want)
    solve("cell", -1, cell=0)
    solve("cell_lstm", -1, cell=1)
    solve("D12", -1, D=12)
    solve("T0", -1, T=0)
    solve("B0", -1, B=0)
    solve("dtype", -2, dt=7)
    solve("no_u", -1, u=None)
    solve("no_h", -1, h=None)
    solve("lam_for_gru", -1, lam=0x2000)
    solve("decay_without_lam", -1, cell=dec)
    solve("kappa_zero", -1, cell=dec, lam=0x2000, kappa=0.0)
    solve("kappa_nan", -1, cell=dec, lam=0x2000, kappa=float("nan"))
    solve("kappa_inf", -1, cell=dec, lam=0x2000, kappa=float("inf"))
    solve("stride_odd", -1, st=36)
    solve("stride_negative", -1, sg=-32)
    solve("u_misaligned", -5, u=0x1008)
    solve("h_misaligned", -5, h=0x3008)
    solve("bias_misaligned", -5, bias=0x2002)
    solve("h0_misaligned", -5, h0=0x2002)
    solve("too_large", -6, B=1 << 20, T=1 << 20, D=8)
    solve("T_too_large", -6, T=(1 << 30) + 1, D=8)

    def adj(name, want, **o):
        a = dict(cell=dec, u=0x1000, dt=bf16, sb=128, st=64, sg=32, lam=0x2000, bias=None, h0=None, reset=None,
                 h=0x3000, g=0x4000, du=0x5000, ddt=bf16, dlam=None, dbias=None, dh0=None, B=1, T=2, D=32,
                 kappa=8.0, ws=0x10000, wsb=1 << 20, stream=None)
        a.update(o)
        C["adjoint_" + name] = ("pararnn_linrec_adjoint", list(a.values()), want)
    adj("cell", -1, cell=0)
    adj("no_du", -1, du=None)
    adj("no_g", -1, g=None)
    adj("no_ws", -1, ws=None)
    adj("dlam_for_gru", -1, cell=gru, lam=None, dlam=0x6000)
    adj("du_dtype", -2, ddt=5)
    adj("bf16_du_of_f32_u", -2, dt=f32)
    adj("g_misaligned", -5, g=0x4004)
    adj("dlam_misaligned", -5, dlam=0x6001)
    adj("ws_misaligned", -5, ws=0x10040)
    adj("ws_too_small", -3, wsb=64)

    def step(name, want, **o):
        a = dict(cell=gru, u=0x1000, dt=f32, sb=64, sg=32, lam=None, bias=None, hp=None, hn=0x3000, B=1, D=32,
                 kappa=8.0, stream=None)
        a.update(o)
        C["step_" + name] = ("pararnn_linrec_step", list(a.values()), want)
    step("cell", -1, cell=9)
    step("no_out", -1, hn=None)
    step("D4", -1, D=4)
    step("too_large", -6, B=1 << 30, D=1 << 8)
    step("out_misaligned", -5, hn=0x3002)
    step("prev_misaligned", -5, hp=0x3001)

    def norm(name, want, **o):
        a = dict(h=0x1000, hd=f32, lh=64, g=None, gd=0, lg=0, act=0, wpost=None, r=None, rd=0, lr=0, sc=None,
                 wpre=0x2000, s=0x3000, sd=bf16, x=0x4000, xd=bf16, eps=1e-6, N=2, D=64, stream=None)
        a.update(o)
        C["norm_" + name] = ("pararnn_block_norm", list(a.values()), want)
    norm("no_h", -1, h=None)
    norm("N0", -1, N=0)
    norm("D60", -1, D=60)
    norm("D_too_large", -6, D=8200, lh=8200)
    norm("N_too_large", -6, N=1 << 31)
    norm("eps0", -1, eps=0.0)
    norm("eps_nan", -1, eps=float("nan"))
    norm("act", -1, g=0x5000, lg=64, act=2)
    norm("x_without_w_pre", -1, wpre=None)
    norm("w_pre_without_x", -1, x=None)
    norm("nothing_out", -1, wpre=None, x=None, s=None)
    norm("dtype_h", -2, hd=3)
    norm("dtype_g", -2, g=0x5000, gd=-1, lg=64)
    norm("dtype_x", -2, xd=4)
    norm("stride", -1, lh=60)
    norm("in_place_other_type", -1, r=0x3000, rd=f32, lr=64)
    norm("in_place_strided", -1, r=0x3000, rd=bf16, lr=128)
    norm("h_misaligned", -5, h=0x1008)
    norm("w_misaligned", -5, wpre=0x2004)

    def nadj(name, want, **o):
        a = dict(h=0x1000, hd=f32, lh=64, g=None, gd=0, lg=0, act=0, wpost=None, r=None, rd=0, lr=0, sc=None,
                 wpre=0x2000, ds=0x3000, dsd=bf16, lds=64, dx=0x4000, dxd=bf16, ldx=64, dh=0x5000, dg=None,
                 dres=None, dwpost=None, dsc=None, dwpre=None, eps=1e-6, N=2, D=64, ws=0x10000, wsb=1 << 22,
                 stream=None)
        a.update(o)
        C["norm_adjoint_" + name] = ("pararnn_block_norm_adjoint", list(a.values()), want)
    nadj("no_dh", -1, dh=None)
    nadj("no_dx", -1, dx=None)
    nadj("dx_without_w_pre", -1, wpre=None)
    nadj("no_gradient", -1, wpre=None, dx=None, ds=None)
    nadj("gate_without_dgate", -1, g=0x6000, lg=64)
    nadj("dres_without_res", -1, dres=0x6000)
    nadj("dscale_without_scale", -1, dsc=0x6000)
    nadj("dw_post_without_w_post", -1, dwpost=0x6000)
    nadj("dtype_ds", -2, dsd=9)
    nadj("stride_dx", -1, ldx=4)
    nadj("dh_misaligned", -5, dh=0x5004)
    nadj("ws_misaligned", -5, ws=0x10010)
    nadj("ws_too_small", -3, wsb=16)
    return C


def _main():
    if os.environ.get("CUDA_VISIBLE_DEVICES", None) != "":
        print("refusing: these calls pass made-up device addresses", file=sys.stderr)
        return 2
    lib = pr.load_library()
    print(json.dumps({k: int(getattr(lib, fn)(*a)) for k, (fn, a, _) in _host_cases().items()}))
    return 0


@pytest.fixture(scope="module")
def host_rcs():
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="", PYTHONPATH=ROOT)
    r = subprocess.run([sys.executable, os.path.abspath(__file__)], env=env, capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    return json.loads(r.stdout.strip().splitlines()[-1])


@pytest.mark.parametrize("case", sorted(_host_cases()))
def test_layer_entry_points_reject_bad_arguments_on_host(host_rcs, case):
    assert host_rcs[case] == _host_cases()[case][2]


def test_layer_workspace_sizes():
    w = pr.pararnn_linrec_workspace_size(pr.PARARNN_LIN_DECAY, 8, 4096, 1024)
    assert w >= 8 * 4 * 1024 * 4 and w % 256 == 0
    assert pr.pararnn_linrec_workspace_size(pr.PARARNN_GRU, 8, 4096, 1024) == 0
    assert pr.pararnn_linrec_workspace_size(pr.PARARNN_LIN_GRU, 1, 1, 12) == 0
    assert pr.pararnn_linrec_workspace_size(pr.PARARNN_LIN_GRU, 1, 0, 16) == 0
    assert pr.pararnn_block_norm_workspace_size(1, 64) >= 3 * 64 * 4
    assert pr.pararnn_block_norm_workspace_size(0, 64) == 0
    assert pr.pararnn_block_norm_workspace_size(4, 8200) == 0


def test_nonlinear_entry_points_refuse_the_linear_cells():
    for cell in (pr.PARARNN_LIN_GRU, pr.PARARNN_LIN_DECAY):
        assert pr.pararnn_workspace_size(cell, 1, 256, 64, 0, 0) == 0
        assert pr.pararnn_workspace_size(cell, 1, 256, 64, 0, 1) == 0
        assert pr.pararnn_unfused_workspace_size(cell, 1, 16, 16) == 0


def test_wrappers_refuse_host_tensors_and_unknown_cells():
    u = torch.zeros((1, 4, 2, 8))
    with pytest.raises(ValueError):
        pr.linrec_solve(pr.PARARNN_LIN_GRU, u)
    with pytest.raises(pr.PararnnError):
        pr.linrec_solve(pr.PARARNN_GRU, u)
    with pytest.raises(ValueError):
        pr.linrec_step(pr.PARARNN_LIN_GRU, u[:, 0])
    with pytest.raises(ValueError):
        pr.block_norm(torch.zeros((2, 8)))


if __name__ == "__main__":
    sys.exit(_main())
