"""GPU parity of the block norm and its adjoint against the fp64 restatement in
oracle/layer.py (tolerances: DELTA_NORM times the magnitude there, and half a
step of the output's type), and a run of the layer's operators together."""
import numpy as np
import pytest
import torch

import nonlinear_rnn_paragru_b200 as pr
from oracle import layer as ol

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


def draw(N, D, h=F32, gate=None, post=False, res=None, scale=False, pre=False, s=None, x=BF16, wide=False,
         seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *k: torch.randn(k, generator=g)  # noqa: E731

    def rows(dt, k=1.0):
        if dt is None:
            return None
        if wide:    # part of a wider projection
            return (k * r(N, D + 24)).clamp_(-7, 7).to(dt).cuda()[:, 8:8 + D]
        return (k * r(N, D)).clamp_(-7, 7).to(dt).cuda()
    st = s or res or BF16
    return (dict(h=rows(h), gate=rows(gate), w_post=(1 + 0.2 * r(D)).cuda() if post else None, res=rows(res, 2.0),
                 scale=(0.5 + 0.2 * r(D)).cuda() if scale else None,
                 w_pre=(1 + 0.2 * r(D)).cuda() if pre else None),
            dict(ds=rows(st), dx=rows(x) if pre else None), st, x)


def close(got, want, mag, chain=0.0, what=""):
    tol = (ol.DELTA_NORM + chain) * mag + HALF[got.dtype] * (np.abs(want) + ol.DELTA_NORM * mag) + 1e-37
    err = np.abs(got.double().cpu().numpy() - want)
    bad = ~(err <= tol)         # a NaN is off too
    assert not bad.any(), (what, float((err / tol).max()), np.argwhere(bad)[:3])


def check(p, d, st, xt, act="silu", eps=1e-6):
    s, x = pr.block_norm(**p, act=act, eps=eps, s_dtype=st, x_dtype=xt)
    want = ol.block_norm(**p, act=act, eps=eps)
    assert s.dtype == st and (x is None) == (p["w_pre"] is None)
    close(s, *want["s"], what="s")
    if x is not None:
        assert x.dtype == xt
        close(x, *want["x"], what="x")
    got = pr.block_norm_adjoint(ds=d["ds"], dx=d["dx"], **p, act=act, eps=eps)
    want = ol.block_norm_adjoint(ds=d["ds"], dx=d["dx"], act=act, eps=eps, **p)
    assert {k for k, v in got.items() if v is not None} == set(want)
    N = p["h"].shape[0]
    for k, (v, m) in want.items():
        # a sum over N rows goes through at most N additions
        close(got[k], v, m, N * 2.0 ** -24 if v.ndim == 1 else 0.0, what=k)
    return s, x, got


FULL = dict(gate=BF16, post=True, res=BF16, scale=True, pre=True)
KINDS = {
    "pre": dict(h=BF16, pre=True), "res_pre": dict(h=BF16, res=F32, pre=True),
    "post_gate": dict(gate=BF16, post=True), "full": FULL,
    "full_f32": dict(gate=F32, post=True, res=F32, scale=True, pre=True, x=F32),
    "gate": dict(gate=F32, s=F32), "scale_res": dict(h=BF16, scale=True, res=BF16), "none": dict(s=F32),
    "both": dict(gate=BF16, post=True, res=F32, pre=True), "pre_f32": dict(h=F32, res=F32, pre=True, x=F32),
    "mixed": dict(h=BF16, gate=F32, post=True, res=BF16, scale=True, pre=True, s=F32, x=F32),
    "post_f32_out": dict(h=BF16, post=True, s=F32), "gate_scale_pre": dict(gate=BF16, scale=True, pre=True),
}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("N,D", [(1, 8), (5, 264), (33, 1000)])
def test_parts_match_the_oracle(cuda_ok, kind, N, D):
    check(*draw(N, D, **KINDS[kind], seed=N), act=["silu", "sigmoid"][N % 2])


@pytest.mark.parametrize("D", [8, 16, 248, 256, 264, 512, 776, 1024, 2048, 4096, 4104, 6000, 8192])
def test_widths_match_the_oracle(cuda_ok, D):
    check(*draw(7, D, **FULL, wide=True, seed=D))


@pytest.mark.parametrize("kind,D", [("full_f32", 4096), ("full_f32", 5600), ("full_f32", 8192), ("full", 8192),
                                    ("full", 4096), ("post_gate", 8192), ("res_pre", 8192), ("post_gate", 1000),
                                    ("res_pre", 1000), ("res_pre", 4096), ("pre_f32", 4096), ("pre_f32", 520),
                                    ("both", 1000), ("mixed", 1000), ("full_f32", 776), ("full", 136), ("post_gate", 136),
                                    ("res_pre", 72), ("full_f32", 200), ("both", 24), ("mixed", 256)])
def test_wide_rows_of_several_rounds(cuda_ok, kind, D):
    # more rows than blocks, at the widths where the adjoint's ring holds four
    # rows, three, two and one
    check(*draw(330 if D > 600 else 1300 if D > 256 else 6000, D, **KINDS[kind], seed=D))


def test_only_one_of_the_gradients(cuda_ok):
    p, d, st, xt = draw(700, 520, **FULL)
    for ds, dx, w in ((None, d["dx"], p["w_pre"]), (d["ds"], None, None)):
        q = {**p, "w_pre": w}
        got = pr.block_norm_adjoint(ds=ds, dx=dx, **q)
        for k, (v, m) in ol.block_norm_adjoint(ds=ds, dx=dx, **q).items():
            close(got[k], v, m, 700 * 2.0 ** -24 if v.ndim == 1 else 0.0, what=k)


@pytest.mark.parametrize("N", [1, 2, 8, 9, 147, 1000, 5000])
def test_row_counts_match_the_oracle(cuda_ok, N):
    check(*draw(N, 72, **FULL, seed=N))
    if N >= 1000:
        check(*draw(N, 520, **KINDS["res_pre"], seed=N))


def test_rows_of_zeros_and_cancelled_rows(cuda_ok):
    p, d, st, xt = draw(4, 64, **KINDS["full_f32"])
    p["h"][0] = 0
    p["res"][0] = 0          # s = 0: x = 0, the root is 1 / sqrt(eps)
    s, x, g = check(p, d, st, xt, eps=1e-3)
    assert (s[0] == 0).all() and (x[0] == 0).all() and torch.isfinite(g["dh"]).all()


def test_nan_and_infinities_stay_in_their_row(cuda_ok):
    p, d, st, xt = draw(40, 72, **KINDS["full_f32"])
    clean = pr.block_norm(**p, s_dtype=st, x_dtype=xt)
    cg = pr.block_norm_adjoint(ds=d["ds"], dx=d["dx"], **p)
    p["h"][3, 5], p["gate"][11, 0], p["res"][20, 1] = float("nan"), float("inf"), float("-inf")
    rows = [r for r in range(40) if r not in (3, 11, 20)]
    for a, b in zip(pr.block_norm(**p, s_dtype=st, x_dtype=xt), clean):
        assert torch.equal(a[rows], b[rows])
    g = pr.block_norm_adjoint(ds=d["ds"], dx=d["dx"], **p)
    for k in ("dh", "dgate", "dres"):
        assert torch.equal(g[k][rows], cg[k][rows])


def test_in_place_residual_and_given_outputs(cuda_ok):
    p, d, st, xt = draw(50, 520, **FULL)
    s, x = pr.block_norm(**p)
    big = torch.full((50 * 520 + 32,), 3.0, dtype=BF16, device="cuda")
    xo = big[16:-16].view(50, 520)
    res = p["res"].clone()
    s2, x2 = pr.block_norm(**{**p, "res": res}, out=(res, xo))
    assert s2 is res and x2 is xo and torch.equal(res, s) and torch.equal(xo, x)
    assert (big[:16] == 3).all() and (big[-16:] == 3).all()
    s3, x3 = pr.block_norm(**p, want_s=False)
    assert s3 is None and torch.equal(x3, x)


def test_leading_axes_and_broadcast_rows(cuda_ok):
    p, d, st, xt = draw(6, 64, **FULL)
    flat = pr.block_norm(**p)
    q = {k: v.view(2, 3, 64) if v is not None and v.dim() == 2 else v for k, v in p.items()}
    for a, b in zip(pr.block_norm(**q), flat):
        assert a.shape == (2, 3, 64) and torch.equal(a.view(6, 64), b)
    g1 = pr.block_norm_adjoint(ds=d["ds"], dx=d["dx"], **p)
    g2 = pr.block_norm_adjoint(ds=d["ds"].view(2, 3, 64), dx=d["dx"].view(2, 3, 64), **q)
    assert all(torch.equal(g1[k], g2[k].view(g1[k].shape)) for k in g1)
    one = {**p, "res": p["res"][:1].expand(6, 64)}          # one residual row for all
    for a, b in zip(pr.block_norm(**one), pr.block_norm(**{**p, "res": one["res"].contiguous()})):
        assert torch.equal(a, b)


def test_equal_calls_streams_and_graphs(cuda_ok):
    p, d, st, xt = draw(700, 520, **FULL)
    s, x = pr.block_norm(**p)
    g = pr.block_norm_adjoint(ds=d["ds"], dx=d["dx"], **p)
    torch.cuda.synchronize()
    st1, st2 = torch.cuda.Stream(), torch.cuda.Stream()
    r1 = pr.block_norm_adjoint(ds=d["ds"], dx=d["dx"], **p, stream=st1)
    r2 = pr.block_norm_adjoint(ds=d["ds"], dx=d["dx"], **p, stream=st2)
    torch.cuda.synchronize()
    for r in (r1, r2):
        assert all(torch.equal(r[k], g[k]) for k in g)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gs, gx = pr.block_norm(**p)
        gg = pr.block_norm_adjoint(ds=d["ds"], dx=d["dx"], **p)
    p2, d2, _, _ = draw(700, 520, **FULL, seed=5)
    for a, b in list(zip(p.values(), p2.values())) + list(zip(d.values(), d2.values())):
        a.copy_(b)
    graph.replay()
    s, x = pr.block_norm(**p)
    g = pr.block_norm_adjoint(ds=d["ds"], dx=d["dx"], **p)
    assert torch.equal(gs, s) and torch.equal(gx, x) and all(torch.equal(gg[k], g[k]) for k in g)


def test_refusals(cuda_ok):
    p, d, st, xt = draw(4, 64, **FULL)
    for bad in (dict(gate=p["gate"][:3]), dict(res=p["res"].cpu()), dict(w_post=p["w_post"][:8]),
                dict(act="relu"), dict(h=p["h"].t()), dict(out=(p["res"][:, :32], None))):
        with pytest.raises(ValueError):
            pr.block_norm(**{**p, **bad})
    with pytest.raises(TypeError):
        pr.block_norm(**{**p, "scale": p["scale"].double()})
    for bad in (dict(h=p["h"].half()), dict(eps=0.0), dict(eps=float("inf"))):
        with pytest.raises(pr.PararnnError):
            pr.block_norm(**{**p, **bad})
    for shape in ((0, 64), (4, 60), (1, 8200)):
        with pytest.raises(pr.PararnnError):
            pr.block_norm(torch.zeros(shape, device="cuda"))
    with pytest.raises(ValueError):
        pr.block_norm_adjoint(ds=d["ds"], dx=None, **p)
    with pytest.raises(pr.PararnnError):
        pr.block_norm_adjoint(ds=None, dx=None, **{**p, "w_pre": None})
    wide = torch.zeros((4, 68), device="cuda")[:, 4:]       # rows 272 bytes apart, 16 bytes in
    with pytest.raises(pr.PararnnError):
        pr.block_norm(wide)


# ------------------------------------------------------------ a whole layer --
@pytest.mark.parametrize("cell", ["lin_gru", "lin_decay", "gru"])
def test_a_layer_forward_backward_and_decode(cuda_ok, cell):
    """Pre-norm, projection, recurrence, gated norm added to the residual
    stream with the next pre-norm: the fp64 forward and its gradients, then the
    same tokens one at a time."""
    B, T, C, D = 2, 40, 48, 64
    G = 2 if cell == "lin_gru" else 3
    code = {"lin_gru": pr.PARARNN_LIN_GRU, "lin_decay": pr.PARARNN_LIN_DECAY}.get(cell)
    gen = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(s, generator=gen).cuda()  # noqa: E731
    stream = r(B, T, D)
    W = r((G + 1) * D, D) / D ** 0.5
    w0, w_post, scale, w_pre = (1 + 0.1 * r(D) for _ in range(4))
    bias, lam = 0.1 * r(G, D), r(D) - 5 if cell == "lin_decay" else None
    a3 = 0.5 * r(3, D) if cell == "gru" else None
    ds, dx = r(B, T, D), r(B, T, D)

    # forward, fp32 throughout (the types' roundings are other tests' matter)
    _, x0 = pr.block_norm(stream, w_pre=w0, x_dtype=F32, want_s=False)
    proj = x0 @ W.t()
    u, gate = proj[..., :G * D].unflatten(-1, (G, D)), proj[..., G * D:]
    if cell == "gru":
        uc = u.contiguous()
        h, st, _ = pr.gru_solve(uc, a3, bias)
        assert pr.read_stats(st)["status"] == "converged"
    else:
        h = pr.linrec_solve(code, u, lam, bias)
    parts = dict(gate=gate, w_post=w_post, res=stream, scale=scale, w_pre=w_pre)
    s, x = pr.block_norm(h, **parts, x_dtype=F32)

    # backward
    gn = pr.block_norm_adjoint(h, ds, dx, **parts)
    h0 = torch.zeros((B, D), device="cuda")
    if cell == "gru":
        gr = pr.adjoint(pr.PARARNN_GRU, uc, a3, bias, h0, h, gn["dh"])
    else:
        gr = pr.linrec_adjoint(code, u, lam, bias, None, h, gn["dh"])
    dproj = torch.cat([gr["du"].flatten(2), gn["dgate"]], -1)
    dW = dproj.flatten(0, 1).t() @ x0.flatten(0, 1)
    g0 = pr.block_norm_adjoint(stream, None, dproj @ W, w_pre=w0)
    dstream = gn["dres"] + g0["dh"]

    # the same in float64 with autograd
    v = {k: t.double().cpu().requires_grad_(True) for k, t in
         dict(stream=stream, W=W, w0=w0, w_post=w_post, scale=scale, w_pre=w_pre, bias=bias).items()}
    lam64 = None if lam is None else lam.double().cpu().requires_grad_(True)
    a64 = None if a3 is None else a3.double().cpu().requires_grad_(True)
    rms = lambda t: t / torch.sqrt(t.pow(2).mean(-1, keepdim=True) + 1e-6)  # noqa: E731
    p = (rms(v["stream"]) * v["w0"]) @ v["W"].t()
    q, gt = p[..., :G * D].unflatten(-1, (G, D)) + v["bias"], p[..., G * D:]
    hs, hh = [], torch.zeros((B, D), dtype=torch.float64)
    for t in range(T):
        if cell == "lin_gru":
            z = torch.sigmoid(q[:, t, 0])
            hh = (1 - z) * hh + z * torch.tanh(q[:, t, 1])
        elif cell == "gru":
            z, rr = torch.sigmoid(a64[0] * hh + q[:, t, 0]), torch.sigmoid(a64[1] * hh + q[:, t, 1])
            hh = (1 - z) * hh + z * torch.tanh(a64[2] * (rr * hh) + q[:, t, 2])
        else:
            la = -8 * torch.nn.functional.softplus(lam64) * torch.sigmoid(q[:, t, 0])
            hh = la.exp() * hh + torch.sqrt(-torch.expm1(2 * la)) * torch.sigmoid(q[:, t, 1]) * q[:, t, 2]
        hs.append(hh)
    H = torch.stack(hs, 1)
    S = v["stream"] + v["scale"] * rms(H) * v["w_post"] * torch.nn.functional.silu(gt)
    X = rms(S) * v["w_pre"]
    leaves = list(v.values()) + [t for t in (lam64, a64) if t is not None]
    grads = torch.autograd.grad((S * ds.double().cpu()).sum() + (X * dx.double().cpu()).sum(), leaves)
    want = dict(zip(list(v) + (["lam"] if lam is not None else ["a"]), grads))
    # states within 1e-4 and gradients within 1e-3 of the tensor's largest value: the library's contract for a
    # solve and its adjoint, which every value here went through
    assert (s.double().cpu() - S).abs().max() < 1e-4 * S.abs().max()
    assert (x.double().cpu() - X).abs().max() < 1e-3 * X.abs().max()
    got = dict(stream=dstream, W=dW, w0=g0["dw_pre"], w_post=gn["dw_post"], scale=gn["dscale"], w_pre=gn["dw_pre"],
               bias=gr["dbias"], lam=gr.get("dlam"), a=gr.get("da"))
    for k, w in want.items():
        assert (got[k].double().cpu() - w).abs().max() < 1e-3 * w.abs().max(), k

    # one token at a time
    state = torch.zeros((B, D), device="cuda")
    for t in range(T):
        _, y0 = pr.block_norm(stream[:, t].contiguous(), w_pre=w0, x_dtype=F32, want_s=False)
        pt = y0 @ W.t()
        ut = pt[:, :G * D].unflatten(-1, (G, D))
        if cell == "gru":
            pr.gru_step(ut.contiguous(), a3, bias, state, out=state)
        else:
            pr.linrec_step(code, ut, lam, bias, state, out=state)
        st_, xt_ = pr.block_norm(state, gate=pt[:, G * D:], w_post=w_post, res=stream[:, t].contiguous(),
                                 scale=scale, w_pre=w_pre, x_dtype=F32)
        assert (st_.double().cpu() - S[:, t]).abs().max() < 1e-4 * S.abs().max()
        assert (xt_.double().cpu() - X[:, t]).abs().max() < 1e-3 * X.abs().max()
