"""GPU parity of the gated linear recurrence (solve, adjoint, decode step)
against the fp64 restatement in oracle/layer.py, whose error bounds (a
recurrence over the roundings of each step) are the tolerances."""
import numpy as np
import pytest
import torch

import nonlinear_rnn_paragru_b200 as pr
from oracle import layer as ol

pytestmark = pytest.mark.gpu

GRU, DECAY = pr.PARARNN_LIN_GRU, pr.PARARNN_LIN_DECAY
HALF = torch.finfo(torch.bfloat16).eps / 2     # a rounding to bf16 is off by at most this, relatively


def draw(cell, B, T, D, dtype="bf16", docs=0, fused=False, params=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    G = 2 if cell == GRU else 3
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    if fused:   # part of a projection that also holds another G + 1st input
        u = r(B, T, (G + 1) * D).clamp_(-5, 5).to(dt)
    else:
        u = r(B, T, G * D).clamp_(-5, 5).to(dt)
    x = dict(u=u.cuda()[..., :G * D].unflatten(-1, (G, D)), lam=None, bias=None, h0=None, reset=None)
    if cell == DECAY:   # decays of 0.9 to 0.9995 at r = 1
        a = 0.9 + 0.0995 * torch.rand(D, generator=g)
        x["lam"] = torch.log(torch.expm1(-torch.log(a) / 8)).cuda()
    if params:
        x["bias"], x["h0"] = (0.2 * r(G, D)).clamp_(-1, 1).cuda(), r(B, D).cuda()
    if docs:
        x["reset"] = (torch.rand((B, T), generator=g) < 1.0 / docs).cuda()
    x["dLdh"] = r(B, T, D).cuda()
    return x


def ref(cell, x, **kw):
    return ol.lin_seq(cell, x["u"], x["lam"], x["bias"], x["h0"], x["reset"], **kw)


def solve(cell, x, **kw):
    return pr.linrec_solve(cell, x["u"], x["lam"], x["bias"], x["h0"], reset=x["reset"], **kw)


def adjoint(cell, x, h, **kw):
    return pr.linrec_adjoint(cell, x["u"], x["lam"], x["bias"], x["h0"], h, x["dLdh"], reset=x["reset"], **kw)


def check_states(h, H, E, what=""):
    err = np.abs(h.cpu().numpy().astype(np.float64) - H)
    bad = ~(err <= E + 1e-37)   # a NaN is off too
    assert not bad.any(), (what, float((err / (E + 1e-37)).max()), np.argwhere(bad)[:3])


def check_adjoint(got, want, rounded):
    for k, (v, e) in want.items():
        g = got[k].double().cpu().numpy()
        tol = e + 1e-37 + (HALF * (np.abs(v) + e) if k == "du" and rounded else 0)
        bad = ~(np.abs(g - v) <= tol)
        assert not bad.any(), (k, float((np.abs(g - v) / tol).max()), np.argwhere(bad)[:3])


# one token; a warp's steps and their neighbours; the first cluster sizes; many
# rounds; one lane pair, a partial tile, several tiles
SHAPES = [(1, 1, 8), (3, 1, 200), (1, 2, 64), (2, 7, 72), (1, 8, 64), (1, 9, 8), (5, 63, 24), (1, 64, 64),
          (1, 65, 128), (2, 129, 200), (1, 500, 1000), (3, 1531, 136), (1, 4099, 64), (7, 33, 520),
          (300, 3, 72),
          # tiles enough for the wide kernels: clusters of 8, 4, 2 and 1, rounds
          # that end inside a group, a warp and a CTA
          (20, 700, 72), (1, 602, 2048), (38, 260, 136), (150, 70, 200), (30, 150, 640), (10, 129, 1000), (1, 2999, 1216)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cell", [GRU, DECAY], ids=["gru", "decay"])
@pytest.mark.parametrize("B,T,D", SHAPES)
def test_solve_and_adjoint_match_the_oracle(cuda_ok, cell, B, T, D, dtype):
    x = draw(cell, B, T, D, dtype, docs=[0, 3, 40][(B + T) % 3], fused=T % 2 == 1, seed=T)
    H, E = ref(cell, x)
    h = solve(cell, x)
    check_states(h, H, E)
    got = adjoint(cell, x, h)
    want = ol.lin_adjoint(cell, x["u"], x["lam"], x["bias"], x["h0"], h, x["dLdh"], x["reset"])
    assert got["du"].dtype == x["u"].dtype and got["du"].is_contiguous()
    check_adjoint(got, want, dtype == "bf16")


@pytest.mark.parametrize("cell", [GRU, DECAY], ids=["gru", "decay"])
def test_without_bias_state_and_sums(cuda_ok, cell):
    x = draw(cell, 2, 100, 72, params=False, seed=3)
    h = solve(cell, x)
    check_states(h, *ref(cell, x))
    got = adjoint(cell, x, h, want_params=False, want_dh0=False, du_dtype=torch.float32)
    assert got["dlam"] is None and got["dbias"] is None and got["dh0"] is None
    want = ol.lin_adjoint(cell, x["u"], x["lam"], x["bias"], x["h0"], h, x["dLdh"], x["reset"])
    check_adjoint({"du": got["du"]}, {"du": want["du"]}, False)


@pytest.mark.parametrize("cell", [GRU, DECAY], ids=["gru", "decay"])
def test_slow_decays_over_a_long_sequence(cuda_ok, cell):
    # 20000 steps that remember thousands of steps, with steady gates, so that
    # a rounding of a = 1 - m would add up in one direction: the bound holds
    # no such term
    B, T, D = 1, 20000, 64
    x = draw(cell, B, T, D, "f32", seed=9)
    if cell == GRU:
        x["u"][:, :, 0] = -4.0 + 0.01 * x["u"][:, :, 0]
        x["bias"][0] = -1.0
    else:
        x["u"][:, :, 0] = 0.01 * x["u"][:, :, 0]
        x["lam"][:] = torch.linspace(-12, -7, D)
    h = solve(cell, x)
    check_states(h, *ref(cell, x))
    got = adjoint(cell, x, h)
    want = ol.lin_adjoint(cell, x["u"], x["lam"], x["bias"], x["h0"], h, x["dLdh"], x["reset"])
    check_adjoint(got, want, False)


@pytest.mark.parametrize("T", [1, 70, 1000])
def test_a_reset_at_every_step_leaves_the_inputs(cuda_ok, T):
    x = draw(DECAY, 2, T, 64, seed=T)
    x["reset"] = torch.ones((2, T), dtype=torch.uint8, device="cuda")
    x["h0"][:] = float("nan")
    h = solve(DECAY, x)
    _, b = ol.lin_coef(DECAY, x["u"], x["lam"], x["bias"])
    assert np.abs(h.cpu().numpy() - b).max() <= 48 * 2.0 ** -24 * np.abs(b).max()
    got = adjoint(DECAY, x, h)
    assert (got["dh0"] == 0).all()
    assert torch.isfinite(got["du"].float()).all()


@pytest.mark.parametrize("cell", [GRU, DECAY], ids=["gru", "decay"])
def test_infinities_and_nan_stay_in_their_document(cuda_ok, cell):
    T, cut = 700, 333
    x = draw(cell, 2, T, 72, "f32", seed=5)
    clean = {k: v.clone() if torch.is_tensor(v) else v for k, v in x.items()}
    r = torch.zeros((2, T), dtype=torch.bool, device="cuda")
    r[0, cut] = True
    x["reset"] = clean["reset"] = r
    x["u"][0, 17, :, 3] = float("nan")
    x["u"][0, 18, -1, 4] = float("inf")
    x["h0"][0, 5] = float("-inf")
    x["dLdh"][0, 500, 6] = float("nan")
    h, hc = solve(cell, x), solve(cell, clean)
    assert torch.isnan(h[0, 17:cut, 3]).all()
    assert torch.equal(h[0, cut:], hc[0, cut:]) and torch.equal(h[1], hc[1])
    others = [c for c in range(72) if c not in (3, 4, 5)]
    assert torch.equal(h[0][:, others], hc[0][:, others])
    # the gradient of the second document never enters the first
    got, want = adjoint(cell, x, hc), adjoint(cell, clean, hc)
    assert torch.isnan(got["du"][0, cut:501, :, 6].float()).any()
    assert torch.equal(got["du"][0, 19:cut], want["du"][0, 19:cut])
    assert torch.equal(got["dh0"][0, 7:], want["dh0"][0, 7:])


def test_gates_at_infinity_keep_or_replace_the_state(cuda_ok):
    T, D = 50, 64
    u = torch.zeros((1, T, 2, D), device="cuda")
    h0 = torch.randn((1, D), device="cuda")
    u[:, :, 0] = float("-inf")
    u[:, :, 1] = 3.0
    assert torch.equal(pr.linrec_solve(GRU, u, h0=h0), h0[:, None].expand(1, T, D))
    u[:, :, 0] = float("inf")
    want = torch.tanh(torch.tensor(3.0, dtype=torch.float64)).item()
    got = pr.linrec_solve(GRU, u, h0=h0)
    assert (got.double() - want).abs().max() < 16 * 2.0 ** -24
    u[:, :, 0], u[:, :, 1] = 0.0, float("inf")        # candidate 1
    got = pr.linrec_solve(GRU, u, h0=torch.zeros_like(h0))[0, :, 0].double().cpu()
    assert (got - (1 - 0.5 ** torch.arange(1, T + 1, dtype=torch.float64))).abs().max() < 8 * 2.0 ** -24
    v = torch.zeros((1, T, 3, D), device="cuda")
    v[:, :, 0], v[:, :, 2] = float("-inf"), 5.0       # r = 0: the state stays
    lam = torch.zeros(D, device="cuda")
    assert torch.equal(pr.linrec_solve(DECAY, v, lam, h0=h0), h0[:, None].expand(1, T, D))
    g = pr.linrec_adjoint(DECAY, v, lam, None, h0, h0[:, None].expand(1, T, D).contiguous(),
                          torch.ones((1, T, D), device="cuda"))
    assert (g["du"] == 0).all() and (g["dlam"] == 0).all() and (g["dh0"] == T).all()


def test_lin_gru_equals_paragru_without_recurrent_weights(cuda_ok):
    # both within 1e-4 of the exact trajectory is the solves' contract; here
    # both are exact cells, so the states agree to the linear solve's bound
    # plus the Newton tolerance, which the recurrence can grow by 1 / min z
    x = draw(GRU, 2, 300, 64, seed=11)
    u3 = torch.stack([x["u"][:, :, 0], torch.zeros_like(x["u"][:, :, 0]), x["u"][:, :, 1]], 2).contiguous()
    b3 = torch.stack([x["bias"][0], torch.zeros_like(x["bias"][0]), x["bias"][1]])
    a = torch.zeros((3, 64), device="cuda")
    hn, st, _ = pr.gru_solve(u3, a, b3, x["h0"])
    assert pr.read_stats(st)["status"] == "converged"
    h = solve(GRU, x)
    assert (h - hn).abs().max() < 1e-4
    gl = adjoint(GRU, x, hn, du_dtype=torch.float32)
    gn = pr.adjoint(pr.PARARNN_GRU, u3, a, b3, x["h0"], hn, x["dLdh"])
    for i, j in ((0, 0), (1, 2)):
        scale = gn["du"][:, :, j].abs().max()
        assert (gl["du"][:, :, i] - gn["du"][:, :, j]).abs().max() < 1e-3 * scale
    assert (gl["dh0"] - gn["dh0"]).abs().max() < 1e-3 * gn["dh0"].abs().max()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cell", [GRU, DECAY], ids=["gru", "decay"])
def test_steps_continue_the_solve(cuda_ok, cell, dtype):
    B, T, D, T0 = 3, 90, 40, 70
    x = draw(cell, B, T, D, dtype, fused=True, seed=2)
    H, E = ref(cell, x)
    h = pr.linrec_solve(cell, x["u"][:, :T0], x["lam"], x["bias"], x["h0"])
    state = h[:, -1].contiguous()
    out = []
    for t in range(T0, T):
        if t % 2:
            assert pr.linrec_step(cell, x["u"][:, t], x["lam"], x["bias"], state, out=state) is state
        else:
            state = pr.linrec_step(cell, x["u"][:, t], x["lam"], x["bias"], state)
        out.append(state.clone())
    check_states(torch.cat([h, torch.stack(out, 1)], 1), H, E)


def test_step_from_nothing_and_large_batch(cuda_ok):
    for B, D in ((1, 8), (513, 1000)):
        x = draw(DECAY, B, 1, D, params=False, seed=B)
        x["h0"] = None
        H, E = ref(DECAY, x)
        check_states(pr.linrec_step(DECAY, x["u"][:, 0], x["lam"])[:, None], H, E)


def test_equal_calls_return_equal_bits_and_nothing_else_is_written(cuda_ok):
    B, T, D = 2, 1000, 72
    x = draw(DECAY, B, T, D, docs=100, seed=8)
    big = torch.full((B * T * D + 128,), 7.5, device="cuda")
    out = big[64:-64].view(B, T, D)
    h1 = solve(DECAY, x, out=out)
    assert h1 is out and (big[:64] == 7.5).all() and (big[-64:] == 7.5).all()
    h2 = solve(DECAY, x)
    assert torch.equal(h1, h2)
    a, b = adjoint(DECAY, x, h2), adjoint(DECAY, x, h2)
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_broadcast_batch_and_gradient_of_every_row(cuda_ok):
    # one u for all rows (stride 0): each row's gradient is its own
    x = draw(GRU, 1, 60, 64, seed=4)
    x["u"] = x["u"].expand(4, 60, 2, 64)
    x["h0"] = torch.randn((4, 64), device="cuda")
    x["dLdh"] = torch.randn((4, 60, 64), device="cuda")
    h = solve(GRU, x)
    check_states(h, *ref(GRU, x))
    want = ol.lin_adjoint(GRU, x["u"], None, x["bias"], x["h0"], h, x["dLdh"])
    check_adjoint(adjoint(GRU, x, h), want, True)


def test_other_streams_and_two_calls_at_once(cuda_ok):
    xs = [draw(DECAY, 2, 800, 128, seed=s) for s in (1, 2)]
    want = []
    for x in xs:
        h = solve(DECAY, x)
        want.append((h, adjoint(DECAY, x, h)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        got = []
        for x, s in zip(xs, streams):
            h = solve(DECAY, x, stream=s)
            got.append((h, adjoint(DECAY, x, h, stream=s)))
        torch.cuda.synchronize()
        for (h, g), (hw, gw) in zip(got, want):
            assert torch.equal(h, hw)
            assert all(torch.equal(g[k], gw[k]) for k in g)
    raw = solve(DECAY, xs[0], stream=streams[0].cuda_stream)
    torch.cuda.synchronize()
    assert torch.equal(raw, want[0][0])


def test_captured_graphs_replay_on_new_inputs(cuda_ok):
    xs = [draw(DECAY, 2, 300, 128, seed=s) for s in (1, 2)]
    graphs = []
    for x in xs:          # two graphs, each with its own scratch
        solve(DECAY, x)
        adjoint(DECAY, x, solve(DECAY, x))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            h = solve(DECAY, x)
            out = adjoint(DECAY, x, h)
            nxt = pr.linrec_step(DECAY, x["u"][:, 0], x["lam"], x["bias"], x["h0"])
        graphs.append((g, h, out, nxt))
    new = [draw(DECAY, 2, 300, 128, seed=s) for s in (3, 4)]
    for x, n in zip(xs, new):
        for k in ("u", "lam", "bias", "h0", "dLdh"):
            x[k].copy_(n[k])
    for g, *_ in graphs:
        g.replay()
    for (g, h, out, nxt), x in zip(graphs, xs):
        hw = solve(DECAY, x)
        gw = adjoint(DECAY, x, hw)
        assert torch.equal(h, hw) and torch.equal(nxt, pr.linrec_step(DECAY, x["u"][:, 0], x["lam"],
                                                                      x["bias"], x["h0"]))
        assert all(torch.equal(out[k], gw[k]) for k in gw)


def test_refusals(cuda_ok):
    x = draw(DECAY, 2, 16, 64)
    u, lam, bias, h0 = x["u"], x["lam"], x["bias"], x["h0"]
    bad = [dict(lam=None), dict(lam=lam[:32]), dict(bias=bias[:2]), dict(h0=h0[:1]), dict(h0=h0.cpu()),
           dict(reset=torch.zeros((2, 15), dtype=torch.bool, device="cuda")),
           dict(out=torch.empty((2, 16, 32), device="cuda")), dict(u=u[..., ::2]), dict(u=u[:, :, :2])]
    for b in bad:
        a = {**dict(u=u, lam=lam, bias=bias, h0=h0, reset=None, out=None), **b}
        with pytest.raises(ValueError):
            pr.linrec_solve(DECAY, a["u"], a["lam"], a["bias"], a["h0"], reset=a["reset"], out=a["out"])
    for b in (dict(bias=bias.double()), dict(h0=h0.bfloat16()),
              dict(reset=torch.zeros((2, 16), device="cuda"))):
        a = {**dict(bias=bias, h0=h0, reset=None), **b}
        with pytest.raises(TypeError):
            pr.linrec_solve(DECAY, u, lam, a["bias"], a["h0"], reset=a["reset"])
    for bu in (u.half(), u[..., :60], u[:, :0], torch.empty((2, 16, 3, 72), dtype=u.dtype, device="cuda")[..., 4:68]):
        with pytest.raises((pr.PararnnError, ValueError)):
            pr.linrec_solve(DECAY, bu, torch.zeros(bu.shape[-1], device="cuda"))
    with pytest.raises(ValueError):
        pr.linrec_solve(GRU, u[:, :, :2], lam)
    h = solve(DECAY, x)
    with pytest.raises(ValueError):
        pr.linrec_adjoint(DECAY, u, lam, bias, h0, h[:, :8], x["dLdh"])
    with pytest.raises(ValueError):
        pr.linrec_adjoint(DECAY, u, lam, bias, h0, h, None)
    with pytest.raises(pr.PararnnError):
        pr.linrec_solve(DECAY, u, lam, kappa=-1.0)
