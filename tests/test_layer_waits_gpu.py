"""The bounded waits of the layer operators: a part of an exchange is withheld,
so that the waits for it run out after a short limit.  The call then ends, says
so in its status word, leaves NaN where a value depends on what never came and
the right values elsewhere, and the next call is not touched by it."""
import pytest
import torch

import nonlinear_rnn_paragru_b200 as pr

pytestmark = pytest.mark.gpu

GRU, DECAY = pr.PARARNN_LIN_GRU, pr.PARARNN_LIN_DECAY
TIMEOUT = 3


def withhold(at, us=20000):
    return pr._opts(flags=pr.PARARNN_FLAG_INJECT_WITHHOLD, inject_chunk=at, timeout_us=us)


def word():
    return torch.full((1,), 77, dtype=torch.int32, device="cuda")


def draw(cell, B, T, D, dtype, reset=False, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    G = 2 if cell == GRU else 3
    x = dict(u=r(B, T, G, D).to(dtype).cuda(), lam=(r(D) - 4).cuda() if cell == DECAY else None,
             bias=(0.2 * r(G, D)).cuda(), h0=r(B, D).cuda())
    return x, (torch.rand((B, T), generator=g) < 0.005).cuda() if reset else None, r(B, T, D).cuda()


# clusters of 8, 4 and 2 on 64-channel tiles and of 8 on narrow ones, several
# rounds each; bf16 u, and fp32 u, whose solve publishes a round ahead
SHAPES = [(1, 14000, 24), (20, 2100, 72), (30, 1500, 72), (74, 1100, 64)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("cell", [GRU, DECAY], ids=["gru", "decay"])
@pytest.mark.parametrize("B,T,D", SHAPES)
def test_solve_whose_cluster_waits_run_out(cuda_ok, cell, B, T, D, dtype):
    x, _, _ = draw(cell, B, T, D, dtype, seed=T)
    st = word()
    want = pr.linrec_solve(cell, **x, status=st)
    assert st.item() == 0
    for turn, rank in ((0, 0), (1, 1), (1, 0), (2, 1)):
        h = pr.linrec_solve(cell, **x, status=st, opts=withhold(8 * turn + rank))
        torch.cuda.synchronize()
        if st.item() == 0:      # the cluster has fewer rounds, or one CTA
            assert torch.equal(h, want)
            assert (B, turn, rank) != (1, 0, 0) and (B, turn, rank) != (1, 1, 1)
            continue
        assert st.item() == TIMEOUT
        lost = torch.isnan(h).all(-1)                           # [B, T]
        first = int(lost[0].int().argmax())
        assert (first > 0) == (turn > 0)
        assert not lost[:, :first].any() and lost[:, first:].all()
        assert torch.equal(h[:, :first], want[:, :first])
        assert torch.equal(pr.linrec_solve(cell, **x, status=st), want) and st.item() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("cell", [GRU, DECAY], ids=["gru", "decay"])
@pytest.mark.parametrize("B,T,D", SHAPES)
def test_adjoint_whose_cluster_waits_run_out(cuda_ok, cell, B, T, D, dtype):
    x, _, g = draw(cell, B, T, D, dtype, seed=T)
    h, st = pr.linrec_solve(cell, **x), word()
    want = pr.linrec_adjoint(cell, **x, h=h, dLdh=g, status=st)
    assert st.item() == 0
    for turn, rank in ((0, 1), (1, 0), (2, 1)):
        got = pr.linrec_adjoint(cell, **x, h=h, dLdh=g, status=st, opts=withhold(8 * turn + rank))
        torch.cuda.synchronize()
        if st.item() == 0:
            assert all(got[k] is None or torch.equal(got[k], want[k]) for k in got)
            assert (B, turn) not in ((1, 0), (1, 1))
            continue
        assert st.item() == TIMEOUT
        lost = torch.isnan(got["du"]).all(-1).all(-1)           # [B, T]
        last = T - int(lost[0].flip(0).int().argmax())          # steps below it are lost
        assert (last < T) == (turn > 0)
        assert not lost[:, last:].any() and lost[:, :last].all()
        assert torch.equal(got["du"][:, last:], want["du"][:, last:])
        for k in ("dh0", "dbias", "dlam"):
            assert got[k] is None or torch.isnan(got[k]).all(), k
        again = pr.linrec_adjoint(cell, **x, h=h, dLdh=g, status=st)
        assert st.item() == 0
        assert all(again[k] is None or torch.equal(again[k], want[k]) for k in again)


@pytest.mark.parametrize("cell", [GRU, DECAY], ids=["gru", "decay"])
def test_what_a_reset_cuts_off_is_not_lost(cuda_ok, cell):
    x, reset, g = draw(cell, 1, 14000, 24, torch.bfloat16, reset=True)
    want = pr.linrec_solve(cell, **x, reset=reset)
    wantg = pr.linrec_adjoint(cell, **x, h=want, dLdh=g, reset=reset)
    st = word()
    h = pr.linrec_solve(cell, **x, reset=reset, status=st, opts=withhold(8))
    assert st.item() == TIMEOUT
    bad = torch.isnan(h)
    assert bad.any() and torch.equal(h[~bad], want[~bad])
    got = pr.linrec_adjoint(cell, **x, h=want, dLdh=g, reset=reset, status=st, opts=withhold(8))
    assert st.item() == TIMEOUT
    bad = torch.isnan(got["du"])
    assert bad.any() and torch.equal(got["du"][~bad], wantg["du"][~bad])


def test_a_cluster_of_one_waits_for_nobody(cuda_ok):
    x, _, g = draw(GRU, 300, 30, 64, torch.bfloat16)   # no more steps than the shortest round of one CTA
    h, st = pr.linrec_solve(GRU, **x), word()
    assert torch.equal(pr.linrec_solve(GRU, **x, status=st, opts=withhold(0)), h) and st.item() == 0
    want = pr.linrec_adjoint(GRU, **x, h=h, dLdh=g)
    got = pr.linrec_adjoint(GRU, **x, h=h, dLdh=g, status=st, opts=withhold(0))
    assert st.item() == 0 and all(got[k] is None or torch.equal(got[k], want[k]) for k in got)


def test_status_in_a_graph_and_through_the_plain_bindings(cuda_ok):
    x, _, g = draw(DECAY, 1, 14000, 24, torch.bfloat16)
    h = torch.empty((1, 14000, 24), device="cuda")
    st = word()
    pr.pararnn_linrec_solve_ex(DECAY, x["u"], x["lam"], x["bias"], x["h0"], None, h, st, withhold(8))
    assert st.item() == TIMEOUT and torch.isnan(h).any()
    pr.pararnn_linrec_solve_ex(DECAY, x["u"], x["lam"], x["bias"], x["h0"], None, h, st, None)
    assert st.item() == 0 and torch.equal(h, pr.linrec_solve(DECAY, **x))
    st.fill_(77)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h2 = pr.linrec_solve(DECAY, **x, status=st)
    for _ in range(2):
        st.fill_(77)
        graph.replay()
        assert st.item() == 0 and torch.equal(h2, h)
    with pytest.raises(TypeError):
        pr.linrec_solve(DECAY, **x, status=torch.zeros(1, device="cuda"))
    with pytest.raises(ValueError):
        pr.linrec_solve(DECAY, **x, status=torch.zeros(1, dtype=torch.int32))


# rings of four rows, three, two and one; a norm first, a norm last, neither
NORMS = {"full": (dict(gate=1, post=1, res=1, scale=1, pre=1), (1000, 4096, 8192)),
         "pre": (dict(res=1, pre=1), (520, 4096)), "post": (dict(gate=1, post=1), (1000, 8192)),
         "plain": (dict(gate=1, scale=1), (1000,))}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind,D", [(k, D) for k, (_, Ds) in NORMS.items() for D in Ds])
def test_norm_adjoint_whose_copies_never_come(cuda_ok, kind, D, dtype):
    parts, N = NORMS[kind][0], 4000     # several rows a block, at any width
    gen = torch.Generator().manual_seed(D)
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    row = lambda k: r(N, D).to(dtype).cuda() if parts.get(k) else None  # noqa: E731
    vec = lambda k: (1 + 0.1 * r(D)).cuda() if parts.get(k) else None  # noqa: E731
    p = dict(gate=row("gate"), w_post=vec("post"), res=row("res"), scale=vec("scale"), w_pre=vec("pre"))
    h, ds, dx = r(N, D).cuda(), r(N, D).to(dtype).cuda(), row("pre")
    st = word()
    want = pr.block_norm_adjoint(h, ds, dx, **p, status=st)
    assert st.item() == 0
    for at in (0, 700, 3999):
        got = pr.block_norm_adjoint(h, ds, dx, **p, status=st, opts=withhold(at))
        torch.cuda.synchronize()
        assert st.item() == TIMEOUT
        for k in ("dh", "dgate", "dres"):
            if got[k] is None:
                continue
            lost = torch.isnan(got[k])
            rows = lost.any(-1)
            # whole rows: the one withheld and some that the block had after it
            # (or, where a row's wait is taken a row ahead, the one before it)
            assert rows[at] and torch.equal(rows, lost.all(-1)), k
            assert torch.equal(got[k][~rows], want[k][~rows]), k
            assert int(rows.sum()) < N // 20, k
        for k in ("dw_post", "dscale", "dw_pre"):
            assert got[k] is None or torch.isnan(got[k]).all(), k
        again = pr.block_norm_adjoint(h, ds, dx, **p, status=st)
        assert st.item() == 0
        assert all(again[k] is None or torch.equal(again[k], want[k]) for k in again)


def test_norm_adjoint_status_through_the_plain_binding(cuda_ok):
    N, D = 600, 520
    h, ds, w = torch.randn(N, D, device="cuda"), torch.randn(N, D, device="cuda"), torch.ones(D, device="cuda")
    ws = torch.empty(pr.pararnn_block_norm_workspace_size(N, D), dtype=torch.uint8, device="cuda")
    dh, dw, st = torch.empty_like(h), torch.empty_like(w), word()
    for opts, want in ((None, 0), (withhold(1), TIMEOUT), (None, 0)):
        pr.pararnn_block_norm_adjoint_ex(h, D, None, 0, 0, w, None, 0, None, None, ds, D, None, 0, dh, None,
                                         None, dw, None, None, 1e-6, N, D, st, ws, opts)
        assert st.item() == want and bool(torch.isnan(dh).any()) == (want != 0)
    ref = pr.block_norm_adjoint(h, ds, None, w_post=w)
    assert torch.equal(dh, ref["dh"]) and torch.equal(dw, ref["dw_post"])
