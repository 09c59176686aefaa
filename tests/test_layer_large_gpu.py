"""The layer operators on tensors whose offsets pass 2^31 elements (and 2^32
bytes), in windows at those places and at the end, and with broadcast rows."""
import gc

import numpy as np
import pytest
import torch

import nonlinear_rnn_paragru_b200 as pr
from oracle import layer as ol
from test_block_norm_gpu import FULL, close, draw

pytestmark = pytest.mark.gpu

GRU = pr.PARARNN_LIN_GRU
HALF = 2.0 ** -8        # half a step of bf16, relatively


@pytest.fixture
def room(cuda_ok):
    gc.collect()
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    yield
    gc.collect()
    torch.cuda.empty_cache()


def within(got, want, err, rounded):
    got = got.double().cpu().numpy()
    tol = err + 1e-37 + (HALF * (np.abs(want) + err) if rounded else 0)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (float((np.abs(got - want) / tol).max()), np.argwhere(bad)[:3])


def test_a_sequence_of_a_million_steps(room):
    T, D = 1050000, 2048            # h passes 2^31 elements at step 1048576, u 2^31 at 349525 and 2^32 at 699050
    gen = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s: torch.randn(s, generator=gen, device="cuda")  # noqa: E731
    wide = torch.randn((1, T, 3 * D), generator=gen, device="cuda", dtype=torch.bfloat16).clamp_(-5, 5)
    u = wide[..., :2 * D].unflatten(-1, (2, D))
    bias, h0, g = (0.1 * r(2, D)).clamp_(-1, 1), r(1, D), r(1, T, D)
    h = pr.linrec_solve(GRU, u, None, bias, h0)
    out = pr.linrec_adjoint(GRU, u, None, bias, h0, h, g, want_params=False)
    for t0 in (0, 349500, 699020, 1048540, T - 264):
        # 264 steps, of which the later 200 decide what reaches the first 64 from behind: products of 200
        # factors 1 - z are far below a rounding
        at = slice(t0, t0 + 264)
        before = h0 if t0 == 0 else h[:, t0 - 1]
        H, E = ol.lin_seq(GRU, u[:, at], None, bias, before)
        within(h[:, at], H, E, False)
        want = ol.lin_adjoint(GRU, u[:, at], None, bias, before, h[:, at], g[:, at])["du"]
        n = 264 if t0 + 264 == T else 64
        within(out["du"][:, t0:t0 + n], want[0][:, :n], want[1][:, :n], True)
        if t0 == 0:
            want = ol.lin_adjoint(GRU, u[:, at], None, bias, before, h[:, at], g[:, at])["dh0"]
            within(out["dh0"], *want, False)


@pytest.mark.parametrize("N,D", [(300000, 8192), (30000000, 72)])
def test_rows_beyond_2_31_elements(room, N, D):
    gen = torch.Generator(device="cuda").manual_seed(2)
    rows = lambda: torch.randn((N, D), generator=gen, device="cuda", dtype=torch.bfloat16).clamp_(-7, 7)  # noqa: E731
    h, ds = rows(), rows()
    gate = rows() if D > 256 else None
    w = 1 + 0.1 * torch.randn(D, generator=gen, device="cuda")
    s, _ = pr.block_norm(h, gate=gate, w_post=w)
    got = pr.block_norm_adjoint(h, ds, None, gate=gate, w_post=w)
    edge = (1 << 31) // D
    for at in (slice(0, 40), slice(edge - 20, edge + 20), slice(N - 40, N)):
        p = dict(h=h[at], gate=None if gate is None else gate[at], w_post=w)
        close(s[at], *ol.block_norm(**p)["s"], what="s")
        want = ol.block_norm_adjoint(ds=ds[at], dx=None, **p)
        for k in ("dh", "dgate"):
            assert (k in want) == (got[k] is not None)
            if k in want:
                close(got[k][at], *want[k], what=k)


@pytest.mark.parametrize("N,D", [(9, 72), (700, 520)])
def test_gradients_with_broadcast_rows(cuda_ok, N, D):
    # one row (stride 0) for all of each input in turn: every row's gradient is its own
    p, d, st, xt = draw(N, D, **FULL)
    for name in ("h", "gate", "res", "ds", "dx"):
        q, e = dict(p), dict(d)
        where = q if name in q else e
        where[name] = where[name][:1].expand(N, D)
        got = pr.block_norm_adjoint(**e, **q)
        for k, (v, m) in ol.block_norm_adjoint(**e, **q).items():
            assert got[k].shape == v.shape and got[k].is_contiguous()
            close(got[k], v, m, N * 2.0 ** -24 if v.ndim == 1 else 0.0, what=(name, k))
