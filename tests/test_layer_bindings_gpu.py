"""The layer operators through the bindings that carry the C names: what they
return equals the wrappers' results, and what they refuse."""
import pytest
import torch

import nonlinear_rnn_paragru_b200 as pr

pytestmark = pytest.mark.gpu

DECAY = pr.PARARNN_LIN_DECAY


@pytest.fixture
def x():
    g = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(s, generator=g).cuda()  # noqa: E731
    B, T, D = 2, 150, 72
    return dict(u=r(B, T, 3, D).bfloat16(), lam=r(D) - 4, bias=r(3, D), h0=r(B, D), g=r(B, T, D),
                reset=(torch.rand((B, T), generator=g) < 0.05).cuda())


def test_linrec_bindings_equal_the_wrappers(cuda_ok, x):
    B, T, G, D = x["u"].shape
    for reset in (None, x["reset"], x["reset"].to(torch.uint8)):
        h = torch.empty((B, T, D), device="cuda")
        pr.pararnn_linrec_solve(DECAY, x["u"], x["lam"], x["bias"], x["h0"], reset, h)
        want = pr.linrec_solve(DECAY, x["u"], x["lam"], x["bias"], x["h0"], reset=reset)
        assert torch.equal(h, want)
        out = dict(du=torch.empty_like(x["u"]), dlam=torch.empty_like(x["lam"]),
                   dbias=torch.empty_like(x["bias"]), dh0=torch.empty_like(x["h0"]))
        ws = torch.empty(pr.pararnn_linrec_workspace_size(DECAY, B, T, D), dtype=torch.uint8, device="cuda")
        want = pr.linrec_adjoint(DECAY, x["u"], x["lam"], x["bias"], x["h0"], h, x["g"], reset=reset)
        pr.pararnn_linrec_adjoint(DECAY, x["u"], x["lam"], x["bias"], x["h0"], reset, h, x["g"],
                                  *out.values(), ws)
        assert all(torch.equal(out[k], want[k]) for k in want)
        given = {k: torch.full_like(v, 7.0) for k, v in out.items()}
        got = pr.linrec_adjoint(DECAY, x["u"], x["lam"], x["bias"], x["h0"], h, x["g"], reset=reset, out=given)
        assert all(got[k] is given[k] and torch.equal(got[k], want[k]) for k in want)
    nxt = torch.empty_like(x["h0"])
    pr.pararnn_linrec_step(DECAY, x["u"][:, 3], x["lam"], x["bias"], x["h0"], nxt)
    assert torch.equal(nxt, pr.linrec_step(DECAY, x["u"][:, 3], x["lam"], x["bias"], x["h0"]))


@pytest.mark.parametrize("dtype", [torch.int64, torch.int32, torch.float32, torch.bfloat16])
def test_linrec_bindings_take_masks_of_bytes_only(cuda_ok, x, dtype):
    B, T, G, D = x["u"].shape
    h, reset = torch.empty((B, T, D), device="cuda"), x["reset"].to(dtype)
    du, ws = torch.empty_like(x["u"]), torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    with pytest.raises(TypeError):
        pr.pararnn_linrec_solve(DECAY, x["u"], x["lam"], None, None, reset, h)
    with pytest.raises(TypeError):
        pr.pararnn_linrec_solve_ex(DECAY, x["u"], x["lam"], None, None, reset, h, None, None)
    with pytest.raises(TypeError):
        pr.pararnn_linrec_adjoint(DECAY, x["u"], x["lam"], None, None, reset, h, h, du, None, None, None, ws)
    with pytest.raises(TypeError):
        pr.pararnn_linrec_adjoint_ex(DECAY, x["u"], x["lam"], None, None, reset, h, h, du, None, None, None,
                                     None, ws, None)


def test_block_norm_bindings_equal_the_wrappers(cuda_ok, x):
    N, D = 300, 72
    h, res, w, ds = x["g"].view(N, D), x["u"].view(N * 3, D)[:N], x["lam"], x["u"].view(N * 3, D)[N:2 * N]
    s, y = torch.empty_like(res), torch.empty_like(res)
    pr.pararnn_block_norm(h, D, res, D, 1, w, res, D, None, w, s, y, 1e-6, N, D)
    parts = dict(gate=res, act="sigmoid", w_post=w, res=res, w_pre=w)
    want = pr.block_norm(h, **parts)
    assert torch.equal(s, want[0]) and torch.equal(y, want[1])
    want = pr.block_norm_adjoint(h, ds, ds, **parts)
    out = {k: torch.empty_like(v) for k, v in want.items() if v is not None}
    ws = torch.empty(pr.pararnn_block_norm_workspace_size(N, D), dtype=torch.uint8, device="cuda")
    pr.pararnn_block_norm_adjoint(h, D, res, D, 1, w, res, D, None, w, ds, D, ds, D, out["dh"], out["dgate"],
                                  out["dres"], out["dw_post"], None, out["dw_pre"], 1e-6, N, D, ws)
    assert all(torch.equal(out[k], want[k]) for k in out)
