"""The gated linear recurrence's adjoint where its gates saturate."""
import numpy as np
import pytest
import torch

import nonlinear_rnn_paragru_b200 as pr
from oracle import layer as ol

pytestmark = pytest.mark.gpu

GRU, DECAY = pr.PARARNN_LIN_GRU, pr.PARARNN_LIN_DECAY


def within(got, want, err):
    got = got.double().cpu().numpy()
    bad = ~(np.abs(got - want) <= err + 1e-37)      # a NaN is off too
    assert not bad.any(), (float((np.abs(got - want) / (err + 1e-37)).max()), np.argwhere(bad)[:3])


@pytest.mark.parametrize("T", [1, 37, 900])
@pytest.mark.parametrize("sign", [1, -1])
def test_candidates_far_out_have_their_gradient(cuda_ok, sign, T):
    # |y| of 7 to 10.  An fp32 slope 4 t / (1 + t)^2, t = e^2y: three roundings of 2y (20) make 60, ex2, the
    # reciprocal, 1 + t and the products 11 more; z (arguments up to 6: 24) and lambda's factors 5: 100
    # roundings, below 2 x 64
    B, D = 2, 72
    g = torch.Generator().manual_seed(T)
    u = torch.randn((B, T, 2, D), generator=g).clamp_(-5, 5)
    u[:, :, 1] = sign * (7 + 3 * torch.rand((B, T, D), generator=g))
    h0, dLdh = torch.randn((B, D), generator=g), torch.randn((B, T, D), generator=g)
    u, h0, dLdh = u.cuda(), h0.cuda(), dLdh.cuda()
    h = pr.linrec_solve(GRU, u, h0=h0)
    got = pr.linrec_adjoint(GRU, u, None, None, h0, h, dLdh)
    want = ol.lin_adjoint(GRU, u, None, None, h0, h, dLdh, delta=64 * 2.0 ** -24)
    for k in ("du", "dbias", "dh0"):
        within(got[k], *want[k])
    # and nowhere is it rounded away
    assert (got["du"][:, :, 1] != 0).all()


def test_infinite_candidates_have_no_gradient(cuda_ok):
    u = torch.zeros((1, 3, 2, 8), device="cuda")
    u[:, :, 1, :4], u[:, :, 1, 4:] = float("inf"), float("-inf")
    h = pr.linrec_solve(GRU, u)
    got = pr.linrec_adjoint(GRU, u, None, None, None, h, torch.ones_like(h))
    assert (got["du"][:, :, 1] == 0).all() and torch.isfinite(got["du"]).all()


@pytest.mark.parametrize("T", [1, 33, 700])
def test_channels_that_forget_at_once_have_their_gradient(cuda_ok, T):
    # w = -log a up to 8 softplus(3) = 24.4, a down to 2.5e-11.  An fp32 w is off by up to 24 roundings of its
    # sigmoid, 6 of softplus and the products: a by 24.4 x 30 of itself, and the gradient of r by that and
    # the 48 roundings of its other factors: 780
    B, D = 2, 72
    g = torch.Generator().manual_seed(T)
    u = torch.randn((B, T, 3, D), generator=g).clamp_(-5, 5).cuda()
    u[:, :, 0] = u[:, :, 0].abs()
    lam = torch.linspace(-4, 3, D).cuda()
    h0, dLdh = torch.randn((B, D), generator=g).cuda(), torch.randn((B, T, D), generator=g).cuda()
    h = pr.linrec_solve(DECAY, u, lam, h0=h0)
    got = pr.linrec_adjoint(DECAY, u, lam, None, h0, h, dLdh)
    want = ol.lin_adjoint(DECAY, u, lam, None, h0, h, dLdh, delta=780 * 2.0 ** -24)
    for k in ("du", "dlam", "dbias"):
        within(got[k], *want[k])


def test_lam_where_its_softplus_is_denormal(cuda_ok):
    # softplus(-95) is 5.5e-42, some 3900 of fp32's smallest step: expf, log1pf and their quotient are off by
    # 3 steps of 3900, the products with kappa, log2 e, r and ln 2 by less: 2e-3 covers them
    T, D = 40, 72
    g = torch.Generator().manual_seed(1)
    u = torch.zeros((1, T, 3, D))                     # x = 0: the states are h0's, and the first term is 0
    u[:, :, 0] = torch.randn((1, T, D), generator=g).abs().clamp_(0, 5)
    u = u.cuda()
    h0 = 1e10 * (1 + torch.rand((1, D), generator=g)).cuda()
    dLdh = 1e10 * (1 + torch.rand((1, T, D), generator=g)).cuda()
    for x in (-88.0, -92.0, -95.0):
        lam = torch.full((D,), x, device="cuda")
        h = pr.linrec_solve(DECAY, u, lam, h0=h0)
        got = pr.linrec_adjoint(DECAY, u, lam, None, h0, h, dLdh)["dlam"].double().cpu().numpy()
        want = ol.lin_adjoint(DECAY, u, lam, None, h0, h, dLdh)["dlam"][0]
        assert (np.abs(got - want) <= 2e-3 * np.abs(want)).all(), (x, float(got[0]), float(want[0]))
