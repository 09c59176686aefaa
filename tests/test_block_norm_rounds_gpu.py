"""Narrow rows (several a block) over more than one round of the blocks: the
adjoint's ring used again, the rows ahead of the forward, a last round in part."""
import pytest
import torch

import nonlinear_rnn_paragru_b200 as pr
from oracle import layer as ol
from test_block_norm_gpu import KINDS, close, draw

pytestmark = pytest.mark.gpu

SMS, THREADS = 148, 256


def rows_a_block(D):
    threads = 1
    while 8 * threads < D:
        threads *= 2
    return THREADS // threads


@pytest.mark.parametrize("kind", ["full", "post_gate", "res_pre", "full_f32", "mixed", "gate_scale_pre"])
@pytest.mark.parametrize("D", [8, 16, 24, 40, 64, 136, 248])
def test_narrow_rows_of_several_rounds(cuda_ok, kind, D):
    slots = rows_a_block(D)
    ahead, back = SMS * 4 * slots, SMS * 2 * slots      # rows of a round, forward and adjoint, at most
    N = 2 * ahead + slots // 2 + 3
    assert N > 2 * ahead and N > 4 * back and N % slots != 0
    p, d, st, xt = draw(N, D, **KINDS[kind], seed=D)
    s, x = pr.block_norm(**p, s_dtype=st, x_dtype=xt)
    want = ol.block_norm(**p)
    close(s, *want["s"], what="s")
    if x is not None:
        close(x, *want["x"], what="x")
    got = pr.block_norm_adjoint(ds=d["ds"], dx=d["dx"], **p)
    want = ol.block_norm_adjoint(ds=d["ds"], dx=d["dx"], **p)
    assert {k for k, v in got.items() if v is not None} == set(want)
    # additions that a value of a sum goes through, at most: the rounds, the block's rows, the blocks 32 deep
    chain = (N // back + 1 + slots + (SMS * 2 + 31) // 32 + 8) * 2.0 ** -24
    for k, (v, m) in want.items():
        close(got[k], v, m, chain if v.ndim == 1 else 0.0, what=k)
