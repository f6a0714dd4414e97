"""db of sigmoid and silu over many rows.

Tolerance, per column. D = dy act'(p) is off by dD = |dy| ((k + 4) 2^-23 S + 2^-18), S the sizes of p's sum
(tests/test_gpu_linear.py). dy is drawn apart from everything else with a random sign, so these add up like
independent values of mean 0: six times the root of the sum of their squares. The sum itself is kept in fp32:
a column's terms go through at most rows / (148 128) + 3 additions in a tile's and the tiles' sums and 600 in
joining the parts, each off by 2^-23 of a partial sum, which is under six root sums of squares of D. Then one
rounding, 2^-8 of db. For each size here that is a few per cent of db's spread, the root sum of squares of D.
"""
import numpy as np
import pytest
import torch

import pair_representation_b200 as tm
from oracle.linear import linear_backward as oracle_backward
from test_gpu_linear import E, U, dev, draw

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from pair_representation_b200 import build
    build.build()
    tm.lib()


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("held", [False, True])
@pytest.mark.parametrize("rows,k,n", [(19021, 128, 128), (60001, 64, 200), (19021, 128, 392), (60001, 320, 72),
                                      (30001, 160, 520)])
def test_db_over_many_rows(rows, k, n, act, held):
    x, w, b, dy = draw(rows, k, n, 41)
    xt = dev(x)
    if held:
        xt = tm.act8_pack(xt)
        x = tm.act8_unpack(xt).float().cpu().numpy()
    db = tm.linear_backward(xt, dev(w), dev(dy), bias=dev(b), act=act)[2].double().cpu().numpy()
    _, _, rb, D = oracle_backward(x, w, dy, b, act)
    dD = np.abs(dy) * ((k + 4) * E * (np.abs(x) @ np.abs(w).T + np.abs(b)) + 2.0 ** -18)
    spread = np.sqrt((D ** 2).sum(0))
    tol = U * np.abs(rb) + 6 * np.sqrt((dD ** 2).sum(0)) + (rows / (148 * 128) + 603) * E * 6 * spread
    assert (tol - U * np.abs(rb)).max() < 0.05 * spread.min()  # the check says something
    assert (np.abs(db - rb) <= tol).all(), float((np.abs(db - rb) / tol).max())
    assert np.linalg.norm(db - rb) <= U * np.linalg.norm(rb)
