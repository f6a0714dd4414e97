"""Sums over more rows than one accumulator takes. All values are whole numbers small enough that every sum
is exact in fp32 (under 2^24): one rounding, no tolerance."""
import pytest
import torch

import pair_representation_b200 as tm

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from pair_representation_b200 import build
    build.build()
    tm.lib()


def check(rows, k, n, act, held=False):
    gen = torch.Generator(device=DEV).manual_seed(rows + n)
    whole = lambda *s: torch.randint(-1, 2, s, generator=gen, device=DEV, dtype=torch.int8).to(torch.bfloat16)  # noqa: E731
    x, w, dy = whole(rows, k), whole(n, k), whole(rows, n)
    b = torch.full((n,), 0.5, device=DEV, dtype=torch.bfloat16)  # no relu in doubt
    ws = torch.zeros(tm.trimul_linear_backward_workspace_size(rows, k, n, tm.ACTS[act], held), dtype=torch.uint8, device=DEV)
    dx, dw, db = tm.linear_backward(tm.act8_pack(x) if held else x, w, dy, b, act, workspace=ws)
    assert tm.device_status(ws)[0] == 0
    rw, rb = torch.zeros(n, k, dtype=torch.float64, device=DEV), torch.zeros(n, dtype=torch.float64, device=DEV)
    for i in range(0, rows, 1 << 20):
        xs, D = x[i:i + (1 << 20)].double(), dy[i:i + (1 << 20)].double()
        if act == "relu":
            D = D * (xs @ w.double().T + 0.5 > 0)
        assert torch.equal(dx[i:i + (1 << 20)], (D @ w.double()).to(torch.bfloat16))
        rw += D.T @ xs
        rb += D.sum(0)
    assert torch.equal(dw, rw.to(torch.bfloat16)) and torch.equal(db, rb.to(torch.bfloat16))


@pytest.mark.parametrize("rows,k,n,act,held", [
    (148 * 512 * 128 + 1000, 8, 8, "relu", False), (148 * 512 * 128 + 77, 8, 8, "none", False),
    (148 * 512 * 128 + 77, 32, 8, "relu", True), (74 * 512 * 128 + 77, 8, 264, "relu", False),
    (65536 + 100, 1280, 1280, "none", False), (65536 + 64, 1280, 1288, "relu", False), (140000, 160, 1280, "none", False)])
def test_more_rows_than_one_accumulator(rows, k, n, act, held):
    check(rows, k, n, act, held)
