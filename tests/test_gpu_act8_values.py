"""Activations in 8 bits that the caller made: what every code and scale byte stands for (E4M3 times E8M0 of OCP
Microscaling: 2^(s - 127), and NaN where s is 255), alone and in the backward that takes them."""
import numpy as np
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


def same(a, b):
    return torch.equal(a.isnan(), b.isnan()) and torch.equal(a.nan_to_num(0, 1e38, -1e38), b.nan_to_num(0, 1e38, -1e38))


def test_every_code_with_every_scale():
    c = np.arange(256)
    e, m = c >> 3 & 15, c & 7
    size = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    value = np.where(c & 127 == 127, np.nan, np.where(c > 127, -size, size))
    scale = np.where(c == 255, np.nan, 2.0 ** (c - 127.0))
    # At most 4 bits, at least 2^-136: exact in fp32, so one rounding to bf16.
    want = torch.from_numpy(scale[:, None] * value[None]).to(torch.bfloat16)
    codes = torch.arange(256, dtype=torch.uint8, device=DEV).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.uint8, device=DEV)[:, None].repeat(1, 8).contiguous()
    assert same(tm.act8_unpack(tm.Act8(codes, scales)).cpu(), want)


@pytest.mark.parametrize("act", ["none", "relu", "sigmoid"])
@pytest.mark.parametrize("k,n", [(64, 72), (128, 136), (96, 264), (160, 72)])
def test_a_scale_of_255_in_the_backward(k, n, act):
    """The gradients at the values that act8_unpack gives, bit for bit."""
    gen = torch.Generator(device=DEV).manual_seed(k)
    rnd = lambda *s: torch.randn(*s, generator=gen, device=DEV).to(torch.bfloat16)  # noqa: E731
    a, w, dy = tm.act8_pack(rnd(300, k)), rnd(n, k), rnd(300, n)
    a.scales[7, k // 32 - 1] = 255
    a.codes[7, k - 32:] = 56  # 1: no NaN among the codes
    x = tm.act8_unpack(a)
    assert x[7, k - 32:].isnan().all() and x.isnan().sum() == 32
    for g, r in zip(tm.linear_backward(a, w, dy, act=act), tm.linear_backward(x, w, dy, act=act)):
        assert same(g, r)
