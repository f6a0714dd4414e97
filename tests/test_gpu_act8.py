"""GPU tests of activations kept in 8 bits (trimul_act8_pack / unpack, through the C ABI): codes,
scales and values bit for bit against the oracle's MX quantiser (oracle/mx.py)."""
import numpy as np
import pytest
import torch

import pair_inputs as pi
import pair_representation_b200 as tm
from gpu_helpers import as_bf16
from oracle.mx import mx_quantize_blocks

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from pair_representation_b200 import build
    build.build()
    tm.lib()


def check(x):
    """x: float32 numpy of bf16 values, finite."""
    t = torch.from_numpy(x).to(DEV).to(torch.bfloat16)
    a = tm.act8_pack(t)
    p, e, values = mx_quantize_blocks(x, -1)
    assert torch.equal(a.scales.cpu(), torch.from_numpy((e + 127).astype(np.uint8)))
    codes = a.codes.cpu().view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(codes, p) and np.array_equal(np.signbit(codes), np.signbit(p))
    got = tm.act8_unpack(a)
    # Exact in bf16 but under its smallest normal number, where the nearest is taken.
    want = torch.from_numpy(values).to(torch.bfloat16)
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("rows,channels", [(1, 32), (1, 96), (3, 64), (7, 160), (1001, 96), (31, 1024), (129, 128),
                                           (2048, 512)])
def test_bits(rows, channels):
    rng = np.random.default_rng([rows, channels])
    check(as_bf16(rng.standard_normal((rows, channels)) * np.exp2(rng.integers(-20, 20, size=(rows, 1)))))


def test_every_bf16_pattern_of_a_sign_and_ties():
    """Blocks made of all finite bf16 values, largest and smallest included, in several orders."""
    bits = np.arange(0x7F80, dtype=np.uint16)
    both = np.concatenate([bits, bits | 0x8000])
    x = torch.from_numpy(both.astype(np.int16)).view(torch.bfloat16).float().numpy()
    rng = np.random.default_rng(5)
    check(x.reshape(-1, 32))
    check(rng.permutation(x).reshape(-1, 96))
    mixed = np.sort(np.abs(x))[::-1].reshape(32, -1).T.copy()  # each block spans the whole range
    check(np.ascontiguousarray(mixed))


def test_zero_blocks():
    check(np.zeros((5, 64), np.float32))
    x = np.zeros((2, 64), np.float32)
    x[1, 40] = -3.0
    check(x)


def test_infinities_and_nan_stay_with_their_value():
    rng = np.random.default_rng(6)
    x = as_bf16(rng.standard_normal((40, 64)))
    y = x.copy()
    y[3, 5], y[3, 9], y[7, 40], y[8, :32] = np.inf, -np.inf, np.nan, np.inf
    t = torch.from_numpy(y).to(DEV).to(torch.bfloat16)
    got = tm.act8_unpack(tm.act8_pack(t)).float().cpu().numpy()
    bad = ~np.isfinite(y)
    assert np.isnan(got[bad]).all()
    z = np.where(bad, 0, y).astype(np.float32)
    want = tm.act8_unpack(tm.act8_pack(torch.from_numpy(z).to(DEV).to(torch.bfloat16))).float().cpu().numpy()
    assert np.array_equal(got[~bad], want[~bad])


def test_shapes_streams_and_out():
    x = torch.randn(3, 5, 7, 64, device=DEV).to(torch.bfloat16)
    a = tm.act8_pack(x)
    assert a.codes.shape == x.shape and a.scales.shape == (3, 5, 7, 2)
    ref = tm.act8_unpack(a)
    out = torch.empty_like(x)
    assert tm.act8_unpack(a, out=out) is out and torch.equal(out, ref)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    b = tm.act8_pack(x, stream=side)
    got = tm.act8_unpack(b, stream=side)
    side.synchronize()
    assert torch.equal(got, ref)
    empty = tm.act8_pack(x[:0].contiguous())
    assert tm.act8_unpack(empty).shape == (0, 5, 7, 64)


def test_nothing_behind_the_arrays_is_written():
    x = torch.randn(13, 96, device=DEV).to(torch.bfloat16)
    codes = torch.full((13 * 96 + 64,), 9, dtype=torch.uint8, device=DEV)
    scales = torch.full((13 * 3 + 64,), 9, dtype=torch.uint8, device=DEV)
    tm.trimul_act8_pack(x, 13, 96, codes, scales)
    y = torch.full((13 * 96 + 64,), 7.0, dtype=torch.bfloat16, device=DEV)
    tm.trimul_act8_unpack(codes, scales, 13, 96, y)
    torch.cuda.synchronize()
    assert (codes[13 * 96:] == 9).all() and (scales[39:] == 9).all() and (y[13 * 96:] == 7).all()
    a = tm.act8_pack(x)
    assert torch.equal(codes[:13 * 96].view(13, 96), a.codes) and torch.equal(scales[:39].view(13, 3), a.scales)


def test_triangle_backward_from_the_kept_z():
    """layer.backward(Act8 of z) = layer.backward(the values it stands for), bit for bit in dz."""
    N = 72
    case = pi.random_case(N, 31, bf16=True, affine=True, mask="random")
    sd = {key: torch.from_numpy(case[field]) for field, key, _ in tm.STATE_KEYS if field in case}
    layer = tm.TriangleMultiplicationOutgoing(128, 128).load_state_dict(sd).to(DEV, torch.bfloat16)
    z = torch.from_numpy(case["z"]).to(DEV).to(torch.bfloat16)
    dout = torch.randn(N, N, 128, device=DEV).to(torch.bfloat16)
    mask = torch.from_numpy(case["mask"]).to(DEV)
    a = tm.act8_pack(z)
    dz, grads = layer.backward(a, dout, mask)
    dz2, grads2 = layer.backward(tm.act8_unpack(a), dout, mask)
    assert torch.equal(dz, dz2)
    for f in ("w_a", "w_ag", "w_b", "w_bg", "w_g", "w_o"):
        assert torch.equal(grads[f], grads2[f]), f
    with pytest.raises(ValueError):
        layer.backward(a, dout, mask, reuse_forward=True)
