"""What the layers' calls refuse before any work is enqueued, and the sizes they ask for (no GPU needed)."""
import pytest
import torch

import pair_representation_b200 as tm
from pair_representation_b200 import build as tmbuild

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    tmbuild.build()


def _attention_arguments():
    """Right shapes, one wrong at a time: a kernel takes each tensor's size from q's."""
    q = torch.zeros(2, 70, 3, 32, dtype=BF16)
    bias, mask = torch.zeros(2, 3, 3, 32, 128, dtype=BF16), torch.ones(2, 70, dtype=BF16)
    yield q, bias[:1], mask, None
    yield q, bias[:, :2], mask, None
    yield q, bias[:, :, :2], mask, None
    yield q, bias[..., :96], mask, None
    yield q, bias.reshape(-1), mask, None
    yield q, bias, mask[:, :32], None
    yield q, bias, mask[:1], None
    yield q, bias, mask.reshape(-1), None
    yield q, None, mask[:, :69], None
    yield q, bias, mask, torch.zeros(2, 70, 3, 16, dtype=BF16)
    yield q, bias, mask, torch.zeros(1, 70, 3, 32, dtype=BF16)
    yield q, bias, mask, torch.zeros(2, 70, 3, 32)


@pytest.mark.parametrize("case", range(12))
def test_attention_refuses_other_shapes(case):
    q, bias, mask, out = list(_attention_arguments())[case]
    with pytest.raises(ValueError) as e:
        tm.atom_attention(q, q, q, bias, mask, out=out)
    assert "CUDA device" not in str(e.value)  # found before the tensors' place


def test_attention_refuses_tensors_of_the_host():
    q = torch.zeros(1, 40, 2, 32, dtype=BF16)
    with pytest.raises(ValueError, match="CUDA device"):
        tm.atom_attention(q, q, q)


@pytest.mark.parametrize("case", range(5))
def test_the_layer_refuses_a_bias_or_mask_of_another_shape(case, monkeypatch):
    """The layer's calls give the core their bias and mask as they came: with the projections taken out, on the CPU."""
    _, bias, mask, _ = list(_attention_arguments())[(0, 1, 3, 5, 6)[case]]
    layer = tm.AtomAttention(64, 3)
    monkeypatch.setattr(layer, "_linear", lambda name, x, residual=None: torch.zeros(2, 70, 96, dtype=BF16))
    x = torch.zeros(2, 70, 64, dtype=BF16)
    for call in (lambda: layer(x, bias, mask), lambda: layer.backward(x, x, bias, mask)):
        with pytest.raises(ValueError, match="must be"):
            call()


BASE = 1 << 32  # fake device addresses: never dereferenced by host checks
X, Y, W, B, WS, DY, DX, DW, DB, ST = (BASE + (i << 28) for i in range(1, 11))


def test_a_status_word_of_the_callers():
    """Aligned and apart from the tensors; a call that needs no scratch then needs no workspace."""
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    E = tm.ERR
    passed = [E["TRIMUL_ERR_CUDA"], E["TRIMUL_ERR_UNSUPPORTED"]]  # what a valid call returns where there is no GPU

    def calls(rows, status, ws=None, size=0):
        p = tm.LinearParams(rows, 128, 64, 3, W, B, ws, size, 0, status)
        a = tm.AtomAttnParams(2, 100, 4, 32, X, Y, W, B, None, ws, size, 0, status)
        yield tm.trimul_linear_forward(X, None, p, DX, stream=0, check=False)
        yield tm.trimul_linear_backward(X, None, DY, p, DX, DW, DB, stream=0, check=False)
        yield tm.atomattn_forward(a, DX, stream=0, check=False)
        yield tm.atomattn_backward(a, DY, tm.AtomAttnGrads(DX, DW, DB, None), stream=0, check=False)

    assert all(rc in passed for rc in calls(100, ST))
    assert list(calls(100, None)) == [E["TRIMUL_ERR_WORKSPACE"]] * 4
    assert list(calls(100, ST + 8)) == [E["TRIMUL_ERR_MISALIGNED"]] * 4
    assert list(calls(100, DX + 16)) == [E["TRIMUL_ERR_ALIAS"]] * 4
    assert list(calls(100, X + 16)) == [E["TRIMUL_ERR_ALIAS"]] * 4
    rcs = list(calls(100000, ST))
    assert rcs[1] == E["TRIMUL_ERR_WORKSPACE"] and all(rc in passed for rc in rcs[:1] + rcs[2:])
    need = tm.trimul_linear_backward_workspace_size(100000, 128, 64, 3)
    assert all(rc in passed for rc in calls(100000, ST, WS, need))
    assert list(calls(100000, WS + 512, WS, need))[1] == E["TRIMUL_ERR_ALIAS"]
    assert tm.lib().trimul_status_word(None) == E["TRIMUL_ERR_INVALID_ARG"]
    assert tm.lib().trimul_status_take(None, None, None) == E["TRIMUL_ERR_INVALID_ARG"]
    assert tm.lib().trimul_status_take(ST + 4, None, None) == E["TRIMUL_ERR_MISALIGNED"]


@pytest.mark.parametrize("k,n,act", [(8, 8, 0), (8, 8, 3), (128, 512, 1), (1280, 1280, 0), (160, 1280, 3), (4096, 4096, 0)])
@pytest.mark.parametrize("rows", [65537, 1 << 20, 10000000, 1 << 30])
def test_no_sum_over_more_rows_than_a_part(k, n, act, rows):
    """dW of each part of at most 65536 rows has its place in the workspace, beside what the call needs anyhow."""
    parts = -(-rows // 65536)
    d = rows * n * 2 if act and (k > 128 or n > 512) else 0  # D, where it is a product of its own
    assert tm.trimul_linear_backward_workspace_size(rows, k, n, act) >= 256 + d + parts * n * (k + 1) * 4


class _Stream:
    """What the calls look at of a torch stream."""

    def __init__(self, index):
        self.device, self.cuda_stream = torch.device("cuda", index), 0


def test_a_stream_of_another_device_is_refused(monkeypatch):
    """Work on device 0's tensors has nothing to do on device 1's streams: the call had run on another stream than
    the one it was given."""
    monkeypatch.setattr(torch.cuda, "device", lambda index: pytest.fail("a device was entered"))
    ran = []
    with pytest.raises(ValueError, match="stream"):
        tm._run_on(0, _Stream(1), (), lambda: ran.append(1))
    assert not ran


def test_the_triangle_layer_refuses_a_mask_or_out_of_another_size():
    """The kernels take both sizes from z."""
    layer = tm.TriangleMultiplicationOutgoing(128, 128)
    layer.tensors, layer.dtype, layer.device = {}, BF16, torch.device("cpu")
    z = torch.zeros(6, 6, 128, dtype=BF16)
    for mask in (torch.ones(5, 6), torch.ones(6), torch.ones(0, 6)):
        for call in (lambda: layer(z, mask), lambda: layer.backward(z, z, mask)):
            with pytest.raises(ValueError, match="mask"):
                call()
    for out in (z[:5], z.float(), z.transpose(0, 1)):
        with pytest.raises(ValueError, match="out"):
            layer(z, None, out=out)
