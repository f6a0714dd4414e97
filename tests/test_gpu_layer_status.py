"""The status word of calls that are given no workspace: kept by the library, one for each device, holding the
first failure until it is asked for. A failure is planted from the host (its code written into the word), as
a wait that ran out would have left it."""
import ctypes
import subprocess
import sys

import pytest
import torch

import pair_representation_b200 as tm

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda", 0)
TIMEOUT = tm.ERR["TRIMUL_ERR_TIMEOUT"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from pair_representation_b200 import build
    build.build()
    tm.lib()


class _Raw:
    """16 bytes of device memory at an address, as torch takes foreign memory."""

    def __init__(self, at):
        self.__cuda_array_interface__ = dict(shape=(4,), typestr="<i4", data=(at, False), version=3)


def word():
    return torch.as_tensor(_Raw(tm.trimul_status_word()), device=DEV)


def rnd(*s):
    return torch.randn(*s, device=DEV).to(torch.bfloat16)


def calls():
    """Each call without a workspace, with scratch of its own and without."""
    x, w, dy = rnd(20000, 64), rnd(72, 64), rnd(20000, 72)
    v, u, dv = rnd(20000, 160), rnd(72, 160), rnd(20000, 72)
    q, bias = rnd(1, 333, 2, 32), rnd(1, 11, 2, 32, 128)
    layer = tm.AtomAttention(64, 2).load_state_dict(
        {f"linear_{n}.weight": torch.randn(64, 64) / 8 for n in "qkvo"}).to(DEV)
    a, da = rnd(1, 333, 64), rnd(1, 333, 64)
    return dict(
        linear=lambda: tm.linear(x, w, act="silu"),
        one_team=lambda: tm.linear_backward(x[:100], w, dy[:100]),
        one_pass=lambda: tm.linear_backward(x, w, dy, act="silu"),
        held=lambda: tm.linear_backward(tm.act8_pack(x), w, dy, act="silu"),
        products=lambda: tm.linear_backward(v, u, dv, act="silu"),
        products_held=lambda: tm.linear_backward(tm.act8_pack(v), u, dv),
        dx_alone=lambda: tm.linear_backward(tm.act8_pack(v), u, dv, need_dw=False, need_db=False),
        nothing=lambda: tm.linear_backward(v, u, dv, need_dx=False, need_dw=False, need_db=False),
        attention=lambda: tm.atom_attention_backward(q, q, q, q, bias),
        layer=lambda: layer(a),
        layer_backward=lambda: layer.backward(a, da))


def test_a_failure_outlives_the_calls_after_it():
    assert tm.device_status(DEV)[0] in (0, TIMEOUT)  # whatever was there: taken
    assert tm.device_status(DEV) == (0, [0, 0, 0, 0])
    for name, call in calls().items():
        word().copy_(torch.tensor([1, 0x52, 7, 3], dtype=torch.int32))
        call()
        assert tm.device_status(DEV) == (TIMEOUT, [1, 0x52, 7, 3]), name
        assert tm.device_status(DEV) == (0, [0, 0, 0, 0]), name
        call()
        assert tm.device_status(DEV)[0] == 0, name


def test_a_workspace_has_its_own():
    """Cleared by each call that is given it; the device's word is not that call's."""
    x, w, dy = rnd(700, 64), rnd(72, 64), rnd(700, 72)
    ws = torch.zeros(tm.trimul_linear_backward_workspace_size(700, 64, 72, 3), dtype=torch.uint8, device=DEV)
    fail = torch.tensor([1, 0x52, 7, 3], dtype=torch.int32)
    q = rnd(1, 100, 2, 32)
    for call in (lambda: tm.linear(x, w, act="silu", workspace=ws),
                 lambda: tm.linear_backward(x, w, dy, act="silu", workspace=ws),
                 lambda: tm.atom_attention_backward(q, q, q, q, workspace=ws)):
        ws[:16].view(torch.int32).copy_(fail)
        assert tm.device_status(ws)[0] == TIMEOUT
        call()
        assert tm.device_status(ws)[0] == 0
    assert tm.device_status(DEV)[0] == 0


def test_a_word_of_the_callers():
    """params.status: kept by every call, also where the workspace is there."""
    x, w, dy = rnd(700, 160), rnd(72, 160), rnd(700, 72)
    dx, dw, y = torch.empty_like(x), torch.empty_like(w), torch.empty_like(dy)
    need = tm.trimul_linear_backward_workspace_size(700, 160, 72, 3)
    ws = torch.full((need,), 9, dtype=torch.uint8, device=DEV)
    st = torch.tensor([1, 0x52, 7, 3], dtype=torch.int32, device=DEV)
    p = tm.LinearParams(700, 160, 72, 3, w.data_ptr(), None, ws.data_ptr(), need, 0, st.data_ptr())
    q = rnd(1, 100, 2, 32)
    out, grads = torch.empty_like(q), [torch.empty_like(q) for _ in range(3)]
    a = tm.AtomAttnParams(1, 100, 2, 32, q.data_ptr(), q.data_ptr(), q.data_ptr(), None, None, None, 0, 0, st.data_ptr())
    for call in (lambda: tm.trimul_linear_forward(x, None, p, y), lambda: tm.trimul_linear_backward(x, None, dy, p, dx, dw, None),
                 lambda: tm.atomattn_forward(a, out),
                 lambda: tm.atomattn_backward(a, q, tm.AtomAttnGrads(*(g.data_ptr() for g in grads), None))):
        call()
        assert st.tolist() == [1, 0x52, 7, 3]
        assert tm.trimul_linear_device_status(p) == (TIMEOUT, [1, 0x52, 7, 3])
    assert tm.atomattn_device_status(a) == (TIMEOUT, [1, 0x52, 7, 3])
    assert (ws[:256] == 9).all()  # the word is elsewhere
    st.zero_()
    assert tm.trimul_linear_device_status(p)[0] == 0


FIRST = """
import torch, pair_representation_b200 as tm
d = torch.device("cuda", 0)
x, w = torch.ones(300, 64, device=d, dtype=torch.bfloat16), torch.ones(72, 64, device=d, dtype=torch.bfloat16)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    y = tm.linear(x, w)
    dx, dw, db = tm.linear_backward(x, w, y)
g.replay()
torch.cuda.synchronize()
assert (y == 64).all() and (dx == 64 * 72).all()
assert tm.device_status(d) == (0, [0, 0, 0, 0])
class Raw:
    __cuda_array_interface__ = dict(shape=(4,), typestr="<i4", data=(tm.trimul_status_word(), False), version=3)
word = torch.as_tensor(Raw(), device=d)
word.copy_(torch.tensor([1, 2, 3, 4], dtype=torch.int32))
g.replay()
assert tm.device_status(d) == (tm.ERR["TRIMUL_ERR_TIMEOUT"], [1, 2, 3, 4])
"""


def test_a_process_whose_first_call_is_captured():
    """The replays' failures are the device's too."""
    done = subprocess.run([sys.executable, "-c", FIRST], capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


def test_take_needs_a_word():
    assert tm.lib().trimul_status_take(None, None, None) == tm.ERR["TRIMUL_ERR_INVALID_ARG"]
    host = (ctypes.c_int * 4)()
    assert tm.lib().trimul_status_take(ctypes.addressof(host), None, None) == tm.ERR["TRIMUL_ERR_INVALID_ARG"]
