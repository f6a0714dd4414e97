"""Host-side checks of the linear layer's, the 8-bit activations' and atom attention's backward entry
points: sizes and refusals, before any CUDA call (no GPU needed)."""
import ctypes

import pytest

import pair_representation_b200 as tm
from pair_representation_b200 import build as tmbuild

E = tm.ERR
BASE = 1 << 32  # fake device addresses: never dereferenced by host checks
X, Y, R, W, B, WS = (BASE + (i << 28) for i in range(1, 7))
DX, DW, DB, DY, CODES, SCALES = (BASE + (i << 28) for i in range(7, 13))
PASSED = ("TRIMUL_ERR_CUDA", "TRIMUL_ERR_UNSUPPORTED")  # what a valid call returns where there is no GPU


@pytest.fixture(scope="module")
def L():
    tmbuild.build()
    return tm.lib()


@pytest.fixture(scope="module")
def no_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")


def _p(rows=100, k=128, n=64, act=0, **kw):
    p = tm.LinearParams(rows, k, n, act, W, B, WS, 1 << 27, 0)
    for f, v in kw.items():
        setattr(p, f, v)
    return p


def _fwd(p, x=X, r=R, y=Y):
    return tm.trimul_linear_forward(x, r, p, y, stream=0, check=False)


def _bwd(p, x=X, x8=None, dy=DY, dx=DX, dw=DW, db=DB):
    return tm.trimul_linear_backward(x, x8, dy, p, dx, dw, db, stream=0, check=False)


def test_linear_sizes(L):
    assert tm.trimul_linear_workspace_size() == 256
    for act in range(4):
        for rows in (1, 63, 64, 65, 5000):
            a = tm.trimul_linear_backward_workspace_size(rows, 128, 64, act)
            assert a >= 256  # the status word, and nothing else where one team of CTAs does it all
            assert tm.trimul_linear_backward_workspace_size(rows, 128, 64, act, True) >= a
    for bad in ((0, 128, 64, 0), (-1, 128, 64, 0), (1 << 31, 128, 64, 0), (10, 0, 64, 0), (10, 12, 64, 0),
                (10, 128, 20, 0), (10, 128, 64, 4), (10, 128, 64, -1), (10, 16392, 64, 0)):
        assert tm.trimul_linear_backward_workspace_size(*bad) == 0, bad
    assert tm.trimul_linear_backward_workspace_size(10, 40, 64, 0, True) == 0


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_linear_argument_checks(L, call):
    for kw, code in ((dict(rows=0), "INVALID_ARG"), (dict(rows=(1 << 30) + 1), "INVALID_ARG"),
                     (dict(in_features=0), "INVALID_ARG"), (dict(out_features=16392), "INVALID_ARG"),
                     (dict(in_features=129), "UNSUPPORTED"), (dict(out_features=4), "UNSUPPORTED"),
                     (dict(act=4), "INVALID_ARG"), (dict(act=-1), "INVALID_ARG"), (dict(weight=None), "INVALID_ARG"),
                     (dict(weight=W + 8), "MISALIGNED"), (dict(bias=B + 1), "MISALIGNED"),
                     (dict(workspace=None), "WORKSPACE"), (dict(workspace_bytes=255), "WORKSPACE"),
                     (dict(workspace=WS + 16), "MISALIGNED")):
        assert call(_p(**kw)) == E["TRIMUL_ERR_" + code], kw
    assert call(_p(), x=None) == E["TRIMUL_ERR_INVALID_ARG"]
    assert call(_p(), x=X + 2) == E["TRIMUL_ERR_MISALIGNED"]


def test_linear_forward_checks(L, no_gpu):
    assert tm.lib().trimul_linear_forward(X, None, None, Y, None) == E["TRIMUL_ERR_INVALID_ARG"]
    assert _fwd(_p(), y=None) == E["TRIMUL_ERR_INVALID_ARG"]
    for kw in (dict(r=R + 8), dict(y=Y + 4)):
        assert _fwd(_p(), **kw) == E["TRIMUL_ERR_MISALIGNED"]
    yb = 100 * 64 * 2
    for y in (X, W, B, WS, R + 16, R + yb - 16, X + 100 * 128 * 2 - 16):
        assert _fwd(_p(), y=y) == E["TRIMUL_ERR_ALIAS"], hex(y)
    assert _fwd(_p(workspace=X)) == E["TRIMUL_ERR_ALIAS"]
    passed = [E[c] for c in PASSED]
    assert _fwd(_p()) in passed and _fwd(_p(), y=R) in passed and _fwd(_p(bias=None), r=None) in passed


def test_linear_backward_checks(L, no_gpu):
    x8 = tm.Act8Ptrs(CODES, SCALES)
    assert tm.lib().trimul_linear_backward(X, None, DY, None, DX, DW, DB, None) == E["TRIMUL_ERR_INVALID_ARG"]
    assert _bwd(_p(), x8=x8) == E["TRIMUL_ERR_INVALID_ARG"]          # both forms of x
    assert _bwd(_p(), dy=None) == E["TRIMUL_ERR_INVALID_ARG"]
    assert _bwd(_p(), x=None, x8=tm.Act8Ptrs(CODES, None)) == E["TRIMUL_ERR_INVALID_ARG"]
    assert _bwd(_p(in_features=40), x=None, x8=x8) == E["TRIMUL_ERR_UNSUPPORTED"]
    for kw in (dict(dy=DY + 8), dict(dx=DX + 8), dict(dw=DW + 2), dict(db=DB + 1)):
        assert _bwd(_p(), **kw) == E["TRIMUL_ERR_MISALIGNED"], kw
    assert _bwd(_p(), x=None, x8=tm.Act8Ptrs(CODES + 8, SCALES)) == E["TRIMUL_ERR_MISALIGNED"]
    for kw in (dict(dx=X), dict(dx=DY), dict(dw=W), dict(dw=DX), dict(db=DW), dict(db=WS + 64), dict(dx=WS + 4096),
               dict(dy=WS)):
        assert _bwd(_p(), **kw) == E["TRIMUL_ERR_ALIAS"], kw
    for act, from8 in ((0, False), (3, False), (0, True), (3, True)):
        need = tm.trimul_linear_backward_workspace_size(100, 128, 64, act, from8)
        kw = dict(x=None, x8=x8) if from8 else {}
        assert _bwd(_p(act=act, workspace_bytes=need - 1), **kw) == E["TRIMUL_ERR_WORKSPACE"]
        passed = [E[c] for c in PASSED]
        assert _bwd(_p(act=act, workspace_bytes=need), **kw) in passed
        assert _bwd(_p(act=act, workspace_bytes=need), dx=None, dw=None, db=None, **kw) in passed


def test_act8_checks(L, no_gpu):
    pack = lambda x=X, rows=10, c=64, codes=CODES, scales=SCALES: tm.trimul_act8_pack(  # noqa: E731
        x, rows, c, codes, scales, stream=0, check=False)
    unpack = lambda x=X, rows=10, c=64, codes=CODES, scales=SCALES: tm.trimul_act8_unpack(  # noqa: E731
        codes, scales, rows, c, x, stream=0, check=False)
    for f in (pack, unpack):
        assert f(x=None) == f(codes=None) == f(scales=None) == f(rows=0) == f(c=0) == E["TRIMUL_ERR_INVALID_ARG"]
        assert f(c=48) == E["TRIMUL_ERR_UNSUPPORTED"]
        assert f(x=X + 8) == f(codes=CODES + 8) == f(scales=SCALES + 1) == E["TRIMUL_ERR_MISALIGNED"]
        assert f(codes=X + 640) == f(scales=X) == f(scales=CODES + 624) == E["TRIMUL_ERR_ALIAS"]
        assert f() in [E[c] for c in PASSED]


def _attn():
    p = tm.AtomAttnParams(2, 100, 4, 32, X, Y, R, W, B, WS, 256, 0)
    return p, tm.AtomAttnGrads(DX, DW, DB, CODES)


def _abwd(p, g, dout=DY):
    return tm.atomattn_backward(p, dout, g, stream=0, check=False)


def test_attention_backward_checks(L, no_gpu):
    p, g = _attn()
    assert tm.lib().atomattn_backward(None, DY, ctypes.byref(g), None) == E["TRIMUL_ERR_INVALID_ARG"]
    assert tm.lib().atomattn_backward(ctypes.byref(p), DY, None, None) == E["TRIMUL_ERR_INVALID_ARG"]
    assert _abwd(p, g, dout=None) == E["TRIMUL_ERR_INVALID_ARG"]
    for f in ("dq", "dk", "dv"):
        _, h = _attn()
        setattr(h, f, None)
        assert _abwd(p, h) == E["TRIMUL_ERR_INVALID_ARG"], f
    q, h = _attn()
    q.bias = None
    assert _abwd(q, h) == E["TRIMUL_ERR_INVALID_ARG"]    # dbias of no bias
    h.dbias = None
    assert _abwd(q, h) in [E[c] for c in PASSED]
    assert _abwd(p, h) in [E[c] for c in PASSED]         # dbias not wanted
    q, _ = _attn()
    q.head_dim = 64
    assert _abwd(q, g) == E["TRIMUL_ERR_UNSUPPORTED"]
    for f in ("dq", "dk", "dv", "dbias"):
        _, h = _attn()
        setattr(h, f, getattr(h, f) + 8)
        assert _abwd(p, h) == E["TRIMUL_ERR_MISALIGNED"], f
        for at in (X, Y, R, W + 4096, DY, WS):
            setattr(h, f, at)
            assert _abwd(p, h) == E["TRIMUL_ERR_ALIAS"], (f, hex(at))
    assert _abwd(p, g, dout=DY + 8) == E["TRIMUL_ERR_MISALIGNED"]
    _, h = _attn()
    h.dk = h.dq
    assert _abwd(p, h) == E["TRIMUL_ERR_ALIAS"]
    assert _abwd(p, g) in [E[c] for c in PASSED]


def test_python_refusals_without_a_gpu():
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(32, 64, dtype=torch.bfloat16)
    q = torch.zeros(1, 40, 2, 32, dtype=torch.bfloat16)
    for f in (lambda: tm.linear(x, w), lambda: tm.linear_backward(x, w, x[:, :32].contiguous()),
              lambda: tm.act8_pack(x), lambda: tm.atom_attention_backward(q, q, q, q),
              lambda: tm.atom_attention_backward(q, q, q, q[:, :3]),
              lambda: tm.Act8(torch.zeros(2, 33, dtype=torch.uint8), torch.zeros(2, 1, dtype=torch.uint8)),
              lambda: tm.Act8(torch.zeros(2, 64, dtype=torch.uint8), torch.zeros(2, 1, dtype=torch.uint8)),
              lambda: tm.act8_unpack(tm.Act8(torch.zeros(2, 32, dtype=torch.uint8), torch.zeros(2, 1, dtype=torch.uint8)))):
        with pytest.raises(ValueError):
            f()
