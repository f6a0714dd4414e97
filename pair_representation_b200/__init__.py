"""Python binding of the B200 triangle multiplicative update (libtrimul_b200.so).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels (see include/trimul.h). PyTorch supplies device memory and streams.
There is no CPU fallback: if the library is missing or no sm_100 GPU is
present, calls raise.

Two levels:
  * C-ABI mirrors with the same names as the header (``trimul_forward``,
    ``trimul_prologue``, ``trimul_contract``, ``trimul_epilogue``,
    ``trimul_workspace_size`` ...) taking ``TrimulParams`` and raw pointers or
    tensors.
  * ``TriangleMultiplicationOutgoing`` / ``TriangleMultiplicationIncoming``:
    the layer as the pages use it (construct with the channel size, load a
    state dict, call ``layer(z, mask)``), holding device weights and the
    workspace.
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libtrimul_b200.so")

OUTGOING, INCOMING = 0, 1
DTYPE_F32, DTYPE_BF16 = 0, 1
DEBUG_STALL_CONTRACT = 0x1
BWD_REUSE_FORWARD = 0x1

STATUS = {
    0: "TRIMUL_OK", -1: "TRIMUL_ERR_INVALID_ARG", -2: "TRIMUL_ERR_UNSUPPORTED", -3: "TRIMUL_ERR_MISALIGNED",
    -4: "TRIMUL_ERR_ALIAS", -5: "TRIMUL_ERR_WORKSPACE", -6: "TRIMUL_ERR_CUDA", -7: "TRIMUL_ERR_TIMEOUT",
    -8: "TRIMUL_ERR_DEVICE",
}
ERR = {v: k for k, v in STATUS.items()}

# Every symbol include/trimul.h, include/atomattn.h and include/linear.h declare.
EXPORTS = ("trimul_workspace_size", "trimul_workspace_size_dtype", "trimul_forward", "trimul_prologue",
           "trimul_contract", "trimul_epilogue", "trimul_workspace_views", "trimul_device_status",
           "trimul_status_word", "trimul_status_take",
           "trimul_error_string", "trimul_last_error_detail", "trimul_version", "trimul_forward_noalloc",
           "trimul_backward", "trimul_backward_workspace_size", "trimul_backward_workspace_size_rows",
           "trimul_backward_block_rows",
           "trimul_workspace_size_mxfp8", "trimul_forward_mxfp8", "trimul_contract_mxfp8", "trimul_mxfp8_views",
           "trimul_prologue_mxfp8", "trimul_mma_mxfp8",
           "trimul_shard_workspace_size", "trimul_prologue_rows", "trimul_contract_channels", "trimul_epilogue_rows",
           "atomattn_forward", "atomattn_workspace_size", "atomattn_device_status", "atomattn_backward",
           "trimul_linear_workspace_size", "trimul_linear_forward", "trimul_linear_backward_workspace_size",
           "trimul_linear_backward", "trimul_linear_device_status", "trimul_act8_pack", "trimul_act8_unpack")

# trimul_linear_params.act
ACTS = {"none": 0, "relu": 1, "sigmoid": 2, "silu": 3}

# Gradient outputs of trimul_grads, in struct order; each is "d_" + a TrimulParams field.
GRAD_FIELDS = ("d_w_a", "d_w_ag", "d_w_b", "d_w_bg", "d_w_g", "d_w_o", "d_b_a", "d_b_ag", "d_b_b", "d_b_bg",
               "d_b_g", "d_b_o", "d_ln_in_w", "d_ln_in_b", "d_ln_out_w", "d_ln_out_b")


class TrimulError(RuntimeError):
    def __init__(self, code: int, what: str = ""):
        self.code = code
        detail = ""
        try:
            detail = lib().trimul_last_error_detail().decode()
        except Exception:  # noqa: BLE001 - best effort only
            pass
        super().__init__(f"{what}: {STATUS.get(code, code)}" + (f" ({detail})" if detail else ""))


class TrimulParams(ctypes.Structure):
    """Mirror of ``trimul_params`` in include/trimul.h."""

    _fields_ = [
        ("N", ctypes.c_int), ("c_z", ctypes.c_int), ("c_h", ctypes.c_int), ("dtype", ctypes.c_int),
        ("ln_eps", ctypes.c_float),
        ("ln_in_w", ctypes.c_void_p), ("ln_in_b", ctypes.c_void_p),
        ("w_a", ctypes.c_void_p), ("w_ag", ctypes.c_void_p), ("w_b", ctypes.c_void_p), ("w_bg", ctypes.c_void_p),
        ("b_a", ctypes.c_void_p), ("b_ag", ctypes.c_void_p), ("b_b", ctypes.c_void_p), ("b_bg", ctypes.c_void_p),
        ("w_g", ctypes.c_void_p), ("b_g", ctypes.c_void_p),
        ("ln_out_w", ctypes.c_void_p), ("ln_out_b", ctypes.c_void_p),
        ("w_o", ctypes.c_void_p), ("b_o", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t),
        ("timeout_ms", ctypes.c_uint32), ("debug_flags", ctypes.c_uint32),
    ]


class TrimulGrads(ctypes.Structure):
    """Mirror of ``trimul_grads`` in include/trimul.h (fp32 gradient outputs + backward workspace)."""

    _fields_ = [(f, ctypes.c_void_p) for f in GRAD_FIELDS] + [
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t), ("flags", ctypes.c_uint32)]


class AtomAttnParams(ctypes.Structure):
    """Mirror of ``atomattn_params`` in include/atomattn.h."""

    _fields_ = [
        ("batch", ctypes.c_int), ("n_atoms", ctypes.c_int), ("heads", ctypes.c_int), ("head_dim", ctypes.c_int),
        ("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
        ("bias", ctypes.c_void_p), ("atom_mask", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t), ("timeout_ms", ctypes.c_uint32),
        ("status", ctypes.c_void_p),
    ]


class AtomAttnGrads(ctypes.Structure):
    """Mirror of ``atomattn_grads`` in include/atomattn.h."""

    _fields_ = [("dq", ctypes.c_void_p), ("dk", ctypes.c_void_p), ("dv", ctypes.c_void_p), ("dbias", ctypes.c_void_p)]


class LinearParams(ctypes.Structure):
    """Mirror of ``trimul_linear_params`` in include/linear.h."""

    _fields_ = [
        ("rows", ctypes.c_longlong), ("in_features", ctypes.c_int), ("out_features", ctypes.c_int),
        ("act", ctypes.c_int), ("weight", ctypes.c_void_p), ("bias", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_size_t), ("timeout_ms", ctypes.c_uint32),
        ("status", ctypes.c_void_p),
    ]


class Act8Ptrs(ctypes.Structure):
    """Mirror of ``trimul_act8`` in include/linear.h."""

    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


_lib = None


def lib():
    """Load libtrimul_b200.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with `python -m pair_representation_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        PP = ctypes.POINTER(TrimulParams)
        L.trimul_workspace_size.argtypes = [I, I, I]
        L.trimul_workspace_size.restype = S
        L.trimul_workspace_size_dtype.argtypes = [I, I, I, I]
        L.trimul_workspace_size_dtype.restype = S
        L.trimul_forward.argtypes = [P, P, PP, I, P, P]
        L.trimul_forward_noalloc.argtypes = [P, P, PP, I, P, P]
        L.trimul_prologue.argtypes = [P, P, PP, P]
        L.trimul_contract.argtypes = [PP, I, P]
        L.trimul_epilogue.argtypes = [P, PP, P, P]
        L.trimul_workspace_views.argtypes = [PP, ctypes.POINTER(P), ctypes.POINTER(P), ctypes.POINTER(P),
                                             ctypes.POINTER(S)]
        L.trimul_device_status.argtypes = [PP, P, ctypes.POINTER(ctypes.c_int)]
        L.trimul_status_word.argtypes = [ctypes.POINTER(P)]
        L.trimul_status_take.argtypes = [P, P, ctypes.POINTER(ctypes.c_int)]
        L.trimul_error_string.argtypes = [I]
        L.trimul_error_string.restype = ctypes.c_char_p
        L.trimul_last_error_detail.argtypes = []
        L.trimul_last_error_detail.restype = ctypes.c_char_p
        L.trimul_version.argtypes = []
        L.trimul_backward_workspace_size.argtypes = [I, I, I]
        L.trimul_backward_workspace_size.restype = S
        L.trimul_backward_workspace_size_rows.argtypes = [I, I, I, I]
        L.trimul_backward_workspace_size_rows.restype = S
        L.trimul_backward_block_rows.argtypes = [I, I, I, S]
        L.trimul_backward.argtypes = [P, P, PP, I, P, P, ctypes.POINTER(TrimulGrads), P]
        L.trimul_workspace_size_mxfp8.argtypes = [I, I, I]
        L.trimul_workspace_size_mxfp8.restype = S
        L.trimul_forward_mxfp8.argtypes = [P, P, PP, I, P, P]
        L.trimul_contract_mxfp8.argtypes = [PP, I, P]
        L.trimul_prologue_mxfp8.argtypes = [P, P, PP, I, P]
        L.trimul_mma_mxfp8.argtypes = [PP, P]
        L.trimul_mxfp8_views.argtypes = [PP] + [ctypes.POINTER(P)] * 4 + [ctypes.POINTER(S)]
        L.trimul_shard_workspace_size.argtypes = [I, I]
        L.trimul_shard_workspace_size.restype = S
        L.trimul_prologue_rows.argtypes = [P, P, PP, I, P, P, P]
        L.trimul_contract_channels.argtypes = [PP, I, I, P, P, P, P]
        L.trimul_epilogue_rows.argtypes = [P, P, PP, I, P, P]
        AP = ctypes.POINTER(AtomAttnParams)
        L.atomattn_workspace_size.argtypes = []
        L.atomattn_workspace_size.restype = S
        L.atomattn_forward.argtypes = [AP, P, P]
        L.atomattn_device_status.argtypes = [AP, P, ctypes.POINTER(ctypes.c_int)]
        L.atomattn_backward.argtypes = [AP, P, ctypes.POINTER(AtomAttnGrads), P]
        LP, LL = ctypes.POINTER(LinearParams), ctypes.c_longlong
        L.trimul_linear_workspace_size.argtypes = []
        L.trimul_linear_workspace_size.restype = S
        L.trimul_linear_forward.argtypes = [P, P, LP, P, P]
        L.trimul_linear_backward_workspace_size.argtypes = [LL, I, I, I, I]
        L.trimul_linear_backward_workspace_size.restype = S
        L.trimul_linear_backward.argtypes = [P, ctypes.POINTER(Act8Ptrs), P, LP, P, P, P, P]
        L.trimul_linear_device_status.argtypes = [LP, P, ctypes.POINTER(ctypes.c_int)]
        L.trimul_act8_pack.argtypes = [P, LL, I, P, P, P]
        L.trimul_act8_unpack.argtypes = [P, P, LL, I, P, P]
        for f in ("atomattn_backward", "trimul_linear_forward", "trimul_linear_backward", "trimul_linear_device_status",
                  "trimul_act8_pack", "trimul_act8_unpack"):
            getattr(L, f).restype = I
        for f in ("trimul_forward", "trimul_forward_noalloc", "trimul_prologue", "trimul_contract", "trimul_epilogue",
                  "trimul_workspace_views", "trimul_device_status", "trimul_status_word", "trimul_status_take",
                  "trimul_version", "trimul_backward",
                  "atomattn_forward", "atomattn_device_status", "trimul_forward_mxfp8", "trimul_contract_mxfp8",
                  "trimul_mxfp8_views", "trimul_prologue_mxfp8", "trimul_mma_mxfp8", "trimul_prologue_rows", "trimul_contract_channels", "trimul_epilogue_rows"):
            getattr(L, f).restype = I
        _lib = L
    return _lib


def _ptr(t):
    """Device address of a tensor, an int address, or None."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int, what: str):
    if rc != 0:
        raise TrimulError(rc, what)


# ---- C-ABI mirrors ---------------------------------------------------------

def trimul_workspace_size(N: int, c_z: int = 128, c_h: int = 128) -> int:
    return lib().trimul_workspace_size(N, c_z, c_h)


def trimul_workspace_size_dtype(N: int, c_z: int, c_h: int, dtype: int) -> int:
    return lib().trimul_workspace_size_dtype(N, c_z, c_h, dtype)


def trimul_forward(z, mask, params: TrimulParams, direction: int, out, stream=None, check=True) -> int:
    rc = lib().trimul_forward(_ptr(z), _ptr(mask), ctypes.byref(params), direction, _ptr(out), _stream(stream))
    if check:
        _check(rc, "trimul_forward")
    return rc


def trimul_forward_noalloc(z, mask, params: TrimulParams, direction: int, out, stream=None, check=True) -> int:
    """trimul_forward with the library's static scratch instead of params.workspace.

    For callers that cannot allocate device memory; limited to bf16 N <= 128
    and fp32 N <= 88. Overlapping calls share the scratch and race.
    """
    rc = lib().trimul_forward_noalloc(_ptr(z), _ptr(mask), ctypes.byref(params), direction, _ptr(out),
                                      _stream(stream))
    if check:
        _check(rc, "trimul_forward_noalloc")
    return rc


def trimul_prologue(z, mask, params: TrimulParams, stream=None, check=True) -> int:
    rc = lib().trimul_prologue(_ptr(z), _ptr(mask), ctypes.byref(params), _stream(stream))
    if check:
        _check(rc, "trimul_prologue")
    return rc


def trimul_contract(params: TrimulParams, direction: int, stream=None, check=True) -> int:
    rc = lib().trimul_contract(ctypes.byref(params), direction, _stream(stream))
    if check:
        _check(rc, "trimul_contract")
    return rc


def trimul_epilogue(z, params: TrimulParams, out, stream=None, check=True) -> int:
    rc = lib().trimul_epilogue(_ptr(z), ctypes.byref(params), _ptr(out), _stream(stream))
    if check:
        _check(rc, "trimul_epilogue")
    return rc


def trimul_backward_workspace_size(N: int, c_z: int = 128, c_h: int = 128) -> int:
    return lib().trimul_backward_workspace_size(N, c_z, c_h)


def trimul_backward_workspace_size_rows(N: int, rows: int, c_z: int = 128, c_h: int = 128) -> int:
    return lib().trimul_backward_workspace_size_rows(N, c_z, c_h, rows)


def trimul_backward_block_rows(N: int, workspace_bytes: int, c_z: int = 128, c_h: int = 128) -> int:
    return lib().trimul_backward_block_rows(N, c_z, c_h, workspace_bytes)


def trimul_backward(z, mask, params: TrimulParams, direction: int, dout, dz, grads: TrimulGrads, stream=None,
                    check=True) -> int:
    """dz and the fp32 parameter gradients of sum(out * dout); see trimul_backward in the header."""
    rc = lib().trimul_backward(_ptr(z), _ptr(mask), ctypes.byref(params), direction, _ptr(dout), _ptr(dz),
                               ctypes.byref(grads), _stream(stream))
    if check:
        _check(rc, "trimul_backward")
    return rc


def trimul_workspace_size_mxfp8(N: int, c_z: int = 128, c_h: int = 128) -> int:
    return lib().trimul_workspace_size_mxfp8(N, c_z, c_h)


def trimul_forward_mxfp8(z, mask, params: TrimulParams, direction: int, out, stream=None, check=True) -> int:
    """The layer with the contraction in MXFP8 (E4M3 in blocks of 32 along k, E8M0 scales)."""
    rc = lib().trimul_forward_mxfp8(_ptr(z), _ptr(mask), ctypes.byref(params), direction, _ptr(out), _stream(stream))
    if check:
        _check(rc, "trimul_forward_mxfp8")
    return rc


def trimul_contract_mxfp8(params: TrimulParams, direction: int, stream=None, check=True) -> int:
    rc = lib().trimul_contract_mxfp8(ctypes.byref(params), direction, _stream(stream))
    if check:
        _check(rc, "trimul_contract_mxfp8")
    return rc


def trimul_prologue_mxfp8(z, mask, params: TrimulParams, direction: int, stream=None, check=True) -> int:
    """The quantising prologue: z, mask -> E4M3 operands and scales of `direction`'s contraction."""
    rc = lib().trimul_prologue_mxfp8(_ptr(z), _ptr(mask), ctypes.byref(params), direction, _stream(stream))
    if check:
        _check(rc, "trimul_prologue_mxfp8")
    return rc


def trimul_mma_mxfp8(params: TrimulParams, stream=None, check=True) -> int:
    """The block-scaled contraction of the MXFP8 operands in the workspace -> x."""
    rc = lib().trimul_mma_mxfp8(ctypes.byref(params), _stream(stream))
    if check:
        _check(rc, "trimul_mma_mxfp8")
    return rc


def trimul_mxfp8_views(params: TrimulParams):
    """(aq, bq, sa, sb, ldq): device addresses of the quantised operands and scales in the workspace."""
    ptrs = [ctypes.c_void_p() for _ in range(4)]
    ldq = ctypes.c_size_t()
    _check(lib().trimul_mxfp8_views(ctypes.byref(params), *[ctypes.byref(x) for x in ptrs], ctypes.byref(ldq)),
           "trimul_mxfp8_views")
    return ptrs[0].value, ptrs[1].value, ptrs[2].value, ptrs[3].value, ldq.value


def trimul_shard_workspace_size(N: int, rows: int) -> int:
    return lib().trimul_shard_workspace_size(N, rows)


def trimul_prologue_rows(z_rows, mask_rows, params: TrimulParams, rows: int, a, b, stream=None, check=True) -> int:
    rc = lib().trimul_prologue_rows(_ptr(z_rows), _ptr(mask_rows), ctypes.byref(params), rows, _ptr(a), _ptr(b),
                                    _stream(stream))
    if check:
        _check(rc, "trimul_prologue_rows")
    return rc


def trimul_contract_channels(params: TrimulParams, direction: int, channels: int, a, b, x, stream=None,
                             check=True) -> int:
    rc = lib().trimul_contract_channels(ctypes.byref(params), direction, channels, _ptr(a), _ptr(b), _ptr(x),
                                        _stream(stream))
    if check:
        _check(rc, "trimul_contract_channels")
    return rc


def trimul_epilogue_rows(z_rows, x_rows, params: TrimulParams, rows: int, out_rows, stream=None, check=True) -> int:
    rc = lib().trimul_epilogue_rows(_ptr(z_rows), _ptr(x_rows), ctypes.byref(params), rows, _ptr(out_rows),
                                    _stream(stream))
    if check:
        _check(rc, "trimul_epilogue_rows")
    return rc


def trimul_workspace_views(params: TrimulParams):
    """(a, b, x, ld): device addresses of the workspace sections and their leading dimension."""
    a, b, x = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_void_p()
    ld = ctypes.c_size_t()
    _check(lib().trimul_workspace_views(ctypes.byref(params), ctypes.byref(a), ctypes.byref(b),
                                        ctypes.byref(x), ctypes.byref(ld)), "trimul_workspace_views")
    return a.value, b.value, x.value, ld.value


def trimul_device_status(params: TrimulParams, stream=None):
    """(code, [code, site, block, aux]) of the workspace status word (synchronises)."""
    d = (ctypes.c_int * 4)()
    rc = lib().trimul_device_status(ctypes.byref(params), _stream(stream), d)
    return rc, list(d)


def trimul_status_word() -> int:
    """Device address of the status word that the library keeps for the current device."""
    word = ctypes.c_void_p()
    _check(lib().trimul_status_word(ctypes.byref(word)), "trimul_status_word")
    return word.value


def trimul_status_take(word: int, stream=None):
    """(code, [code, site, block, aux]) of a status word that calls do not clear, set back to 0 (synchronises)."""
    d = (ctypes.c_int * 4)()
    rc = lib().trimul_status_take(word, _stream(stream), d)
    return rc, list(d)


# ---- sequence-local atom attention -------------------------------------------

def atomattn_workspace_size() -> int:
    return lib().atomattn_workspace_size()


def atomattn_forward(params: AtomAttnParams, out, stream=None, check=True) -> int:
    rc = lib().atomattn_forward(ctypes.byref(params), _ptr(out), _stream(stream))
    if check:
        _check(rc, "atomattn_forward")
    return rc


def atomattn_device_status(params: AtomAttnParams, stream=None):
    """(code, [code, site, block, aux]) of the status word (synchronises)."""
    d = (ctypes.c_int * 4)()
    rc = lib().atomattn_device_status(ctypes.byref(params), _stream(stream), d)
    return rc, list(d)


def atomattn_backward(params: AtomAttnParams, dout, grads: AtomAttnGrads, stream=None, check=True) -> int:
    rc = lib().atomattn_backward(ctypes.byref(params), _ptr(dout), ctypes.byref(grads), _stream(stream))
    if check:
        _check(rc, "atomattn_backward")
    return rc


# torch and what the calls below need of it, and the library: looked up by the first of them. Small
# calls are bound by the host, so these functions keep names, attributes and allocations few.
_T = _L = _BF16 = _U8 = _current_device = _raw_stream = None


def _load():
    global _T, _L, _BF16, _U8, _current_device, _raw_stream
    import torch
    _L = lib()
    _BF16, _U8 = torch.bfloat16, torch.uint8
    _current_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
    _T = torch
    return torch


def _need_bf16(what: str, index: int, tensors):
    """Every tensor (None passes) must be contiguous bf16 on CUDA device `index`."""
    if index < 0:
        raise ValueError(f"{what}: tensors must be on a CUDA device")
    for t in tensors:
        if t is not None:
            if t.dtype is not _BF16 or not t.is_contiguous():
                raise ValueError(f"{what}: tensors must be contiguous bf16")
            if t.get_device() != index:
                raise ValueError(f"{what}: tensors must be on one CUDA device")


def _need_workspace(what: str, index: int, workspace):
    if workspace.dtype is not _U8 or not workspace.is_contiguous() or workspace.get_device() != index:
        raise ValueError(f"{what}: workspace must be contiguous uint8 on the tensors' device")


def _run_on(index: int, stream, tensors, call):
    """call() with device `index` current and, where one is given, `stream` current too, so that
    what the call allocates belongs to it. `tensors` may be another stream's: they are marked as
    used on this one, so that their memory is not handed out again before this work is done."""
    torch = _T or _load()
    if stream is not None and not isinstance(stream, int) and stream.device.index != index:
        raise ValueError(f"stream must be one of device {index}, where the tensors are")
    with torch.cuda.device(index):
        if stream is None:
            return call()
        s = torch.cuda.ExternalStream(stream, device=index) if isinstance(stream, int) else stream
        with torch.cuda.stream(s):
            out = call()
            for t in tensors:
                if t is not None:
                    t.record_stream(s)
            return out


_words = {}  # device index -> the library's status word there, of the calls that are given no workspace


def _status_word(index: int) -> int:
    """Looked up with device `index` current. Its memory is the library's: a captured call's replays write it too."""
    word = _words.get(index)
    if word is None:
        word = _words[index] = trimul_status_word()
    return word


def _attention_shape(what, q, bias, atom_mask, like):
    """q's batch, atoms and heads; the kernels take every other tensor's size from these."""
    shape = q.shape
    if len(shape) != 4 or shape[3] != 32:
        raise ValueError(f"{what}: q must be [batch, n_atoms, heads, 32]")
    for t in like:
        if t is not None and t.shape != shape:
            raise ValueError(f"{what}: q, k, v, dout and out must be of one shape")
    B, n, H, _ = shape
    if bias is not None and bias.shape != (B, (n + 31) // 32, H, 32, 128):
        raise ValueError(f"{what}: bias must be [batch, ceil(n_atoms / 32), heads, 32, 128]")
    if atom_mask is not None and atom_mask.shape != (B, n):
        raise ValueError(f"{what}: atom_mask must be [batch, n_atoms]")
    return B, n, H


def atom_attention(q, k, v, bias=None, atom_mask=None, out=None, workspace=None, stream=None):
    """Windowed atom attention (include/atomattn.h) on bf16 device tensors.

    q, k, v: [batch][n_atoms][heads][32]; bias: [batch][ceil(n_atoms/32)][heads][32][128]
    or None; atom_mask: [batch][n_atoms] or None. Returns out (allocated if None) and the call's
    AtomAttnParams, whose status atomattn_device_status reads."""
    torch = _T or _load()
    B, n, H = _attention_shape("atom_attention", q, bias, atom_mask, (k, v, out))
    if out is not None and out.dtype is not _BF16:
        raise ValueError("atom_attention: tensors must be contiguous bf16")
    index = q.get_device()
    _need_bf16("atom_attention", index, (q, k, v, bias, atom_mask, out))
    if workspace is not None:
        _need_workspace("atom_attention", index, workspace)
    if _current_device() != index or stream is not None and (
            _stream(stream) != _raw_stream(index) or not isinstance(stream, int) and stream.device.index != index):
        return _run_on(index, stream, (q, k, v, bias, atom_mask, out, workspace),
                       lambda: atom_attention(q, k, v, bias, atom_mask, out, workspace))
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        workspace = torch.zeros(atomattn_workspace_size(), dtype=torch.uint8, device=q.device)
    p = AtomAttnParams(B, n, H, 32, q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(bias), _ptr(atom_mask),
                       workspace.data_ptr(), workspace.numel(), 0)
    p.kept = workspace  # its memory stays while the status may be asked for
    atomattn_forward(p, out, _raw_stream(index))
    return out, p


def _attention_core(q, k, v, bias, atom_mask):
    """atom_attention's result alone, its failures kept by the device's status word."""
    torch = _T or _load()
    B, n, H = _attention_shape("atom_attention", q, bias, atom_mask, (k, v))
    index = q.get_device()
    _need_bf16("atom_attention", index, (q, k, v, bias, atom_mask))
    if _current_device() != index:
        return _run_on(index, None, (), lambda: _attention_core(q, k, v, bias, atom_mask))
    out = torch.empty_like(q)
    p = AtomAttnParams(B, n, H, 32, q.data_ptr(), k.data_ptr(), v.data_ptr(), _ptr(bias), _ptr(atom_mask), None, 0, 0,
                       _status_word(index))
    atomattn_forward(p, out, _raw_stream(index))
    return out


def atom_attention_backward(q, k, v, dout, bias=None, atom_mask=None, workspace=None, stream=None):
    """Gradients of sum(atom_attention(q, k, v, bias, atom_mask) * dout) (include/atomattn.h).

    Arguments as for atom_attention, dout like q. Returns (dq, dk, dv, dbias), dbias None
    without bias. `workspace` (atomattn_workspace_size() bytes): where device_status finds this
    call's status; without one, the device's status word keeps a failure."""
    torch = _T or _load()
    B, n, H = _attention_shape("atom_attention_backward", q, bias, atom_mask, (k, v, dout))
    index = q.get_device()
    _need_bf16("atom_attention_backward", index, (q, k, v, dout, bias, atom_mask))
    if workspace is not None:
        _need_workspace("atom_attention_backward", index, workspace)
    if stream is not None or _current_device() != index:
        return _run_on(index, stream, (q, k, v, dout, bias, atom_mask, workspace),
                       lambda: atom_attention_backward(q, k, v, dout, bias, atom_mask, workspace))
    dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    dbias = None if bias is None else torch.empty_like(bias)
    ws, size, word = (None, 0, _status_word(index)) if workspace is None else (workspace.data_ptr(), workspace.numel(), None)
    p = AtomAttnParams(B, n, H, 32, q.data_ptr(), k.data_ptr(), v.data_ptr(), None if bias is None else bias.data_ptr(),
                       None if atom_mask is None else atom_mask.data_ptr(), ws, size, 0, word)
    g = AtomAttnGrads(dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), None if bias is None else dbias.data_ptr())
    rc = _L.atomattn_backward(p, dout.data_ptr(), g, _raw_stream(index))
    if rc:
        raise TrimulError(rc, "atomattn_backward")
    return dq, dk, dv, dbias


# ---- linear layers and activations in 8 bits (include/linear.h) -----------------

def trimul_linear_workspace_size() -> int:
    return lib().trimul_linear_workspace_size()


def trimul_linear_backward_workspace_size(rows: int, in_features: int, out_features: int, act: int,
                                          from8: bool = False) -> int:
    return lib().trimul_linear_backward_workspace_size(rows, in_features, out_features, act, int(from8))


def trimul_linear_forward(x, residual, params: LinearParams, y, stream=None, check=True) -> int:
    rc = lib().trimul_linear_forward(_ptr(x), _ptr(residual), ctypes.byref(params), _ptr(y), _stream(stream))
    if check:
        _check(rc, "trimul_linear_forward")
    return rc


def trimul_linear_backward(x, x8, dout, params: LinearParams, dx, dw, db, stream=None, check=True) -> int:
    rc = lib().trimul_linear_backward(_ptr(x), None if x8 is None else ctypes.byref(x8), _ptr(dout),
                                      ctypes.byref(params), _ptr(dx), _ptr(dw), _ptr(db), _stream(stream))
    if check:
        _check(rc, "trimul_linear_backward")
    return rc


def trimul_linear_device_status(params: LinearParams, stream=None):
    """(code, [code, site, block, aux]) of the status word (synchronises)."""
    d = (ctypes.c_int * 4)()
    rc = lib().trimul_linear_device_status(ctypes.byref(params), _stream(stream), d)
    return rc, list(d)


def trimul_act8_pack(x, rows: int, channels: int, codes, scales, stream=None, check=True) -> int:
    rc = lib().trimul_act8_pack(_ptr(x), rows, channels, _ptr(codes), _ptr(scales), _stream(stream))
    if check:
        _check(rc, "trimul_act8_pack")
    return rc


def trimul_act8_unpack(codes, scales, rows: int, channels: int, x, stream=None, check=True) -> int:
    rc = lib().trimul_act8_unpack(_ptr(codes), _ptr(scales), rows, channels, _ptr(x), _stream(stream))
    if check:
        _check(rc, "trimul_act8_unpack")
    return rc


def device_status(workspace, stream=None):
    """(code, [code, site, block, aux]) that the last linear, linear_backward or
    atom_attention_backward call with this workspace left (synchronises). With a device in the
    workspace's place: the first failure since this was last asked among that device's calls that were
    given no workspace, AtomAttention's and captured ones included. Only `stream` (by default the
    current one) is waited for: work on others may still add one."""
    torch = _T or _load()
    if not isinstance(workspace, torch.Tensor):
        device = torch.device(workspace)
        index = torch.cuda.current_device() if device.index is None else device.index
        return _run_on(index, stream, (), lambda: trimul_status_take(_status_word(index)))
    p = LinearParams()
    p.workspace, p.workspace_bytes = workspace.data_ptr(), workspace.numel()
    return _run_on(workspace.get_device(), stream, (), lambda: trimul_linear_device_status(p))


class Act8:
    """A bf16 tensor kept in 8 bits: E4M3 codes (its shape, uint8) and one E8M0 scale per 32
    channels (last dimension / 32, uint8). Made by act8_pack; act8_unpack gives the values, and
    linear_backward and the triangle layers' backward take it in the tensor's place."""

    __slots__ = ("codes", "scales")

    def __init__(self, codes, scales):
        _T or _load()
        shape, c = codes.shape, codes.shape[-1] if codes.dim() else 0
        if c == 0 or c % 32 or scales.shape != shape[:-1] + (c // 32,):
            raise ValueError("codes must be [..., channels] and scales [..., channels / 32]")
        for t in (codes, scales):
            if t.dtype is not _U8 or not t.is_contiguous():
                raise ValueError("codes and scales must be contiguous uint8")
        if codes.get_device() != scales.get_device():
            raise ValueError("codes and scales must be on one device")
        self.codes, self.scales = codes, scales

    @property
    def shape(self):
        return self.codes.shape

    @property
    def device(self):
        return self.codes.device


def act8_pack(x, stream=None) -> Act8:
    """Keep a bf16 tensor [..., channels] (channels a multiple of 32) in 33/32 bytes per value."""
    torch = _T or _load()
    shape = x.shape
    c = shape[-1] if len(shape) else 0
    if c == 0 or c % 32:
        raise ValueError("x must be [..., channels], channels a multiple of 32")
    index = x.get_device()
    _need_bf16("act8_pack", index, (x,))
    if stream is not None or _current_device() != index:
        return _run_on(index, stream, (x,), lambda: act8_pack(x))
    codes = torch.empty_like(x, dtype=_U8)
    scales = codes.new_empty(shape[:-1] + (c // 32,))
    count = codes.numel()
    if count:
        rc = _L.trimul_act8_pack(x.data_ptr(), count // c, c, codes.data_ptr(), scales.data_ptr(), _raw_stream(index))
        if rc:
            raise TrimulError(rc, "trimul_act8_pack")
    a = Act8.__new__(Act8)  # nothing to check: these are ours
    a.codes, a.scales = codes, scales
    return a


def act8_unpack(a: Act8, out=None, stream=None):
    """The values an Act8 stands for, as a bf16 tensor (written to `out` if given)."""
    torch = _T or _load()
    codes, scales = a.codes, a.scales
    index = codes.get_device()
    if out is not None and out.shape != codes.shape:
        raise ValueError("out must have the codes' shape")
    _need_bf16("act8_unpack", index, (out,))
    if stream is not None or _current_device() != index:
        return _run_on(index, stream, (codes, scales, out), lambda: act8_unpack(a, out))
    x = torch.empty_like(codes, dtype=_BF16) if out is None else out
    count = x.numel()
    if count:
        c = codes.shape[-1]
        rc = _L.trimul_act8_unpack(codes.data_ptr(), scales.data_ptr(), count // c, c, x.data_ptr(), _raw_stream(index))
        if rc:
            raise TrimulError(rc, "trimul_act8_unpack")
    return x


def _linear_shape(what, x_shape, weight, bias, act):
    """Shape of the layer's result."""
    w = weight.shape
    if len(w) != 2 or len(x_shape) < 1 or x_shape[-1] != w[1] or w[1] == 0:
        raise ValueError(f"{what}: x must be [..., in_features] and weight [out_features, in_features]")
    if bias is not None and bias.shape != w[:1]:
        raise ValueError(f"{what}: bias must be [out_features]")
    if act not in ACTS:
        raise ValueError(f"{what}: act must be one of {', '.join(ACTS)}")
    return x_shape[:-1] + w[:1]


def linear(x, weight, bias=None, residual=None, act="none", out=None, workspace=None, stream=None):
    """act(x weight^T + bias) + residual in one kernel (include/linear.h), on bf16 device tensors.

    x: [..., in_features]; weight: [out_features, in_features] (both multiples of 8); bias:
    [out_features] or None; residual: like the result, or None; act: "none", "relu",
    "sigmoid" or "silu". Returns out (allocated if None; it may be the residual itself). Not
    recorded by autograd: linear_backward gives the gradients. `workspace`
    (trimul_linear_workspace_size() bytes): where device_status finds this call's status;
    without one, the device's status word keeps a failure."""
    torch = _T or _load()
    shape = _linear_shape("linear", x.shape, weight, bias, act)
    index = x.get_device()
    _need_bf16("linear", index, (x, weight, bias, residual, out))
    if workspace is not None:
        _need_workspace("linear", index, workspace)
    if residual is not None and residual.shape != shape:
        raise ValueError("linear: residual must have the result's shape")
    if out is not None and out.shape != shape:
        raise ValueError("linear: out must have the result's shape")
    if stream is not None or _current_device() != index:
        return _run_on(index, stream, (x, weight, bias, residual, out, workspace),
                       lambda: linear(x, weight, bias, residual, act, out, workspace))
    n, k = weight.shape
    y = out if out is not None else torch.empty_like(x) if n == k else x.new_empty(shape)
    rows = x.numel() // k
    if rows and n:
        ws, size, word = (None, 0, _status_word(index)) if workspace is None else (workspace.data_ptr(), workspace.numel(), None)
        p = LinearParams(rows, k, n, ACTS[act], weight.data_ptr(), None if bias is None else bias.data_ptr(), ws, size, 0, word)
        rc = _L.trimul_linear_forward(x.data_ptr(), None if residual is None else residual.data_ptr(), p, y.data_ptr(),
                                      _raw_stream(index))
        if rc:
            raise TrimulError(rc, "trimul_linear_forward")
    return y


def linear_backward(x, weight, dout, bias=None, act="none", need_dx=True, need_dw=True, need_db=True, workspace=None,
                    stream=None):
    """Gradients of sum(linear(x, weight, bias, act=act) * dout): (dx, dw, db), bf16 (include/linear.h).

    x is the forward's input, or the Act8 that kept it. What is not needed is not computed
    and comes back as None; db is computed without bias too (a bias of zeros). The
    residual's gradient is dout itself. `workspace`: trimul_linear_backward_workspace_size
    bytes, for callers that keep one or want the call's status (device_status)."""
    torch = _T or _load()
    held = isinstance(x, Act8)
    shape = _linear_shape("linear_backward", x.shape, weight, bias, act)
    if dout.shape != shape:
        raise ValueError("linear_backward: dout must be [..., out_features] with x's leading dimensions")
    index = weight.get_device()
    _need_bf16("linear_backward", index, (weight, None if held else x, dout, bias))
    if workspace is not None:
        _need_workspace("linear_backward", index, workspace)
    if held and x.codes.get_device() != index:
        raise ValueError("linear_backward: tensors must be on one CUDA device")
    if stream is not None or _current_device() != index:
        tensors = (x.codes, x.scales) if held else (x,)
        return _run_on(index, stream, tensors + (weight, dout, bias, workspace),
                       lambda: linear_backward(x, weight, dout, bias, act, need_dx, need_dw, need_db, workspace))
    n, k = weight.shape
    dx = None if not need_dx else torch.empty_like(x) if not held else torch.empty_like(x.codes, dtype=_BF16)
    dw = torch.empty_like(weight) if need_dw else None
    db = None if not need_db else torch.empty_like(bias) if bias is not None else weight.new_empty(n)
    rows = dout.numel() // n if n else 0
    if rows == 0:  # no rows, or no columns: nothing to sum over
        for t in (dx, dw, db):
            if t is not None:
                t.zero_()
        return dx, dw, db
    code, ws, word = ACTS[act], workspace, None
    if ws is None:
        word = _status_word(index)
        need = _L.trimul_linear_backward_workspace_size(rows, k, n, code, held)
        if need > 256:  # more than a status word
            ws = weight.new_empty(need, dtype=_U8)
    p = LinearParams(rows, k, n, code, weight.data_ptr(), None if bias is None else bias.data_ptr(),
                     None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(), 0, word)
    rc = _L.trimul_linear_backward(None if held else x.data_ptr(),
                                   Act8Ptrs(x.codes.data_ptr(), x.scales.data_ptr()) if held else None, dout.data_ptr(), p,
                                   dx.data_ptr() if need_dx else None, dw.data_ptr() if need_dw else None,
                                   db.data_ptr() if need_db else None, _raw_stream(index))
    if rc:
        raise TrimulError(rc, "trimul_linear_backward")
    return dx, dw, db


# ---- the layer as the pages use it ------------------------------------------

# State-dict keys: (params field, key, required)
STATE_KEYS = (
    ("ln_in_w", "layer_norm_in.weight", False), ("ln_in_b", "layer_norm_in.bias", False),
    ("w_a", "linear_a_p.weight", True), ("b_a", "linear_a_p.bias", False),
    ("w_ag", "linear_a_g.weight", True), ("b_ag", "linear_a_g.bias", False),
    ("w_b", "linear_b_p.weight", True), ("b_b", "linear_b_p.bias", False),
    ("w_bg", "linear_b_g.weight", True), ("b_bg", "linear_b_g.bias", False),
    ("w_g", "linear_g.weight", True), ("b_g", "linear_g.bias", False),
    ("ln_out_w", "layer_norm_out.weight", False), ("ln_out_b", "layer_norm_out.bias", False),
    ("w_o", "linear_z.weight", True), ("b_o", "linear_z.bias", False),
)


class _TriangleMultiplication:
    """Holds device weights and a workspace; ``layer(z, mask)`` returns the update."""

    direction = OUTGOING

    def __init__(self, c_z: int = 128, c_hidden: int = 128, eps: float = 1e-5):
        self.c_z, self.c_h, self.eps = c_z, c_hidden, eps
        self.tensors = {}
        self.device = None
        self.dtype = None
        self._ws = None
        self.timeout_ms = 0
        self.debug_flags = 0

    def load_state_dict(self, sd: dict):
        """Take weights by the keys in STATE_KEYS (torch tensors or numpy arrays)."""
        import torch
        t = {}
        for field, key, required in STATE_KEYS:
            if key in sd and sd[key] is not None:
                v = sd[key]
                t[field] = v if isinstance(v, torch.Tensor) else torch.as_tensor(v)
            elif required:
                raise KeyError(key)
        self.tensors = t
        return self

    def to(self, device=None, dtype=None):
        import torch
        dtype = dtype or next(iter(self.tensors.values())).dtype
        if dtype not in (torch.float32, torch.bfloat16):
            raise ValueError("dtype must be float32 or bfloat16")
        self.tensors = {k: v.to(device=device, dtype=dtype).contiguous() for k, v in self.tensors.items()}
        self.device = self.tensors["w_a"].device  # resolved (cuda -> cuda:0)
        self.dtype = dtype
        return self

    def params(self, N: int) -> TrimulParams:
        import torch
        p = TrimulParams()
        p.N, p.c_z, p.c_h = N, self.c_z, self.c_h
        p.dtype = DTYPE_BF16 if self.dtype == torch.bfloat16 else DTYPE_F32
        p.ln_eps = self.eps
        for field, _, _ in STATE_KEYS:
            setattr(p, field, _ptr(self.tensors.get(field)))
        need = trimul_workspace_size_dtype(N, self.c_z, self.c_h, p.dtype)
        if self._ws is None or self._ws.numel() < need:
            self._ws = torch.empty(need, dtype=torch.uint8, device=self.device)
        p.workspace = self._ws.data_ptr()
        p.workspace_bytes = self._ws.numel()
        p.timeout_ms = self.timeout_ms
        p.debug_flags = self.debug_flags
        return p

    def _mask(self, z, mask):
        if mask is None:
            return None
        if mask.numel() != z.shape[0] * z.shape[1]:
            raise ValueError("mask must be [N, N]")
        return mask.to(dtype=self.dtype).contiguous()

    def __call__(self, z, mask=None, out=None, stream=None):
        import torch
        if z.dim() != 3 or z.shape[0] != z.shape[1] or z.shape[2] != self.c_z:
            raise ValueError("z must be [N, N, c_z]")
        if z.dtype != self.dtype or z.device != self.device:
            raise ValueError("z must match the layer's dtype and device")
        z = z.contiguous()
        mask = self._mask(z, mask)
        if out is None:
            out = torch.empty_like(z)
        elif out.shape != z.shape or out.dtype != z.dtype or out.device != z.device or not out.is_contiguous():
            raise ValueError("out must be contiguous, of z's shape, dtype and device")
        p = self.params(z.shape[0])
        trimul_forward(z, mask, p, self.direction, out, stream)
        return out

    def backward(self, z, dout, mask=None, stream=None, reuse_forward=False, block_rows=None):
        """Gradients of sum(layer(z, mask) * dout): (dz, {params field: fp32 gradient}).

        Every parameter gets a gradient, including the optional ones the state
        dict left out (taken as bias 0, gamma 1, beta 0 in the forward). With
        reuse_forward the call relies on the layer's last forward call having
        been ``layer(z, mask)`` with this z and mask (its a, b and x are still in
        the workspace) and does not recompute them. block_rows gives the call
        only the workspace for blocks of that many rows
        (trimul_backward_workspace_size_rows); the library then uses the largest
        block that fits in it. z may be the Act8 that kept it since the forward
        (33/32 bytes per value instead of 2): the gradients are then those at the
        values it stands for."""
        import torch
        if isinstance(z, Act8):
            if reuse_forward:
                raise ValueError("reuse_forward needs the z of the forward call, not the 8 bits kept of it")
            z = act8_unpack(z, stream=stream)
        if z.dim() != 3 or z.shape[0] != z.shape[1] or z.shape[2] != self.c_z:
            raise ValueError("z must be [N, N, c_z]")
        if z.dtype != self.dtype or z.device != self.device or dout.shape != z.shape or dout.dtype != z.dtype:
            raise ValueError("z and dout must match each other and the layer's dtype and device")
        z, dout = z.contiguous(), dout.contiguous()
        mask = self._mask(z, mask)
        N = z.shape[0]
        p = self.params(N)
        g = TrimulGrads()
        need = (trimul_backward_workspace_size(N, self.c_z, self.c_h) if block_rows is None
                else trimul_backward_workspace_size_rows(N, block_rows, self.c_z, self.c_h))
        if need == 0:
            raise ValueError("no backward workspace size for these arguments")
        if getattr(self, "_bws", None) is None or self._bws.numel() < need:
            self._bws = torch.empty(need, dtype=torch.uint8, device=self.device)
        g.workspace, g.workspace_bytes = self._bws.data_ptr(), need
        g.flags = BWD_REUSE_FORWARD if reuse_forward else 0
        cz, ch = self.c_z, self.c_h
        shapes = {"w_a": (ch, cz), "w_ag": (ch, cz), "w_b": (ch, cz), "w_bg": (ch, cz), "w_g": (cz, cz),
                  "w_o": (cz, ch), "b_a": (ch,), "b_ag": (ch,), "b_b": (ch,), "b_bg": (ch,), "b_g": (cz,),
                  "b_o": (cz,), "ln_in_w": (cz,), "ln_in_b": (cz,), "ln_out_w": (ch,), "ln_out_b": (ch,)}
        grads = {}
        for f in GRAD_FIELDS:
            grads[f[2:]] = torch.empty(shapes[f[2:]], dtype=torch.float32, device=self.device)
            setattr(g, f, grads[f[2:]].data_ptr())
        dz = torch.empty_like(z)
        trimul_backward(z, mask, p, self.direction, dout, dz, g, stream)
        return dz, grads

    def forward_host(self, z_host, mask_host=None, out_host=None, stream=None):
        """End to end from host memory: copy z (and the mask) in, run, copy out back."""
        import torch
        s = stream or torch.cuda.current_stream()
        with torch.cuda.stream(s):
            z = z_host.to(self.device, non_blocking=True)
            mask = None if mask_host is None else mask_host.to(self.device, non_blocking=True)
            out = self(z, mask, stream=s)
            if out_host is None:
                out_host = torch.empty(out.shape, dtype=out.dtype, pin_memory=True)
            out_host.copy_(out, non_blocking=True)
        return out_host


class TriangleMultiplicationOutgoing(_TriangleMultiplication):
    """x_ij = sum_k a_ik * b_jk."""
    direction = OUTGOING


class TriangleMultiplicationIncoming(_TriangleMultiplication):
    """x_ij = sum_k a_ki * b_kj."""
    direction = INCOMING


# ---- the atom attention as a trainable layer ---------------------------------

class AtomAttention:
    """Windowed atom attention with its projections: x + W_o attention(W_q x, W_k x, W_v x) + b_o.

    x: [batch, n_atoms, c_atom] bf16; heads of 32 channels; bias and atom_mask as for
    atom_attention. The projections and the residual run in `linear`, the core in
    atom_attention; ``backward`` runs linear_backward and atom_attention_backward and keeps
    nothing of the forward but x, which may have been kept in 8 bits (act8_pack)."""

    KEYS = tuple(f"linear_{n}.{p}" for n in "qkvo" for p in ("weight", "bias"))

    def __init__(self, c_atom: int = 128, heads: int = 4):
        self.c_atom, self.heads = c_atom, heads
        self.tensors = {}

    def load_state_dict(self, sd: dict):
        """Take linear_q, linear_k, linear_v, linear_o .weight ([heads * 32, c_atom], o transposed) and,
        where present, .bias."""
        import torch
        c, d = self.c_atom, self.heads * 32
        t = {}
        for key in self.KEYS:
            out, inn = (c, d) if key.startswith("linear_o") else (d, c)
            if sd.get(key) is None:
                if key.endswith("weight"):
                    raise KeyError(key)
                continue
            v = sd[key] if isinstance(sd[key], torch.Tensor) else torch.as_tensor(sd[key])
            if tuple(v.shape) != ((out, inn) if key.endswith("weight") else (out,)):
                raise ValueError(f"{key}: shape {tuple(v.shape)}")
            t[key] = v
        self.tensors = t
        return self

    def to(self, device=None, dtype=None):
        import torch
        if dtype not in (None, torch.bfloat16):
            raise ValueError("dtype must be bfloat16")
        self.tensors = {k: v.to(device=device, dtype=torch.bfloat16).contiguous() for k, v in self.tensors.items()}
        return self

    def _linear(self, name, x, residual=None):
        return linear(x, self.tensors[f"linear_{name}.weight"], self.tensors.get(f"linear_{name}.bias"), residual)

    def _core(self, x, bias, atom_mask):
        shape = tuple(x.shape[:2]) + (self.heads, 32)
        q, k, v = (self._linear(n, x).view(shape) for n in "qkv")
        return q, k, v, _attention_core(q, k, v, bias, atom_mask)

    def _check(self, x):
        if len(x.shape) != 3 or x.shape[2] != self.c_atom:
            raise ValueError("x must be [batch, n_atoms, c_atom]")

    def __call__(self, x, bias=None, atom_mask=None):
        self._check(x)
        o = self._core(x, bias, atom_mask)[3]
        return self._linear("o", o.view(*x.shape[:2], self.heads * 32), residual=x)

    def backward(self, x, dout, bias=None, atom_mask=None):
        """Gradients of sum(layer(x, bias, atom_mask) * dout): (dx, dbias, {state-dict key: gradient}).

        x is the forward's input or the Act8 that kept it (the gradients are then those at the values it
        stands for). q, k, v and the attention's output are recomputed from it. Every parameter gets a
        gradient, biases the state dict left out included."""
        self._check(x)
        held = isinstance(x, Act8)
        q, k, v, o = self._core(act8_unpack(x) if held else x, bias, atom_mask)
        rows = tuple(x.shape[:2]) + (self.heads * 32,)
        grads = {}

        def back(name, inp, d):
            dx, grads[f"linear_{name}.weight"], grads[f"linear_{name}.bias"] = linear_backward(
                inp, self.tensors[f"linear_{name}.weight"], d, self.tensors.get(f"linear_{name}.bias"))
            return dx

        do = back("o", o.view(rows), dout).view(o.shape)
        dq, dk, dv, dbias = atom_attention_backward(q, k, v, do, bias, atom_mask)
        dx = dout.float()  # the residual's gradient; the four are added in fp32 and rounded once
        for name, d in (("q", dq), ("k", dk), ("v", dv)):
            dx += back(name, x, d.view(rows))
        return dx.to(dout.dtype), dbias, grads
