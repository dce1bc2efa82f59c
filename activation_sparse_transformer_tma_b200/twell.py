"""Thin ctypes binding of libtwell.so (argument marshalling only).

Every function here has the name of the C entry point it calls and does no
arithmetic of its own: it checks that the tensors are contiguous CUDA tensors,
packs their device pointers and sizes, calls the library on the current torch
stream, and raises ``TwellError`` on a non-OK status.  The small ``Twell`` and
``Hybrid`` classes only allocate the caller-owned buffers of the two sparse
formats with torch.  If the library cannot be loaded the first call raises:
there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtwell.so")

TW_F32, TW_BF16 = 0, 1
STATUS = ["TW_OK", "TW_ERR_INVALID_ARG", "TW_ERR_UNSUPPORTED", "TW_ERR_ALIGNMENT",
          "TW_ERR_CUDA", "TW_ERR_SPILL_CAPACITY", "TW_ERR_BACKUP_CAPACITY",
          "TW_ERR_TIMEOUT", "TW_ERR_WORKSPACE"]
EXPORTS = ["twell_gate_gemm", "twell_fused_updown_workspace_size", "twell_fused_updown",
           "twell_fused_updown_noalloc", "twell_ffn_small_batch_workspace_size",
           "twell_ffn_small_batch", "twell_to_hybrid", "hybrid_ffn_forward_workspace_size",
           "hybrid_ffn_forward",
           "hybrid_ffn_backward_workspace_size", "hybrid_ffn_backward", "dense_ffn_forward",
           "dense_ffn_train_workspace_size", "dense_ffn_train_saved_bytes",
           "dense_ffn_train_forward", "dense_ffn_train_backward",
           "gated_ffn_workspace_size", "gated_ffn_forward",
           "gated_ffn_backward_workspace_size", "gated_ffn_backward",
           "norm_residual_forward", "norm_residual_backward_workspace_size",
           "norm_residual_backward", "adamw_step",
           "tw_test_withhold_next_gate_loads", "tw_test_withhold_next_gated_ffn_loads",
           "tw_measure_row_gather", "tw_measure_stream_read", "tw_status_string",
           "twell_version"]


class TwellError(RuntimeError):
    def __init__(self, fn, code):
        name = STATUS[code] if 0 <= code < len(STATUS) else str(code)
        super().__init__(f"{fn} returned {name}")
        self.code = code


class TwTwellC(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("F", ctypes.c_int32), ("W", ctypes.c_int32),
                ("C", ctypes.c_int32), ("dtype", ctypes.c_int), ("val", ctypes.c_void_p),
                ("idx", ctypes.c_void_p), ("cnt", ctypes.c_void_p),
                ("spill_ref", ctypes.c_void_p), ("spill_cap", ctypes.c_int32),
                ("spill_tk", ctypes.c_void_p), ("spill_val", ctypes.c_void_p),
                ("spill_n", ctypes.c_void_p)]


class TwHybridC(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("F", ctypes.c_int32), ("C_h", ctypes.c_int32),
                ("dtype", ctypes.c_int), ("ell_g", ctypes.c_void_p), ("ell_u", ctypes.c_void_p),
                ("ell_idx", ctypes.c_void_p), ("row_nnz", ctypes.c_void_p),
                ("row_slot", ctypes.c_void_p), ("backup_cap", ctypes.c_int32),
                ("backup_rows", ctypes.c_void_p), ("backup_g", ctypes.c_void_p),
                ("backup_u", ctypes.c_void_p), ("n_backup", ctypes.c_void_p)]


class TwNormBlockC(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("gate_group", ctypes.c_int32),
                ("y_dtype", ctypes.c_int), ("r_dtype", ctypes.c_int), ("n_dtype", ctypes.c_int),
                ("w_dtype", ctypes.c_int), ("res_scale", ctypes.c_float),
                ("block_scale", ctypes.c_float), ("eps", ctypes.c_float),
                ("w_post", ctypes.c_void_p), ("gate", ctypes.c_void_p),
                ("w_pre", ctypes.c_void_p)]


class TwAdamwTensorC(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("p", ctypes.c_void_p), ("master", ctypes.c_void_p),
                ("g", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
                ("m_values", ctypes.c_void_p), ("v_values", ctypes.c_void_p),
                ("p_dtype", ctypes.c_int), ("g_dtype", ctypes.c_int),
                ("values_dtype", ctypes.c_int), ("state_bits", ctypes.c_int32),
                ("weight_decay", ctypes.c_double)]


class TwAdamwArgsC(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("step", ctypes.c_int32), ("lr_dev", ctypes.c_void_p),
                ("step_dev", ctypes.c_void_p), ("grad_scale", ctypes.c_void_p)]


_lib = None


def lib():
    """Load libtwell.so once; raise if it is missing (no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m activation_sparse_transformer_tma_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, st = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int
        PT, PH = ctypes.POINTER(TwTwellC), ctypes.POINTER(TwHybridC)
        L.twell_gate_gemm.argtypes = [vp, vp, i32, i32, i32, ctypes.c_int, PT, vp, vp, vp]
        L.twell_fused_updown_workspace_size.argtypes = [i32, i32]
        L.twell_fused_updown_workspace_size.restype = ctypes.c_size_t
        L.twell_fused_updown.argtypes = [vp, PT, vp, vp, i32, vp, ctypes.c_int, vp,
                                         ctypes.c_size_t, vp, vp]
        L.twell_fused_updown_noalloc.argtypes = [vp, PT, vp, vp, i32, vp, ctypes.c_int, vp, vp]
        L.twell_fused_updown_noalloc.restype = st
        L.twell_ffn_small_batch_workspace_size.argtypes = [i32, i32, i32]
        L.twell_ffn_small_batch_workspace_size.restype = ctypes.c_size_t
        L.twell_ffn_small_batch.argtypes = [vp, vp, vp, vp, i32, i32, i32, PT, vp, vp,
                                            ctypes.c_int, vp, ctypes.c_size_t, vp, vp]
        L.twell_to_hybrid.argtypes = [PT, PH, vp, vp]
        L.hybrid_ffn_forward_workspace_size.argtypes = [i32, i32]
        L.hybrid_ffn_forward_workspace_size.restype = ctypes.c_size_t
        L.hybrid_ffn_forward.argtypes = [vp, PH, vp, vp, i32, vp, ctypes.c_int, vp,
                                         ctypes.c_size_t, vp, vp]
        L.hybrid_ffn_backward_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        L.hybrid_ffn_backward_workspace_size.restype = ctypes.c_size_t
        L.hybrid_ffn_backward.argtypes = [vp, vp, PH, vp, vp, vp, i32, ctypes.c_float, vp,
                                          ctypes.c_int, vp, vp, vp, vp, ctypes.c_size_t, vp, vp]
        L.dense_ffn_forward.argtypes = [vp, vp, vp, vp, i32, i32, i32, vp, vp, vp, vp]
        L.dense_ffn_train_workspace_size.argtypes = [i32, i32]
        L.dense_ffn_train_workspace_size.restype = ctypes.c_size_t
        L.dense_ffn_train_saved_bytes.argtypes = [i32, i32]
        L.dense_ffn_train_saved_bytes.restype = ctypes.c_size_t
        L.dense_ffn_train_forward.argtypes = [vp, vp, vp, vp, i32, i32, i32, vp, ctypes.c_size_t,
                                              vp, vp, vp]
        L.dense_ffn_train_backward.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, ctypes.c_float,
                                               vp, ctypes.c_size_t, vp, vp, vp, vp, vp, vp]
        sz, ci = ctypes.c_size_t, ctypes.c_int
        for name in ("gated_ffn_workspace_size", "gated_ffn_backward_workspace_size"):
            getattr(L, name).argtypes = [i32, i32, i32]
            getattr(L, name).restype = sz
        L.gated_ffn_forward.argtypes = [vp, vp, vp, vp, i32, i32, i32, ci, vp, vp, vp, ci, vp, sz,
                                        vp, vp]
        L.gated_ffn_backward.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, ci, vp, vp, vp, ci, vp,
                                         vp, vp, ci, vp, sz, vp, vp]
        PN = ctypes.POINTER(TwNormBlockC)
        L.norm_residual_forward.argtypes = [PN, vp, vp, vp, vp, vp, vp, vp]
        L.norm_residual_backward_workspace_size.argtypes = [i32, i32, i32]
        L.norm_residual_backward_workspace_size.restype = ctypes.c_size_t
        L.norm_residual_backward.argtypes = [PN, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                             ctypes.c_size_t, vp]
        L.adamw_step.argtypes = [ctypes.POINTER(TwAdamwTensorC), i32,
                                 ctypes.POINTER(TwAdamwArgsC), vp]
        L.tw_test_withhold_next_gate_loads.argtypes = [ctypes.c_uint64]
        L.tw_test_withhold_next_gate_loads.restype = None
        L.tw_test_withhold_next_gated_ffn_loads.argtypes = [ctypes.c_uint64]
        L.tw_test_withhold_next_gated_ffn_loads.restype = None
        L.tw_measure_row_gather.argtypes = [vp, i32, i32, ctypes.c_int64, ctypes.c_uint32, vp,
                                            vp]
        L.tw_measure_row_gather.restype = st
        L.tw_measure_stream_read.argtypes = [vp, ctypes.c_int64, vp, vp]
        L.tw_measure_stream_read.restype = st
        L.tw_status_string.argtypes = [st]
        L.tw_status_string.restype = ctypes.c_char_p
        L.twell_version.restype = i32
        for name in ("twell_gate_gemm", "twell_fused_updown", "twell_ffn_small_batch",
                     "twell_to_hybrid",
                     "hybrid_ffn_forward", "hybrid_ffn_backward", "dense_ffn_forward",
                     "dense_ffn_train_forward", "dense_ffn_train_backward",
                     "gated_ffn_forward", "gated_ffn_backward", "norm_residual_forward",
                     "norm_residual_backward", "adamw_step"):
            getattr(L, name).restype = st
        _lib = L
    return _lib


# ------------------------------------------------------------------ helpers --
_DTYPE_CODES = {torch.bfloat16: TW_BF16, torch.float32: TW_F32, None: TW_F32}  # None: absent


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return TW_BF16
    if t.dtype == torch.float32:
        return TW_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _torch_dtype(code: int):
    return torch.bfloat16 if code == TW_BF16 else torch.float32


def _ptr(t):
    if t is None:
        return None
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("tensors passed to libtwell must be contiguous CUDA tensors")
    return t.data_ptr()


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def _check(fn, code):
    if code != 0:
        raise TwellError(fn, code)


def _addresses(*tensors):
    """The index of the one CUDA device of the tensors, and their addresses (None
    for None)."""
    index, out = None, []
    for t in tensors:
        if t is None:
            out.append(None)
            continue
        i = t.get_device()
        if i < 0 or not t.is_contiguous():
            raise ValueError("tensors passed to libtwell must be contiguous CUDA tensors")
        if i != index:
            if index is not None:
                raise ValueError("tensors passed to libtwell must be on one device")
            index = i
        out.append(t.data_ptr())
    return index, out


def _call_on(index, fn, stream, *args):
    """lib().<fn>(*args, stream) with device `index` current, on its current
    stream unless one is given."""
    f = getattr(_lib or lib(), fn)
    if stream is None:
        # the address alone: building a Stream object costs as much as a launch
        raw = torch._C._cuda_getCurrentRawStream(index)
    elif stream.device.index != index:
        raise ValueError("the stream and the tensors are on different devices")
    else:
        raw = stream.cuda_stream
    if torch.cuda.current_device() == index:
        code = f(*args, raw)
    else:
        with torch.cuda.device(index):
            code = f(*args, raw)
    if code != 0:
        raise TwellError(fn, code)


class Twell:
    """Caller-owned buffers of one TwELL tensor (tile-major, W = 128)."""

    def __init__(self, T, F, C, dtype=torch.bfloat16, spill_cap=None, device="cuda", W=128):
        K = F // W
        if spill_cap is None:
            spill_cap = max(1024, (K * T) // 16)
        self.T, self.F, self.W, self.C, self.spill_cap = T, F, W, C, spill_cap
        self.dtype = dtype
        self.val = torch.zeros((K, T, C), dtype=dtype, device=device) if C else None
        self.idx = torch.zeros((K, T, C), dtype=torch.uint8, device=device) if C else None
        self.cnt = torch.zeros((K, T), dtype=torch.uint8, device=device)
        self.spill_ref = torch.full((K, T), -1, dtype=torch.int32, device=device)
        self.spill_tk = torch.zeros((max(spill_cap, 1), 2), dtype=torch.int32, device=device)
        self.spill_val = torch.zeros((max(spill_cap, 1), W), dtype=dtype, device=device)
        self.spill_n = torch.zeros(1, dtype=torch.int32, device=device)

    def struct(self):
        return TwTwellC(self.T, self.F, self.W, self.C, _dt(self.spill_val), _ptr(self.val),
                        _ptr(self.idx), _ptr(self.cnt), _ptr(self.spill_ref), self.spill_cap,
                        _ptr(self.spill_tk), _ptr(self.spill_val), _ptr(self.spill_n))


class Hybrid:
    """Caller-owned buffers of one hybrid tensor (ELL part + dense backup rows)."""

    def __init__(self, T, F, C_h, dtype=torch.bfloat16, backup_cap=None, device="cuda"):
        if backup_cap is None:
            backup_cap = max(64, T // 8)
        self.T, self.F, self.C_h, self.backup_cap = T, F, C_h, backup_cap
        self.dtype = dtype
        self.ell_g = torch.zeros((T, C_h), dtype=dtype, device=device)
        self.ell_u = torch.zeros((T, C_h), dtype=dtype, device=device)
        self.ell_idx = torch.zeros((T, C_h), dtype=torch.int16, device=device)
        self.row_nnz = torch.zeros(T, dtype=torch.int32, device=device)
        self.row_slot = torch.zeros(T, dtype=torch.int32, device=device)
        self.backup_rows = torch.zeros(max(backup_cap, 1), dtype=torch.int32, device=device)
        self.backup_g = torch.zeros((max(backup_cap, 1), F), dtype=dtype, device=device)
        self.backup_u = torch.zeros((max(backup_cap, 1), F), dtype=dtype, device=device)
        self.n_backup = torch.zeros(1, dtype=torch.int32, device=device)

    def struct(self):
        e = self.ell_g if self.C_h else None
        return TwHybridC(self.T, self.F, self.C_h, _dt(self.backup_g), _ptr(e),
                         _ptr(self.ell_u if self.C_h else None),
                         _ptr(self.ell_idx if self.C_h else None), _ptr(self.row_nnz),
                         _ptr(self.row_slot), self.backup_cap, _ptr(self.backup_rows),
                         _ptr(self.backup_g), _ptr(self.backup_u), _ptr(self.n_backup))


# ------------------------------------------------------------- entry points --
def twell_gate_gemm(x, Wg_t, out: Twell, g_dense_dump=None, dev_status=None, stream=None):
    T, d = x.shape
    F = Wg_t.shape[0]
    s = out.struct()
    _check("twell_gate_gemm", lib().twell_gate_gemm(
        _ptr(x), _ptr(Wg_t), T, d, F, _dt(x), ctypes.byref(s), _ptr(g_dense_dump),
        _ptr(dev_status), _stream(stream)))


def twell_fused_updown_workspace_size(T, d):
    return int(lib().twell_fused_updown_workspace_size(T, d))


def fused_workspace(T, d, device="cuda"):
    """A caller-owned workspace tensor of the size twell_fused_updown needs."""
    return torch.empty(twell_fused_updown_workspace_size(T, d), dtype=torch.uint8, device=device)


def twell_fused_updown(x, g: Twell, Wu_t, Wd, y, ws, dev_status=None, stream=None):
    s = g.struct()
    _check("twell_fused_updown", lib().twell_fused_updown(
        _ptr(x), ctypes.byref(s), _ptr(Wu_t), _ptr(Wd), x.shape[1], _ptr(y), _dt(y), _ptr(ws),
        ws.numel() * ws.element_size(), _ptr(dev_status), _stream(stream)))


def twell_fused_updown_noalloc(x, g: Twell, Wu_t, Wd, y, dev_status=None, stream=None):
    """twell_fused_updown for callers that cannot allocate a workspace: the
    library uses its own fixed device array (see include/twell.h)."""
    s = g.struct()
    _check("twell_fused_updown_noalloc", lib().twell_fused_updown_noalloc(
        _ptr(x), ctypes.byref(s), _ptr(Wu_t), _ptr(Wd), x.shape[1], _ptr(y), _dt(y),
        _ptr(dev_status), _stream(stream)))


def twell_ffn_small_batch_workspace_size(T, d, F):
    return int(lib().twell_ffn_small_batch_workspace_size(T, d, F))


def small_batch_workspace(T, d, F, device="cuda"):
    """A zero-filled workspace for twell_ffn_small_batch (its barrier counters
    must start at zero; each call leaves them at zero)."""
    return torch.zeros(twell_ffn_small_batch_workspace_size(T, d, F), dtype=torch.uint8,
                       device=device)


def twell_ffn_small_batch(x, Wg_t, Wu_t, Wd, g: Twell, y, ws, g_dense_dump=None, dev_status=None,
                          stream=None):
    T, d = x.shape
    F = Wg_t.shape[0]
    s = g.struct()
    _check("twell_ffn_small_batch", lib().twell_ffn_small_batch(
        _ptr(x), _ptr(Wg_t), _ptr(Wu_t), _ptr(Wd), T, d, F, ctypes.byref(s), _ptr(g_dense_dump),
        _ptr(y), _dt(y), _ptr(ws), ws.numel() * ws.element_size(), _ptr(dev_status),
        _stream(stream)))


def twell_to_hybrid(g: Twell, out: Hybrid, dev_status=None, stream=None):
    sg, sh = g.struct(), out.struct()
    _check("twell_to_hybrid", lib().twell_to_hybrid(
        ctypes.byref(sg), ctypes.byref(sh), _ptr(dev_status), _stream(stream)))


def hybrid_ffn_forward_workspace_size(T, d):
    return int(lib().hybrid_ffn_forward_workspace_size(T, d))


def hybrid_ffn_forward(x, gu: Hybrid, Wu_t, Wd, y, ws=None, dev_status=None, stream=None):
    """ws: caller-owned workspace (hybrid_ffn_forward_workspace_size bytes);
    when None, one is allocated with torch for this call."""
    if ws is None:
        ws = torch.empty(hybrid_ffn_forward_workspace_size(x.shape[0], x.shape[1]),
                         dtype=torch.uint8, device=x.device)
    s = gu.struct()
    _check("hybrid_ffn_forward", lib().hybrid_ffn_forward(
        _ptr(x), ctypes.byref(s), _ptr(Wu_t), _ptr(Wd), x.shape[1], _ptr(y), _dt(y), _ptr(ws),
        ws.numel() * ws.element_size(), _ptr(dev_status), _stream(stream)))


def hybrid_ffn_backward_workspace_size(T, d, F, C_h, backup_cap):
    return int(lib().hybrid_ffn_backward_workspace_size(T, d, F, C_h, backup_cap))


def hybrid_ffn_backward(x, dy, gu: Hybrid, Wg_t, Wu_t, Wd, l1_lambda, dx, dWg_t, dWu_t, dWd, ws,
                        dev_status=None, stream=None):
    s = gu.struct()
    _check("hybrid_ffn_backward", lib().hybrid_ffn_backward(
        _ptr(x), _ptr(dy), ctypes.byref(s), _ptr(Wg_t), _ptr(Wu_t), _ptr(Wd), x.shape[1],
        float(l1_lambda), _ptr(dx), _dt(dx), _ptr(dWg_t), _ptr(dWu_t), _ptr(dWd), _ptr(ws),
        ws.numel() * ws.element_size(), _ptr(dev_status), _stream(stream)))


def dense_ffn_forward(x, Wg_t, Wu_t, Wd_dense, h_ws, y, dev_status=None, stream=None):
    T, d = x.shape
    F = Wg_t.shape[0]
    _check("dense_ffn_forward", lib().dense_ffn_forward(
        _ptr(x), _ptr(Wg_t), _ptr(Wu_t), _ptr(Wd_dense), T, d, F, _ptr(h_ws), _ptr(y),
        _ptr(dev_status), _stream(stream)))


def dense_ffn_train_workspace_size(T, F):
    return int(lib().dense_ffn_train_workspace_size(T, F))


def dense_ffn_train_saved_bytes(T, F):
    return int(lib().dense_ffn_train_saved_bytes(T, F))


def dense_train_workspace(T, F, device="cuda"):
    """A caller-owned workspace tensor for the dense training comparator."""
    return torch.empty(dense_ffn_train_workspace_size(T, F), dtype=torch.uint8, device=device)


def dense_ffn_train_forward(x, Wg_t, Wu_t, Wd, ws, y, dev_status=None, stream=None):
    T, d = x.shape
    F = Wg_t.shape[0]
    _check("dense_ffn_train_forward", lib().dense_ffn_train_forward(
        _ptr(x), _ptr(Wg_t), _ptr(Wu_t), _ptr(Wd), T, d, F, _ptr(ws),
        ws.numel() * ws.element_size(), _ptr(y), _ptr(dev_status), _stream(stream)))


def dense_ffn_train_backward(x, dy, Wg_t, Wu_t, Wd, l1_lambda, ws, dx, dWg_t, dWu_t, dWd,
                             dev_status=None, stream=None):
    T, d = x.shape
    F = Wg_t.shape[0]
    _check("dense_ffn_train_backward", lib().dense_ffn_train_backward(
        _ptr(x), _ptr(dy), _ptr(Wg_t), _ptr(Wu_t), _ptr(Wd), T, d, F, float(l1_lambda),
        _ptr(ws), ws.numel() * ws.element_size(), _ptr(dx), _ptr(dWg_t), _ptr(dWu_t), _ptr(dWd),
        _ptr(dev_status), _stream(stream)))


def dense_train_saved(ws, T, F):
    """Views of the g, u, h [T][F] bf16 tensors the training forward saved in ws."""
    part = (T * F * 2 + 255) // 256 * 256
    return [ws[i * part:i * part + T * F * 2].view(torch.bfloat16).view(T, F) for i in range(3)]


ACTIVATIONS = {"relu": 0, "silu": 1, "gelu": 2, "gelu_tanh": 3}


def _all_bf16(*tensors):
    for t in tensors:
        if t is not None and t.dtype != torch.bfloat16:
            raise TypeError(f"bf16 expected, got {t.dtype}")


def _dtype_code(t):
    try:
        return _DTYPE_CODES[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}") from None


def _activation(act):
    if act not in ACTIVATIONS:
        raise ValueError(f"act is one of {sorted(ACTIVATIONS)}, not {act!r}")
    return ACTIVATIONS[act]


_INT32_MAX = 2 ** 31 - 1


def _int32(*values):
    """Refuses what ctypes would cut to 32 bits in silence."""
    for v in values:
        if not -_INT32_MAX <= v <= _INT32_MAX:
            raise ValueError(f"{v} does not fit 32 bits")


def _gate_group(group):
    """T or more is one group: a sentinel past 32 bits stays one."""
    return min(group, _INT32_MAX)


def _check_ffn(x, Wg_t, Wu_t, Wd):
    T, d = x.shape
    F = Wg_t.shape[0]
    if T > _INT32_MAX or d > _INT32_MAX or F > _INT32_MAX:
        _int32(T, d, F)
    for w in (Wg_t, Wu_t, Wd):
        if w.shape != (F, d):
            raise ValueError(f"weights of {tuple(w.shape)} and {(F, d)} for rows of {d}")
    _all_bf16(x, Wg_t, Wu_t, Wd)
    return T, d, F


def gated_ffn_workspace_size(T, d, F):
    _int32(T, d, F)
    return int(lib().gated_ffn_workspace_size(T, d, F))


def gated_ffn_backward_workspace_size(T, d, F):
    _int32(T, d, F)
    return int(lib().gated_ffn_backward_workspace_size(T, d, F))


def gated_ffn_workspace(T, d, F, training=False, device="cuda"):
    """A caller-owned workspace tensor for gated_ffn_forward, and with `training`
    for gated_ffn_backward too."""
    with torch.cuda.device(device):
        size = gated_ffn_workspace_size(T, d, F)
        if training:
            size = max(size, gated_ffn_backward_workspace_size(T, d, F))
    return torch.empty(size, dtype=torch.uint8, device=device)


def gated_ffn_forward(x, Wg_t, Wu_t, Wd, act, y, ws, z=None, u=None, dev_status=None, stream=None):
    """y = (act(x Wg) * (x Wu)) Wd for x [T, d] and weights [F, d], all bf16; act is a key of
    ACTIVATIONS, y bf16 or fp32.  z and u [T, F] bf16 keep what gated_ffn_backward needs."""
    index, (xp, gp, up, dp, yp, wsp, zp, usp, sp) = _addresses(x, Wg_t, Wu_t, Wd, y, ws, z, u,
                                                               dev_status)
    T, d, F = _check_ffn(x, Wg_t, Wu_t, Wd)
    _all_bf16(z, u)
    _same_shape(x, y)
    for t in (z, u):
        if t is not None and t.shape != (T, F):
            raise ValueError(f"z and u of {(T, F)} expected, got {tuple(t.shape)}")
    _call_on(index, "gated_ffn_forward", stream, xp, gp, up, dp, T, d, F, _activation(act), zp, usp,
             yp, _dtype_code(y), wsp, ws.numel() * ws.element_size(), sp)


def gated_ffn_backward(x, dy, Wg_t, Wu_t, Wd, act, z, u, dx, dWg_t, dWu_t, dWd, ws,
                       dev_status=None, stream=None):
    """Gradients of gated_ffn_forward: dx [T, d] and dWg_t, dWu_t, dWd [F, d], bf16 or fp32, from
    dy [T, d] bf16 and the saved z and u."""
    index, (xp, dyp, gp, up, dp, zp, usp, dxp, dgp, dup, ddp, wsp, sp) = _addresses(
        x, dy, Wg_t, Wu_t, Wd, z, u, dx, dWg_t, dWu_t, dWd, ws, dev_status)
    T, d, F = _check_ffn(x, Wg_t, Wu_t, Wd)
    _all_bf16(dy, z, u)
    _same_shape(x, dy, dx)
    _same_shape(Wg_t, dWg_t, dWu_t, dWd)
    if z.shape != (T, F) or u.shape != (T, F):
        raise ValueError(f"z and u of {(T, F)} expected")
    if dWg_t.dtype != dWu_t.dtype or dWg_t.dtype != dWd.dtype:
        raise TypeError("the weight gradients differ in dtype")
    _call_on(index, "gated_ffn_backward", stream, xp, dyp, gp, up, dp, T, d, F, _activation(act),
             zp, usp, dxp, _dtype_code(dx), dgp, dup, ddp, _dtype_code(dWg_t), wsp,
             ws.numel() * ws.element_size(), sp)


def _norm_block(T, d, y_dtype, r_dtype, n_dtype, weights, addresses, gate_group, res_scale,
                block_scale, eps):
    """The shared descriptor of a norm call; weights and addresses of (w_post, gate, w_pre)."""
    w_dtype = None
    if T > _INT32_MAX or d > _INT32_MAX or gate_group > _INT32_MAX:
        _int32(T, d)
        gate_group = _gate_group(gate_group)
    for k, w in enumerate(weights):
        if w is None:
            continue
        rows = 1 if k != 1 else -(-T // gate_group) if gate_group > 0 else 0
        if w.numel() != rows * d:
            raise ValueError(f"a weight of {w.numel()} elements for {rows} rows of {d}")
        if w_dtype is None:
            w_dtype = w.dtype
        elif w.dtype != w_dtype:
            raise TypeError("w_post, gate and w_pre differ in dtype")
    code = _DTYPE_CODES
    try:
        return TwNormBlockC(T, d, gate_group, code[y_dtype], code[r_dtype], code[n_dtype],
                            code[w_dtype], res_scale, block_scale, eps, *addresses)
    except KeyError as e:
        raise TypeError(f"unsupported dtype {e.args[0]}") from None


def _dtype_of(t):
    return None if t is None else t.dtype


def _same_shape(like, *tensors):
    for t in tensors:
        if t is not None and t.shape != like.shape:
            raise ValueError(f"shape {tuple(t.shape)} beside {tuple(like.shape)}")


def _floats(n, *tensors):
    for t in tensors:
        if t is not None and (t.dtype != torch.float32 or t.numel() != n):
            raise ValueError(f"{n} fp32 elements expected, got {t.numel()} of {t.dtype}")


def norm_residual_forward(y, r, w_post, gate, w_pre, r_out, n_out, *, gate_group=0, res_scale=1.0,
                          block_scale=1.0, eps=1e-6, rstd_post=None, rstd_pre=None, stream=None):
    """r_out = res_scale r + block_scale gate norm(y) w_post and n_out = norm(r_out) w_pre, per
    token of [T, d] tensors.  w_post, w_pre [d], gate [ceil(T / gate_group), d]; any of them may
    be None, and y and r_out for the first norm of a network.  rstd_post, rstd_pre [T] fp32 keep
    what norm_residual_backward needs."""
    index, (yp, rp, wpost, gp, wpre, rop, nop, pp, qp) = _addresses(
        y, r, w_post, gate, w_pre, r_out, n_out, rstd_post, rstd_pre)
    _same_shape(r, y, r_out, n_out)
    if r_out is not None and r_out.dtype != r.dtype:
        raise TypeError("r and r_out differ in dtype")
    T, d = r.shape
    _floats(T, rstd_post, rstd_pre)
    b = _norm_block(T, d, _dtype_of(y), r.dtype, _dtype_of(n_out), (w_post, gate, w_pre),
                    (wpost, gp, wpre), gate_group, res_scale, block_scale, eps)
    _call_on(index, "norm_residual_forward", stream, ctypes.byref(b), yp, rp, rop, nop, pp, qp)


def norm_residual_backward_workspace_size(T, d, gate_group=0):
    _int32(T, d)
    return int(lib().norm_residual_backward_workspace_size(T, d, _gate_group(gate_group)))


def norm_residual_backward_workspace(T, d, gate_group=0, device="cuda"):
    """A caller-owned workspace tensor for norm_residual_backward."""
    with torch.cuda.device(device):
        size = norm_residual_backward_workspace_size(T, d, gate_group)
    return torch.empty(size, dtype=torch.uint8, device=device)


def norm_residual_backward(dn, dr_out, y, r_out, w_post, gate, w_pre, rstd_post, rstd_pre, dy, dr,
                           dw_post, dgate, dw_pre, ws, *, gate_group=0, res_scale=1.0,
                           block_scale=1.0, stream=None):
    """Gradients of norm_residual_forward: dy, dr [T, d], dw_post, dw_pre [d] and dgate like gate
    (fp32), from dn and dr_out, the gradients of n_out and r_out (either may be None; dn is None
    exactly when w_pre is)."""
    index, (dnp, drop, yp, rop, wpost, gp, wpre, pp, qp, dyp, drp, dwpost, dgp, dwpre, wsp) = \
        _addresses(dn, dr_out, y, r_out, w_post, gate, w_pre, rstd_post, rstd_pre, dy, dr, dw_post,
                   dgate, dw_pre, ws)
    _same_shape(dr, dn, dr_out, y, r_out, dy)
    for a, b in ((dr_out, dr), (r_out, dr), (dy, y)):
        if a is not None and b is not None and a.dtype != b.dtype:
            raise TypeError("a gradient differs in dtype from its tensor")
    T, d = dr.shape
    _floats(T, rstd_post, rstd_pre)
    _floats(d, dw_post, dw_pre)
    if dgate is not None:
        _floats(0 if gate is None else gate.numel(), dgate)
    b = _norm_block(T, d, _dtype_of(y), dr.dtype, _dtype_of(dn), (w_post, gate, w_pre),
                    (wpost, gp, wpre), gate_group, res_scale, block_scale, 0.0)
    _call_on(index, "norm_residual_backward", stream, ctypes.byref(b), dnp, drop, yp, rop, pp, qp,
             dyp, drp, dwpost, dgp, dwpre, wsp, ws.numel() * ws.element_size())


ADAMW_BLOCK = 256  # elements that share one scale of an 8-bit moment


class AdamWTensors:
    """The tensors of an AdamW step, packed once for many steps.

    ``tensors``: mappings with p, g (bf16 or fp32), m, v and optionally master
    (fp32, for a bf16 p), weight_decay (default 0), and for 8-bit moments
    (m int8, v uint8) m_scale and v_scale (fp32, ``adamw_blocks(n)`` long) and
    m_values, v_values, which receive what the new codes stand for.  The
    tensors stay referenced; a program that puts another storage behind one of
    them builds a new list."""

    def __init__(self, tensors):
        tensors = [dict(t) for t in tensors]
        self._c = (TwAdamwTensorC * max(len(tensors), 1))()
        self.count = len(tensors)
        self._keep = []
        for c, t in zip(self._c, tensors):
            self._pack(c, t)
        self.device = None
        if self._keep:
            index, _ = _addresses(*[x for t, _ in self._keep for x in t])
            self.device = torch.device("cuda", index)
        self._args = TwAdamwArgsC()

    def _pack(self, c, t):
        names = ("p", "master", "g", "m", "v", "m_scale", "v_scale", "m_values", "v_values")
        unknown = set(t) - set(names) - {"weight_decay"}
        if unknown:
            raise TypeError(f"unknown keys {sorted(unknown)}")
        get = {k: t.get(k) for k in names}
        for k in ("p", "g", "m", "v"):
            if get[k] is None:
                raise ValueError(f"{k} is missing")
        n = get["p"].numel()
        small = get["m"].dtype == torch.int8
        want = {"master": torch.float32, "m": torch.int8 if small else torch.float32,
                "v": torch.uint8 if small else torch.float32,
                "m_scale": torch.float32, "v_scale": torch.float32}
        given = {k: x for k, x in get.items() if x is not None}
        for k, x in given.items():
            if k in want and x.dtype != want[k]:
                raise TypeError(f"{k} is {x.dtype}, not {want[k]}")
            if x.numel() != (adamw_blocks(n) if k.endswith("_scale") else n):
                raise ValueError(f"{k} has {x.numel()} elements for a parameter of {n}")
        for k, x in given.items():
            setattr(c, k, _ptr(x))
        c.n = n
        c.p_dtype, c.g_dtype = _dt(get["p"]), _dt(get["g"])
        if get["m_values"] is not None:
            c.values_dtype = _dt(get["m_values"])
            if get["v_values"] is not None and get["v_values"].dtype != get["m_values"].dtype:
                raise TypeError("m_values and v_values differ in dtype")
        c.state_bits = 8 if small else 32
        c.weight_decay = float(t.get("weight_decay", 0.0))
        held = list(given.values())
        # the storages too: an address in the list must not outlive its memory
        self._keep.append((held, [x.untyped_storage() for x in held]))


def adamw_blocks(n):
    """Block scales of an 8-bit moment of n elements."""
    return (n + ADAMW_BLOCK - 1) // ADAMW_BLOCK


def adamw_step(tensors: AdamWTensors, *, lr, beta1=0.9, beta2=0.999, eps=1e-8, step=1, lr_dev=None,
               step_dev=None, grad_scale=None, stream=None):
    """One AdamW step over all tensors of the list, in one launch for up to 256
    of them.  lr_dev (fp32), step_dev (int32) and grad_scale (fp32) are device
    tensors of one element that a captured step reads at each replay."""
    if tensors.count == 0:
        return
    if not 0 <= step <= _INT32_MAX:
        _int32(step)
    for x, dtype in ((lr_dev, torch.float32), (step_dev, torch.int32),
                     (grad_scale, torch.float32)):
        if x is not None and (x.dtype != dtype or x.numel() != 1 or x.device != tensors.device):
            raise ValueError(f"device scalars are one {dtype} on {tensors.device}")
    a = tensors._args
    a.lr, a.beta1, a.beta2, a.eps, a.step = lr, beta1, beta2, eps, step
    a.lr_dev, a.step_dev, a.grad_scale = _ptr(lr_dev), _ptr(step_dev), _ptr(grad_scale)
    _call_on(tensors.device.index, "adamw_step", stream, tensors._c, tensors.count, ctypes.byref(a))


def status_bits(dev_status) -> list:
    """Names of the device-side conditions set in a status word tensor."""
    v = int(dev_status.item())
    return [STATUS[i] for i in range(len(STATUS)) if v & (1 << i)]


def measure_row_gather(mat, n_gathers, seed, checksum, stream=None):
    """Measurement aid (not part of the FFN): n_gathers scattered whole rows of
    the bf16 matrix mat [rows][d]; checksum (an int32 tensor, zeroed by the
    caller) receives the XOR of every 32-bit word read."""
    rows, d = mat.shape
    _check("tw_measure_row_gather", lib().tw_measure_row_gather(
        _ptr(mat), rows, d, int(n_gathers), int(seed) & 0xFFFFFFFF, _ptr(checksum), _stream(stream)))


def measure_stream_read(buf, checksum, stream=None):
    """Measurement aid (not part of the FFN): one launch that reads the whole
    device tensor buf front to back; checksum (an int32 tensor, zeroed by the
    caller) receives the XOR of every 32-bit word read."""
    _check("tw_measure_stream_read", lib().tw_measure_stream_read(
        _ptr(buf), buf.numel() * buf.element_size(), _ptr(checksum), _stream(stream)))
