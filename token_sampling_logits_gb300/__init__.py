"""gsample: batch Gumbel-max / HLG token sampling on GB300 (sm_103a).

Thin ctypes binding over the C ABI of ``libgsample.so`` (declared in
``include/gsample.h``). Every step of the sampling runs in the library's CUDA
kernels; this module only checks tensors, passes device pointers and the
current CUDA stream, and turns status codes into exceptions. PyTorch supplies
device memory and streams.

    import torch, token_sampling_logits_gb300 as gs
    idx = gs.gumbel_argmax(logits, temperature, seed, offset)   # int64 [B]

All calls are asynchronous on ``torch.cuda.current_stream()``.
"""
from __future__ import annotations

import ctypes
import operator
import os
import threading
from dataclasses import dataclass

from . import build as _build

__all__ = [
    "GSampleError", "HlgParams", "PIVOT_TOP", "PIVOT_ENTROPY", "F32", "BF16", "F16",
    "lib", "library_path", "workspace_bytes", "workspace_init", "new_workspace", "argmax",
    "gumbel_argmax", "hlg_gumbel_argmax", "hlg_gumbel_argmax_rows", "hlg_rows_tensor",
    "categorical", "filtered_gumbel_argmax", "status_string", "LogitState", "new_logit_state",
    "state_reset", "history_append", "bias_set", "process_logits", "constrained_gumbel_argmax",
]

F32, BF16, F16 = 0, 1, 2
PIVOT_TOP, PIVOT_ENTROPY = 0, 1
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA = 0, 1, 2, 3, 4

_i64 = ctypes.c_int64
_i32 = ctypes.c_int32
_u32 = ctypes.c_uint32
_u64 = ctypes.c_uint64
_vp = ctypes.c_void_p
_int = ctypes.c_int


class _HlgParamsC(ctypes.Structure):
    _fields_ = [("m", ctypes.c_float), ("w", ctypes.c_float), ("beta_t", ctypes.c_float),
                ("beta_h", ctypes.c_float), ("pivot_offset", ctypes.c_float),
                ("pivot_mode", ctypes.c_int32)]


class _StateC(ctypes.Structure):
    _fields_ = [("history", _vp), ("bias", _vp), ("touched", _vp), ("rows", _i64),
                ("vocab", _i64), ("ld", _i64)]


class _ConstraintsC(ctypes.Structure):
    # state: the address of a _StateC that outlives the call
    _fields_ = [("state", _vp), ("slot", _vp), ("repetition", _vp),
                ("frequency", _vp), ("presence", _vp), ("mask", _vp), ("mask_rows", _i64),
                ("mask_ld", _i64), ("mask_row", _vp)]


@dataclass(frozen=True)
class HlgParams:
    """HLG tone-curve knobs in nats ("HLG sampling", "The transfer function"
    and "The pivot"). w = inf turns the rolloff off."""
    m: float = 1.0
    w: float = 4.0
    beta_t: float = 6.0
    beta_h: float = 4.0
    pivot_offset: float = 6.0
    pivot_mode: int = PIVOT_TOP

    def to_c(self) -> _HlgParamsC:
        return _HlgParamsC(self.m, self.w, self.beta_t, self.beta_h, self.pivot_offset,
                           self.pivot_mode)


class GSampleError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__("%s failed: %s" % (what, status_string(status)))
        self.status = status


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB


def lib() -> ctypes.CDLL:
    """Load libgsample.so (building it first if its sources are newer).
    Raises if the library cannot be built or loaded: there is no fallback."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.build() if _build.is_stale() else _build.LIB
        L = ctypes.CDLL(path)
        sigs = {
            "gsample_workspace_bytes": (ctypes.c_size_t, [_i64]),
            "gsample_workspace_init": (_int, [_vp, _i64, _vp]),
            "gsample_argmax": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp]),
            "gsample_gumbel_argmax": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp,
                                             _vp]),
            "gsample_hlg_gumbel_argmax": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _vp,
                                                 _vp, _vp, _vp]),
            "gsample_hlg_gumbel_argmax_rows": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp,
                                                      _vp, _vp, _vp, _vp]),
            "gsample_categorical": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp]),
            "gsample_debug_categorical_ex": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp,
                                                    _vp, _i32, _vp]),
            "gsample_debug_sample_cluster": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp,
                                                    _vp, _vp, _i32, _vp]),
            "gsample_status_string": (ctypes.c_char_p, [_int]),
            "gsample_debug_philox": (_int, [_u64, _u32, _u64, _i64, _i64, _vp, _vp]),
            "gsample_debug_gumbel": (_int, [_vp, _i64, _vp, _vp, _vp]),
            "gsample_debug_word_test": (_int, [_vp, _vp, _i64, ctypes.c_float, ctypes.c_float, _vp,
                                               _vp, _vp]),
            "gsample_debug_sample_ex": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _vp,
                                               _vp, _vp, _i32, _vp]),
            "gsample_debug_planned_ctas": (_i32, [_int, _i64, _i64, _i64, _vp, _i32]),
            "gsample_debug_philox_rate": (_int, [_i32, _u32, _vp, _vp]),
            "gsample_debug_philox_alu_mix": (_int, [_i32, _u32, _i32, _i32, _vp, _vp]),
            "gsample_debug_blocks_computed": (_int, [_vp, _i32]),
            "gsample_debug_hlg_score": (_int, [_vp, _vp, _i64, _vp, ctypes.c_float, ctypes.c_float,
                                               _vp, _vp]),
            "gsample_gumbel_argmax_static": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp,
                                                    _vp, _vp]),
            "gsample_gumbel_argmax_host": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp,
                                                  _vp, _vp, _vp]),
            "gsample_filtered_gumbel_argmax": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp,
                                                      _vp, _vp, _vp, _vp, _vp]),
            "gsample_logit_state_ld": (_i64, [_i64]),
            "gsample_state_reset": (_int, [_vp, _vp, _i64, _vp]),
            "gsample_history_append": (_int, [_vp, _vp, _i64, _vp, _i64, _vp, _int, _vp]),
            "gsample_bias_set": (_int, [_vp, _vp, _i64, _vp, _vp, _i64, _vp, _vp]),
            "gsample_process_logits": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _vp, _int, _i64,
                                              _vp]),
            "gsample_constrained_gumbel_argmax": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _vp,
                                                         _vp, _vp, _vp, _vp, _vp]),
            "gsample_debug_filtered_ex": (_int, [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _vp,
                                                 _vp, _vp, _vp, _i32, _vp]),
        }
        for name, (res, args) in sigs.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
        return L


def status_string(status: int) -> str:
    return lib().gsample_status_string(status).decode()


def _check(status: int, what: str) -> None:
    if status != OK:
        raise GSampleError(status, what)


# --------------------------------------------------------------------------
# torch marshalling
# --------------------------------------------------------------------------
_torch_mod = None
_DTYPES = {}


def _torch():
    global _torch_mod
    if _torch_mod is None:
        import torch

        _DTYPES.update({torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16})
        _torch_mod = torch
    return _torch_mod


def _dtype_code(t) -> int:
    _torch()
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise TypeError("logits must be float32, bfloat16 or float16, got %s" % t.dtype)
    return code


def _stream_ptr(device) -> int:
    torch = _torch()
    return torch.cuda.current_stream(device).cuda_stream


def _logits_args(logits):
    if not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor")
    if logits.dim() != 2:
        raise ValueError("logits must be 2-D [B, V]")
    ld, inner = logits.stride()
    if inner != 1:
        raise ValueError("logits rows must be contiguous (stride(1) == 1)")
    B, V = logits.shape
    return _dtype_code(logits), B, V, ld if B > 1 else V


def _row_tensor(x, B, dtype, device, name):
    torch = _torch()
    if not isinstance(x, torch.Tensor):
        x = torch.full((B,), x, dtype=dtype, device=device)
    if x.dtype != dtype or x.device != device or x.dim() != 1 or x.numel() != B or \
            not x.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape [%d] on %s" %
                         (name, dtype, B, device))
    return x


def workspace_bytes(B: int) -> int:
    return int(lib().gsample_workspace_bytes(B))


def new_workspace(B: int, device=None):
    """A zeroed workspace for up to B rows (uint8 tensor, 16-byte aligned)."""
    torch = _torch()
    n = max(16, workspace_bytes(B))
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def workspace_init(ws, B: int) -> None:
    _check(lib().gsample_workspace_init(ws.data_ptr(), B, _stream_ptr(ws.device)),
           "gsample_workspace_init")


def _prepare(logits, out, workspace, need_ws: bool = True):
    torch = _torch()
    dt, B, V, ld = _logits_args(logits)
    dev = logits.device
    if out is None:
        out = torch.empty(B, dtype=torch.int64, device=dev)
    elif out.dtype != torch.int64 or out.device != dev or out.shape != (B,) or not out.is_contiguous():
        raise ValueError("out must be a contiguous int64 tensor of shape [B] on the logits' device")
    if not need_ws:
        return dt, B, V, ld, out, None
    if workspace is None:
        workspace = new_workspace(B, dev)
    elif workspace.device != dev or workspace.nbytes < workspace_bytes(B):
        raise ValueError("workspace too small or on another device")
    return dt, B, V, ld, out, workspace


def argmax(logits, out=None, workspace=None):
    """Greedy argmax per row (lowest index on ties; -1 for an all-masked row)."""
    dt, B, V, ld, out, ws = _prepare(logits, out, workspace)
    _check(lib().gsample_argmax(logits.data_ptr(), dt, B, V, ld, out.data_ptr(), ws.data_ptr(),
                                _stream_ptr(logits.device)), "gsample_argmax")
    return out


def gumbel_argmax(logits, temperature, seed, offset, out=None, workspace=None, ctas: int = 0,
                  cluster: int = 0):
    """Gumbel-max sample per row: argmax_i(logits[i]/T + g_i). temperature
    (float32), seed (uint64 as int64 bits) and offset (uint64 as int64 bits)
    are per-row tensors or scalars. Rows with T <= 0 are greedy. Diagnostics:
    ctas > 0 forces the flat split with that many CTAs; cluster > 0 forces the
    cluster-per-row kernel with that many CTAs per row."""
    torch = _torch()
    dt, B, V, ld, out, ws = _prepare(logits, out, workspace)
    dev = logits.device
    T = _row_tensor(temperature, B, torch.float32, dev, "temperature")
    S = _row_tensor(seed, B, torch.int64, dev, "seed")
    O = _row_tensor(offset, B, torch.int64, dev, "offset")
    L = lib()
    if cluster:
        st = L.gsample_debug_sample_cluster(logits.data_ptr(), dt, B, V, ld, T.data_ptr(),
                                            S.data_ptr(), O.data_ptr(), out.data_ptr(),
                                            ws.data_ptr(), cluster, _stream_ptr(dev))
    elif ctas:
        st = L.gsample_debug_sample_ex(logits.data_ptr(), dt, B, V, ld, T.data_ptr(), S.data_ptr(),
                                       O.data_ptr(), None, out.data_ptr(), ws.data_ptr(), ctas,
                                       _stream_ptr(dev))
    else:
        st = L.gsample_gumbel_argmax(logits.data_ptr(), dt, B, V, ld, T.data_ptr(), S.data_ptr(),
                                     O.data_ptr(), out.data_ptr(), ws.data_ptr(), _stream_ptr(dev))
    _check(st, "gsample_gumbel_argmax")
    return out


def filtered_gumbel_argmax(logits, temperature, seed, offset, top_k=None, top_p=None, out=None,
                           workspace=None, cluster: int = 0):
    """Top-k / top-p Gumbel-max sample per row (gsample_filtered_gumbel_argmax):
    the Gumbel-max over the row's filter set K (the top_k largest logits and/or
    the smallest prefix whose softmax mass reaches top_p). top_k (int32) and
    top_p (float32) are per-row tensors, scalars, or None (filter off).
    Diagnostics: cluster > 0 forces that many filter CTAs per row."""
    torch = _torch()
    dt, B, V, ld, out, ws = _prepare(logits, out, workspace)
    dev = logits.device
    T = _row_tensor(temperature, B, torch.float32, dev, "temperature")
    S = _row_tensor(seed, B, torch.int64, dev, "seed")
    O = _row_tensor(offset, B, torch.int64, dev, "offset")
    K = None if top_k is None else _row_tensor(top_k, B, torch.int32, dev, "top_k")
    P = None if top_p is None else _row_tensor(top_p, B, torch.float32, dev, "top_p")
    args = (logits.data_ptr(), dt, B, V, ld, T.data_ptr(), S.data_ptr(), O.data_ptr(),
            None if K is None else K.data_ptr(), None if P is None else P.data_ptr(),
            out.data_ptr(), ws.data_ptr())
    if cluster:
        st = lib().gsample_debug_filtered_ex(*args, cluster, _stream_ptr(dev))
    else:
        st = lib().gsample_filtered_gumbel_argmax(*args, _stream_ptr(dev))
    _check(st, "gsample_filtered_gumbel_argmax")
    return out


def _pinned_row(x, B, dtype, name):
    torch = _torch()
    if not torch.is_tensor(x):
        x = torch.full((B,), x, dtype=dtype).pin_memory()
    if x.dtype != dtype or x.is_cuda or x.shape != (B,) or not x.is_contiguous() or \
            not x.is_pinned():
        raise ValueError("%s must be a contiguous pinned %s host tensor of shape [%d]" %
                         (name, dtype, B))
    return x


def gumbel_argmax_host(logits, temperature, seed, offset, out=None, workspace=None,
                       sync: bool = True):
    """gumbel_argmax on pinned HOST tensors: the kernel reads the logits and the
    per-row arrays over the CPU-GPU link and writes the indices straight into
    `out` (a pinned int64 host tensor), with no device copy of the logits. The
    workspace is a device tensor. With sync=False the call only enqueues on the
    current CUDA stream, and `out` is ready once that stream is synchronised."""
    torch = _torch()
    if logits.is_cuda or not logits.is_pinned():
        raise ValueError("logits must be a pinned host tensor")
    if logits.dim() != 2 or logits.stride(1) != 1:
        raise ValueError("logits must be 2-D [B, V] with contiguous rows")
    dt = _dtype_code(logits)
    B, V = logits.shape
    ld = logits.stride(0) if B > 1 else V
    T = _pinned_row(temperature, B, torch.float32, "temperature")
    S = _pinned_row(seed, B, torch.int64, "seed")
    O = _pinned_row(offset, B, torch.int64, "offset")
    if out is None:
        out = torch.empty(B, dtype=torch.int64).pin_memory()
    else:
        _pinned_row(out, B, torch.int64, "out")
    dev = torch.device("cuda", torch.cuda.current_device())
    if workspace is None:
        workspace = new_workspace(B, dev)
    elif not workspace.is_cuda or workspace.numel() * workspace.element_size() < workspace_bytes(B):
        raise ValueError("workspace must be a device tensor of at least workspace_bytes(B) bytes")
    stream = torch.cuda.current_stream(dev)
    _check(lib().gsample_gumbel_argmax_host(logits.data_ptr(), dt, B, V, ld, T.data_ptr(),
                                            S.data_ptr(), O.data_ptr(), out.data_ptr(),
                                            workspace.data_ptr(), stream.cuda_stream),
           "gsample_gumbel_argmax_host")
    if sync:
        stream.synchronize()
    return out


def hlg_gumbel_argmax(logits, temperature, seed, offset, hlg: HlgParams, out=None,
                      workspace=None, cluster: int = 0):
    """HLG tone curve on the row's log-probs, then Gumbel-max."""
    torch = _torch()
    dt, B, V, ld, out, ws = _prepare(logits, out, workspace)
    dev = logits.device
    T = _row_tensor(temperature, B, torch.float32, dev, "temperature")
    S = _row_tensor(seed, B, torch.int64, dev, "seed")
    O = _row_tensor(offset, B, torch.int64, dev, "offset")
    hp = hlg.to_c()
    L = lib()
    if cluster:
        st = L.gsample_debug_sample_ex(logits.data_ptr(), dt, B, V, ld, T.data_ptr(), S.data_ptr(),
                                       O.data_ptr(), ctypes.byref(hp), out.data_ptr(),
                                       ws.data_ptr(), cluster, _stream_ptr(dev))
    else:
        st = L.gsample_hlg_gumbel_argmax(logits.data_ptr(), dt, B, V, ld, T.data_ptr(),
                                         S.data_ptr(), O.data_ptr(), ctypes.byref(hp),
                                         out.data_ptr(), ws.data_ptr(), _stream_ptr(dev))
    _check(st, "gsample_hlg_gumbel_argmax")
    return out


def categorical(logits, temperature, seed, offset, out=None, cluster: int = 0):
    """The categorical baseline: softmax(logits / T) drawn by the inverse CDF of
    element 0's uniform. cluster: CTAs per row (0 = the library's choice)."""
    torch = _torch()
    dt, B, V, ld, out, _ = _prepare(logits, out, None, need_ws=False)
    dev = logits.device
    T = _row_tensor(temperature, B, torch.float32, dev, "temperature")
    S = _row_tensor(seed, B, torch.int64, dev, "seed")
    O = _row_tensor(offset, B, torch.int64, dev, "offset")
    L = lib()
    if cluster:
        st = L.gsample_debug_categorical_ex(logits.data_ptr(), dt, B, V, ld, T.data_ptr(),
                                            S.data_ptr(), O.data_ptr(), out.data_ptr(), cluster,
                                            _stream_ptr(dev))
    else:
        st = L.gsample_categorical(logits.data_ptr(), dt, B, V, ld, T.data_ptr(), S.data_ptr(),
                                   O.data_ptr(), out.data_ptr(), _stream_ptr(dev))
    _check(st, "gsample_categorical")
    return out


def hlg_rows_tensor(params, device):
    """Per-row curves as the device array gsample_hlg_gumbel_argmax_rows reads:
    B records of 24 bytes (five float32 fields, then the int32 pivot mode)."""
    import numpy as np

    torch = _torch()
    rec = np.dtype([("m", "<f4"), ("w", "<f4"), ("beta_t", "<f4"), ("beta_h", "<f4"),
                    ("pivot_offset", "<f4"), ("pivot_mode", "<i4")])
    a = np.zeros(len(params), dtype=rec)
    for i, h in enumerate(params):
        a[i] = (h.m, h.w, h.beta_t, h.beta_h, h.pivot_offset, h.pivot_mode)
    return torch.from_numpy(a.view(np.uint8).copy()).to(device)


def hlg_gumbel_argmax_rows(logits, temperature, seed, offset, params, out=None, workspace=None):
    """HLG + Gumbel-max with one curve per row. `params`: a list of B HlgParams,
    or a uint8 device tensor from hlg_rows_tensor."""
    torch = _torch()
    dt, B, V, ld, out, ws = _prepare(logits, out, workspace)
    dev = logits.device
    T = _row_tensor(temperature, B, torch.float32, dev, "temperature")
    S = _row_tensor(seed, B, torch.int64, dev, "seed")
    O = _row_tensor(offset, B, torch.int64, dev, "offset")
    if not torch.is_tensor(params):
        params = hlg_rows_tensor(params, dev)
    if params.device != dev or params.dtype != torch.uint8 or params.numel() != 24 * B:
        raise ValueError("per-row HLG parameters: a uint8 tensor of 24*B bytes on the logits' device")
    st = lib().gsample_hlg_gumbel_argmax_rows(logits.data_ptr(), dt, B, V, ld, T.data_ptr(),
                                              S.data_ptr(), O.data_ptr(), params.data_ptr(),
                                              out.data_ptr(), ws.data_ptr(), _stream_ptr(dev))
    _check(st, "gsample_hlg_gumbel_argmax_rows")
    return out


# --------------------------------------------------------------------------
# Logit constraints
# --------------------------------------------------------------------------
class LogitState:
    """What each request slot has seen and its biases (gsample_logit_state): a
    view of caller-owned tensors on one device, zeroed before first use.

    history  int32 [rows, ld]: output count, bit 31 set for a prompt token.
    bias     float32 [rows, ld], or None.
    touched  int32 [rows, ld // 32]: bit v set where history or bias may be
             nonzero.
    ld is `vocab` rounded up to a multiple of 32 (or more). Rows may be copied
    with plain tensor copies (all three tensors): to fork a request, say. The
    calls use the memory that these tensors had here: the attributes cannot be
    assigned."""

    def __init__(self, history, bias, touched, vocab: int):
        torch = _torch()
        if not history.is_cuda or history.dim() != 2 or history.dtype != torch.int32 or \
                not history.is_contiguous():
            raise ValueError("history must be a contiguous int32 CUDA tensor [rows, ld]")
        rows, ld = history.shape
        if ld % 32 or not 1 <= vocab <= ld:
            raise ValueError("ld must be a multiple of 32 and at least vocab")
        dev = history.device
        if bias is not None and (bias.dtype != torch.float32 or bias.device != dev or
                                 bias.shape != (rows, ld) or not bias.is_contiguous()):
            raise ValueError("bias must be a contiguous float32 tensor [rows, ld] on history's "
                             "device, or None")
        if touched.dtype != torch.int32 or touched.device != dev or \
                touched.shape != (rows, ld // 32) or not touched.is_contiguous():
            raise ValueError("touched must be a contiguous int32 tensor [rows, ld // 32] on "
                             "history's device")
        self._history, self._bias, self._touched, self._vocab = history, bias, touched, int(vocab)
        self._rows, self._ld, self._device = rows, ld, dev
        self._c = _StateC(history.data_ptr(), None if bias is None else bias.data_ptr(),
                          touched.data_ptr(), rows, int(vocab), ld)
        self._at = ctypes.addressof(self._c)

    history = property(operator.attrgetter("_history"))
    bias = property(operator.attrgetter("_bias"))
    touched = property(operator.attrgetter("_touched"))
    vocab = property(operator.attrgetter("_vocab"))
    rows = property(operator.attrgetter("_rows"))
    ld = property(operator.attrgetter("_ld"))
    device = property(operator.attrgetter("_device"))


def new_logit_state(rows: int, vocab: int, device=None, bias: bool = True) -> LogitState:
    """An empty state for `rows` request slots."""
    torch = _torch()
    ld = int(lib().gsample_logit_state_ld(vocab))
    dev = device or "cuda"
    return LogitState(torch.zeros((rows, ld), dtype=torch.int32, device=dev),
                      torch.zeros((rows, ld), dtype=torch.float32, device=dev) if bias else None,
                      torch.zeros((rows, ld // 32), dtype=torch.int32, device=dev), vocab)


def _launch(index, what, fn, *args):
    """fn(*args, the current stream of device `index`) with that device as the
    current one (the library launches there)."""
    torch = _torch()
    if torch.cuda.current_device() == index:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if status != OK:
        raise GSampleError(status, what)


def _vector(x, n, dtype, index, name):
    """The address of a contiguous 1-D tensor of n (None: any number of)
    entries on device `index`; None for None."""
    if x is None:
        return None
    if x.dtype != dtype or x.get_device() != index or x.dim() != 1 or \
            (n is not None and x.numel() != n) or not x.is_contiguous():
        raise ValueError("%s must be a contiguous 1-D %s tensor%s on cuda:%d" %
                         (name, dtype, "" if n is None else " of %d entries" % n, index))
    return x.data_ptr()


def _row_at(x, B, dtype, index, name, keep):
    """The address of a per-row array given as a tensor of B entries or as a
    scalar; a tensor made here goes into `keep`."""
    torch = _torch()
    if not isinstance(x, torch.Tensor):
        x = torch.full((B,), x, dtype=dtype, device="cuda:%d" % index)
        keep.append(x)
    return _vector(x, B, dtype, index, name)


def _lists(state, slots, tokens, offsets):
    """n requests: (slot, n, tokens, total, offsets) as the library takes them."""
    torch = _torch()
    index = state.device.index
    tokens_at = _vector(tokens, None, torch.int64, index, "tokens")
    offsets_at = _vector(offsets, None, torch.int64, index, "offsets")
    total = tokens.numel()
    n = total
    if offsets is not None:
        n = offsets.numel() - 1
        if n < 0:
            raise ValueError("offsets has one entry more than there are requests")
    return _vector(slots, n, torch.int32, index, "slots"), n, tokens_at, total, offsets_at


def state_reset(state: LogitState, slots=None) -> None:
    """Clears the state rows in `slots` (int32 device tensor), or all of them."""
    index = state.device.index
    at = _vector(slots, None, _torch().int32, index, "slots")
    _launch(index, "gsample_state_reset", lib().gsample_state_reset, state._at, at,
            state.rows if slots is None else slots.numel())


def history_append(state: LogitState, tokens, slots=None, offsets=None,
                   prompt: bool = False) -> None:
    """Appends tokens (int64 device tensor) to the requests' histories: request
    i owns tokens[offsets[i]:offsets[i + 1]], or tokens[i] alone without
    offsets (the indices a sampler just drew). slots[i] (int32) is its state
    row; without slots, row i. Ids outside the vocabulary are ignored."""
    _launch(state.device.index, "gsample_history_append", lib().gsample_history_append, state._at,
            *_lists(state, slots, tokens, offsets), 0 if prompt else 1)


def bias_set(state: LogitState, tokens, values, slots=None, offsets=None) -> None:
    """Sets the biases of the listed tokens (lists as in history_append,
    values float32). Other entries keep theirs."""
    if state.bias is None:
        raise ValueError("the state was made without biases")
    slot, n, tokens_at, total, offsets_at = _lists(state, slots, tokens, offsets)
    index = state.device.index
    values_at = _vector(values, total, _torch().float32, index, "values")
    _launch(index, "gsample_bias_set", lib().gsample_bias_set, state._at, slot, n, tokens_at,
            values_at, total, offsets_at)


def _constraints(B, V, index, state, slots, repetition, frequency, presence, mask, mask_rows,
                 keep):
    """The C struct; tensors made here that it points into go into `keep`."""
    torch = _torch()
    state_at = slot = rep = freq = pres = None
    if state is not None:
        if state.device.index != index or state.vocab != V:
            raise ValueError("the state must be on the logits' device and of their vocabulary")
        if slots is None and state.rows < B:
            raise ValueError("without slots the state needs a row for every batch row")
        state_at = state._at
        slot = _vector(slots, B, torch.int32, index, "slots")
        f32 = torch.float32
        if repetition is not None:
            rep = _row_at(repetition, B, f32, index, "repetition", keep)
        if frequency is not None:
            freq = _row_at(frequency, B, f32, index, "frequency", keep)
        if presence is not None:
            pres = _row_at(presence, B, f32, index, "presence", keep)
    elif slots is not None or repetition is not None or frequency is not None or \
            presence is not None:
        raise ValueError("slots and penalties need a state")
    mask_at = mask_row = None
    masks = mask_ld = 0
    if mask is not None:
        if mask.dtype != torch.int32 or mask.get_device() != index or mask.dim() != 2:
            raise ValueError("mask must be a 2-D int32 tensor on the logits' device")
        masks, words = mask.shape
        mask_ld, inner = mask.stride()
        if masks <= 1:
            mask_ld = words
        if words < (V + 31) // 32 or (words > 1 and inner != 1) or mask_ld < words:
            raise ValueError("mask must have >= ceil(V / 32) words a row, in contiguous rows that "
                             "do not overlap")
        if mask_rows is None and masks < B:
            raise ValueError("without mask_rows there must be a mask for every batch row")
        mask_at = mask.data_ptr()
        mask_row = _vector(mask_rows, B, torch.int32, index, "mask_rows")
    elif mask_rows is not None:
        raise ValueError("mask_rows needs a mask")
    return _ConstraintsC(state_at, slot, rep, freq, pres, mask_at, masks, mask_ld, mask_row)


def process_logits(logits, state: LogitState | None = None, slots=None, repetition=None,
                   frequency=None, presence=None, mask=None, mask_rows=None, out=None,
                   out_dtype=None):
    """The constrained logits [B, V] (gsample_process_logits): biases,
    repetition / frequency / presence penalties and grammar masks.

    state       LogitState; slots (int32 [B]) names each row's state row, -1
                for none (default: row b uses state row b).
    repetition, frequency, presence   float32 [B] tensors or scalars.
    mask        int32 [masks, >= ceil(V / 32)], bit v & 31 of word v >> 5 set
                where token v is allowed; mask_rows (int32 [B]) names each
                row's mask, -1 for none (default: row b uses mask b).
    out         a [B, V] tensor with contiguous rows, in the logits' type or
                float32; out=logits works in place. Default: a new tensor of
                out_dtype (the logits' type, or torch.float32) whose rows start
                on 32-byte boundaries, as the samplers read them fastest:
                stride(0) is V rounded up."""
    torch = _torch()
    dt, B, V, ld = _logits_args(logits)
    dev = logits.device
    if out is None:
        dtype = out_dtype or logits.dtype
        pitch = -(-V * dtype.itemsize // 32) * 32 // dtype.itemsize
        out = torch.empty_strided((B, V), (pitch, 1), dtype=dtype, device=dev)
    elif out.device != dev or out.shape != (B, V) or (out_dtype or out.dtype) != out.dtype:
        raise ValueError("out must be a [B, V] tensor on the logits' device, of out_dtype")
    odt, _, _, out_ld = _logits_args(out)
    if odt not in (F32, dt):
        raise ValueError("out must be of the logits' type or float32")
    index, keep = dev.index, []
    c = _constraints(B, V, index, state, slots, repetition, frequency, presence, mask, mask_rows,
                     keep)
    _launch(index, "gsample_process_logits", lib().gsample_process_logits, logits.data_ptr(), dt,
            B, V, ld, ctypes.byref(c), out.data_ptr(), odt, out_ld)
    return out


def constrained_gumbel_argmax(logits, temperature, seed, offset, state: LogitState | None = None,
                              slots=None, repetition=None, frequency=None, presence=None,
                              mask=None, mask_rows=None, out=None, workspace=None):
    """gumbel_argmax on the constrained logits (arguments as in process_logits
    and gumbel_argmax), which are never written: the same indices as
    gumbel_argmax(process_logits(..., out_dtype=torch.float32), ...). -1 for a
    row whose constraints leave nothing."""
    torch = _torch()
    dt, B, V, ld, out, ws = _prepare(logits, out, workspace)
    index, keep = logits.get_device(), []
    T = _row_at(temperature, B, torch.float32, index, "temperature", keep)
    S = _row_at(seed, B, torch.int64, index, "seed", keep)
    O = _row_at(offset, B, torch.int64, index, "offset", keep)
    c = _constraints(B, V, index, state, slots, repetition, frequency, presence, mask, mask_rows,
                     keep)
    _launch(index, "gsample_constrained_gumbel_argmax", lib().gsample_constrained_gumbel_argmax,
            logits.data_ptr(), dt, B, V, ld, T, S, O, ctypes.byref(c), out.data_ptr(),
            ws.data_ptr())
    return out


def seeds_as_tensor(seeds, device):
    """uint64 seeds (numpy or ints) as an int64 tensor holding the same bits."""
    import numpy as np

    torch = _torch()
    a = np.ascontiguousarray(np.asarray(seeds, dtype=np.uint64)).view(np.int64)
    return torch.from_numpy(a.copy()).to(device)


def debug_philox(seed: int, row: int, offset: int, group0: int, n_groups: int, device=None):
    """Raw Philox4x32-10 blocks of the kernels' stream -> int32 tensor [n, 4]
    (bit patterns of uint32)."""
    torch = _torch()
    out = torch.empty((n_groups, 4), dtype=torch.int32, device=device or "cuda")
    _check(lib().gsample_debug_philox(seed, row, offset, group0, n_groups, out.data_ptr(),
                                      _stream_ptr(out.device)), "gsample_debug_philox")
    return out


def debug_gumbel(words, with_bound: bool = True):
    """The kernels' binary32 Gumbel transform (and pruning bound) of raw words
    (int32 tensor of uint32 bit patterns)."""
    torch = _torch()
    g = torch.empty(words.shape, dtype=torch.float32, device=words.device)
    bnd = torch.empty_like(g) if with_bound else None
    _check(lib().gsample_debug_gumbel(words.data_ptr(), words.numel(), g.data_ptr(),
                                      bnd.data_ptr() if bnd is not None else None,
                                      _stream_ptr(words.device)), "gsample_debug_gumbel")
    return g, bnd


def planned_ctas(dtype: int, B: int, V: int, ld: int | None = None, ptr: int = 0) -> int:
    return int(lib().gsample_debug_planned_ctas(dtype, B, V, ld or V, ptr or None, 0))
