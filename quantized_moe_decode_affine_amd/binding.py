"""Thin ctypes binding over libq4moe.so (the C ABI in include/q4moe.h).

Argument marshalling only: torch tensors supply device memory and the current
HIP stream; every step of the computation runs in the library's kernels.  The
library must be built (``python -m quantized_moe_decode_affine_amd.build``);
loading fails with an error otherwise, and there is no other code path.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import numpy as np
import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libq4moe.so")

OK, EINVAL, EUNSUPPORTED, EWORKSPACE, EHIP = 0, 1, 2, 3, 4
OUT_F32, OUT_BF16, OUT_BF16_RESIDUAL = 0, 1, 2  # residual: bf16(x + y), moe_ffn_decode only
OP_GEMV, OP_GEMM, OP_ROUTE, OP_PERMUTE, OP_FFN_DECODE, OP_FFN_PREFILL, OP_LMHEAD, OP_FFN_DECODE_BATCH = range(8)
OP_ROUTE_RULE = 8

EXPORTS = ("q4_gemv", "q4_gemm", "moe_route_topk", "moe_route_topk_q8", "moe_permute", "moe_ffn_decode", "moe_ffn_decode_noalloc",
           "moe_ffn_decode_batch",
           "moe_route", "moe_route_logits", "i8_quantize", "i8_gemm", "i8_gemm_workspace_bytes",
           "moe_experts_i8", "moe_experts_i8_workspace_bytes",
           "moe_ffn_prefill", "lmhead_argmax", "q4moe_pack_group_major", "q4moe_workspace_bytes", "q4moe_strerror")


class Q4Error(RuntimeError):
    def __init__(self, fn: str, status: int, message: str):
        super().__init__(f"{fn} failed with status {status}: {message}")
        self.status = status


class q4moe_matrix(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("biases", ctypes.c_void_p),
                ("count", ctypes.c_int64), ("n", ctypes.c_int64), ("k", ctypes.c_int64),
                ("bits", ctypes.c_int32), ("reserved", ctypes.c_int32), ("codes_gm", ctypes.c_void_p)]


class q4moe_layer(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("top_k", ctypes.c_int32), ("router", ctypes.c_void_p),
                ("gate", q4moe_matrix), ("up", q4moe_matrix), ("down", q4moe_matrix),
                ("sh_gate", q4moe_matrix), ("sh_up", q4moe_matrix), ("sh_down", q4moe_matrix),
                ("router_q8", q4moe_matrix), ("sh_gate_w", ctypes.c_void_p)]


class q4moe_i8_matrix(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("count", ctypes.c_int64), ("n", ctypes.c_int64), ("k", ctypes.c_int64)]


class q4moe_i8_experts(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("reserved", ctypes.c_int32),
                ("gate", q4moe_i8_matrix), ("up", q4moe_i8_matrix), ("down", q4moe_i8_matrix),
                ("sh_gate", q4moe_i8_matrix), ("sh_up", q4moe_i8_matrix), ("sh_down", q4moe_i8_matrix)]


class q4moe_routing(ctypes.Structure):
    _fields_ = [("n_experts", ctypes.c_int32), ("hidden", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("score", ctypes.c_int32), ("n_groups", ctypes.c_int32), ("top_groups", ctypes.c_int32),
                ("group_terms", ctypes.c_int32), ("renormalise", ctypes.c_int32), ("scale", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("bias", ctypes.c_void_p), ("router", ctypes.c_void_p),
                ("router_q8", q4moe_matrix)]


_lib = None


def load_library(path: str = _LIB_PATH) -> ctypes.CDLL:
    """Load libq4moe.so (once) and declare the entry points; raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run `python -m quantized_moe_decode_affine_amd.build` "
                           "(the HIP library is the only implementation)")
    lib = ctypes.CDLL(path)
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t
    pm, pl = ctypes.POINTER(q4moe_matrix), ctypes.POINTER(q4moe_layer)
    sigs = {
        "q4_gemv": [pm, vp, vp, ctypes.c_int, vp],
        "q4_gemm": [pm, vp, i64, vp, ctypes.c_int, vp, sz, vp],
        "moe_route_topk": [vp, i32, i32, vp, i64, i32, vp, vp, vp, sz, vp],
        "moe_route_topk_q8": [pm, vp, i64, i32, vp, vp, vp, sz, vp],
        "moe_permute": [vp, i64, i32, i32, vp, vp, vp, vp, sz, vp],
        "moe_ffn_decode": [pl, vp, vp, ctypes.c_int, vp, vp, vp, sz, vp],
        "moe_ffn_decode_noalloc": [pl, vp, vp, ctypes.c_int, vp, vp, vp],
        "moe_ffn_decode_batch": [pl, vp, i64, vp, ctypes.c_int, vp, vp, vp, sz, vp],
        "moe_ffn_prefill": [pl, vp, i64, vp, ctypes.c_int, vp, sz, vp],
        "lmhead_argmax": [pm, vp, i64, vp, vp, vp, sz, vp],
        "q4moe_pack_group_major": [pm, vp, vp],
        "moe_route": [ctypes.POINTER(q4moe_routing), vp, i64, vp, vp, vp, sz, vp],
        "moe_route_logits": [ctypes.POINTER(q4moe_routing), vp, i64, vp, vp, vp],
        "i8_quantize": [vp, i64, i64, vp, vp, vp],
        "i8_gemm": [ctypes.POINTER(q4moe_i8_matrix), vp, i64, vp, ctypes.c_int, vp, sz, vp],
        "moe_experts_i8": [ctypes.POINTER(q4moe_i8_experts), vp, i64, vp, vp, i32, vp, ctypes.c_int, vp, sz, vp],
    }
    for name, args in sigs.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    lib.q4moe_workspace_bytes.argtypes = [ctypes.c_int, pl, pm, i64]
    lib.q4moe_workspace_bytes.restype = sz
    lib.i8_gemm_workspace_bytes.argtypes = [ctypes.POINTER(q4moe_i8_matrix), i64]
    lib.i8_gemm_workspace_bytes.restype = sz
    lib.moe_experts_i8_workspace_bytes.argtypes = [ctypes.POINTER(q4moe_i8_experts), i64, i32]
    lib.moe_experts_i8_workspace_bytes.restype = sz
    lib.q4moe_strerror.argtypes = [ctypes.c_int]
    lib.q4moe_strerror.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _check(fn: str, status: int) -> None:
    if status != OK:
        raise Q4Error(fn, status, load_library().q4moe_strerror(status).decode())


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream() -> int:
    return torch.cuda.current_stream().cuda_stream


# --------------------------------------------------------------- device data --

def _dev(a: np.ndarray, device) -> torch.Tensor:
    """A numpy array of raw bits -> device tensor of the same bytes (uint32 -> int32, uint16 -> int16)."""
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint32:
        a = a.view(np.int32)
    elif a.dtype == np.uint16:
        a = a.view(np.int16)
    return torch.from_numpy(a).to(device)


def bf16_tensor(bits: np.ndarray, device="cuda") -> torch.Tensor:
    """bf16 bit patterns (uint16) -> a torch.bfloat16 device tensor."""
    return _dev(bits, device).view(torch.bfloat16)


def _need(name: str, t: torch.Tensor, dtype: torch.dtype, shape, device: Optional[torch.device] = None) -> None:
    """Raise ValueError unless `t` is a contiguous GPU tensor of this type and shape (on `device`)."""
    if t.dtype != dtype or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: {dtype} of shape {tuple(shape)} wanted, got {t.dtype} of {tuple(t.shape)}")
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name} is on {t.device}, wanted on {device if device is not None else 'a GPU'}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


class DeviceQ4:
    """An affine matrix (or a stack of them) resident on the device: 4-bit codes, or 8-bit
    codes when the code words per row hold 4 columns each (k is taken from the groups)."""

    def __init__(self, codes: np.ndarray, scales: np.ndarray, biases: np.ndarray, device="cuda"):
        if codes.ndim == 2:
            codes, scales, biases = codes[None], scales[None], biases[None]
        self.count, self.n, words = codes.shape
        self.k = scales.shape[-1] * 64
        if words * 8 == self.k:
            self.bits = 4
        elif words * 4 == self.k:
            self.bits = 8
        else:
            raise ValueError(f"{words} code words per row do not hold {self.k} columns at 4 or 8 bits")
        self.codes = _dev(codes, device)
        self.scales = _dev(scales, device)
        self.biases = _dev(biases, device)
        self.codes_gm = None
        self.struct = q4moe_matrix(self.codes.data_ptr(), self.scales.data_ptr(), self.biases.data_ptr(),
                                   self.count, self.n, self.k, self.bits, 0)

    @classmethod
    def from_device(cls, codes: torch.Tensor, scales: torch.Tensor, biases: torch.Tensor) -> "DeviceQ4":
        """The same from tensors that are on the device already: codes int32 words [n][words] or
        [count][n][words], scales and biases bfloat16 [..][k/64], all contiguous."""
        if codes.dim() == 2:
            codes, scales, biases = codes[None], scales[None], biases[None]
        count, n, words = codes.shape
        _need("codes", codes, torch.int32, (count, n, words), codes.device)
        _need("scales", scales, torch.bfloat16, (count, n, scales.shape[-1]), codes.device)
        _need("biases", biases, torch.bfloat16, tuple(scales.shape), codes.device)
        self = cls.__new__(cls)
        self.count, self.n, self.k = count, n, scales.shape[-1] * 64
        self.bits = 4 if words * 8 == self.k else 8
        if words * 32 != self.k * self.bits:
            raise ValueError(f"{words} code words per row do not hold {self.k} columns at 4 or 8 bits")
        self.codes, self.scales, self.biases, self.codes_gm = codes, scales, biases, None
        self.struct = q4moe_matrix(codes.data_ptr(), scales.data_ptr(), biases.data_ptr(), count, n, self.k,
                                   self.bits, 0)
        return self

    def pack_group_major(self) -> None:
        """Add the group-major copy of the codes that the prefill GEMMs read (4-bit only)."""
        if self.bits != 4 or self.codes_gm is not None:
            return
        self.codes_gm = torch.empty_like(self.codes)
        _check("q4moe_pack_group_major", load_library().q4moe_pack_group_major(
            ctypes.byref(self.struct), _ptr(self.codes_gm), _stream()))
        self.struct.codes_gm = self.codes_gm.data_ptr()

    @property
    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.codes, self.scales, self.biases))


class DeviceLayer:
    """MoE layer weights on the device plus the C descriptor that points at them."""

    def __init__(self, layer, device="cuda"):
        self.hidden, self.inter = layer.hidden, layer.inter
        self.n_experts, self.top_k = layer.n_experts, layer.top_k
        self.router = _dev(layer.router, device)
        self.gate = DeviceQ4(layer.gate.codes, layer.gate.scales, layer.gate.biases, device)
        self.up = DeviceQ4(layer.up.codes, layer.up.scales, layer.up.biases, device)
        self.down = DeviceQ4(layer.down.codes, layer.down.scales, layer.down.biases, device)
        self.has_shared = layer.has_shared
        if layer.has_shared:
            self.sh = [DeviceQ4(m.codes, m.scales, m.biases, device) for m in (layer.sh_gate, layer.sh_up, layer.sh_down)]
        else:
            self.sh = []
        rq8 = getattr(layer, "router_q8", None)
        self.router_q8 = DeviceQ4(*rq8, device=device) if rq8 is not None else None
        gw = getattr(layer, "sh_gate_w", None)
        self.sh_gate_w = _dev(gw, device) if gw is not None else None
        self._describe()

    def _describe(self) -> None:
        sh = [m.struct for m in self.sh] if self.has_shared else [q4moe_matrix() for _ in range(3)]
        new = q4moe_layer(self.hidden, self.inter, self.n_experts, self.top_k, self.router.data_ptr(),
                          self.gate.struct, self.up.struct, self.down.struct, *sh,
                          self.router_q8.struct if self.router_q8 is not None else q4moe_matrix(),
                          self.sh_gate_w.data_ptr() if self.sh_gate_w is not None else None)
        if hasattr(self, "struct"):  # rewritten in place: references taken to it stay current
            ctypes.memmove(ctypes.addressof(self.struct), ctypes.addressof(new), ctypes.sizeof(new))
        else:
            self.struct = new

    def pack_group_major(self) -> None:
        """Give every 4-bit expert matrix its group-major copy (moe_ffn_prefill reads those;
        the decode calls keep reading the row-major codes).  Doubles the 4-bit code memory."""
        for m in (self.gate, self.up, self.down, *self.sh):
            m.pack_group_major()
        self._describe()

    @property
    def nbytes(self) -> int:
        total = self.gate.nbytes + self.up.nbytes + self.down.nbytes + sum(m.nbytes for m in self.sh)
        return total + (self.router_q8.nbytes if self.router_q8 is not None else self.router.numel() * 2)


class DeviceI8:
    """A matrix of symmetric 8-bit codes (or a stack of them) on the device: codes int8 [n][k] or
    [count][n][k] and one fp32 scale per row, [n] or [count][n]."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        if codes.dim() == 2:
            codes, scales = codes[None], scales[None]
        self.count, self.n, self.k = codes.shape
        _need("codes", codes, torch.int8, (self.count, self.n, self.k))
        _need("scales", scales, torch.float32, (self.count, self.n), codes.device)
        self.codes, self.scales = codes, scales
        self.struct = q4moe_i8_matrix(codes.data_ptr(), scales.data_ptr(), self.count, self.n, self.k)

    @classmethod
    def quantize(cls, weight: torch.Tensor) -> "DeviceI8":
        """The 8-bit form of bfloat16 weights [n][k] or [count][n][k], a scale per row."""
        codes, scales = i8_quantize(weight.reshape(-1, weight.shape[-1]))
        return cls(codes.view(weight.shape), scales.view(weight.shape[:-1]))

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel() * 4


class DeviceI8Experts:
    """The 8-bit experts of a layer: gate and up [n_experts][inter][hidden], down
    [n_experts][hidden][inter], and optionally the shared expert's (gate, up, down)."""

    def __init__(self, gate: DeviceI8, up: DeviceI8, down: DeviceI8, shared=None):
        self.n_experts, self.inter, self.hidden = gate.count, gate.n, gate.k
        self.matrices = (gate, up, down, *(shared or ()))
        self.has_shared = shared is not None
        if len(self.matrices) not in (3, 6) or any(m.codes.device != gate.codes.device for m in self.matrices):
            raise ValueError("experts: gate, up and down, and as many of the shared expert, on one device")
        for m, count, n, k in zip(self.matrices, (self.n_experts,) * 3 + (1,) * 3, (self.inter, self.inter, self.hidden) * 2,
                                  (self.hidden, self.hidden, self.inter) * 2):
            if (m.count, m.n, m.k) != (count, n, k):
                raise ValueError(f"experts: a matrix of shape {(m.count, m.n, m.k)} where {(count, n, k)} is wanted")
        self.struct = q4moe_i8_experts(self.hidden, self.inter, self.n_experts, 0, *(m.struct for m in self.matrices))

    @property
    def nbytes(self) -> int:
        return sum(m.nbytes for m in self.matrices)


class Routing:
    """A routing rule and its router: bfloat16 [n_experts][hidden], an 8-bit DeviceQ4, or for
    moe_route_logits the number of experts.  See q4moe_routing in include/q4moe.h."""

    SCORES = {"softmax": 0, "sigmoid": 1}

    def __init__(self, router, top_k: int, score: str = "softmax", bias: Optional[torch.Tensor] = None,
                 n_groups: int = 1, top_groups: int = 1, group_terms: int = 2, renormalise: bool = True,
                 scale: float = 1.0):
        if score not in self.SCORES:
            raise ValueError(f"score {score!r}: one of {sorted(self.SCORES)} is wanted")
        self.router, self.bias, self.top_k = router, bias, top_k
        q8, bf16, self.hidden, self.device = q4moe_matrix(), None, 0, None
        if isinstance(router, DeviceQ4):
            q8, self.n_experts, self.hidden, self.device = router.struct, router.n, router.k, router.codes.device
        elif isinstance(router, torch.Tensor):
            self.n_experts, self.hidden = router.shape
            _need("router", router, torch.bfloat16, (self.n_experts, self.hidden))
            bf16, self.device = router.data_ptr(), router.device
        else:
            self.n_experts = int(router)
        if bias is not None:
            _need("bias", bias, torch.float32, (self.n_experts,), self.device)
            self.device = bias.device
        self.struct = q4moe_routing(self.n_experts, self.hidden, top_k, self.SCORES[score], n_groups, top_groups,
                                    group_terms, int(renormalise), scale, 0, _ptr(bias), bf16, q8)


# ---------------------------------------------------------------- workspaces --

def workspace_bytes(op: int, layer: Optional[DeviceLayer] = None, W: Optional[DeviceQ4] = None,
                    rows: int = 0) -> int:
    lib = load_library()
    return lib.q4moe_workspace_bytes(op, ctypes.byref(layer.struct) if layer else None,
                                     ctypes.byref(W.struct) if W else None, rows)


def workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """A zero-filled device byte buffer (torch's allocator returns 256-byte aligned blocks).

    Zero-filled because the decode workspace holds arrival counters and phase
    flags, and the LM-head workspace an arrival counter, that must be zero before
    their first use (each call leaves them ready for the next); the other
    operations do not care."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def _out(shape, out_dtype, device, out=None):
    if out is not None:
        return out
    return torch.empty(shape, dtype=torch.float32 if out_dtype == OUT_F32 else torch.bfloat16, device=device)


# --------------------------------------------------------------- entry points --

def q4_gemv(W: DeviceQ4, x: torch.Tensor, out_dtype: int = OUT_F32, out: Optional[torch.Tensor] = None):
    y = _out((W.count * W.n,), out_dtype, x.device, out)
    _check("q4_gemv", load_library().q4_gemv(ctypes.byref(W.struct), _ptr(x), _ptr(y), out_dtype, _stream()))
    return y


def q4_gemm(W: DeviceQ4, X: torch.Tensor, out_dtype: int = OUT_F32, out=None, ws: Optional[torch.Tensor] = None):
    m = X.shape[0]
    Y = _out((m, W.count * W.n), out_dtype, X.device, out)
    need = workspace_bytes(OP_GEMM, W=W, rows=m)
    ws = ws if ws is not None else workspace(need, X.device)
    _check("q4_gemm", load_library().q4_gemm(ctypes.byref(W.struct), _ptr(X), m, _ptr(Y), out_dtype, _ptr(ws),
                                             ws.numel(), _stream()))
    return Y


def moe_route_topk(router: torch.Tensor, X: torch.Tensor, top_k: int, ws: Optional[torch.Tensor] = None):
    E, H = router.shape
    T = X.shape[0]
    ids = torch.empty((T, top_k), dtype=torch.int32, device=X.device)
    w = torch.empty((T, top_k), dtype=torch.float32, device=X.device)
    if ws is None:
        ws = workspace(load_library().q4moe_workspace_bytes(
            OP_ROUTE, ctypes.byref(q4moe_layer(H, 0, E, top_k)), None, T), X.device)
    _check("moe_route_topk", load_library().moe_route_topk(_ptr(router), E, H, _ptr(X), T, top_k, _ptr(ids),
                                                           _ptr(w), _ptr(ws), ws.numel(), _stream()))
    return ids, w


def moe_route_topk_q8(router_q8: DeviceQ4, X: torch.Tensor, top_k: int, ws: Optional[torch.Tensor] = None):
    """Top-k routing through an affine-Q8 router matrix (n_experts x hidden, 8-bit codes)."""
    E = router_q8.n
    T = X.shape[0]
    ids = torch.empty((T, top_k), dtype=torch.int32, device=X.device)
    w = torch.empty((T, top_k), dtype=torch.float32, device=X.device)
    if ws is None:
        ws = workspace(load_library().q4moe_workspace_bytes(
            OP_ROUTE, ctypes.byref(q4moe_layer(router_q8.k, 0, E, top_k)), None, T), X.device)
    _check("moe_route_topk_q8", load_library().moe_route_topk_q8(ctypes.byref(router_q8.struct), _ptr(X), T, top_k,
                                                                 _ptr(ids), _ptr(w), _ptr(ws), ws.numel(), _stream()))
    return ids, w


def gpu_routing(layer: DeviceLayer, X: torch.Tensor):
    """The layer's routing of the rows X through its own router (bf16 or 8-bit)."""
    if layer.router_q8 is not None:
        return moe_route_topk_q8(layer.router_q8, X, layer.top_k)
    return moe_route_topk(layer.router, X, layer.top_k)


# The current stream's handle of a device by its index: torch's raw form where this torch has it
# (0.1 us instead of the 1.9 us of a Stream object, next to the 4 us of a launch).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(fn: str, device: torch.device, *args) -> None:
    """Call an entry point on `device` and its current stream."""
    f = getattr(load_library(), fn)
    if device.index == torch.cuda.current_device():
        status = f(*args, _raw_stream(device.index))
    else:
        with torch.cuda.device(device):
            status = f(*args, _raw_stream(device.index))
    if status != OK:
        _check(fn, status)


def _result(name: str, out: Optional[torch.Tensor], shape, dtype: torch.dtype, device: torch.device) -> torch.Tensor:
    if out is None:
        return torch.empty(shape, dtype=dtype, device=device)
    _need(name, out, dtype, shape, device)
    return out


def _scratch(ws: Optional[torch.Tensor], nbytes, device: torch.device) -> torch.Tensor:
    """The caller's workspace, or one of nbytes() for this call."""
    if ws is None:
        return torch.empty(max(nbytes(), 256), dtype=torch.uint8, device=device)
    if ws.dtype != torch.uint8 or ws.device != device or not ws.is_contiguous():
        raise ValueError("ws: a contiguous uint8 buffer on the inputs' device is wanted")
    return ws


def _out_type(out_dtype: int) -> torch.dtype:
    if out_dtype not in (OUT_F32, OUT_BF16):
        raise ValueError(f"out_dtype {out_dtype}: OUT_F32 or OUT_BF16 is wanted")
    return torch.float32 if out_dtype == OUT_F32 else torch.bfloat16


def moe_route_workspace(routing: Routing, T: int) -> torch.Tensor:
    """A workspace for moe_route on up to T rows, its arrival counts (the first 256 bytes) zeroed
    as the first call needs them.  moe_route on another buffer whose counts are not zero gives id
    -1 and weight NaN."""
    nbytes = load_library().q4moe_workspace_bytes(
        OP_ROUTE_RULE, ctypes.byref(q4moe_layer(routing.hidden, 0, routing.n_experts, routing.top_k)), None, T)
    ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=routing.device)
    ws[:256].zero_()
    return ws


def moe_route(routing: Routing, X: torch.Tensor, ids: Optional[torch.Tensor] = None,
              weights: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None):
    """Expert ids int32 and weights fp32 [T][top_k] of the rows X by a routing rule."""
    T, dev = X.shape[0], X.device
    _need("X", X, torch.bfloat16, (T, routing.hidden), routing.device)
    ids = _result("ids", ids, (T, routing.top_k), torch.int32, dev)
    weights = _result("weights", weights, (T, routing.top_k), torch.float32, dev)
    if T:
        ws = moe_route_workspace(routing, T) if ws is None else _scratch(ws, None, dev)
        _call("moe_route", dev, ctypes.byref(routing.struct), X.data_ptr(), T, ids.data_ptr(), weights.data_ptr(),
              ws.data_ptr(), ws.numel())
    return ids, weights


def moe_route_logits(routing: Routing, logits: torch.Tensor, ids: Optional[torch.Tensor] = None,
                     weights: Optional[torch.Tensor] = None):
    """moe_route on logits fp32 [T][n_experts] that the caller has."""
    T, dev = logits.shape[0], logits.device
    _need("logits", logits, torch.float32, (T, routing.n_experts), routing.device)
    ids = _result("ids", ids, (T, routing.top_k), torch.int32, dev)
    weights = _result("weights", weights, (T, routing.top_k), torch.float32, dev)
    if T:
        _call("moe_route_logits", dev, ctypes.byref(routing.struct), logits.data_ptr(), T, ids.data_ptr(),
              weights.data_ptr())
    return ids, weights


def moe_permute(ids: torch.Tensor, n_experts: int, ws: Optional[torch.Tensor] = None):
    T, k = ids.shape
    offsets = torch.empty(n_experts + 1, dtype=torch.int32, device=ids.device)
    rows = torch.empty(T * k, dtype=torch.int32, device=ids.device)
    inv = torch.empty(T * k, dtype=torch.int32, device=ids.device)
    if ws is None:
        ws = workspace(load_library().q4moe_workspace_bytes(
            OP_PERMUTE, ctypes.byref(q4moe_layer(0, 0, n_experts, k)), None, T), ids.device)
    _check("moe_permute", load_library().moe_permute(_ptr(ids), T, k, n_experts, _ptr(offsets), _ptr(rows),
                                                     _ptr(inv), _ptr(ws), ws.numel(), _stream()))
    return offsets, rows, inv


# Byte offset of the decode workspace's abandoned-wait counter (include/q4moe.h, moe_ffn_decode).
DECODE_TIMEOUT_OFFSET = 2048


class DecodeTimeout(RuntimeError):
    """A decode launch gave up waiting for a value another workgroup publishes; its result is wrong."""


def decode_timeouts(ws: torch.Tensor) -> int:
    """The abandoned-wait counter of a decode workspace (synchronises with the device)."""
    return int(ws[DECODE_TIMEOUT_OFFSET:DECODE_TIMEOUT_OFFSET + 4].view(torch.int32).item())


def check_decode_workspace(ws: torch.Tensor) -> None:
    """Raise DecodeTimeout when any decode call that used `ws` abandoned a wait."""
    n = decode_timeouts(ws)
    if n:
        raise DecodeTimeout(f"{n} bounded wait(s) inside moe_ffn_decode gave up: the outputs written since the "
                            f"workspace was zeroed are wrong (were all workgroups resident at once?)")


def moe_ffn_decode(layer: DeviceLayer, x: torch.Tensor, out_dtype: int = OUT_F32, out=None,
                   ids_out: Optional[torch.Tensor] = None, w_out: Optional[torch.Tensor] = None,
                   ws: Optional[torch.Tensor] = None):
    """One decode step through the layer.  With a workspace of its own (ws None) the call
    synchronises and raises DecodeTimeout if the launch abandoned a wait; a caller that passes
    `ws` checks it with check_decode_workspace when it synchronises."""
    y = _out((layer.hidden,), out_dtype, x.device, out)
    own = ws is None
    if own:
        ws = workspace(workspace_bytes(OP_FFN_DECODE, layer), x.device)
    _check("moe_ffn_decode", load_library().moe_ffn_decode(ctypes.byref(layer.struct), _ptr(x), _ptr(y), out_dtype,
                                                           _ptr(ids_out), _ptr(w_out), _ptr(ws), ws.numel(),
                                                           _stream()))
    if own:
        check_decode_workspace(ws)
    return y


def moe_ffn_decode_noalloc(layer: DeviceLayer, x: torch.Tensor, out_dtype: int = OUT_F32, out=None,
                           ids_out: Optional[torch.Tensor] = None, w_out: Optional[torch.Tensor] = None):
    """moe_ffn_decode on the library's fixed scratch array (no workspace, nothing allocated
    by the call; `out` must be given for that)."""
    y = _out((layer.hidden,), out_dtype, x.device, out)
    _check("moe_ffn_decode_noalloc", load_library().moe_ffn_decode_noalloc(
        ctypes.byref(layer.struct), _ptr(x), _ptr(y), out_dtype, _ptr(ids_out), _ptr(w_out), _stream()))
    return y


def moe_ffn_decode_batch(layer: DeviceLayer, X: torch.Tensor, out_dtype: int = OUT_F32, out=None,
                         ids_out: Optional[torch.Tensor] = None, w_out: Optional[torch.Tensor] = None,
                         ws: Optional[torch.Tensor] = None):
    B = X.shape[0]
    Y = _out((B, layer.hidden), out_dtype, X.device, out)
    if ws is None:
        ws = workspace(workspace_bytes(OP_FFN_DECODE_BATCH, layer, rows=B), X.device)
    _check("moe_ffn_decode_batch", load_library().moe_ffn_decode_batch(
        ctypes.byref(layer.struct), _ptr(X), B, _ptr(Y), out_dtype, _ptr(ids_out), _ptr(w_out), _ptr(ws),
        ws.numel(), _stream()))
    return Y


def moe_ffn_prefill(layer: DeviceLayer, X: torch.Tensor, out_dtype: int = OUT_F32, out=None,
                    ws: Optional[torch.Tensor] = None):
    T = X.shape[0]
    Y = _out((T, layer.hidden), out_dtype, X.device, out)
    if ws is None:
        ws = workspace(workspace_bytes(OP_FFN_PREFILL, layer, rows=T), X.device)
    _check("moe_ffn_prefill", load_library().moe_ffn_prefill(ctypes.byref(layer.struct), _ptr(X), T, _ptr(Y),
                                                             out_dtype, _ptr(ws), ws.numel(), _stream()))
    return Y


def lmhead_argmax(W: DeviceQ4, X: torch.Tensor, ws: Optional[torch.Tensor] = None, with_max: bool = True):
    B = X.shape[0]
    ids = torch.empty(B, dtype=torch.int32, device=X.device)
    mx = torch.empty(B, dtype=torch.float32, device=X.device) if with_max else None
    if ws is None:
        ws = workspace(workspace_bytes(OP_LMHEAD, W=W, rows=B), X.device)
    _check("lmhead_argmax", load_library().lmhead_argmax(ctypes.byref(W.struct), _ptr(X), B, _ptr(ids), _ptr(mx),
                                                         _ptr(ws), ws.numel(), _stream()))
    return ids, mx


def i8_quantize(X: torch.Tensor):
    """Symmetric 8-bit codes int8 [rows][k] and scales fp32 [rows] of bfloat16 rows."""
    rows, k = X.shape
    _need("X", X, torch.bfloat16, (rows, k))
    codes = torch.empty((rows, k), dtype=torch.int8, device=X.device)
    scales = torch.empty(rows, dtype=torch.float32, device=X.device)
    if rows:
        _call("i8_quantize", X.device, X.data_ptr(), rows, k, codes.data_ptr(), scales.data_ptr())
    return codes, scales


def i8_gemm_workspace(W: DeviceI8, m: int) -> torch.Tensor:
    """A workspace for i8_gemm on up to m rows."""
    return torch.empty(max(256, load_library().i8_gemm_workspace_bytes(ctypes.byref(W.struct), m)),
                       dtype=torch.uint8, device=W.codes.device)


def i8_gemm(W: DeviceI8, X: torch.Tensor, out_dtype: int = OUT_F32, out: Optional[torch.Tensor] = None,
            ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y = X W^T in 8-bit integers: the rows of X (bfloat16) are quantized per token inside the call."""
    m, dev = X.shape[0], W.codes.device
    _need("X", X, torch.bfloat16, (m, W.k), dev)
    Y = _result("out", out, (m, W.count * W.n), _out_type(out_dtype), dev)
    if m:
        ws = _scratch(ws, lambda: load_library().i8_gemm_workspace_bytes(ctypes.byref(W.struct), m), dev)
        _call("i8_gemm", dev, ctypes.byref(W.struct), X.data_ptr(), m, Y.data_ptr(), out_dtype, ws.data_ptr(),
              ws.numel())
    return Y


def moe_experts_i8_workspace(experts: DeviceI8Experts, T: int, top_k: int) -> torch.Tensor:
    """A workspace for moe_experts_i8 on up to T tokens of top_k slots."""
    return torch.empty(max(256, load_library().moe_experts_i8_workspace_bytes(ctypes.byref(experts.struct), T, top_k)),
                       dtype=torch.uint8, device=experts.matrices[0].codes.device)


def moe_experts_i8(experts: DeviceI8Experts, X: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor,
                   out_dtype: int = OUT_F32, out: Optional[torch.Tensor] = None,
                   ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The rows of X through the 8-bit experts of ids [T][top_k] (others than 0..n_experts-1 add
    nothing), weighted by weights [T][top_k], plus the shared expert."""
    T, dev = X.shape[0], experts.matrices[0].codes.device
    _need("X", X, torch.bfloat16, (T, experts.hidden), dev)
    k = ids.shape[1] if ids.dim() == 2 else 0
    _need("ids", ids, torch.int32, (T, k), dev)
    _need("weights", weights, torch.float32, (T, k), dev)
    Y = _result("out", out, (T, experts.hidden), _out_type(out_dtype), dev)
    if T:
        ws = _scratch(ws, lambda: load_library().moe_experts_i8_workspace_bytes(ctypes.byref(experts.struct), T, k), dev)
        _call("moe_experts_i8", dev, ctypes.byref(experts.struct), X.data_ptr(), T, ids.data_ptr(),
              weights.data_ptr(), k, Y.data_ptr(), out_dtype, ws.data_ptr(), ws.numel())
    return Y
