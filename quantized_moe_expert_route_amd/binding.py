"""Python binding of libqmoe.so (ctypes): argument marshalling only.

Every step of the routed-MoE call runs in the library's HIP kernels; torch is
used for device memory and the current stream. The names follow the C ABI in
include/qmoe.h. Importing this module does not load the library; the first
use does, and fails loudly when it has not been built.
"""

from __future__ import annotations

import ctypes
import os
from typing import Dict, Optional

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "libqmoe.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_DEVICE, MOE_ERR_HIP = range(6)
MID_E4M3, MID_MXFP4 = 0, 1  # moe_mid_format
BF16, FP16, FP32 = range(3)  # moe_dtype
ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}  # moe_activation
LAYOUT_W13_PACKED, LAYOUT_W2_PACKED = 1, 2  # moe_weight_layout flags


def layout_for(mid_format: int) -> int:
    """The weight layout calls with this mid format read: gate/up packed, and
    down packed with the MXFP4 mid."""
    return LAYOUT_W13_PACKED | (LAYOUT_W2_PACKED if mid_format == MID_MXFP4 else 0)
NOALLOC_SCRATCH_BYTES = 64 << 20  # MOE_NOALLOC_SCRATCH_BYTES of include/qmoe.h


class moe_shape(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("H", ctypes.c_int64), ("E", ctypes.c_int64), ("I", ctypes.c_int64),
                ("top_k", ctypes.c_int64), ("routed_scaling", ctypes.c_float), ("shared_I", ctypes.c_int64)]


LAYOUT_FIELDS = ["total_bytes", "topk_ids", "topk_w", "count", "offset", "sorted_entry", "xq", "xs", "midq",
                 "mids", "y", "sh_xq", "sh_xs", "sh_hq", "sh_hs", "sh_y"]


class moe_ws_layout(ctypes.Structure):
    _fields_ = [(f, ctypes.c_size_t) for f in LAYOUT_FIELDS]


TP_MAX = 8  # MOE_TP_MAX


class moe_tp_exchange(ctypes.Structure):
    _fields_ = [("tp", ctypes.c_int32), ("rank", ctypes.c_int32), ("epoch", ctypes.c_uint32),
                ("spin_limit", ctypes.c_int32), ("inbox", ctypes.c_void_p), ("inbox_tags", ctypes.c_void_p),
                ("push", ctypes.c_void_p * TP_MAX), ("push_tags", ctypes.c_void_p * TP_MAX),
                ("status", ctypes.c_void_p)]


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_str(status)} (status {status})")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library (built in-tree by quantized_moe_expert_route_amd.build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m quantized_moe_expert_route_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, st = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    L.moe_status_str.restype = ctypes.c_char_p
    L.moe_status_str.argtypes = [st]
    L.moe_stage_count.restype = ctypes.c_int
    L.moe_stage_count.argtypes = []
    L.moe_stage_name.restype = ctypes.c_char_p
    L.moe_stage_name.argtypes = [ctypes.c_int]
    L.moe_shape_workspace_bytes.restype = st
    L.moe_shape_workspace_bytes.argtypes = [ctypes.POINTER(moe_shape), ctypes.POINTER(ctypes.c_size_t)]
    L.moe_plan_create.restype = st
    L.moe_plan_create.argtypes = [ctypes.POINTER(moe_shape), ctypes.POINTER(vp)]
    L.moe_plan_destroy.restype = None
    L.moe_plan_destroy.argtypes = [vp]
    L.moe_plan_workspace_bytes.restype = ctypes.c_size_t
    L.moe_plan_workspace_bytes.argtypes = [vp]
    L.moe_plan_layout.restype = st
    L.moe_plan_layout.argtypes = [vp, ctypes.POINTER(moe_ws_layout)]
    L.moe_plan_set_workspace.restype = st
    L.moe_plan_set_workspace.argtypes = [vp, vp, ctypes.c_size_t, vp]
    L.moe_plan_set_shared.restype = st
    L.moe_plan_set_shared.argtypes = [vp, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    L.moe_plan_shared_pack_bytes.restype = ctypes.c_size_t
    L.moe_plan_shared_pack_bytes.argtypes = [vp]
    L.moe_plan_set_stage_events.restype = st
    L.moe_plan_set_stage_events.argtypes = [vp, ctypes.POINTER(vp), ctypes.c_int]
    L.moe_plan_set_call_events.restype = st
    L.moe_plan_set_call_events.argtypes = [vp, vp, vp]
    L.moe_plan_stage_launches.restype = ctypes.c_int
    L.moe_plan_stage_launches.argtypes = [vp, i64, ctypes.c_int]
    L.moe_forward.restype = st
    L.moe_forward.argtypes = [vp, i64, vp, vp, vp, vp, vp, vp, vp, vp]
    L.moe_forward_noalloc.restype = st
    L.moe_forward_noalloc.argtypes = [vp, i64, vp, vp, vp, vp, vp, vp, vp, vp]
    L.moe_pack_w13.restype = st
    L.moe_pack_w13.argtypes = [vp, vp, i64, i64, i64, vp, vp, vp]
    L.moe_pack_w2.restype = st
    L.moe_pack_w2.argtypes = [vp, vp, i64, i64, i64, vp, vp, vp]
    L.moe_plan_set_shared_slot.restype = st
    L.moe_plan_set_shared_slot.argtypes = [vp, ctypes.c_int]
    L.moe_plan_set_mid_format.restype = st
    L.moe_plan_set_mid_format.argtypes = [vp, ctypes.c_int]
    L.moe_plan_set_weight_layout.restype = st
    L.moe_plan_set_weight_layout.argtypes = [vp, ctypes.c_uint]
    L.moe_router_create.restype = st
    L.moe_router_create.argtypes = [i64, i64, ctypes.c_int, vp, ctypes.c_int, i64, ctypes.POINTER(vp)]
    L.moe_router_destroy.restype = None
    L.moe_router_destroy.argtypes = [vp]
    L.moe_router_forward.restype = st
    L.moe_router_forward.argtypes = [vp, i64, vp, i64, vp, vp]
    for f in (L.moe_router_kernel, L.moe_linear_kernel):
        f.restype = ctypes.c_char_p
        f.argtypes = [vp, i64]
    L.moe_linear_pack_bytes.restype = st
    L.moe_linear_pack_bytes.argtypes = [i64, i64, ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t)]
    L.moe_pack_linear.restype = st
    L.moe_pack_linear.argtypes = [vp, vp, i64, i64, vp, vp, vp]
    L.moe_linear_create.restype = st
    L.moe_linear_create.argtypes = [i64, i64, ctypes.c_int, vp, vp, vp, i64, ctypes.POINTER(vp)]
    L.moe_linear_destroy.restype = None
    L.moe_linear_destroy.argtypes = [vp]
    L.moe_linear_forward.restype = st
    L.moe_linear_forward.argtypes = [vp, i64, vp, i64, vp, i64, vp, i64, ctypes.c_int, vp]
    L.moe_layer_forward.restype = st
    L.moe_layer_forward.argtypes = [vp, vp, i64, vp, vp, vp, vp, vp, vp, vp]
    sz, psz, ph, ci, cf = ctypes.c_size_t, ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(vp), ctypes.c_int, ctypes.c_float
    for name, args in {
        "moe_dense_create": [i64, i64, ci, vp, vp, ci, i64, ph],
        "moe_dense_workspace_bytes": [vp, i64, ci, psz],
        "moe_dense_forward": [vp, i64, vp, i64, vp, i64, vp, i64, ci, vp, i64, ci, vp, sz, vp],
        "moe_dense_backward": [vp, i64, vp, i64, vp, i64, ci, vp, i64, vp, i64, vp, vp, vp, sz, vp],
        "moe_gated_create": [i64, i64, ci, vp, ci, i64, ph],
        "moe_gated_workspace_bytes": [vp, i64, ci, psz],
        "moe_gated_forward": [vp, i64, vp, i64, vp, i64, vp, ci, vp, sz, vp],
        "moe_gated_backward": [vp, i64, vp, i64, vp, ci, vp, i64, vp, i64, vp, vp, sz, vp],
        "moe_scores_create": [i64, i64, ci, i64, ph],
        "moe_scores_workspace_bytes": [vp, i64, psz],
        "moe_scores_forward": [vp, i64, vp, i64, vp, vp, vp, vp, vp, vp, vp, sz, vp],
        "moe_distill_create": [i64, i64, ci, ci, cf, i64, ph],
        "moe_distill_workspace_bytes": [vp, i64, psz],
        "moe_distill_forward": [vp, i64, vp, i64, vp, vp, vp, vp, vp, sz, vp],
        "moe_distill_backward": [vp, i64, vp, i64, vp, vp, vp, vp, vp, i64, vp],
        "moe_distill_forward_backward": [vp, i64, vp, i64, vp, vp, vp, vp, vp, i64, vp, sz, vp],
    }.items():
        f = getattr(L, name)
        f.restype, f.argtypes = st, args
    for f in (L.moe_dense_kernel, L.moe_gated_kernel, L.moe_distill_kernel):
        f.restype, f.argtypes = ctypes.c_char_p, [vp, i64, ci]
    L.moe_scores_kernel.restype, L.moe_scores_kernel.argtypes = ctypes.c_char_p, [vp, i64]
    for f in (L.moe_dense_destroy, L.moe_gated_destroy, L.moe_scores_destroy, L.moe_distill_destroy):
        f.restype, f.argtypes = None, [vp]
    L.moe_plan_set_tp_exchange.restype = st
    L.moe_plan_set_tp_exchange.argtypes = [vp, ctypes.POINTER(moe_tp_exchange)]
    _lib = L
    return L


def status_str(status: int) -> str:
    return lib().moe_status_str(status).decode()


def stage_names():
    L = lib()
    return [L.moe_stage_name(i).decode() for i in range(L.moe_stage_count())]


def shape_workspace_bytes(M, H, E, I, top_k, routed_scaling=2.5, shared_I=0) -> int:
    s = moe_shape(M, H, E, I, top_k, routed_scaling, shared_I)
    out = ctypes.c_size_t(0)
    st = lib().moe_shape_workspace_bytes(ctypes.byref(s), ctypes.byref(out))
    if st != MOE_OK:
        raise MoeError(st, "moe_shape_workspace_bytes")
    return out.value


def _ptr(t) -> int:
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    import torch

    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def pack_w13(w13, s13, out=None, stream=None):
    """Gate/up weights and scales (row-major MXFP4 [E, 2I, H/2] and E8M0
    [E, 2I, H/32], uint8 device tensors) -> (w13_packed, s13_packed) in the
    layout moe_forward reads (moe_pack_w13). Enqueued on `stream`; `out`
    may give the two destination tensors, else they are allocated here."""
    import torch

    E, R, Hh = w13.shape
    if R % 2 or tuple(s13.shape) != (E, R, Hh // 16):
        raise ValueError("w13 must be [E, 2I, H/2] and s13 [E, 2I, H/32]")
    if out is None:
        out = (torch.empty_like(w13), torch.empty_like(s13))
    wp, sp = out
    st = lib().moe_pack_w13(_ptr(w13), _ptr(s13), E, R // 2, 2 * Hh, _ptr(wp), _ptr(sp), _stream(stream))
    if st != MOE_OK:
        raise MoeError(st, "moe_pack_w13")
    return wp, sp


def pack_w2(w2, s2, out=None, stream=None):
    """Down weights and scales (row-major MXFP4 [E, H, I/2] and E8M0
    [E, H, I/32], uint8 device tensors) -> (w2_packed, s2_packed) in the
    layout the MXFP4-mid down reads (moe_pack_w2); s2_packed is [E, H, 16]."""
    import torch

    E, H, Ih = w2.shape
    if tuple(s2.shape) != (E, H, Ih // 16):
        raise ValueError("w2 must be [E, H, I/2] and s2 [E, H, I/32]")
    if out is None:
        out = (torch.empty_like(w2), torch.empty((E, H, 16), dtype=torch.uint8, device=w2.device))
    wp, sp = out
    st = lib().moe_pack_w2(_ptr(w2), _ptr(s2), E, 2 * Ih, H, _ptr(wp), _ptr(sp), _stream(stream))
    if st != MOE_OK:
        raise MoeError(st, "moe_pack_w2")
    return wp, sp


class _Handle:
    """A library handle on one device, destroyed with the object."""

    _h = None
    _destroy = ""

    def _check(self, name, t, dtype, rows, cols, dense=False):
        """The library sees bare pointers: a tensor on another device, of
        another type, smaller than the call, or with strided columns is
        refused here. Returns the elements between its rows."""
        try:
            n, c = t.shape
            if t.dtype is dtype and c == cols and n >= rows and t.is_contiguous() and t.device == self.device:
                return cols  # one expression for the common case: a small call's time is host time
        except (AttributeError, ValueError):
            pass
        import torch

        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch tensor")
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, the weights on {self.device}")
        if t.dtype != dtype:
            raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
        if t.dim() != 2 or t.shape[0] < rows or t.shape[1] != cols:
            raise ValueError(f"{name} is {tuple(t.shape)}, expected at least [{rows}, {cols}]")
        if (t.stride(1) != 1 and cols != 1) or (rows > 1 and t.stride(0) < cols):
            raise ValueError(f"{name} has strides {t.stride()}: columns must be adjacent, rows apart")
        if dense and not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.stride(0) if rows > 1 else cols  # a single row's stride says nothing

    def _rows(self, x, M):
        M = x.shape[0] if M is None else int(M)
        if not 0 <= M <= self.max_M:
            raise ValueError(f"M = {M} outside [0, {self.max_M}]")
        return M

    def kernel(self, M: int) -> str:
        """Which of its kernels a call of M rows launches (profiling aid)."""
        name = getattr(lib(), self._destroy.replace("destroy", "kernel"))(self._h, int(M))
        if name is None:
            raise ValueError(f"M = {M} outside [1, {self.max_M}], or no handle")
        return name.decode()

    def _stream(self, stream):
        return _raw_stream(self.device) if stream is None else stream.cuda_stream

    def close(self):
        if self._h:
            getattr(lib(), self._destroy)(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _raw_stream(device):
    """The hipStream_t of torch's current stream on `device` (without the
    Python stream object where torch has that: 0.1 against 2 us)."""
    import torch

    get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if get is None or device.index is None:
        return torch.cuda.current_stream(device).cuda_stream
    return get(device.index)


def _dtype_code(dtype):
    import torch

    code = {torch.bfloat16: BF16, torch.float16: FP16, torch.float32: FP32}.get(dtype)
    if code is None:
        raise ValueError(f"dtype {dtype} is none of bfloat16, float16, float32")
    return code


class Router(_Handle):
    """Router projection on weights w [E, H] (bf16 or fp32): the fp32 logits
    moe_forward takes, and the routing of Plan.layer."""

    _destroy = "moe_router_destroy"

    def __init__(self, w, x_dtype=None, max_M: int = 1 << 20):
        import torch

        if not isinstance(w, torch.Tensor) or w.dim() != 2 or not w.is_contiguous():
            raise ValueError("w must be a contiguous [E, H] tensor")
        self.x_dtype = torch.bfloat16 if x_dtype is None else x_dtype
        self.device, self.max_M, self.w = w.device, int(max_M), w  # the library keeps w's pointer
        self._fp32 = torch.float32
        self.E, self.H = w.shape
        h = ctypes.c_void_p()
        st = lib().moe_router_create(self.E, self.H, _dtype_code(self.x_dtype), _ptr(w), _dtype_code(w.dtype),
                                     self.max_M, ctypes.byref(h))
        if st != MOE_OK:
            raise MoeError(st, "moe_router_create")
        self._h = h

    def forward(self, x, logits, M: Optional[int] = None, stream=None):
        """logits[:M] = x[:M] w^T, enqueued on `stream` (default: the current
        stream of the weights' device)."""
        M = self._rows(x, M)
        ldx = self._check("x", x, self.x_dtype, M, self.H)
        self._check("logits", logits, self._fp32, M, self.E, dense=True)
        st = lib().moe_router_forward(self._h, M, x.data_ptr(), ldx, logits.data_ptr(), self._stream(stream))
        if st != MOE_OK:
            raise MoeError(st, "moe_router_forward")
        return logits


class Linear(_Handle):
    """Linear layer on MXFP4 weights: row-major codes w [N, K/2] and E8M0
    scales s [N, K/32] (uint8), packed here into buffers this object keeps (w
    and s are free afterwards), with an optional bias [N] of x's type."""

    _destroy = "moe_linear_destroy"

    def __init__(self, w, s, bias=None, x_dtype=None, max_M: int = 1 << 20):
        import torch

        u8 = torch.uint8
        if not isinstance(w, torch.Tensor) or w.dim() != 2 or w.dtype != u8 or not w.is_contiguous():
            raise ValueError("w must be a contiguous uint8 [N, K/2] tensor")
        self.N, self.K = w.shape[0], 2 * w.shape[1]
        if (not isinstance(s, torch.Tensor) or s.dtype != u8 or not s.is_contiguous() or s.device != w.device
                or tuple(s.shape) != (self.N, w.shape[1] // 16) or w.shape[1] % 16):
            raise ValueError("s must be a contiguous uint8 [N, K/32] tensor beside w")
        self.x_dtype = torch.bfloat16 if x_dtype is None else x_dtype
        self._x_code, self._fp32 = _dtype_code(self.x_dtype), torch.float32
        self.device, self.max_M = w.device, int(max_M)
        if bias is not None and (bias.dtype != self.x_dtype or tuple(bias.shape) != (self.N,)
                                 or bias.device != w.device or not bias.is_contiguous()):
            raise ValueError("bias must be a contiguous [N] tensor of x's type beside w")
        nw, ns = ctypes.c_size_t(0), ctypes.c_size_t(0)
        st = lib().moe_linear_pack_bytes(self.N, self.K, ctypes.byref(nw), ctypes.byref(ns))
        if st != MOE_OK:
            raise MoeError(st, "moe_linear_pack_bytes")
        self.w_packed = torch.empty(nw.value, dtype=u8, device=w.device)
        self.s_packed = torch.empty(ns.value, dtype=u8, device=w.device)
        self.bias = bias
        here = torch.cuda.current_stream(self.device)
        st = lib().moe_pack_linear(_ptr(w), _ptr(s), self.N, self.K, _ptr(self.w_packed), _ptr(self.s_packed),
                                   here.cuda_stream)
        if st != MOE_OK:
            raise MoeError(st, "moe_pack_linear")
        here.synchronize()  # load time: calls on any stream find the weights packed
        h = ctypes.c_void_p()
        st = lib().moe_linear_create(self.N, self.K, self._x_code, _ptr(self.w_packed),
                                     _ptr(self.s_packed), None if bias is None else _ptr(bias), self.max_M,
                                     ctypes.byref(h))
        if st != MOE_OK:
            raise MoeError(st, "moe_linear_create")
        self._h = h

    def forward(self, x, out, residual=None, M: Optional[int] = None, stream=None):
        """out[:M] = x[:M] w^T (+ bias) (+ residual[:M]); out is of x's type or
        float32, residual of out's; residual may be out itself."""
        M = self._rows(x, M)
        ldx = self._check("x", x, self.x_dtype, M, self.K)
        wide = getattr(out, "dtype", None) is self._fp32
        y_dtype = self._fp32 if wide else self.x_dtype
        ldy = self._check("out", out, y_dtype, M, self.N)
        ldr = 0 if residual is None else self._check("residual", residual, y_dtype, M, self.N)
        st = lib().moe_linear_forward(
            self._h, M, x.data_ptr(), ldx, None if residual is None else residual.data_ptr(), ldr, out.data_ptr(), ldy,
            FP32 if wide else self._x_code, self._stream(stream))
        if st != MOE_OK:
            raise MoeError(st, "moe_linear_forward")
        return out


class _Sized(_Handle):
    """A handle whose calls may take a workspace: a uint8 tensor of at least
    workspace_bytes(M) for the call's M (a smaller M may need more), the caller's; calls that
    may overlap need one each."""

    def _create(self, name, *args):
        h = ctypes.c_void_p()
        st = getattr(lib(), name)(*args, ctypes.byref(h))
        if st != MOE_OK:
            raise MoeError(st, name)
        self._h = h

    def _bytes(self, name, *args):
        n = ctypes.c_size_t(0)
        st = getattr(lib(), name)(self._h, *args, ctypes.byref(n))
        if st != MOE_OK:
            raise MoeError(st, name)
        return n.value

    def _call(self, name, *args):
        st = getattr(lib(), name)(self._h, *args)
        if st != MOE_OK:
            raise MoeError(st, name)

    def _workspace(self, t):
        """(pointer, bytes) of a workspace tensor or None."""
        if t is None:
            return None, 0
        import torch  # (a module loaded long before: a dictionary's look-up)

        if not isinstance(t, torch.Tensor) or t.dtype is not torch.uint8 or not t.is_contiguous() or t.device != self.device:
            raise ValueError(f"workspace must be a contiguous uint8 tensor on {self.device}")
        return t.data_ptr(), t.numel()

    def _vector(self, name, t, dtype, n):
        """Pointer of a dense vector of at least n elements."""
        try:
            if t.dtype is dtype and t.dim() == 1 and t.shape[0] >= n and t.device == self.device and t.is_contiguous():
                return t.data_ptr()
        except AttributeError:
            raise TypeError(f"{name} must be a torch tensor") from None
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of at least {n} elements on {self.device}")


class _Product(_Sized):
    """What Dense and Gated share."""

    def _pre(self, pre, M, cols, dense=False):
        """Row distance and type of the saved arguments: of x's type or float32."""
        import torch

        wide = getattr(pre, "dtype", None) is torch.float32
        ld = self._check("pre", pre, torch.float32 if wide else self.dtype, M, cols, dense=dense)
        return ld, FP32 if wide else self._code

    def kernel(self, M: int, product: int = 0) -> str:
        """Which of its kernels a call of M rows launches for the forward product (0),
        the input's gradient (1) or the weight's (2) (profiling aid)."""
        name = getattr(lib(), self._destroy.replace("destroy", "kernel"))(self._h, int(M), int(product))
        if name is None:
            raise ValueError(f"M = {M} outside [1, {self.max_M}], product {product} not 0, 1 or 2, or no handle")
        return name.decode()


def _weight(name, w, rows_even=False):
    import torch

    if (not isinstance(w, torch.Tensor) or w.dim() != 2 or not w.is_contiguous()
            or w.dtype not in (torch.bfloat16, torch.float16) or (rows_even and w.shape[0] % 2)):
        raise ValueError(f"{name} must be a contiguous 2-d bfloat16 or float16 tensor" + (" of 2 I rows" if rows_even else ""))


def _activation(name):
    if name not in ACTIVATIONS:
        raise ValueError(f"activation {name!r} is none of {', '.join(ACTIVATIONS)}")
    return ACTIVATIONS[name]


class Dense(_Product):
    """Matrix product on 16-bit weights w [N, K] with bias [N], activation and
    residual in its epilogue, and its backward pass. w and bias are kept by
    reference: an optimizer may update them in place."""

    _destroy = "moe_dense_destroy"

    def __init__(self, w, bias=None, activation: str = "none", max_M: int = 1 << 20):
        _weight("w", w)
        act = _activation(activation)
        self.N, self.K = w.shape
        if bias is not None and (bias.dtype != w.dtype or tuple(bias.shape) != (self.N,) or bias.device != w.device
                                 or not bias.is_contiguous()):
            raise ValueError("bias must be a contiguous [N] tensor of w's type beside it")
        self.w, self.bias, self.dtype, self.device, self.max_M = w, bias, w.dtype, w.device, int(max_M)
        self.activation, self._code = activation, _dtype_code(w.dtype)
        self._create("moe_dense_create", self.N, self.K, self._code, _ptr(w), None if bias is None else _ptr(bias), act,
                     self.max_M)

    def workspace_bytes(self, M: int, train: bool = False, plain: bool = False) -> int:
        """Workspace of forward, with `train` of backward too, for M rows (fewer rows may
        need more); `plain`: of backward calls without dbias that read dy as it is, for
        which no activation, N and dy's row distance multiples of 8 and dy on 16 bytes are needed."""
        return self._bytes("moe_dense_workspace_bytes", int(M), 2 if train and plain else int(bool(train)))

    def forward(self, x, out, residual=None, pre=None, workspace=None, M: Optional[int] = None, stream=None):
        """out[:M] = act(x[:M] w^T + bias) (+ residual[:M]); out is of x's type or
        float32, residual of out's, and may be out itself. `pre` [M, N] of x's type or
        float32 takes the activation's argument, for backward."""
        import torch

        M = self._rows(x, M)
        ldx = self._check("x", x, self.dtype, M, self.K)
        wide = getattr(out, "dtype", None) is torch.float32
        y_dtype = torch.float32 if wide else self.dtype
        ldy = self._check("out", out, y_dtype, M, self.N)
        ldr = 0 if residual is None else self._check("residual", residual, y_dtype, M, self.N)
        ldp, p_code = (0, self._code) if pre is None else self._pre(pre, M, self.N)
        ws, nws = self._workspace(workspace)
        self._call("moe_dense_forward", M, x.data_ptr(), ldx, None if residual is None else residual.data_ptr(), ldr,
                   out.data_ptr(), ldy, FP32 if wide else self._code, None if pre is None else pre.data_ptr(), ldp, p_code, ws,
                   nws, self._stream(stream))
        return out

    def backward(self, dy, x, dx=None, dw=None, dbias=None, pre=None, workspace=None, M: Optional[int] = None, stream=None):
        """The gradients of x into dx[:M], of w into dw and of the bias into dbias
        (each may be None), for dy[:M] = the gradient of forward's out (in w's type);
        x may be None without dw, `pre` is what forward saved, needed with an activation."""
        M = self._rows(dy, M)
        lddy = self._check("dy", dy, self.dtype, M, self.N)
        ldx = 0 if x is None and dw is None else self._check("x", x, self.dtype, M, self.K)
        ldp, lddx, p_code = 0, 0, self._code
        if self.activation != "none":
            if pre is None:
                raise ValueError("backward through an activation needs pre")
            ldp, p_code = self._pre(pre, M, self.N)
        else:
            pre = None
        if dx is not None:
            lddx = self._check("dx", dx, self.dtype, M, self.K)
        if dw is not None:
            self._check("dw", dw, self.dtype, self.N, self.K, dense=True)
        ws, nws = self._workspace(workspace)
        self._call("moe_dense_backward", M, dy.data_ptr(), lddy, None if pre is None else pre.data_ptr(), ldp, p_code,
                   None if x is None else x.data_ptr(), ldx, None if dx is None else dx.data_ptr(), lddx,
                   None if dw is None else dw.data_ptr(),
                   None if dbias is None else self._vector("dbias", dbias, self.dtype, self.N), ws, nws, self._stream(stream))


class Gated(_Product):
    """Gated feed-forward block on 16-bit weights w13 [2I, H] (rows [0, I) gate, [I,
    2I) up): h = act(x Wg^T) * (x Wu^T), and its backward pass. w13 is kept by reference."""

    _destroy = "moe_gated_destroy"

    def __init__(self, w13, activation: str = "silu", max_M: int = 1 << 20):
        _weight("w13", w13, rows_even=True)
        act = _activation(activation)
        self.I, self.H = w13.shape[0] // 2, w13.shape[1]
        self.w13, self.dtype, self.device, self.max_M = w13, w13.dtype, w13.device, int(max_M)
        self.activation, self._code = activation, _dtype_code(w13.dtype)
        self._create("moe_gated_create", self.I, self.H, self._code, _ptr(w13), act, self.max_M)

    def workspace_bytes(self, M: int, train: bool = False) -> int:
        """Workspace of forward, with `train` of backward too, for M rows."""
        return self._bytes("moe_gated_workspace_bytes", int(M), int(bool(train)))

    def forward(self, x, out, pre=None, workspace=None, M: Optional[int] = None, stream=None):
        """out[:M] [M, I]; `pre` [M, 2I] (contiguous, of x's type or float32) takes [g u],
        for backward (float32 where the gradients' precision counts: 1.4 roundings of their type
        for 1.8)."""
        M = self._rows(x, M)
        ldx = self._check("x", x, self.dtype, M, self.H)
        ldh = self._check("out", out, self.dtype, M, self.I)
        p_code = self._code if pre is None else self._pre(pre, M, 2 * self.I, dense=True)[1]
        ws, nws = self._workspace(workspace)
        self._call("moe_gated_forward", M, x.data_ptr(), ldx, out.data_ptr(), ldh, None if pre is None else pre.data_ptr(),
                   p_code, ws, nws, self._stream(stream))
        return out

    def backward(self, dh, x, pre, dx=None, dw=None, workspace=None, M: Optional[int] = None, stream=None):
        """The gradients of x into dx[:M] and of w13 into dw (one may be None), for
        dh[:M] = the gradient of forward's out, `pre` what forward saved; x may be None without dw."""
        M = self._rows(dh, M)
        lddh = self._check("dh", dh, self.dtype, M, self.I)
        ldx = 0 if x is None and dw is None else self._check("x", x, self.dtype, M, self.H)
        p_code = self._pre(pre, M, 2 * self.I, dense=True)[1]
        lddx = 0 if dx is None else self._check("dx", dx, self.dtype, M, self.H)
        if dw is not None:
            self._check("dw", dw, self.dtype, 2 * self.I, self.H, dense=True)
        ws, nws = self._workspace(workspace)
        self._call("moe_gated_backward", M, dh.data_ptr(), lddh, pre.data_ptr(), p_code,
                   None if x is None else x.data_ptr(), ldx, None if dx is None else dx.data_ptr(), lddx,
                   None if dw is None else dw.data_ptr(), ws, nws, self._stream(stream))


class _Head(_Sized):
    """What TokenScores and Distill share: logits [M, V] of one type on one device."""

    def _init(self, V, dtype, device, max_M):
        import torch

        self.V, self.max_M = int(V), int(max_M)
        self.dtype = torch.float32 if dtype is None else dtype
        device = torch.device("cuda") if device is None else torch.device(device)
        if device.type == "cuda" and device.index is None and torch.cuda.is_available():
            device = torch.device("cuda", torch.cuda.current_device())
        self.device, self._i32, self._fp32 = device, torch.int32, torch.float32

    def _create_here(self, name, *args):
        import torch

        if self.device.type == "cuda" and torch.cuda.is_available():
            with torch.cuda.device(self.device):
                return self._create(name, *args)
        return self._create(name, *args)

    def _out(self, name, t, M, dtype=None):
        return None if t is None else self._vector(name, t, dtype or self._fp32, M)


class TokenScores(_Head):
    """Scores of given tokens from logits [M, V] of `dtype`: their log probabilities,
    the rows' entropies and top_k largest alternatives."""

    _destroy = "moe_scores_destroy"

    def __init__(self, V: int, top_k: int = 0, dtype=None, device=None, max_M: int = 1 << 20):
        self._init(V, dtype, device, max_M)
        self.top_k = int(top_k)
        self._create_here("moe_scores_create", self.V, self.top_k, _dtype_code(self.dtype), self.max_M)

    def workspace_bytes(self, M: int) -> int:
        return self._bytes("moe_scores_workspace_bytes", int(M))

    def forward(self, logits, tokens, logprobs, entropy=None, lse=None, top_logprobs=None, top_ids=None, workspace=None,
                M: Optional[int] = None, stream=None):
        """tokens (int32 [M]) to their logprobs [M], float32; entropy and lse [M] where
        given; top_logprobs and top_ids (int32) [M, top_k], equal logits by rising id.
        tokens and logprobs may both be None."""
        M = self._rows(logits, M)
        ldz = self._check("logits", logits, self.dtype, M, self.V)
        if self.top_k and (top_logprobs is None or top_ids is None):
            raise ValueError("top_logprobs and top_ids are needed with top_k above 0")
        tp = ti = None
        if self.top_k:
            self._check("top_logprobs", top_logprobs, self._fp32, M, self.top_k, dense=True)
            self._check("top_ids", top_ids, self._i32, M, self.top_k, dense=True)
            tp, ti = top_logprobs.data_ptr(), top_ids.data_ptr()
        ws, nws = self._workspace(workspace)
        self._call("moe_scores_forward", M, logits.data_ptr(), ldz, self._out("tokens", tokens, M, self._i32),
                   self._out("logprobs", logprobs, M), self._out("entropy", entropy, M), self._out("lse", lse, M), tp, ti, ws,
                   nws, self._stream(stream))
        return logprobs


class Distill(_Head):
    """Distillation of logits [M, V] from a teacher's k logits a row (t [M, k] float32 at
    tokens ids [M, k] int32, a negative id an empty slot) at a temperature."""

    _destroy = "moe_distill_destroy"

    def __init__(self, V: int, k: int, dtype=None, grad_dtype=None, temperature: float = 1.0, device=None,
                 max_M: int = 1 << 20):
        self._init(V, dtype, device, max_M)
        self.k, self.temperature = int(k), float(temperature)
        self.grad_dtype = self.dtype if grad_dtype is None else grad_dtype
        self._create_here("moe_distill_create", self.V, self.k, _dtype_code(self.dtype), _dtype_code(self.grad_dtype),
                          self.temperature, self.max_M)

    def workspace_bytes(self, M: int) -> int:
        return self._bytes("moe_distill_workspace_bytes", int(M))

    def kernel(self, M: int, step: int = 2) -> str:
        """Which of its kernels a call of M rows launches forward (0), backward (1) or for both
        at once (2), there with the gradient's rows as the logits' (profiling aid)."""
        name = lib().moe_distill_kernel(self._h, int(M), int(step))
        if name is None:
            raise ValueError(f"M = {M} outside [1, {self.max_M}], step {step} not 0, 1 or 2, or no handle")
        return name.decode()

    def _inputs(self, logits, ids, t, M):
        M = self._rows(logits, M)
        ldz = self._check("logits", logits, self.dtype, M, self.V)
        self._check("ids", ids, self._i32, M, self.k, dense=True)
        self._check("t", t, self._fp32, M, self.k, dense=True)
        return M, (logits.data_ptr(), ldz, ids.data_ptr(), t.data_ptr())

    def forward(self, logits, ids, t, loss, lse=None, workspace=None, M: Optional[int] = None, stream=None):
        """The rows' losses [M], and lse [M] for backward, float32."""
        M, args = self._inputs(logits, ids, t, M)
        ws, nws = self._workspace(workspace)
        self._call("moe_distill_forward", M, *args, self._vector("loss", loss, self._fp32, M), self._out("lse", lse, M), ws,
                   nws, self._stream(stream))
        return loss

    def backward(self, logits, ids, t, lse, weight, grad, M: Optional[int] = None, stream=None):
        """The logits' gradient into grad[:M] (may be logits itself), for weight [M] =
        the gradient of the rows' losses, lse what forward wrote."""
        M, args = self._inputs(logits, ids, t, M)
        ldg = self._check("grad", grad, self.grad_dtype, M, self.V)
        self._call("moe_distill_backward", M, *args, self._vector("lse", lse, self._fp32, M),
                   self._vector("weight", weight, self._fp32, M), grad.data_ptr(), ldg, self._stream(stream))
        return grad

    def forward_backward(self, logits, ids, t, weight, loss, grad, workspace=None, M: Optional[int] = None, stream=None):
        """Losses and gradient at once, for weights known beforehand."""
        M, args = self._inputs(logits, ids, t, M)
        ldg = self._check("grad", grad, self.grad_dtype, M, self.V)
        ws, nws = self._workspace(workspace)
        self._call("moe_distill_forward_backward", M, *args, self._vector("weight", weight, self._fp32, M),
                   self._vector("loss", loss, self._fp32, M), grad.data_ptr(), ldg, ws, nws, self._stream(stream))
        return loss


class Plan:
    """A plan for one shape, owning a device workspace allocated through torch."""

    def __init__(self, M: int, H: int, E: int, I: int, top_k: int, routed_scaling: float = 2.5,
                 shared_I: int = 0, device=None, weight_layout: int = LAYOUT_W13_PACKED):
        import torch

        self.shape = moe_shape(M, H, E, I, top_k, routed_scaling, shared_I)
        self._h = ctypes.c_void_p()
        st = lib().moe_plan_create(ctypes.byref(self.shape), ctypes.byref(self._h))
        if st != MOE_OK:
            raise MoeError(st, "moe_plan_create")
        self.device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        nbytes = lib().moe_plan_workspace_bytes(self._h)
        self.workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=self.device)
        st = lib().moe_plan_set_workspace(self._h, _ptr(self.workspace), self.workspace.numel(), _stream(None))
        if st != MOE_OK:
            raise MoeError(st, "moe_plan_set_workspace")
        self._shared = None
        self._events = None
        self._layout = LAYOUT_W13_PACKED
        self.set_weight_layout(weight_layout)

    def set_weight_layout(self, layout: int):
        """Declare the layout of the weights later calls pass (LAYOUT_W13_PACKED:
        w13/s13 from pack_w13, the only gate/up layout served; | LAYOUT_W2_PACKED:
        w2/s2 from pack_w2, required by and only by the MXFP4 mid)."""
        st = lib().moe_plan_set_weight_layout(self._h, int(layout))
        if st != MOE_OK:
            raise MoeError(st, "moe_plan_set_weight_layout")
        self._layout = int(layout)

    def _tensor(self, name, t, dtypes, numel=None, rows=None, cols=None, min_numel=None):
        """The library sees bare pointers: a tensor on another device, of
        another element type, strided, or smaller than the plan's shape would
        be read or written out of bounds, so each is checked here."""
        import torch

        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch tensor")
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, the plan on {self.device}")
        if t.dtype not in dtypes:
            raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if numel is not None and t.numel() != numel:
            raise ValueError(f"{name} holds {t.numel()} elements, the plan's shape needs {numel}")
        if min_numel is not None and t.numel() < min_numel:
            raise ValueError(f"{name} holds {t.numel()} elements, at least {min_numel} are needed")
        if cols is not None and (t.dim() != 2 or t.shape[1] != cols or t.shape[0] < rows):
            raise ValueError(f"{name} is {tuple(t.shape)}, expected at least [{rows}, {cols}]")

    def _check_call(self, M, x, logits, w13, s13, w2, s2, out):
        import torch

        s = self.shape
        if not 0 <= int(M) <= s.M:
            raise ValueError(f"M = {M} outside [0, {s.M}] (the plan's shape)")
        H, E, I = s.H, s.E, s.I
        bf16 = (torch.int16, torch.bfloat16)
        self._tensor("x", x, bf16, rows=M, cols=H)
        self._tensor("logits", logits, (torch.float32,), rows=M, cols=E)
        self._tensor("out", out, bf16, rows=M, cols=H)
        u8 = (torch.uint8,)
        self._tensor("w13", w13, u8, numel=E * 2 * I * H // 2)
        self._tensor("s13", s13, u8, numel=E * 2 * I * H // 32)
        self._tensor("w2", w2, u8, numel=E * H * I // 2)
        self._tensor("s2", s2, u8, numel=E * H * (16 if self._layout & LAYOUT_W2_PACKED else I // 32))

    def layout(self) -> Dict[str, int]:
        L = moe_ws_layout()
        st = lib().moe_plan_layout(self._h, ctypes.byref(L))
        if st != MOE_OK:
            raise MoeError(st, "moe_plan_layout")
        return {f: getattr(L, f) for f in LAYOUT_FIELDS}

    def set_shared(self, ws13, ss13, ws2, ss2, stream=None):
        """Bind the block-FP8 shared expert: row-major E4M3 ws13 [2 Is, H] and
        ws2 [H, Is] (uint8), fp32 block scales ss13 [2 Is/128, H/128] and ss2
        [H/128, Is/128]. The library packs the weights into a buffer this
        object allocates and keeps (with the scales)."""
        import torch

        H, Is = self.shape.H, self.shape.shared_I
        self._tensor("ws13", ws13, (torch.uint8,), numel=2 * Is * H)
        self._tensor("ss13", ss13, (torch.float32,), numel=(2 * Is // 128) * (H // 128))
        self._tensor("ws2", ws2, (torch.uint8,), numel=H * Is)
        self._tensor("ss2", ss2, (torch.float32,), numel=(H // 128) * (Is // 128))
        nbytes = lib().moe_plan_shared_pack_bytes(self._h)
        packed = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=self.device)
        st = lib().moe_plan_set_shared(self._h, _ptr(ws13), _ptr(ss13), _ptr(ws2), _ptr(ss2), _ptr(packed),
                                       packed.numel(), _stream(stream))
        if st != MOE_OK:
            raise MoeError(st, "moe_plan_set_shared")
        self._shared = (ss13, ss2, packed)  # kept alive while the plan uses them

    def set_shared_slot(self, on: bool):
        """Expert E-1 as the shared expert, fused as the last slot of every token."""
        st = lib().moe_plan_set_shared_slot(self._h, int(bool(on)))
        if st != MOE_OK:
            raise MoeError(st, "moe_plan_set_shared_slot")

    def set_tp_exchange(self, tp=None, rank=0, epoch=1, inbox=None, inbox_tags=None, push=(), push_tags=(),
                        status=None, spin_limit=1 << 20):
        """Tensor-parallel exchange epilogue (moe_plan_set_tp_exchange); tp=None
        turns it off. inbox: float64 [tp, M, H], inbox_tags: int32 [tp, M, H/512],
        push / push_tags: per rank (None at this rank), status: int32 [1]."""
        if tp is None:
            st = lib().moe_plan_set_tp_exchange(self._h, None)
            self._tpx = None
        else:
            import torch

            M, H = self.shape.M, self.shape.H
            tags = (torch.int32, torch.uint32)
            self._tensor("inbox", inbox, (torch.float64,), numel=tp * M * H)
            self._tensor("inbox_tags", inbox_tags, tags, numel=tp * M * (H // 512))
            self._tensor("status", status, tags, min_numel=1)
            for p in range(tp):
                if p != rank:
                    self._tensor(f"push[{p}]", push[p], (torch.float64,), min_numel=M * H)
                    self._tensor(f"push_tags[{p}]", push_tags[p], tags, min_numel=M * (H // 512))
            x = moe_tp_exchange()
            x.tp, x.rank, x.epoch, x.spin_limit = tp, rank, epoch, spin_limit
            x.inbox, x.inbox_tags, x.status = _ptr(inbox), _ptr(inbox_tags), _ptr(status)
            for p in range(tp):
                if p != rank:
                    x.push[p] = _ptr(push[p])
                    x.push_tags[p] = _ptr(push_tags[p])
            st = lib().moe_plan_set_tp_exchange(self._h, ctypes.byref(x))
            self._tpx = (inbox, inbox_tags, tuple(push), tuple(push_tags), status)  # kept alive
        if st != MOE_OK:
            raise MoeError(st, "moe_plan_set_tp_exchange")

    def set_mid_format(self, fmt: int):
        """MID_E4M3 (default) or MID_MXFP4 for the plan's later calls (the
        MXFP4 mid reads packed down weights: declare them with
        set_weight_layout(LAYOUT_W13_PACKED | LAYOUT_W2_PACKED))."""
        st = lib().moe_plan_set_mid_format(self._h, int(fmt))
        if st != MOE_OK:
            raise MoeError(st, "moe_plan_set_mid_format")

    def set_stage_events(self, events):
        """events: raw hipEvent_t handles (ints), [start0, stop0, start1, stop1, ...]
        for every stage; None clears."""
        if events is None:
            st = lib().moe_plan_set_stage_events(self._h, None, 0)
            self._events = None
        else:
            arr = (ctypes.c_void_p * len(events))(*events)
            st = lib().moe_plan_set_stage_events(self._h, arr, len(events))
            self._events = arr
        if st != MOE_OK:
            raise MoeError(st, "moe_plan_set_stage_events")

    def set_call_events(self, start, stop):
        """start/stop: raw hipEvent_t handles (ints) recorded at the first
        kernel's start and the last kernel's end of every call; None clears."""
        st = lib().moe_plan_set_call_events(self._h, start, stop)
        if st != MOE_OK:
            raise MoeError(st, "moe_plan_set_call_events")
        if start is not None:
            self._events = None

    def forward(self, x, logits, w13, s13, w2, s2, out, M: Optional[int] = None, stream=None):
        """Enqueue the call on `stream` (default: torch's current stream)."""
        if M is None:
            M = x.shape[0]
        self._check_call(M, x, logits, w13, s13, w2, s2, out)
        st = lib().moe_forward(self._h, int(M), _ptr(x), _ptr(logits), _ptr(w13), _ptr(s13), _ptr(w2),
                               _ptr(s2), _ptr(out), _stream(stream))
        if st != MOE_OK:
            raise MoeError(st, "moe_forward")
        return out

    def forward_noalloc(self, x, logits, w13, s13, w2, s2, out, M: Optional[int] = None, stream=None):
        """moe_forward_noalloc: the same call on the library's static device
        scratch instead of this plan's workspace (nothing is allocated)."""
        if M is None:
            M = x.shape[0]
        self._check_call(M, x, logits, w13, s13, w2, s2, out)
        st = lib().moe_forward_noalloc(self._h, int(M), _ptr(x), _ptr(logits), _ptr(w13), _ptr(s13), _ptr(w2),
                                       _ptr(s2), _ptr(out), _stream(stream))
        if st != MOE_OK:
            raise MoeError(st, "moe_forward_noalloc")
        return out

    def layer(self, x, router, w13, s13, w2, s2, out, M: Optional[int] = None, stream=None):
        """The whole layer of up to 16 tokens from their hidden states x
        (moe_layer_forward): `router` is a Router on [E, H] weights, the expert
        weights are those of forward (E4M3 mid). Leaves topk_ids and topk_w."""
        import torch

        if not isinstance(router, Router):
            raise TypeError("router must be a Router")
        M = x.shape[0] if M is None else int(M)
        s = self.shape
        if not 0 <= M <= s.M:
            raise ValueError(f"M = {M} outside [0, {s.M}] (the plan's shape)")
        H, codes = s.H, s.E * s.I * s.H
        bf16, u8 = (torch.int16, torch.bfloat16), (torch.uint8,)
        for name, t in (("x", x), ("out", out)):
            self._tensor(name, t, bf16, rows=M, cols=H)
        for name, t, n in (("w13", w13, codes), ("s13", s13, codes // 16), ("w2", w2, codes // 2),
                           ("s2", s2, codes // 32)):
            self._tensor(name, t, u8, numel=n)
        st = lib().moe_layer_forward(self._h, router._h, M, _ptr(x), _ptr(w13), _ptr(s13), _ptr(w2), _ptr(s2),
                                     _ptr(out), router._stream(stream))
        if st != MOE_OK:
            raise MoeError(st, "moe_layer_forward")
        return out

    def stage_launches(self, M: int):
        """Kernels each stage launches for a call of M tokens."""
        return [lib().moe_plan_stage_launches(self._h, int(M), i) for i in range(lib().moe_stage_count())]

    def view(self, name: str, dtype, shape):
        """A torch view of an intermediate inside the workspace (see moe_ws_layout)."""
        import math

        import torch

        off = self.layout()[name]
        itemsize = torch.empty(0, dtype=dtype).element_size()
        n = math.prod(shape)
        return self.workspace[off:off + n * itemsize].view(dtype).view(*shape)

    def close(self):
        if self._h:
            lib().moe_plan_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class HipEvents:
    """A few raw hipEvent_t handles from libamdhip64 (for per-stage timing)."""

    def __init__(self, n: int):
        self._hip = ctypes.CDLL("libamdhip64.so")
        self._hip.hipEventCreate.argtypes = [ctypes.POINTER(ctypes.c_void_p)]
        self._hip.hipEventElapsedTime.argtypes = [ctypes.POINTER(ctypes.c_float), ctypes.c_void_p, ctypes.c_void_p]
        self._hip.hipEventSynchronize.argtypes = [ctypes.c_void_p]
        self._hip.hipEventDestroy.argtypes = [ctypes.c_void_p]
        self._hip.hipEventRecord.argtypes = [ctypes.c_void_p, ctypes.c_void_p]
        self.handles = []
        for _ in range(n):
            h = ctypes.c_void_p()
            if self._hip.hipEventCreate(ctypes.byref(h)) != 0:
                raise RuntimeError("hipEventCreate failed")
            self.handles.append(h.value)

    def record(self, i: int, stream) -> None:
        """Record event i on a torch stream (or a raw hipStream_t)."""
        h = stream.cuda_stream if hasattr(stream, "cuda_stream") else stream
        if self._hip.hipEventRecord(self.handles[i], h) != 0:
            raise RuntimeError("hipEventRecord failed")

    def elapsed_ms(self, i: int, j: int) -> float:
        self._hip.hipEventSynchronize(self.handles[j])
        ms = ctypes.c_float(0)
        if self._hip.hipEventElapsedTime(ctypes.byref(ms), self.handles[i], self.handles[j]) != 0:
            raise RuntimeError("hipEventElapsedTime failed")
        return ms.value

    def close(self):
        for h in self.handles:
            self._hip.hipEventDestroy(h)
        self.handles = []
