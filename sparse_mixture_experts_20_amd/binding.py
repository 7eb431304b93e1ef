"""ctypes binding of the C ABI in ``include/moe.h`` (argument marshalling only).

Every step of the layer runs in ``libmoe.so``'s HIP kernels; this module only
turns torch device tensors into ``moe_tensor`` descriptors, passes torch's
current HIP stream, and raises :class:`MoeError` on a non-zero return code.
There is no fallback: if the library is missing, :func:`lib` raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import struct
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_F32, MOE_BF16 = 0, 1
MOE_MAX_EXPERTS, MOE_MAX_TOPK = 256, 16

#: every function the header declares
EXPORTS = ("moe_forward", "moe_workspace_size", "moe_capacity", "moe_error_string",
           "moe_router", "moe_router_workspace_size", "moe_dispatch", "moe_experts",
           "moe_expert_up", "moe_expert_down", "moe_expert_workspace_size", "moe_combine",
           "moe_forward_ex", "moe_experts_ex", "moe_expert_up_ex", "moe_expert_down_ex",
           "moe_backward", "moe_backward_ex", "moe_backward_workspace_size",
           "moe_forward_train", "moe_backward_after_forward", "moe_dispatch_workspace_size",
           "moe_expert_kernel_name", "moe_dispatch_noalloc", "moe_expert_down_compact",
           "moe_combine_compact", "moe_forward_few", "moe_few_workspace_size", "moe_linear",
           "moe_linear_workspace_size", "moe_linear_backward",
           "moe_linear_backward_workspace_size", "moe_layer_norm", "moe_layer_norm_backward",
           "moe_layer_norm_backward_workspace_size", "moe_quantize", "moe_dequantize",
           "moe_linear_quant", "moe_linear_quant_workspace_size", "moe_experts_quant",
           "moe_experts_quant_workspace_size", "moe_router_ex", "moe_router_ex_workspace_size",
           "moe_router_backward", "moe_router_backward_workspace_size", "moe_forward_routed",
           "moe_backward_routed")

MOE_ACT_RELU, MOE_ACT_GELU, MOE_ACT_NONE = 0, 1, 2
ACTS = {"relu": MOE_ACT_RELU, "gelu": MOE_ACT_GELU}
LINEAR_ACTS = {"none": MOE_ACT_NONE, "relu": MOE_ACT_RELU, "gelu": MOE_ACT_GELU}
MOE_FEW_MAX_TOKENS, MOE_NORM_MAX_WIDTH = 64, 16384


class MoeTensor(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("ndim", ctypes.c_int32),
                ("shape", ctypes.c_int64 * 4)]


class MoeStats(ctypes.Structure):
    _fields_ = [("stream", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t),
                ("topk_idx", ctypes.c_void_p), ("topk_gate", ctypes.c_void_p),
                ("slot", ctypes.c_void_p), ("used_capacity", ctypes.c_void_p),
                ("capacity", ctypes.c_int64),
                ("expert_demand", ctypes.c_void_p), ("expert_drops", ctypes.c_void_p),
                ("expert_gate_sum", ctypes.c_void_p), ("aux_stream", ctypes.c_void_p)]


class MoeExpertOpts(ctypes.Structure):
    _fields_ = [("activation", ctypes.c_int32), ("b_up", ctypes.c_void_p),
                ("b_down", ctypes.c_void_p), ("dropout", ctypes.c_float),
                ("dropout_seed", ctypes.c_uint64), ("dropout_offset", ctypes.c_uint64)]


class MoeQ4(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("zero", ctypes.c_void_p),
                ("group", ctypes.c_int32), ("ndim", ctypes.c_int32), ("shape", ctypes.c_int64 * 3)]


class MoeRouterOpts(ctypes.Structure):
    _fields_ = [("score", ctypes.c_int32), ("bias", ctypes.c_void_p), ("groups", ctypes.c_int32),
                ("keep_groups", ctypes.c_int32), ("group_best", ctypes.c_int32),
                ("renormalize", ctypes.c_int32), ("scale", ctypes.c_float),
                ("gates", ctypes.c_void_p)]


class MoeError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: error {code} ({error_string(code)})")


_lib = None
_T = ctypes.POINTER(MoeTensor)
_Q = ctypes.POINTER(MoeQ4)
_D = ctypes.c_char_p
_vp = ctypes.c_void_p
_i64 = ctypes.c_int64


def lib():
    """Load ``libmoe.so`` (built in-tree by ``sparse_mixture_experts_20_amd.build``)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it first "
                               "(python -m sparse_mixture_experts_20_amd.build)")
        L = ctypes.CDLL(LIB_PATH)
        L.moe_forward.argtypes = [_T, _T, _T, _T, _T, ctypes.c_int, ctypes.c_float, _T,
                                  ctypes.POINTER(MoeStats)]
        L.moe_forward.restype = ctypes.c_int
        L.moe_forward_ex.argtypes = [_T, _T, _T, _T, _T, ctypes.POINTER(MoeExpertOpts),
                                     ctypes.c_int, ctypes.c_float, _T, ctypes.POINTER(MoeStats)]
        L.moe_forward_ex.restype = ctypes.c_int
        L.moe_experts_ex.argtypes = [_T, _T, _T, ctypes.POINTER(MoeExpertOpts), ctypes.c_int,
                                     _i64, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
        L.moe_experts_ex.restype = ctypes.c_int
        L.moe_expert_up_ex.argtypes = [_T, _T, ctypes.POINTER(MoeExpertOpts), ctypes.c_int, _i64,
                                       _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
        L.moe_expert_up_ex.restype = ctypes.c_int
        L.moe_expert_down_ex.argtypes = [_i64, _T, ctypes.POINTER(MoeExpertOpts), ctypes.c_int,
                                         _i64, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_size_t,
                                         _vp]
        L.moe_expert_down_ex.restype = ctypes.c_int
        L.moe_expert_down_compact.argtypes = [_i64, _T, ctypes.POINTER(MoeExpertOpts),
                                              ctypes.c_int, _i64, _vp, _vp, _vp, _vp, _vp, _vp,
                                              _vp, ctypes.c_size_t, _vp]
        L.moe_expert_down_compact.restype = ctypes.c_int
        L.moe_backward.argtypes = [_T, _T, _T, _T, _T, ctypes.c_int, ctypes.c_float, _T, _T, _T,
                                   _T, _T, ctypes.POINTER(MoeStats)]
        L.moe_backward.restype = ctypes.c_int
        L.moe_backward_ex.argtypes = [_T, _T, _T, _T, _T, ctypes.POINTER(MoeExpertOpts),
                                      ctypes.c_int, ctypes.c_float, _T, _T, _T, _T, _T, _T, _T,
                                      ctypes.POINTER(MoeStats)]
        L.moe_backward_ex.restype = ctypes.c_int
        L.moe_backward_after_forward.argtypes = L.moe_backward_ex.argtypes
        L.moe_backward_after_forward.restype = ctypes.c_int
        L.moe_forward_train.argtypes = [_T, _T, _T, _T, _T, ctypes.POINTER(MoeExpertOpts),
                                        ctypes.c_int, ctypes.c_float, _T,
                                        ctypes.POINTER(MoeStats)]
        L.moe_forward_train.restype = ctypes.c_int
        L.moe_backward_workspace_size.argtypes = [_i64, _i64, _i64, _i64, ctypes.c_int,
                                                  ctypes.c_float, ctypes.c_int32]
        L.moe_backward_workspace_size.restype = ctypes.c_size_t
        L.moe_workspace_size.argtypes = [_i64, _i64, _i64, _i64, ctypes.c_int, ctypes.c_float,
                                         ctypes.c_int32]
        L.moe_workspace_size.restype = ctypes.c_size_t
        L.moe_capacity.argtypes = [_i64, _i64, ctypes.c_int, ctypes.c_float]
        L.moe_capacity.restype = _i64
        L.moe_error_string.argtypes = [ctypes.c_int]
        L.moe_error_string.restype = ctypes.c_char_p
        L.moe_router.argtypes = [_T, _T, _T, ctypes.c_int, _vp, _vp, _vp, ctypes.c_size_t, _vp]
        L.moe_router.restype = ctypes.c_int
        L.moe_router_workspace_size.argtypes = [_i64, _i64, _i64, ctypes.c_int32]
        L.moe_router_workspace_size.restype = ctypes.c_size_t
        L.moe_dispatch.argtypes = [_i64, _i64, ctypes.c_int, _i64, _vp, _vp, _vp, _vp, _vp, _vp,
                                   _vp, _vp, _vp, _vp, ctypes.c_size_t, _vp]
        L.moe_dispatch.restype = ctypes.c_int
        L.moe_dispatch_noalloc.argtypes = [_i64, _i64, ctypes.c_int, _i64, _vp, _vp, _vp, _vp,
                                           _vp, _vp, _vp, _vp, _vp, _vp]
        L.moe_dispatch_noalloc.restype = ctypes.c_int
        L.moe_dispatch_workspace_size.argtypes = [_i64, _i64, ctypes.c_int]
        L.moe_dispatch_workspace_size.restype = ctypes.c_size_t
        L.moe_expert_kernel_name.argtypes = [_i64, _i64, _i64, _i64, ctypes.c_int, ctypes.c_float,
                                             ctypes.c_int32, ctypes.c_int, ctypes.c_int,
                                             ctypes.c_char_p, ctypes.c_size_t]
        L.moe_expert_kernel_name.restype = ctypes.c_int
        L.moe_experts.argtypes = [_T, _T, _T, ctypes.c_int, _i64, _vp, _vp, _vp, _vp, _vp, _vp,
                                  ctypes.c_size_t, _vp]
        L.moe_experts.restype = ctypes.c_int
        L.moe_expert_up.argtypes = [_T, _T, ctypes.c_int, _i64, _vp, _vp, _vp, _vp, _vp,
                                    ctypes.c_size_t, _vp]
        L.moe_expert_up.restype = ctypes.c_int
        L.moe_expert_down.argtypes = [_i64, _T, ctypes.c_int, _i64, _vp, _vp, _vp, _vp, _vp, _vp,
                                      ctypes.c_size_t, _vp]
        L.moe_expert_down.restype = ctypes.c_int
        L.moe_expert_workspace_size.argtypes = [ctypes.c_int32]
        L.moe_expert_workspace_size.restype = ctypes.c_size_t
        L.moe_combine.argtypes = [_i64, _i64, ctypes.c_int, _T, _vp, _vp, _T, _vp]
        L.moe_combine.restype = ctypes.c_int
        L.moe_combine_compact.argtypes = [_i64, _i64, ctypes.c_int, _vp, _vp, _vp, _vp, _T, _vp]
        L.moe_combine_compact.restype = ctypes.c_int
        # (tensor descriptors of these calls are packed bytes, see _pack)
        L.moe_forward_few.argtypes = [_D, _D, _D, _D, _D, ctypes.POINTER(MoeExpertOpts),
                                      ctypes.c_int, ctypes.c_float, _D, ctypes.POINTER(MoeStats)]
        L.moe_forward_few.restype = ctypes.c_int
        L.moe_few_workspace_size.argtypes = L.moe_workspace_size.argtypes
        L.moe_few_workspace_size.restype = ctypes.c_size_t
        L.moe_linear.argtypes = [_D, _D, _D, ctypes.c_int32, _D, _D, _D, _vp, ctypes.c_size_t,
                                 _vp]
        L.moe_linear.restype = ctypes.c_int
        L.moe_linear_workspace_size.argtypes = [_i64, _i64, _i64]
        L.moe_linear_workspace_size.restype = ctypes.c_size_t
        L.moe_linear_backward.argtypes = [_D, _D, _D, ctypes.c_int32, _D, _D, _D, _D, _vp,
                                          ctypes.c_size_t, _vp]
        L.moe_linear_backward.restype = ctypes.c_int
        L.moe_linear_backward_workspace_size.argtypes = [_i64, _i64, _i64, ctypes.c_int32]
        L.moe_linear_backward_workspace_size.restype = ctypes.c_size_t
        L.moe_layer_norm.argtypes = [_D, _D, _D, _D, ctypes.c_float, _D, _D, _D, _D, _vp]
        L.moe_layer_norm.restype = ctypes.c_int
        L.moe_layer_norm_backward.argtypes = [_D, _D, _D, _D, _D, _D, _D, _D, _D, _vp,
                                              ctypes.c_size_t, _vp]
        L.moe_layer_norm_backward.restype = ctypes.c_int
        L.moe_layer_norm_backward_workspace_size.argtypes = [_i64, _i64]
        L.moe_layer_norm_backward_workspace_size.restype = ctypes.c_size_t
        L.moe_quantize.argtypes = [_D, _Q, _vp]
        L.moe_quantize.restype = ctypes.c_int
        L.moe_dequantize.argtypes = [_Q, _D, _vp]
        L.moe_dequantize.restype = ctypes.c_int
        L.moe_linear_quant.argtypes = [_D, _Q, _D, ctypes.c_int32, _D, _D, _vp, ctypes.c_size_t, _vp]
        L.moe_linear_quant.restype = ctypes.c_int
        L.moe_linear_quant_workspace_size.argtypes = [_i64, _i64, _i64, ctypes.c_int32]
        L.moe_linear_quant_workspace_size.restype = ctypes.c_size_t
        L.moe_experts_quant.argtypes = [_D, _vp, _vp, ctypes.c_int, _Q, _Q,
                                     ctypes.POINTER(MoeExpertOpts), _D, _vp, ctypes.c_size_t, _vp]
        L.moe_experts_quant.restype = ctypes.c_int
        L.moe_experts_quant_workspace_size.argtypes = [_i64, _i64, _i64, _i64, ctypes.c_int,
                                                    ctypes.c_int32]
        L.moe_experts_quant_workspace_size.restype = ctypes.c_size_t
        _O = ctypes.POINTER(MoeRouterOpts)
        L.moe_router_ex.argtypes = [_D, _D, _D, _O, ctypes.c_int, _vp, _vp, _D, _vp,
                                    ctypes.c_size_t, _vp]
        L.moe_router_ex.restype = ctypes.c_int
        L.moe_router_ex_workspace_size.argtypes = [_i64, _i64, _i64, ctypes.c_int32]
        L.moe_router_ex_workspace_size.restype = ctypes.c_size_t
        L.moe_router_backward.argtypes = [_D, _D, _O, ctypes.c_int, _vp, _D, _D, _D, _D, _D, _D,
                                          _vp, ctypes.c_size_t, _vp]
        L.moe_router_backward.restype = ctypes.c_int
        L.moe_router_backward_workspace_size.argtypes = [_i64, _i64, _i64, ctypes.c_int]
        L.moe_router_backward_workspace_size.restype = ctypes.c_size_t
        L.moe_forward_routed.argtypes = [_D, _D, _D, ctypes.POINTER(MoeExpertOpts), ctypes.c_int,
                                         ctypes.c_float, _D, ctypes.POINTER(MoeStats)]
        L.moe_forward_routed.restype = ctypes.c_int
        L.moe_backward_routed.argtypes = [_D, _D, _D, ctypes.POINTER(MoeExpertOpts), ctypes.c_int,
                                          ctypes.c_float, _D, _D, _D, _D, _D, _D, _D,
                                          ctypes.POINTER(MoeStats)]
        L.moe_backward_routed.restype = ctypes.c_int
        _lib = L
    return _lib


def error_string(code: int) -> str:
    return lib().moe_error_string(code).decode()


def _check(rc: int, where: str):
    if rc != 0:
        raise MoeError(rc, where)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return MOE_F32
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def desc(t: Optional[torch.Tensor]):
    """A ``moe_tensor`` for a contiguous device tensor (None -> NULL)."""
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    if t.dim() > 4:
        raise ValueError("at most 4 dimensions")
    shape = (ctypes.c_int64 * 4)(*(list(t.shape) + [0] * (4 - t.dim())))
    return MoeTensor(ctypes.c_void_p(t.data_ptr()), _dtype_code(t), t.dim(), shape)


def _ref(d):
    return None if d is None else ctypes.byref(d)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


_AUX_STREAMS = {}   # device index -> the binding's second stream for "auto"


def _aux_stream(aux, device):
    """The backward's second stream: ``"auto"`` takes the binding's own stream
    of the tensors' device (created once at the default priority and reused:
    creating a stream per call would cost more than the overlap gains), None
    runs the call on one stream, or pass a ``torch.cuda.Stream``. Returns
    (stream object or None, handle)."""
    if isinstance(aux, str):
        if aux != "auto":
            raise ValueError("aux_stream must be 'auto', None or a torch.cuda.Stream")
        dev = torch.device(device)
        index = dev.index if dev.index is not None else torch.cuda.current_device()
        aux = _AUX_STREAMS.get(index)
        if aux is None:
            aux = _AUX_STREAMS[index] = torch.cuda.Stream(device=index)
    return aux, (None if aux is None else ctypes.c_void_p(aux.cuda_stream))


class ExpertOpts:
    """``moe_expert_opts`` for an activation name, optional fp32 bias tensors
    (b_up [E, d_ff], b_down [E, d]) and an optional training-mode dropout
    ``(p, seed, offset)`` on the expert outputs; keeps the descriptors alive."""

    def __init__(self, act: str = "relu", b_up: Optional[torch.Tensor] = None,
                 b_down: Optional[torch.Tensor] = None, dropout=None):
        if act not in ACTS:
            raise ValueError("act must be 'relu' or 'gelu'")
        p, seed, offset = dropout if dropout is not None else (0.0, 0, 0)
        self._d = (desc(b_up), desc(b_down))
        self.c = MoeExpertOpts(ACTS[act],
                               None if self._d[0] is None else ctypes.addressof(self._d[0]),
                               None if self._d[1] is None else ctypes.addressof(self._d[1]),
                               float(p), int(seed), int(offset))

    def ref(self):
        return ctypes.byref(self.c)


def _opts(act, b_up, b_down, dropout=None):
    if act == "relu" and b_up is None and b_down is None and (dropout is None or
                                                              dropout[0] == 0.0):
        return None
    return ExpertOpts(act, b_up, b_down, dropout)


def capacity(N: int, E: int, k: int, capacity_factor: float) -> int:
    return int(lib().moe_capacity(N, E, k, capacity_factor))


def workspace_size(N: int, d: int, E: int, d_ff: int, k: int, capacity_factor: float,
                   dtype: torch.dtype) -> int:
    code = MOE_BF16 if dtype == torch.bfloat16 else MOE_F32
    return int(lib().moe_workspace_size(N, d, E, d_ff, k, capacity_factor, code))


def alloc_workspace(nbytes: int, device="cuda") -> torch.Tensor:
    # torch's caching allocator returns 256-byte (or better) aligned blocks
    return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)


class Stats:
    """Exported routing arrays (device tensors or None) and the capacity; with
    router statistics, demand / drops (int32 [E]) and gate_sum (fp32 [E])."""

    def __init__(self, idx, gate, slot, used, capacity, demand=None, drops=None, gate_sum=None):
        self.idx, self.gate, self.slot, self.used, self.capacity = idx, gate, slot, used, capacity
        self.demand, self.drops, self.gate_sum = demand, drops, gate_sum


def _router_stats(E, dev, on):
    if not on:
        return None, None, None
    return (torch.empty((E,), dtype=torch.int32, device=dev),
            torch.empty((E,), dtype=torch.int32, device=dev),
            torch.empty((E,), dtype=torch.float32, device=dev))


def forward(x: torch.Tensor, W_g: torch.Tensor, noise: Optional[torch.Tensor],
            W_up: torch.Tensor, W_down: torch.Tensor, k: int, capacity_factor: float,
            out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
            export: bool = True, stream=None, act: str = "relu",
            b_up: Optional[torch.Tensor] = None, b_down: Optional[torch.Tensor] = None,
            dropout=None, router_stats: bool = False):
    """Run ``moe_forward`` (``moe_forward_ex`` for an expert variant; dropout:
    ``(p, seed, offset)`` or None). Returns ``(out, Stats)``; with ``export=False`` the
    routing arrays stay in the workspace and Stats only carries the capacity;
    ``router_stats`` also exports the per-expert demand, drops and gate sums."""
    N = x.numel() // x.shape[-1]
    d = x.shape[-1]
    E, d_ff = W_up.shape[0], W_up.shape[1]
    if out is None:
        out = torch.empty_like(x)
    if workspace is None:
        workspace = alloc_workspace(workspace_size(N, d, E, d_ff, k, capacity_factor, x.dtype),
                                    x.device)
    dev = x.device
    idx = gate = slot = used = None
    if export:
        idx = torch.empty((N, k), dtype=torch.int32, device=dev)
        gate = torch.empty((N, k), dtype=torch.float32, device=dev)
        slot = torch.empty((N, k), dtype=torch.int32, device=dev)
        used = torch.empty((E,), dtype=torch.int32, device=dev)
    dem, drp, gsum = _router_stats(E, dev, router_stats)
    st = MoeStats(_stream(stream), ctypes.c_void_p(workspace.data_ptr()), workspace.numel(),
                  _ptr(idx), _ptr(gate), _ptr(slot), _ptr(used), -1, _ptr(dem), _ptr(drp),
                  _ptr(gsum), None)
    dx, dg, dn, du, dd, do = desc(x), desc(W_g), desc(noise), desc(W_up), desc(W_down), desc(out)
    o = _opts(act, b_up, b_down, dropout)
    if o is None:
        rc = lib().moe_forward(_ref(dx), _ref(dg), _ref(dn), _ref(du), _ref(dd), k,
                               capacity_factor, _ref(do), ctypes.byref(st))
    else:
        rc = lib().moe_forward_ex(_ref(dx), _ref(dg), _ref(dn), _ref(du), _ref(dd), o.ref(), k,
                                  capacity_factor, _ref(do), ctypes.byref(st))
    _check(rc, "moe_forward")
    return out, Stats(idx, gate, slot, used, int(st.capacity), dem, drp, gsum)


def backward_workspace_size(N: int, d: int, E: int, d_ff: int, k: int, capacity_factor: float,
                            dtype: torch.dtype) -> int:
    code = MOE_BF16 if dtype == torch.bfloat16 else MOE_F32
    return int(lib().moe_backward_workspace_size(N, d, E, d_ff, k, capacity_factor, code))


def backward(x, W_g, noise, W_up, W_down, k: int, capacity_factor: float, dout,
             workspace=None, stream=None, export: bool = False, act: str = "relu",
             b_up: Optional[torch.Tensor] = None, b_down: Optional[torch.Tensor] = None,
             dropout=None, aux_stream="auto"):
    """Run ``moe_backward`` (``moe_backward_ex`` for GELU, biases or dropout): returns
    (dx [N, d], dW_g [E, d], dW_up [E, d_ff, d], dW_down [E, d, d_ff]), all
    fp32, followed by db_up [E, d_ff] and db_down [E, d] (None where the layer
    has no such bias) when the layer has a bias. With ``export=True`` returns
    ``(grads, Stats)`` with the recomputed routing, as ``forward`` does."""
    N, d = x.numel() // x.shape[-1], x.shape[-1]
    E, d_ff = W_up.shape[0], W_up.shape[1]
    dev = x.device
    dx = torch.empty((N, d), dtype=torch.float32, device=dev)
    dwg = torch.empty((E, d), dtype=torch.float32, device=dev)
    dwu = torch.empty((E, d_ff, d), dtype=torch.float32, device=dev)
    dwd = torch.empty((E, d, d_ff), dtype=torch.float32, device=dev)
    dbu = None if b_up is None else torch.empty((E, d_ff), dtype=torch.float32, device=dev)
    dbd = None if b_down is None else torch.empty((E, d), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = alloc_workspace(
            backward_workspace_size(N, d, E, d_ff, k, capacity_factor, x.dtype), dev)
    idx = gate = slot = used = None
    if export:
        idx = torch.empty((N, k), dtype=torch.int32, device=dev)
        gate = torch.empty((N, k), dtype=torch.float32, device=dev)
        slot = torch.empty((N, k), dtype=torch.int32, device=dev)
        used = torch.empty((E,), dtype=torch.int32, device=dev)
    aux, aux_h = _aux_stream(aux_stream, dev)
    st = MoeStats(_stream(stream), ctypes.c_void_p(workspace.data_ptr()), workspace.numel(),
                  _ptr(idx), _ptr(gate), _ptr(slot), _ptr(used), -1, None, None, None, aux_h)
    ds = [desc(t) for t in (x, W_g, noise, W_up, W_down, dout, dx, dwg, dwu, dwd, dbu, dbd)]
    o = _opts(act, b_up, b_down, dropout)
    r = [_ref(a) for a in ds]
    if o is None:
        rc = lib().moe_backward(r[0], r[1], r[2], r[3], r[4], k, capacity_factor, r[5], r[6],
                                r[7], r[8], r[9], ctypes.byref(st))
    else:
        rc = lib().moe_backward_ex(r[0], r[1], r[2], r[3], r[4], o.ref(), k, capacity_factor,
                                   r[5], r[6], r[7], r[8], r[9], r[10], r[11], ctypes.byref(st))
    _check(rc, "moe_backward")
    grads = (dx, dwg, dwu, dwd)
    if b_up is not None or b_down is not None:
        grads = grads + (dbu, dbd)
    if export:
        return grads, Stats(idx, gate, slot, used, int(st.capacity))
    return grads


class Forward:
    """A reusable call: descriptors, workspace and stats built once, so that
    timing loops measure only the enqueue of the kernels."""

    def __init__(self, x, W_g, noise, W_up, W_down, k, capacity_factor, out=None,
                 export=False, stream=None, act="relu", b_up=None, b_down=None,
                 dropout=None, router_stats=False):
        self.tensors = (x, W_g, noise, W_up, W_down)
        N, d = x.numel() // x.shape[-1], x.shape[-1]
        E, d_ff = W_up.shape[0], W_up.shape[1]
        self.out = torch.empty_like(x) if out is None else out
        self.workspace = alloc_workspace(
            workspace_size(N, d, E, d_ff, k, capacity_factor, x.dtype), x.device)
        dev = x.device
        self.idx = self.gate = self.slot = self.used = None
        if export:
            self.idx = torch.empty((N, k), dtype=torch.int32, device=dev)
            self.gate = torch.empty((N, k), dtype=torch.float32, device=dev)
            self.slot = torch.empty((N, k), dtype=torch.int32, device=dev)
            self.used = torch.empty((E,), dtype=torch.int32, device=dev)
        self.k, self.cf = k, capacity_factor
        self._d = [desc(x), desc(W_g), desc(noise), desc(W_up), desc(W_down), desc(self.out)]
        self.demand, self.drops, self.gate_sum = _router_stats(E, dev, router_stats)
        self.stats = MoeStats(_stream(stream), ctypes.c_void_p(self.workspace.data_ptr()),
                              self.workspace.numel(), _ptr(self.idx), _ptr(self.gate),
                              _ptr(self.slot), _ptr(self.used), -1, _ptr(self.demand),
                              _ptr(self.drops), _ptr(self.gate_sum), None)
        self._args = [_ref(a) for a in self._d]
        self._opts = _opts(act, b_up, b_down, dropout)
        self._biases = (b_up, b_down)
        self._fn = lib().moe_forward if self._opts is None else lib().moe_forward_ex

    def __call__(self):
        a = self._args
        if self._opts is None:
            rc = self._fn(a[0], a[1], a[2], a[3], a[4], self.k, self.cf, a[5],
                          ctypes.byref(self.stats))
        else:
            rc = self._fn(a[0], a[1], a[2], a[3], a[4], self._opts.ref(), self.k, self.cf, a[5],
                          ctypes.byref(self.stats))
        if rc != 0:
            raise MoeError(rc, "moe_forward")
        return self.out


class Backward:
    """A prepared ``moe_backward`` / ``moe_backward_ex`` call: the gradient
    tensors, workspace and descriptors are built once, so repeated calls only
    cross the C ABI."""

    def __init__(self, x, W_g, noise, W_up, W_down, k, capacity_factor, dout, stream=None,
                 act="relu", b_up=None, b_down=None, dropout=None, aux_stream="auto"):
        N, d = x.numel() // x.shape[-1], x.shape[-1]
        E, d_ff = W_up.shape[0], W_up.shape[1]
        dev = x.device
        self.tensors = (x, W_g, noise, W_up, W_down, dout, b_up, b_down)
        self.dx = torch.empty((N, d), dtype=torch.float32, device=dev)
        self.dW_g = torch.empty((E, d), dtype=torch.float32, device=dev)
        self.dW_up = torch.empty((E, d_ff, d), dtype=torch.float32, device=dev)
        self.dW_down = torch.empty((E, d, d_ff), dtype=torch.float32, device=dev)
        self.db_up = None if b_up is None else torch.empty((E, d_ff), dtype=torch.float32,
                                                           device=dev)
        self.db_down = None if b_down is None else torch.empty((E, d), dtype=torch.float32,
                                                               device=dev)
        self.workspace = alloc_workspace(
            backward_workspace_size(N, d, E, d_ff, k, capacity_factor, x.dtype), dev)
        self.k, self.cf = k, capacity_factor
        self._d = [desc(t) for t in (x, W_g, noise, W_up, W_down, dout, self.dx, self.dW_g,
                                     self.dW_up, self.dW_down, self.db_up, self.db_down)]
        self._args = [_ref(a) for a in self._d]
        self._opts = _opts(act, b_up, b_down, dropout)
        self.aux, aux_h = _aux_stream(aux_stream, dev)
        self.stats = MoeStats(_stream(stream), ctypes.c_void_p(self.workspace.data_ptr()),
                              self.workspace.numel(), None, None, None, None, -1, None, None,
                              None, aux_h)

    def __call__(self):
        a = self._args
        if self._opts is None:
            rc = lib().moe_backward(a[0], a[1], a[2], a[3], a[4], self.k, self.cf, a[5], a[6],
                                    a[7], a[8], a[9], ctypes.byref(self.stats))
        else:
            rc = lib().moe_backward_ex(a[0], a[1], a[2], a[3], a[4], self._opts.ref(), self.k,
                                       self.cf, a[5], a[6], a[7], a[8], a[9], a[10], a[11],
                                       ctypes.byref(self.stats))
        if rc != 0:
            raise MoeError(rc, "moe_backward")
        return self.dx, self.dW_g, self.dW_up, self.dW_down


class TrainStep:
    """``moe_forward_train`` + ``moe_backward_after_forward`` on one shared
    workspace: ``forward()`` returns out and keeps the forward state,
    ``backward(dout)`` returns (dx, dW_g, dW_up, dW_down[, db_up, db_down])
    from it. Tensors, workspace and descriptors are built once."""

    def __init__(self, x, W_g, noise, W_up, W_down, k, capacity_factor, stream=None,
                 act="relu", b_up=None, b_down=None, dropout=None, export=False,
                 aux_stream="auto"):
        N, d = x.numel() // x.shape[-1], x.shape[-1]
        E, d_ff = W_up.shape[0], W_up.shape[1]
        dev = x.device
        self.tensors = (x, W_g, noise, W_up, W_down, b_up, b_down)
        self.out = torch.empty_like(x)
        self.dx = torch.empty((N, d), dtype=torch.float32, device=dev)
        self.dW_g = torch.empty((E, d), dtype=torch.float32, device=dev)
        self.dW_up = torch.empty((E, d_ff, d), dtype=torch.float32, device=dev)
        self.dW_down = torch.empty((E, d, d_ff), dtype=torch.float32, device=dev)
        self.db_up = None if b_up is None else torch.empty((E, d_ff), dtype=torch.float32,
                                                           device=dev)
        self.db_down = None if b_down is None else torch.empty((E, d), dtype=torch.float32,
                                                               device=dev)
        self.workspace = alloc_workspace(
            backward_workspace_size(N, d, E, d_ff, k, capacity_factor, x.dtype), dev)
        self.idx = self.gate = self.slot = self.used = None
        if export:
            self.idx = torch.empty((N, k), dtype=torch.int32, device=dev)
            self.gate = torch.empty((N, k), dtype=torch.float32, device=dev)
            self.slot = torch.empty((N, k), dtype=torch.int32, device=dev)
            self.used = torch.empty((E,), dtype=torch.int32, device=dev)
        self.k, self.cf = k, capacity_factor
        self._opts = ExpertOpts(act, b_up, b_down, dropout)
        self._d = [desc(t) for t in (x, W_g, noise, W_up, W_down, self.out, self.dx, self.dW_g,
                                     self.dW_up, self.dW_down, self.db_up, self.db_down)]
        self._a = [_ref(a) for a in self._d]
        self._dout = None
        self.aux, aux_h = _aux_stream(aux_stream, dev)
        self.stats = MoeStats(_stream(stream), ctypes.c_void_p(self.workspace.data_ptr()),
                              self.workspace.numel(), _ptr(self.idx), _ptr(self.gate),
                              _ptr(self.slot), _ptr(self.used), -1, None, None, None, aux_h)

    def forward(self):
        a = self._a
        _check(lib().moe_forward_train(a[0], a[1], a[2], a[3], a[4], self._opts.ref(), self.k,
                                       self.cf, a[5], ctypes.byref(self.stats)),
               "moe_forward_train")
        return self.out

    def backward(self, dout):
        if self._dout is None or self._dout[0] is not dout:
            self._dout = (dout, desc(dout))
        a = self._a
        _check(lib().moe_backward_after_forward(
            a[0], a[1], a[2], a[3], a[4], self._opts.ref(), self.k, self.cf,
            ctypes.byref(self._dout[1]), a[6], a[7], a[8], a[9], a[10], a[11],
            ctypes.byref(self.stats)), "moe_backward_after_forward")
        g = (self.dx, self.dW_g, self.dW_up, self.dW_down)
        if self.db_up is not None or self.db_down is not None:
            g = g + (self.db_up, self.db_down)
        return g


def router_workspace_size(N: int, d: int, E: int, dtype: torch.dtype) -> int:
    code = MOE_BF16 if dtype == torch.bfloat16 else MOE_F32
    return int(lib().moe_router_workspace_size(N, d, E, code))


def router(x, W_g, noise, k, idx=None, gate=None, workspace=None, stream=None):
    N = x.numel() // x.shape[-1]
    if idx is None:
        idx = torch.empty((N, k), dtype=torch.int32, device=x.device)
    if gate is None:
        gate = torch.empty((N, k), dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace = alloc_workspace(router_workspace_size(N, x.shape[-1], W_g.shape[0], x.dtype),
                                    x.device)
    dx, dg, dn = desc(x), desc(W_g), desc(noise)
    _check(lib().moe_router(_ref(dx), _ref(dg), _ref(dn), k, _ptr(idx), _ptr(gate),
                            _ptr(workspace), workspace.numel(), _stream(stream)), "moe_router")
    return idx, gate


def expert_kernel_name(N: int, d: int, E: int, d_ff: int, k: int, capacity_factor: float,
                       dtype: torch.dtype, product: int, dropout: bool = False) -> str:
    """Name of the kernel instantiation the library launches for the up
    (product 0) or down (product 1) expert product of such a layer."""
    code = MOE_BF16 if dtype == torch.bfloat16 else MOE_F32
    buf = ctypes.create_string_buffer(256)
    n = lib().moe_expert_kernel_name(N, d, E, d_ff, k, capacity_factor, code, product,
                                     int(dropout), buf, 256)
    _check(min(n, 0), "moe_expert_kernel_name")
    return buf.value.decode()


def dispatch_workspace_size(N: int, E: int, k: int) -> int:
    return int(lib().moe_dispatch_workspace_size(N, E, k))


def dispatch(idx: torch.Tensor, E: int, capacity_: int, stream=None, gate=None,
             router_stats: bool = False, workspace=None):
    """Returns (slot [N,k], used [E], slot_token [E, min(C,N)], tiles [2(E+1)]);
    with ``router_stats`` also (demand [E], drops [E], gate_sum [E]) (gate_sum
    needs ``gate``, else it is None)."""
    N, k = idx.shape
    ceff = min(capacity_, N)
    dev = idx.device
    slot = torch.empty((N, k), dtype=torch.int32, device=dev)
    used = torch.empty((E,), dtype=torch.int32, device=dev)
    slot_token = torch.full((E, max(ceff, 1)), -1, dtype=torch.int32, device=dev)
    tiles = torch.empty((2 * (E + 1),), dtype=torch.int32, device=dev)
    dem, drp, gsum = _router_stats(E, dev, router_stats)
    if gate is None:
        gsum = None
    if workspace is None:
        n = dispatch_workspace_size(N, E, k)
        workspace = alloc_workspace(n, dev) if n > 0 else None
    wp, wn = _ws_args(workspace)
    _check(lib().moe_dispatch(N, E, k, capacity_, _ptr(idx), _ptr(gate), _ptr(slot), _ptr(used),
                              _ptr(slot_token), _ptr(tiles), _ptr(dem), _ptr(drp), _ptr(gsum),
                              wp, wn, _stream(stream)), "moe_dispatch")
    if router_stats:
        return slot, used, slot_token, tiles, (dem, drp, gsum)
    return slot, used, slot_token, tiles


def expert_workspace_size(dtype: torch.dtype) -> int:
    code = MOE_BF16 if dtype == torch.bfloat16 else MOE_F32
    return int(lib().moe_expert_workspace_size(code))


def _expert_ws(workspace, dtype, device):
    """``"auto"``: scratch of moe_expert_workspace_size(); None: no K-split."""
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be 'auto', None or a uint8 device tensor")
        n = expert_workspace_size(dtype)
        return alloc_workspace(n, device) if n > 0 else None
    return workspace


def _ws_args(ws):
    return (None, 0) if ws is None else (ctypes.c_void_p(ws.data_ptr()), ws.numel())


def experts(x, W_up, W_down, k, capacity_, used, slot_token, tiles, H=None, Y=None,
            workspace="auto", stream=None, act="relu", b_up=None, b_down=None,
            dropout=None):
    """Returns (H [E, min(C,N), d_ff] in x's dtype and Y [N*k, d] fp32)."""
    N, d = x.numel() // x.shape[-1], x.shape[-1]
    E, d_ff = W_up.shape[0], W_up.shape[1]
    ceff = min(capacity_, N)
    if H is None:
        H = torch.zeros((E, max(ceff, 1), d_ff), dtype=x.dtype, device=x.device)
    if Y is None:
        Y = torch.zeros((N * k, d), dtype=torch.float32, device=x.device)
    dx, du, dd = desc(x), desc(W_up), desc(W_down)
    if not slot_token.is_contiguous():
        raise ValueError("slot_token must be a contiguous [E, min(C, N)] tensor")
    wp, wn = _ws_args(_expert_ws(workspace, x.dtype, x.device))
    o = _opts(act, b_up, b_down, dropout)
    if o is None:
        _check(lib().moe_experts(_ref(dx), _ref(du), _ref(dd), k, capacity_, _ptr(used),
                                 _ptr(slot_token), _ptr(tiles), _ptr(H), _ptr(Y), wp, wn,
                                 _stream(stream)),
               "moe_experts")
    else:
        _check(lib().moe_experts_ex(_ref(dx), _ref(du), _ref(dd), o.ref(), k, capacity_,
                                    _ptr(used), _ptr(slot_token), _ptr(tiles), _ptr(H), _ptr(Y),
                                    wp, wn, _stream(stream)),
               "moe_experts_ex")
    return H, Y


def expert_up(x, W_up, k, capacity_, used, slot_token, tiles, H, workspace="auto",
              stream=None, act="relu", b_up=None):
    dx, du = desc(x), desc(W_up)
    wp, wn = _ws_args(_expert_ws(workspace, x.dtype, x.device))
    o = _opts(act, b_up, None)
    if o is None:
        rc = lib().moe_expert_up(_ref(dx), _ref(du), k, capacity_, _ptr(used), _ptr(slot_token),
                                 _ptr(tiles), _ptr(H), wp, wn, _stream(stream))
    else:
        rc = lib().moe_expert_up_ex(_ref(dx), _ref(du), o.ref(), k, capacity_, _ptr(used),
                                    _ptr(slot_token), _ptr(tiles), _ptr(H), wp, wn,
                                    _stream(stream))
    _check(rc, "moe_expert_up")
    return H


def expert_down(N, W_down, k, capacity_, used, slot_token, tiles, H, Y, workspace="auto",
                stream=None, b_down=None, dropout=None):
    dd = desc(W_down)
    wp, wn = _ws_args(_expert_ws(workspace, W_down.dtype, W_down.device))
    o = _opts("relu", None, b_down, dropout)
    if o is None:
        rc = lib().moe_expert_down(N, _ref(dd), k, capacity_, _ptr(used), _ptr(slot_token),
                                   _ptr(tiles), _ptr(H), _ptr(Y), wp, wn, _stream(stream))
    else:
        rc = lib().moe_expert_down_ex(N, _ref(dd), o.ref(), k, capacity_, _ptr(used),
                                      _ptr(slot_token), _ptr(tiles), _ptr(H), _ptr(Y), wp, wn,
                                      _stream(stream))
    _check(rc, "moe_expert_down")
    return Y


def y_groups(d):
    """Shift bytes per compact expert output row (one per 32 columns)."""
    return (d + 31) // 32


def expert_down_compact(N, W_down, k, capacity_, used, slot_token, tiles, H, Y16=None,
                        Ysh=None, workspace="auto", stream=None, b_down=None, dropout=None):
    """The down product writing compact rows, as the fused bf16 layer keeps
    them: returns (Y16 [N*k, d] float16, Ysh [N, ceil(d/32), k] int8); the
    value of Y16[t*k + j, c] is Y16[t*k + j, c] * 2**-Ysh[t, c // 32, j]."""
    import torch
    d = W_down.shape[1]
    if Y16 is None:
        Y16 = torch.zeros((N * k, d), dtype=torch.float16, device=W_down.device)
    if Ysh is None:
        Ysh = torch.zeros((N, y_groups(d), k), dtype=torch.int8, device=W_down.device)
    dd = desc(W_down)
    wp, wn = _ws_args(_expert_ws(workspace, W_down.dtype, W_down.device))
    o = _opts("relu", None, b_down, dropout) or ExpertOpts("relu", None, b_down)
    rc = lib().moe_expert_down_compact(N, _ref(dd), o.ref(), k, capacity_, _ptr(used),
                                       _ptr(slot_token), _ptr(tiles), _ptr(H), _ptr(Y16),
                                       _ptr(Ysh), wp, wn, _stream(stream))
    _check(rc, "moe_expert_down_compact")
    return Y16, Ysh


def combine_compact(Y16, Ysh, gate, slot, out, stream=None):
    """Combine over compact rows (expert_down_compact's Y16, Ysh)."""
    N, k = gate.shape
    d = out.shape[-1]
    do = desc(out)
    _check(lib().moe_combine_compact(N, d, k, _ptr(Y16), _ptr(Ysh), _ptr(gate), _ptr(slot),
                                     _ref(do), _stream(stream)), "moe_combine_compact")
    return out


def combine(Y, gate, slot, out, stream=None):
    """Y: [N*k, d] fp32 or bf16 expert outputs, assignment-major."""
    N, k = gate.shape
    d = out.shape[-1]
    dy, do = desc(Y), desc(out)
    _check(lib().moe_combine(N, d, k, _ref(dy), _ptr(gate), _ptr(slot), _ref(do),
                             _stream(stream)), "moe_combine")
    return out


# --------------------------------------------------------------------------
# The rest of the feed-forward half: the layer for a few tokens, the linear
# product, the layer norm
# --------------------------------------------------------------------------
# A call of these takes a few microseconds on the GPU, so its arguments are
# marshalled with little Python: a descriptor is the 48 bytes of a moe_tensor
# (pointer, dtype, rank, extents), handed over as a bytes object.
_PACK = [struct.Struct("=Qii%dq%dx" % (n, 8 * (4 - n))).pack for n in range(5)]
_CODE = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}


def _pack(t: Optional[torch.Tensor], index: int):
    """The ``moe_tensor`` of a contiguous tensor on device ``index`` as bytes
    (None -> NULL)."""
    if t is None:
        return None
    if t.get_device() != index:
        raise ValueError(f"a tensor on {t.device}, others on cuda:{index}: the library takes "
                         "device pointers of one GPU")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    code = _CODE.get(t.dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {t.dtype}")
    shape = t.shape
    n = len(shape)
    if n > 4:
        raise ValueError("at most 4 dimensions")
    return _PACK[n](t.data_ptr(), code, n, *shape)


def _device_of(t: torch.Tensor) -> int:
    index = t.get_device()
    if index < 0:
        raise ValueError("tensors must be on a HIP device")
    return index


def _scratch(workspace, index: int):
    """(pointer, bytes) of a workspace tensor, or (None, 0)."""
    if workspace is None:
        return None, 0
    if workspace.get_device() != index:
        raise ValueError("the workspace is on another device")
    if not workspace.is_contiguous():
        raise ValueError("the workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _stream_of(index: int):
    # (the handle of torch's current stream without building a Stream object)
    return torch._C._cuda_getCurrentRawStream(index)


def _on_stream(fn):
    """``stream=``: the call and everything it allocates belong to that stream
    (memory allocated for one stream and used on another could be handed out
    again while the call still runs)."""
    @functools.wraps(fn)
    def call(*args, stream=None, **kw):
        if stream is None:
            return fn(*args, **kw)
        for t in (*args, *kw.values()):
            if isinstance(t, Q4):
                t = t.data
            if isinstance(t, torch.Tensor):
                if t.get_device() != stream.device.index:
                    raise ValueError(f"a tensor on {t.device}, the stream on {stream.device}")
                break
        with torch.cuda.stream(stream):
            return fn(*args, **kw)
    return call


def _run(index: int, where: str, fn, *args):
    """Call ``fn(*args)`` with the tensors' device current."""
    if index == torch.cuda.current_device():
        rc = fn(*args)
    else:
        with torch.cuda.device(index):
            rc = fn(*args)
    if rc != 0:
        raise MoeError(rc, where)


def few_workspace_size(N: int, d: int, E: int, d_ff: int, k: int, capacity_factor: float,
                       dtype: torch.dtype) -> int:
    code = MOE_BF16 if dtype == torch.bfloat16 else MOE_F32
    return int(lib().moe_few_workspace_size(N, d, E, d_ff, k, capacity_factor, code))


@_on_stream
def forward_few(x: torch.Tensor, W_g: torch.Tensor, noise: Optional[torch.Tensor],
                W_up: torch.Tensor, W_down: torch.Tensor, k: int, capacity_factor: float,
                out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                export: bool = True, act: str = "relu",
                b_up: Optional[torch.Tensor] = None, b_down: Optional[torch.Tensor] = None,
                router_stats: bool = False):
    """Run ``moe_forward_few`` (at most ``MOE_FEW_MAX_TOKENS`` tokens): the
    arguments and results of :func:`forward`, without dropout."""
    N, d = x.numel() // x.shape[-1], x.shape[-1]
    E, d_ff = W_up.shape[0], W_up.shape[1]
    dev, index = x.device, _device_of(x)
    if out is None:
        out = torch.empty_like(x)
    if workspace is None:
        workspace = alloc_workspace(few_workspace_size(N, d, E, d_ff, k, capacity_factor, x.dtype),
                                    dev)
    idx = gate = slot = used = None
    if export:
        idx = torch.empty((N, k), dtype=torch.int32, device=dev)
        gate = torch.empty((N, k), dtype=torch.float32, device=dev)
        slot = torch.empty((N, k), dtype=torch.int32, device=dev)
        used = torch.empty((E,), dtype=torch.int32, device=dev)
    dem, drp, gsum = _router_stats(E, dev, router_stats)
    ws, wn = _scratch(workspace, index)
    st = MoeStats(_stream_of(index), ws, wn, _ptr(idx), _ptr(gate), _ptr(slot),
                  _ptr(used), -1, _ptr(dem), _ptr(drp), _ptr(gsum), None)
    _pack(b_up, index), _pack(b_down, index)   # (same checks as every tensor)
    o = _opts(act, b_up, b_down)
    _run(index, "moe_forward_few", lib().moe_forward_few, _pack(x, index), _pack(W_g, index),
         _pack(noise, index), _pack(W_up, index), _pack(W_down, index),
         None if o is None else o.ref(), k, capacity_factor, _pack(out, index), ctypes.byref(st))
    return out, Stats(idx, gate, slot, used, int(st.capacity), dem, drp, gsum)


class FewLayer:
    """A layer kept for decoding: the weights' descriptors, the workspace and
    (with ``export``) the routing buffers are built once, for up to
    ``max_tokens`` tokens; ``layer(x, noise=None, out=None)`` runs
    ``moe_forward_few`` on the current stream and returns ``(out, Stats)``.
    Calls share the workspace and the routing buffers, so they must not overlap
    (calls on one stream do not; between streams, order them with events).
    The layer keeps the memory of the weights it was given: it sees updates in
    place, and not memory that a tensor is given later (``W.data = ...``).
    ``out`` is a new tensor unless given. The routing in a returned ``Stats`` is
    the layer's own buffers: valid until the next call."""

    def __init__(self, W_g, W_up, W_down, k, capacity_factor, act="relu", b_up=None, b_down=None,
                 max_tokens=MOE_FEW_MAX_TOKENS, export=False, router_stats=False):
        E, d_ff, d = W_up.shape
        dev, index = W_up.device, _device_of(W_up)
        # the memory that the descriptors point at, whatever becomes of the tensors
        self.tensors = tuple(t if t is None else t.detach() for t in
                             (W_g, W_up, W_down, b_up, b_down))
        self.k, self.cf, self.max_tokens, self.index = k, capacity_factor, max_tokens, index
        n = few_workspace_size(max_tokens, d, E, d_ff, k, capacity_factor, W_up.dtype)
        if n == 0:
            raise ValueError("sizes outside moe_forward_few's limits")
        self.workspace = alloc_workspace(n, dev)
        self._w = [_pack(t, index) for t in (W_g, W_up, W_down)]
        _pack(b_up, index), _pack(b_down, index)   # (same checks as every tensor)
        self._opts = _opts(act, b_up, b_down)
        self._o = None if self._opts is None else self._opts.ref()
        idx = gate = slot = used = None
        if export:
            idx = torch.empty((max_tokens, k), dtype=torch.int32, device=dev)
            gate = torch.empty((max_tokens, k), dtype=torch.float32, device=dev)
            slot = torch.empty((max_tokens, k), dtype=torch.int32, device=dev)
            used = torch.empty((E,), dtype=torch.int32, device=dev)
        self._routing = (idx, gate, slot, used)
        self._counts = _router_stats(E, dev, router_stats)
        dem, drp, gsum = self._counts
        self.stats = MoeStats(None, self.workspace.data_ptr(), self.workspace.numel(), _ptr(idx),
                              _ptr(gate), _ptr(slot), _ptr(used), -1, _ptr(dem), _ptr(drp),
                              _ptr(gsum), None)
        self._sref = ctypes.byref(self.stats)
        self._fn = lib().moe_forward_few
        self._home = _stream_of(index)   # the stream the buffers were allocated for

    def __call__(self, x, noise=None, out=None, stream=None):
        if stream is not None:
            if stream.device.index != self.index:
                raise ValueError(f"the layer is on cuda:{self.index}, the stream on "
                                 f"{stream.device}")
            with torch.cuda.stream(stream):
                return self(x, noise, out)
        N = x.numel() // x.shape[-1]
        if N > self.max_tokens:
            raise ValueError(f"{N} tokens: this layer was built for {self.max_tokens}")
        if out is None:
            out = torch.empty_like(x)
        index, w, st = self.index, self._w, self.stats
        handle = _stream_of(index)   # (a ctypes field reads a handle of 0 back as None)
        st.stream = handle
        if handle != self._home:
            # keep the buffers until that stream is done, should the layer go first
            s = torch.cuda.current_stream(index)
            for b in (self.workspace, *self._routing, *self._counts):
                if b is not None:
                    b.record_stream(s)
        _run(index, "moe_forward_few", self._fn, _pack(x, index), w[0], _pack(noise, index), w[1],
             w[2], self._o, self.k, self.cf, _pack(out, index), self._sref)
        idx, gate, slot, used = self._routing
        if idx is not None and N != self.max_tokens:
            idx, gate, slot = idx[:N], gate[:N], slot[:N]
        return out, Stats(idx, gate, slot, used, st.capacity, *self._counts)


def _linear_act(act):
    if act not in LINEAR_ACTS:
        raise ValueError("act must be 'none', 'relu' or 'gelu'")
    return LINEAR_ACTS[act]


def linear_workspace_size(N: int, K: int, M: int) -> int:
    return int(lib().moe_linear_workspace_size(N, K, M))


@_on_stream
def linear(x, W, bias=None, act: str = "none", residual=None, out=None, keep_z: bool = False,
           workspace=None):
    """``act(x W^T + bias) + residual`` (bf16; x [..., K], W [M, K]): returns
    ``(out, z)``, z the bf16 pre-activations with ``keep_z``, else None."""
    K, M = x.shape[-1], W.shape[0]
    index = _device_of(x)
    if out is None:
        out = torch.empty((*x.shape[:-1], M), dtype=x.dtype, device=x.device)
    z = torch.empty_like(out) if keep_z else None
    if workspace is None:
        n = linear_workspace_size(x.numel() // K, K, M)
        workspace = alloc_workspace(n, x.device) if n else None
    ws, wn = _scratch(workspace, index)
    _run(index, "moe_linear", lib().moe_linear, _pack(x, index), _pack(W, index),
         _pack(bias, index), _linear_act(act), _pack(residual, index), _pack(out, index),
         _pack(z, index), ws, wn, _stream_of(index))
    return out, z


def linear_backward_workspace_size(N: int, K: int, M: int, act: str = "none") -> int:
    return int(lib().moe_linear_backward_workspace_size(N, K, M, _linear_act(act)))


@_on_stream
def linear_backward(x, W, z, dout, act: str = "none", bias: bool = True, need_dx: bool = True,
                    need_dW: bool = True, dx_dtype=torch.float32, dW_dtype=torch.float32,
                    workspace=None):
    """Gradients of :func:`linear` for ``dout``: ``(dx, dW, dbias)``, None for
    the ones not asked for; z is the forward's (None without an activation)."""
    N, K, M = x.numel() // x.shape[-1], x.shape[-1], W.shape[0]
    dev, index = x.device, _device_of(x)
    dx = torch.empty(x.shape, dtype=dx_dtype, device=dev) if need_dx else None
    dW = torch.empty((M, K), dtype=dW_dtype, device=dev) if need_dW else None
    db = torch.empty((M,), dtype=torch.float32, device=dev) if bias else None
    if workspace is None:
        n = linear_backward_workspace_size(N, K, M, act)
        workspace = alloc_workspace(n, dev) if n else None
    ws, wn = _scratch(workspace, index)
    _run(index, "moe_linear_backward", lib().moe_linear_backward, _pack(x, index),
         _pack(W, index), _pack(z, index), _linear_act(act), _pack(dout, index),
         _pack(dx, index), _pack(dW, index), _pack(db, index), ws, wn, _stream_of(index))
    return dx, dW, db


@_on_stream
def layer_norm(x, weight, bias=None, eps: float = 1e-5, residual=None, h=None, out=None,
               stats: bool = False):
    """Layer norm of ``x`` (of ``h = x + residual`` when given, h returned):
    ``(out, h, mean, rstd)``; h is x without a residual, mean and rstd (fp32,
    one per row: what the backward needs) are None unless ``stats``."""
    index = _device_of(x)
    if out is None:
        out = torch.empty_like(x)
    if residual is not None and h is None:
        h = torch.empty_like(x)
    mean = rstd = None
    if stats:
        N = x.numel() // x.shape[-1]
        mean = torch.empty(N, dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
    _run(index, "moe_layer_norm", lib().moe_layer_norm, _pack(x, index), _pack(residual, index),
         _pack(weight, index), _pack(bias, index), eps, _pack(h, index), _pack(out, index),
         _pack(mean, index), _pack(rstd, index), _stream_of(index))
    return out, (x if h is None else h), mean, rstd


def layer_norm_backward_workspace_size(N: int, d: int) -> int:
    return int(lib().moe_layer_norm_backward_workspace_size(N, d))


@_on_stream
def layer_norm_backward(h, weight, mean, rstd, dout, dres=None, bias: bool = True, dx=None,
                        workspace=None):
    """Gradients of :func:`layer_norm` for ``dout`` (and ``dres``, what reaches
    h along the residual path): ``(dx, dweight, dbias)``, dbias None without
    ``bias``. h, mean and rstd are the forward's."""
    d = h.shape[-1]
    index = _device_of(h)
    if dx is None:
        dx = torch.empty_like(h)
    dw = torch.empty(d, dtype=torch.float32, device=h.device)
    db = torch.empty_like(dw) if bias else None
    if workspace is None:
        n = layer_norm_backward_workspace_size(h.numel() // d, d)
        workspace = alloc_workspace(n, h.device) if n else None
    ws, wn = _scratch(workspace, index)
    _run(index, "moe_layer_norm_backward", lib().moe_layer_norm_backward, _pack(h, index),
         _pack(weight, index), _pack(mean, index), _pack(rstd, index), _pack(dout, index),
         _pack(dres, index), _pack(dx, index), _pack(dw, index), _pack(db, index), ws, wn,
         _stream_of(index))
    return dx, dw, db


# --------------------------------------------------------------------------
# Weights of 4 bits with group scales
# --------------------------------------------------------------------------
class Q4:
    """4-bit weights: ``data`` uint8 [.., M, K / 2] (even column in the low
    half of a byte), ``scale`` bf16 [.., M, K / group] and ``zero`` bf16 like
    it, or None (8 everywhere), of one matrix or of E: the values
    ``(q - zero) * scale``. Keeps the memory of the tensors it was given."""

    def __init__(self, data, scale, zero=None, group=128):
        if data.dtype != torch.uint8:
            raise TypeError("data must be uint8, two weights to a byte")
        if data.dim() not in (2, 3):
            raise ValueError("data must have 2 or 3 dimensions")
        if group not in (32, 64, 128):
            raise ValueError("group must be 32, 64 or 128")
        K = data.shape[-1] * 2
        index = _device_of(data)
        for t in (scale, zero):
            if t is None:
                continue
            if t.dtype != torch.bfloat16:
                raise TypeError("scale and zero must be bfloat16")
            if K % group or tuple(t.shape) != (*data.shape[:-1], K // group):
                raise ValueError(f"scale and zero must be {(*data.shape[:-1], K // group)}")
            if t.get_device() != index:
                raise ValueError("the tensors are on different devices")
        if not all(t is None or t.is_contiguous() for t in (data, scale, zero)):
            raise ValueError("tensors must be contiguous")
        self.data, self.scale = data.detach(), scale.detach()
        self.zero = None if zero is None else zero.detach()
        self.group, self.index = group, index
        self.shape = (*data.shape[:-1], K)
        self._c = MoeQ4(data.data_ptr(), scale.data_ptr(),
                        None if zero is None else zero.data_ptr(), group, data.dim(),
                        (ctypes.c_int64 * 3)(*self.shape))
        self._ref = ctypes.byref(self._c)

    def ref(self, index: int):
        """The ``moe_q4`` for a call on device ``index``."""
        if index != self.index:
            raise ValueError(f"weights on cuda:{self.index}, other tensors on cuda:{index}: the "
                             "library takes device pointers of one GPU")
        return self._ref


@_on_stream
def quantize_q4(W, group: int = 128, zero: bool = False) -> Q4:
    """The nearest 4-bit weights of ``W`` (fp32 or bf16, [M, K] or [E, M, K]),
    with zero points or symmetric: a :class:`Q4`."""
    index = _device_of(W)
    if group not in (32, 64, 128) or W.shape[-1] % group:
        raise ValueError("group must be 32, 64 or 128 and divide the last dimension")
    lead, K = W.shape[:-1], W.shape[-1]
    data = torch.empty((*lead, K // 2), dtype=torch.uint8, device=W.device)
    scale = torch.empty((*lead, K // group), dtype=torch.bfloat16, device=W.device)
    q = Q4(data, scale, torch.empty_like(scale) if zero else None, group)
    _run(index, "moe_quantize", lib().moe_quantize, _pack(W, index), q.ref(index),
         _stream_of(index))
    return q


@_on_stream
def dequantize_q4(q: Q4, out=None, dtype=torch.bfloat16):
    """The weights that ``q`` stands for (``out``, or a new tensor of ``dtype``)."""
    index = q.index
    if out is None:
        out = torch.empty(q.shape, dtype=dtype, device=q.data.device)
    _run(index, "moe_dequantize", lib().moe_dequantize, q.ref(index), _pack(out, index),
         _stream_of(index))
    return out


def linear_q4_workspace_size(N: int, K: int, M: int, group: int = 128) -> int:
    return int(lib().moe_linear_quant_workspace_size(N, K, M, group))


@_on_stream
def linear_q4(x, W: Q4, bias=None, act: str = "none", residual=None, out=None, workspace=None):
    """``act(x W^T + bias) + residual`` of at most ``MOE_FEW_MAX_TOKENS`` rows
    (bf16; x [..., K]) with 4-bit weights [M, K]."""
    M, K = W.shape[-2], x.shape[-1]
    index = _device_of(x)
    if out is None:
        out = torch.empty((*x.shape[:-1], M), dtype=x.dtype, device=x.device)
    if workspace is None:
        n = linear_q4_workspace_size(x.numel() // K, K, M, W.group)
        workspace = alloc_workspace(n, x.device) if n else None
    ws, wn = _scratch(workspace, index)
    _run(index, "moe_linear_quant", lib().moe_linear_quant, _pack(x, index), W.ref(index),
         _pack(bias, index), _linear_act(act), _pack(residual, index), _pack(out, index), ws, wn,
         _stream_of(index))
    return out


def experts_q4_workspace_size(N: int, d: int, E: int, d_ff: int, k: int, group: int = 128) -> int:
    return int(lib().moe_experts_quant_workspace_size(N, d, E, d_ff, k, group))


def _routing_ptrs(idx, gate, N, k, index):
    """Pointers of a caller's routing: ids int32 and gates fp32 [N, k]."""
    for t, dt, name in ((idx, torch.int32, "idx"), (gate, torch.float32, "gate")):
        if t.dtype != dt:
            raise TypeError(f"{name} must be {dt}")
        if t.numel() != N * k or t.shape[-1] != k or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [{N}, {k}] tensor")
        if t.get_device() != index:
            raise ValueError(f"{name} is on another device")
    return idx.data_ptr(), gate.data_ptr()


@_on_stream
def experts_q4(x, idx, gate, W_up: Q4, W_down: Q4, act: str = "relu", b_up=None, b_down=None,
               out=None, workspace=None):
    """The routed experts of at most ``MOE_FEW_MAX_TOKENS`` tokens with 4-bit
    weights (W_up [E, d_ff, d], W_down [E, d, d_ff]) for the routing ``idx``
    (int32) and ``gate`` (fp32) [N, k] of :func:`router` or :func:`route`."""
    N, d, k = x.numel() // x.shape[-1], x.shape[-1], idx.shape[-1]
    index = _device_of(x)
    ip, gp = _routing_ptrs(idx, gate, N, k, index)
    if out is None:
        out = torch.empty_like(x)
    if workspace is None:
        n = experts_q4_workspace_size(N, d, W_up.shape[0], W_up.shape[-2], k, W_up.group)
        workspace = alloc_workspace(n, x.device) if n else None
    ws, wn = _scratch(workspace, index)
    _pack(b_up, index), _pack(b_down, index)   # (same checks as every tensor)
    o = _opts(act, b_up, b_down)
    _run(index, "moe_experts_quant", lib().moe_experts_quant, _pack(x, index), ip, gp, k,
         W_up.ref(index), W_down.ref(index), None if o is None else o.ref(), _pack(out, index),
         ws, wn, _stream_of(index))
    return out


# --------------------------------------------------------------------------
# Routing with a balance bias, groups and renormalised gates; the layer for a
# routing that the caller has
# --------------------------------------------------------------------------
SCORES = {"softmax": 0, "sigmoid": 1}


def _route_opts(score, bias, groups, keep_groups, group_best, renormalize, scale, index,
                gates=None):
    """(``moe_router_opts`` by reference, what it points at)."""
    if score not in SCORES:
        raise ValueError("score must be 'softmax' or 'sigmoid'")
    b = _pack(bias, index)
    # (the bias' descriptor: the packed bytes, kept alive by the caller)
    at = None if b is None else ctypes.cast(ctypes.c_char_p(b), ctypes.c_void_p)
    o = MoeRouterOpts(SCORES[score], at, groups, keep_groups, group_best, int(renormalize), scale,
                      gates)
    return ctypes.byref(o), (o, b)


def route_workspace_size(N: int, d: int, E: int, dtype: torch.dtype) -> int:
    code = MOE_BF16 if dtype == torch.bfloat16 else MOE_F32
    return int(lib().moe_router_ex_workspace_size(N, d, E, code))


@_on_stream
def route(x, W_g, k: int, noise=None, bias=None, score: str = "softmax", groups: int = 1,
          keep_groups: int = 0, group_best: int = 1, renormalize: bool = False,
          scale: float = 1.0, export_scores: bool = False, workspace=None):
    """Run ``moe_router_ex``: ``(idx, gate, scores)``, idx int32 and gate fp32
    [N, k], scores the fp32 [N, E] softmax or sigmoid scores with
    ``export_scores`` (what the backward, of bf16 x alone, needs), else None."""
    N, d, E = x.numel() // x.shape[-1], x.shape[-1], W_g.shape[0]
    index, dev = _device_of(x), x.device
    idx = torch.empty((N, k), dtype=torch.int32, device=dev)
    gate = torch.empty((N, k), dtype=torch.float32, device=dev)
    scores = torch.empty((N, E), dtype=torch.float32, device=dev) if export_scores else None
    if workspace is None:
        n = route_workspace_size(N, d, E, x.dtype)
        workspace = alloc_workspace(n, dev) if n else None
    ws, wn = _scratch(workspace, index)
    o, keep = _route_opts(score, bias, groups, keep_groups, group_best, renormalize, scale, index)
    _run(index, "moe_router_ex", lib().moe_router_ex, _pack(x, index), _pack(W_g, index),
         _pack(noise, index), o, k, idx.data_ptr(), gate.data_ptr(), _pack(scores, index), ws, wn,
         _stream_of(index))
    return idx, gate, scores


def route_backward_workspace_size(N: int, d: int, E: int, k: int) -> int:
    return int(lib().moe_router_backward_workspace_size(N, d, E, k))


@_on_stream
def route_backward(x, W_g, idx, scores, dgate, dscores=None, dres=None, score: str = "softmax",
                   renormalize: bool = False, scale: float = 1.0, need_dx: bool = True,
                   need_dW: bool = True, dx_dtype=torch.float32, dx=None, workspace=None,
                   gate=None):
    """Gradients of :func:`route` for ``dgate`` [N, k] (and ``dscores`` [N, E],
    what an auxiliary loss gives the scores): ``(dx, dW_g)``, None for the ones
    not asked for; ``dres`` is added to dx. idx and scores are the forward's, and
    gate, if given: renormalised softmax gates of experts whose scores underflow
    (chosen by a bias far above them) have their gradient from it alone."""
    N, d, E, k = x.numel() // x.shape[-1], x.shape[-1], W_g.shape[0], idx.shape[-1]
    index, dev = _device_of(x), x.device
    ip, _ = _routing_ptrs(idx, dgate, N, k, index)
    if dx is None and need_dx:
        dx = torch.empty(x.shape, dtype=dx_dtype, device=dev)
    dW = torch.empty((E, d), dtype=torch.float32, device=dev) if need_dW else None
    if workspace is None:
        n = route_backward_workspace_size(N, d, E, k)
        workspace = alloc_workspace(n, dev) if n else None
    ws, wn = _scratch(workspace, index)
    gp = None if gate is None else _routing_ptrs(idx, gate, N, k, index)[1]
    o, keep = _route_opts(score, None, 1, 0, 1, renormalize, scale, index, gp)
    _run(index, "moe_router_backward", lib().moe_router_backward, _pack(x, index),
         _pack(W_g, index), o, k, ip, _pack(scores, index), _pack(dgate, index),
         _pack(dscores, index), _pack(dres, index), _pack(dx, index), _pack(dW, index), ws, wn,
         _stream_of(index))
    return dx, dW


@_on_stream
def forward_routed(x, idx, gate, W_up, W_down, capacity_factor: float, out=None, workspace=None,
                   act: str = "relu", b_up=None, b_down=None, dropout=None,
                   router_stats: bool = False):
    """Run ``moe_forward_routed``: :func:`forward` for the routing ``idx`` (int32)
    and ``gate`` (fp32) [N, k]. Returns ``(out, Stats)``."""
    N, d, k = x.numel() // x.shape[-1], x.shape[-1], idx.shape[-1]
    E, d_ff = W_up.shape[0], W_up.shape[1]
    index, dev = _device_of(x), x.device
    ip, gp = _routing_ptrs(idx, gate, N, k, index)
    if out is None:
        out = torch.empty_like(x)
    if workspace is None:
        workspace = alloc_workspace(workspace_size(N, d, E, d_ff, k, capacity_factor, x.dtype),
                                    dev)
    slot = torch.empty((N, k), dtype=torch.int32, device=dev)
    used = torch.empty((E,), dtype=torch.int32, device=dev)
    dem, drp, gsum = _router_stats(E, dev, router_stats)
    ws, wn = _scratch(workspace, index)
    st = MoeStats(_stream_of(index), ws, wn, ip, gp, _ptr(slot), _ptr(used), -1, _ptr(dem),
                  _ptr(drp), _ptr(gsum), None)
    _pack(b_up, index), _pack(b_down, index)   # (same checks as every tensor)
    o = _opts(act, b_up, b_down, dropout)
    _run(index, "moe_forward_routed", lib().moe_forward_routed, _pack(x, index),
         _pack(W_up, index), _pack(W_down, index), None if o is None else o.ref(), k,
         capacity_factor, _pack(out, index), ctypes.byref(st))
    return out, Stats(idx, gate, slot, used, int(st.capacity), dem, drp, gsum)


@_on_stream
def backward_routed(x, idx, gate, W_up, W_down, capacity_factor: float, dout, workspace=None,
                    act: str = "relu", b_up=None, b_down=None, dropout=None, aux_stream=None):
    """Run ``moe_backward_routed``: ``(dx, dgate, dW_up, dW_down, db_up, db_down)``,
    fp32 (None for a bias the layer lacks); dx is the experts' part, to be passed
    to :func:`route_backward` as ``dres`` with ``dgate``."""
    N, d, k = x.numel() // x.shape[-1], x.shape[-1], idx.shape[-1]
    E, d_ff = W_up.shape[0], W_up.shape[1]
    index, dev = _device_of(x), x.device
    ip, gp = _routing_ptrs(idx, gate, N, k, index)
    f32 = dict(dtype=torch.float32, device=dev)
    dx, dgate = torch.empty(x.shape, **f32), torch.empty((N, k), **f32)
    dwu, dwd = torch.empty((E, d_ff, d), **f32), torch.empty((E, d, d_ff), **f32)
    dbu = None if b_up is None else torch.empty((E, d_ff), **f32)
    dbd = None if b_down is None else torch.empty((E, d), **f32)
    if workspace is None:
        workspace = alloc_workspace(
            backward_workspace_size(N, d, E, d_ff, k, capacity_factor, x.dtype), dev)
    ws, wn = _scratch(workspace, index)
    aux, handle = _aux_stream(aux_stream, dev)
    st = MoeStats(_stream_of(index), ws, wn, ip, gp, None, None, -1, None, None, None, handle)
    _pack(b_up, index), _pack(b_down, index)   # (same checks as every tensor)
    o = _opts(act, b_up, b_down, dropout)
    _run(index, "moe_backward_routed", lib().moe_backward_routed, _pack(x, index),
         _pack(W_up, index), _pack(W_down, index), None if o is None else o.ref(), k,
         capacity_factor, _pack(dout, index), _pack(dx, index), _pack(dgate, index),
         _pack(dwu, index), _pack(dwd, index), _pack(dbu, index), _pack(dbd, index),
         ctypes.byref(st))
    return dx, dgate, dwu, dwd, dbu, dbd
