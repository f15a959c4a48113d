"""ctypes binding of libmoe.so: the same entry points as include/moe.h, argument marshalling only.

Every step of the layer runs in the CUDA library; nothing here computes.  If the library is
missing this module raises on import -- there is no fallback of any kind.

Device pointers are passed as ints (``tensor.data_ptr()``); ``stream`` is a cudaStream_t as an
int (``torch.cuda.current_stream().cuda_stream``) or None for the default stream.
"""
from __future__ import annotations

import ctypes
from pathlib import Path

_PKG = Path(__file__).resolve().parent
LIB_PATH = _PKG / "libmoe.so"

if not LIB_PATH.exists():
    raise ImportError(f"{LIB_PATH} is not built: run `python -m expert_ffn_token_b200.build`")

_lib = ctypes.CDLL(str(LIB_PATH))

OK = 0
ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_ALIGNMENT, ERR_CUDA = 1, 2, 3, 4
ERR_NONFINITE, ERR_BOUNDS, ERR_TIMEOUT, ERR_WORKSPACE = 5, 6, 7, 8

FMT_Q4_K, FMT_Q5_K, FMT_Q8_0, FMT_Q5_1, FMT_Q6_K = 0, 1, 2, 3, 4

F_DETERMINISTIC = 1
F_FORCE_DECODE = 2
F_FORCE_PREFILL = 4
F_KEEP_H = 8
F_LOOKAHEAD = 16
F_TC_I8 = 32

DT_F32, DT_BF16, DT_F16 = 0, 1, 2
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1

EXPORTED = ["moe_arena_create", "moe_arena_destroy", "moe_workspace_size", "moe_quantize_act",
            "moe_route_workspace_size", "moe_route_topk", "moe_forward", "moe_ws_views",
            "moe_read_status", "moe_debug_dequant", "moe_status_string",
            "moe_kernels_enqueued", "moe_forward_noalloc", "moe_set_timing_events",
            "moe_router_logits", "moe_shared_gate", "moe_set_wait_limit",
            "moe_forward_routed", "moe_chain_workspace_size", "moe_chain_forward",
            "moe_chain_status", "moe_route_scored", "moe_scaled_quantize",
            "moe_scaled_matmul_workspace_size", "moe_scaled_matmul",
            "moe_scaled_experts_workspace_size", "moe_scaled_experts",
            "moe_scaled_set_wait_limit"]


class ExpertDesc(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("off", ctypes.c_uint64 * 3), ("stride", ctypes.c_uint64 * 3)]


class WsView(ctypes.Structure):
    _fields_ = [("status", ctypes.c_void_p), ("xq", ctypes.c_void_p), ("xd", ctypes.c_void_p),
                ("xs", ctypes.c_void_p), ("ids", ctypes.c_void_p), ("w", ctypes.c_void_p),
                ("counts", ctypes.c_void_p), ("offsets", ctypes.c_void_p),
                ("perm", ctypes.c_void_p), ("inv_perm", ctypes.c_void_p),
                ("hq", ctypes.c_void_p), ("hd", ctypes.c_void_p), ("hs", ctypes.c_void_p),
                ("h", ctypes.c_void_p), ("slots", ctypes.c_int32), ("hpad", ctypes.c_int32),
                ("counters", ctypes.c_void_p)]


class ChainLayer(ctypes.Structure):
    _fields_ = [("arena", ctypes.c_void_p), ("d_router", ctypes.c_void_p),
                ("d_gate_row", ctypes.c_void_p), ("d_norm_weight", ctypes.c_void_p)]


class ChainTrace(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("xn", ctypes.c_void_p), ("logits", ctypes.c_void_p),
                ("ids", ctypes.c_void_p),
                ("w", ctypes.c_void_p), ("gate", ctypes.c_void_p), ("out", ctypes.c_void_p),
                ("early", ctypes.c_void_p)]


class RouteRule(ctypes.Structure):
    """moe_route_rule: score, expert groups, renormalisation, scale and an optional bias: a
    contiguous fp32 CUDA tensor [E], which the rule keeps, or a device pointer to such memory,
    which the caller keeps."""
    _fields_ = [("score", ctypes.c_int32), ("n_group", ctypes.c_int32),
                ("topk_group", ctypes.c_int32), ("group_top", ctypes.c_int32),
                ("renorm", ctypes.c_int32), ("scale", ctypes.c_float),
                ("d_bias", ctypes.c_void_p)]

    def __init__(self, score=SCORE_SOFTMAX, n_group=1, topk_group=1, group_top=1, renorm=True,
                 scale=1.0, d_bias=None):
        self.bias = None
        if d_bias is not None and not isinstance(d_bias, int):
            import torch
            self.bias = _contiguous(d_bias, "d_bias", (d_bias.numel(),), torch.float32,
                                    d_bias.get_device())
            d_bias = d_bias.data_ptr()
        super().__init__(score, n_group, topk_group, group_top, int(renorm), scale, d_bias)


class ScaledWeights(ctypes.Structure):
    """moe_scaled_weights."""
    _fields_ = [("hidden", ctypes.c_int32), ("ffn", ctypes.c_int32),
                ("n_experts", ctypes.c_int32), ("shared", ctypes.c_int32),
                ("d_gate", ctypes.c_void_p), ("d_up", ctypes.c_void_p),
                ("d_down", ctypes.c_void_p), ("d_gate_s", ctypes.c_void_p),
                ("d_up_s", ctypes.c_void_p), ("d_down_s", ctypes.c_void_p)]


_P = ctypes.c_void_p
_I = ctypes.c_int
_L = ctypes.c_int64
_S = ctypes.c_size_t
_U = ctypes.c_uint32

_lib.moe_status_string.restype = ctypes.c_char_p
_lib.moe_status_string.argtypes = [_I]
_lib.moe_arena_create.argtypes = [_P, _S, _I, _I, _I, _I, _P, ctypes.POINTER(_P)]
_lib.moe_arena_destroy.argtypes = [_P]
_lib.moe_arena_destroy.restype = None
_lib.moe_workspace_size.argtypes = [_P, _I, _I, _U, ctypes.POINTER(_S)]
_lib.moe_quantize_act.argtypes = [_P, _I, _I, _P, _P, _P, _P, _P]
_lib.moe_route_workspace_size.argtypes = [_I, _I, _I, ctypes.POINTER(_S)]
_lib.moe_route_topk.argtypes = [_P, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _S, _P]
_lib.moe_forward.argtypes = [_P, _P, _P, _I, _I, _P, _P, _S, _U, _P]
_lib.moe_ws_views.argtypes = [_P, _P, _I, _I, _U, ctypes.POINTER(WsView)]
_lib.moe_read_status.argtypes = [_P, _P, _I, ctypes.POINTER(_I)]
_lib.moe_debug_dequant.argtypes = [_P, _I, _I, _P, _P]
_lib.moe_forward_noalloc.argtypes = [_P, _P, _P, _I, _I, _P, _P, _P]
_lib.moe_set_timing_events.argtypes = [_P, _P, _P, _P]
_lib.moe_router_logits.argtypes = [_P, _I, _I, _P, _I, _P, _P]
_lib.moe_shared_gate.argtypes = [_P, _I, _I, _P, _P, _P]
_lib.moe_set_wait_limit.argtypes = [_P, ctypes.c_uint64]
_lib.moe_forward_routed.argtypes = [_P, _P, _I, _I, _P, _P, _P, _P, _P, _P, _S, _U, _P]
_lib.moe_chain_workspace_size.argtypes = [_P, _I, _I, _I, _U, ctypes.POINTER(_S)]
_lib.moe_chain_forward.argtypes = [_P, _I, _P, _I, _I, _P, _P, _S, _U, _P, _P]
_lib.moe_chain_status.argtypes = [_P, _I, _P, _I, _I, _U, ctypes.POINTER(_P)]
_lib.moe_route_scored.argtypes = [_P, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _S, _P]
_lib.moe_scaled_quantize.argtypes = [_P, _I, _I, _I, _L, _P, _L, _P, _L, _P, _P]
_lib.moe_scaled_matmul_workspace_size.argtypes = [_I, _I, _I, ctypes.POINTER(_S)]
_lib.moe_scaled_matmul.argtypes = [_P, _L, _P, _L, _I, _I, _P, _L, _P, _I, _P, _I, _L, _P, _P,
                                   _S, _P]
_lib.moe_scaled_experts_workspace_size.argtypes = [_P, _I, _I, ctypes.POINTER(_S)]
_lib.moe_scaled_experts.argtypes = [_P, _P, _I, _I, _I, _P, _P, _P, _P, _P, _P, _I, _P, _P, _S,
                                    _P]
_lib.moe_scaled_set_wait_limit.argtypes = [ctypes.c_uint64]
_lib.moe_kernels_enqueued.argtypes = []
_lib.moe_kernels_enqueued.restype = ctypes.c_uint64


class MoeError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {status_string(code)} ({code})")
        self.code = code


def status_string(code: int) -> str:
    return _lib.moe_status_string(code).decode()


def _check(code: int, where: str) -> None:
    if code != OK:
        raise MoeError(code, where)


def library():
    """The loaded CDLL (for symbol checks)."""
    return _lib


def arena_create(d_arena: int, arena_bytes: int, hidden: int, ffn: int, n_experts: int,
                 shared_expert: int, descs) -> int:
    """descs: sequence of (fmt, (off_gate, off_up, off_down), (stride_gate, stride_up, stride_down))."""
    arr = (ExpertDesc * len(descs))()
    for i, (fmt, off, stride) in enumerate(descs):
        arr[i].fmt = int(fmt)
        arr[i].reserved = 0
        for t in range(3):
            arr[i].off[t] = int(off[t])
            arr[i].stride[t] = int(stride[t])
    h = _P()
    _check(_lib.moe_arena_create(d_arena, arena_bytes, hidden, ffn, n_experts, shared_expert,
                                 ctypes.cast(arr, _P), ctypes.byref(h)), "moe_arena_create")
    return h.value


def arena_destroy(arena: int) -> None:
    _lib.moe_arena_destroy(arena)


def workspace_size(arena: int, max_tokens: int, k: int, flags: int = 0) -> int:
    n = _S()
    _check(_lib.moe_workspace_size(arena, max_tokens, k, flags, ctypes.byref(n)),
           "moe_workspace_size")
    return n.value


def quantize_act(d_x: int, T: int, H: int, d_q: int, d_d: int, d_s: int, d_status=None,
                 stream=None) -> None:
    _check(_lib.moe_quantize_act(d_x, T, H, d_q, d_d, d_s, d_status, stream), "moe_quantize_act")


def route_workspace_size(T: int, E: int, k: int) -> int:
    n = _S()
    _check(_lib.moe_route_workspace_size(T, E, k, ctypes.byref(n)), "moe_route_workspace_size")
    return n.value


def router_logits(d_x: int, T: int, H: int, d_router: int, E: int, d_logits: int,
                  stream=None) -> None:
    _check(_lib.moe_router_logits(d_x, T, H, d_router, E, d_logits, stream), "moe_router_logits")


def router_logits_status(d_x, T, H, d_router, E, d_logits, stream=None) -> int:
    return _lib.moe_router_logits(d_x, T, H, d_router, E, d_logits, stream)


def shared_gate(d_x: int, T: int, H: int, d_gate_row: int, d_gate: int, stream=None) -> None:
    _check(_lib.moe_shared_gate(d_x, T, H, d_gate_row, d_gate, stream), "moe_shared_gate")


def route_topk(d_logits: int, T: int, E: int, k: int, d_ids: int, d_w: int, d_counts: int,
               d_offsets: int, d_perm: int, d_inv_perm, d_status, d_ws: int, ws_bytes: int,
               stream=None) -> None:
    _check(_lib.moe_route_topk(d_logits, T, E, k, d_ids, d_w, d_counts, d_offsets, d_perm,
                               d_inv_perm, d_status, d_ws, ws_bytes, stream), "moe_route_topk")


def forward(arena: int, d_x: int, d_logits: int, T: int, k: int, d_out: int, d_ws: int,
            ws_bytes: int, flags: int = 0, stream=None) -> None:
    _check(_lib.moe_forward(arena, d_x, d_logits, T, k, d_out, d_ws, ws_bytes, flags, stream),
           "moe_forward")


def forward_noalloc(arena: int, d_x: int, d_logits: int, T: int, k: int, d_out: int,
                    d_status=None, stream=None) -> None:
    """moe_forward_noalloc: the layer for 1..16 tokens using the library's fixed scratch."""
    _check(_lib.moe_forward_noalloc(arena, d_x, d_logits, T, k, d_out, d_status, stream),
           "moe_forward_noalloc")


def forward_noalloc_status(arena, d_x, d_logits, T, k, d_out, d_status=None, stream=None) -> int:
    """moe_forward_noalloc returning its status code instead of raising."""
    return _lib.moe_forward_noalloc(arena, d_x, d_logits, T, k, d_out, d_status, stream)


def forward_status(arena, d_x, d_logits, T, k, d_out, d_ws, ws_bytes, flags=0, stream=None) -> int:
    """moe_forward returning its status code instead of raising (for error-path tests)."""
    return _lib.moe_forward(arena, d_x, d_logits, T, k, d_out, d_ws, ws_bytes, flags, stream)


def forward_routed(arena: int, d_x: int, T: int, k: int, d_router: int, d_gate_row, d_logits: int,
                   d_gate, d_out: int, d_ws: int, ws_bytes: int, flags: int = 0,
                   stream=None) -> None:
    """moe_forward_routed: router (and optional shared gate) then the layer."""
    _check(forward_routed_status(arena, d_x, T, k, d_router, d_gate_row, d_logits, d_gate, d_out,
                                 d_ws, ws_bytes, flags, stream), "moe_forward_routed")


def forward_routed_status(arena, d_x, T, k, d_router, d_gate_row, d_logits, d_gate, d_out, d_ws,
                          ws_bytes, flags=0, stream=None) -> int:
    return _lib.moe_forward_routed(arena, d_x, T, k, d_router, d_gate_row, d_logits, d_gate, d_out,
                                   d_ws, ws_bytes, flags, stream)


def _chain_layers(layers):
    """layers: sequence of (arena handle, d_router, d_gate_row or None[, d_norm_weight or None])."""
    arr = (ChainLayer * len(layers))()
    for i, ly in enumerate(layers):
        arr[i].arena, arr[i].d_router, arr[i].d_gate_row = ly[0], ly[1], ly[2]
        arr[i].d_norm_weight = ly[3] if len(ly) > 3 else None
    return arr


def chain_workspace_size(layers, max_tokens: int, k: int, flags: int = 0) -> int:
    n = _S()
    _check(_lib.moe_chain_workspace_size(_chain_layers(layers), len(layers), max_tokens, k, flags,
                                         ctypes.byref(n)), "moe_chain_workspace_size")
    return n.value


def chain_forward_status(layers, d_x: int, T: int, k: int, d_x_out: int, d_ws: int,
                         ws_bytes: int, flags: int = 0, trace=None, stream=None) -> int:
    """moe_chain_forward returning its status; trace: dict of device pointers (ChainTrace
    field names) or None."""
    tr = None
    if trace is not None:
        tr = ChainTrace(**{k2: trace.get(k2) for k2, _ in ChainTrace._fields_})
    return _lib.moe_chain_forward(_chain_layers(layers), len(layers), d_x, T, k, d_x_out, d_ws,
                                  ws_bytes, flags, ctypes.byref(tr) if tr is not None else None,
                                  stream)


def chain_forward(layers, d_x: int, T: int, k: int, d_x_out: int, d_ws: int, ws_bytes: int,
                  flags: int = 0, trace=None, stream=None) -> None:
    _check(chain_forward_status(layers, d_x, T, k, d_x_out, d_ws, ws_bytes, flags, trace, stream),
           "moe_chain_forward")


def chain_status_word(layers, d_ws: int, T: int, k: int, flags: int = 0) -> int:
    p = _P()
    _check(_lib.moe_chain_status(_chain_layers(layers), len(layers), d_ws, T, k, flags,
                                 ctypes.byref(p)), "moe_chain_status")
    return p.value


def ws_views(arena: int, d_ws: int, T: int, k: int, flags: int = 0) -> dict:
    v = WsView()
    _check(_lib.moe_ws_views(arena, d_ws, T, k, flags, ctypes.byref(v)), "moe_ws_views")
    return {name: getattr(v, name) for name, _ in WsView._fields_}


def read_status(d_status: int, stream=None, clear: bool = True) -> int:
    s = _I()
    _check(_lib.moe_read_status(d_status, stream, 1 if clear else 0, ctypes.byref(s)),
           "moe_read_status")
    return s.value


def set_timing_events(arena: int, ev_begin=None, ev_mid=None, ev_end=None) -> None:
    """moe_set_timing_events: cudaEvent_t handles (ints) recorded around the tensor-core phases
    of later forwards on this arena, or None to stop."""
    _check(_lib.moe_set_timing_events(arena, ev_begin, ev_mid, ev_end), "moe_set_timing_events")


def set_wait_limit(arena: int, ns: int) -> None:
    """moe_set_wait_limit: limit of every bounded device wait of later calls on this arena."""
    _check(_lib.moe_set_wait_limit(arena, ns), "moe_set_wait_limit")


def kernels_enqueued() -> int:
    return int(_lib.moe_kernels_enqueued())


def debug_dequant(arena: int, expert: int, which: int, d_out: int, stream=None) -> None:
    _check(_lib.moe_debug_dequant(arena, expert, which, d_out, stream), "moe_debug_dequant")


def route_scored(d_logits: int, T: int, E: int, k: int, rule: RouteRule, d_ids: int, d_w: int,
                 d_counts: int, d_offsets: int, d_perm: int, d_inv_perm, d_status, d_ws: int,
                 ws_bytes: int, stream=None) -> None:
    """moe_route_scored: route_topk with a RouteRule (workspace: route_workspace_size)."""
    _check(_lib.moe_route_scored(d_logits, T, E, k, ctypes.addressof(rule), d_ids, d_w, d_counts,
                                 d_offsets, d_perm, d_inv_perm, d_status, d_ws, ws_bytes, stream),
           "moe_route_scored")


def scaled_quantize(d_x: int, dtype: int, T: int, K: int, ldx: int, d_q: int, ldq: int, d_s: int,
                    lds: int, d_status=None, stream=None) -> None:
    _check(_lib.moe_scaled_quantize(d_x, dtype, T, K, ldx, d_q, ldq, d_s, lds, d_status, stream),
           "moe_scaled_quantize")


def scaled_matmul_workspace_size(M: int, N: int, K: int) -> int:
    n = _S()
    _check(_lib.moe_scaled_matmul_workspace_size(M, N, K, ctypes.byref(n)),
           "moe_scaled_matmul_workspace_size")
    return n.value


def scaled_matmul(d_a: int, lda: int, d_as: int, ldas: int, M: int, K: int, d_b: int, ldb: int,
                  d_bs: int, N: int, d_out: int, dtype: int, ldo: int, d_status=None, d_ws=None,
                  ws_bytes: int = 0, stream=None) -> None:
    _check(_lib.moe_scaled_matmul(d_a, lda, d_as, ldas, M, K, d_b, ldb, d_bs, N, d_out, dtype,
                                  ldo, d_status, d_ws, ws_bytes, stream), "moe_scaled_matmul")


def scaled_experts_workspace_size(weights: ScaledWeights, max_tokens: int, k: int) -> int:
    n = _S()
    _check(_lib.moe_scaled_experts_workspace_size(ctypes.addressof(weights), max_tokens, k,
                                                  ctypes.byref(n)),
           "moe_scaled_experts_workspace_size")
    return n.value


def scaled_experts(weights: ScaledWeights, d_x: int, x_dtype: int, T: int, k: int, d_ids: int,
                   d_w: int, d_offsets: int, d_inv_perm: int, d_gate, d_out: int, out_dtype: int,
                   d_status, d_ws: int, ws_bytes: int, stream=None) -> None:
    _check(_lib.moe_scaled_experts(ctypes.addressof(weights), d_x, x_dtype, T, k, d_ids, d_w,
                                   d_offsets, d_inv_perm, d_gate, d_out, out_dtype, d_status,
                                   d_ws, ws_bytes, stream), "moe_scaled_experts")


def scaled_set_wait_limit(ns: int) -> None:
    """moe_scaled_set_wait_limit: limit of every bounded device wait of later scaled_matmul and
    scaled_experts calls of this process."""
    _check(_lib.moe_scaled_set_wait_limit(ns), "moe_scaled_set_wait_limit")


# ------------------------------------------------------------------ torch convenience


_DTYPES: dict = {}
_FLOATS: tuple = ()


def dtype_of(t) -> int:
    """The moe_dtype of a torch tensor (fp32, bf16 or fp16)."""
    if not _DTYPES:
        _fill_dtypes()
    d = _DTYPES.get(t.dtype)
    if d is None:
        raise MoeError(ERR_UNSUPPORTED, f"dtype {t.dtype}")
    return d


def _fill_dtypes() -> None:
    global _FLOATS
    import torch
    _DTYPES.update({torch.float32: DT_F32, torch.bfloat16: DT_BF16, torch.float16: DT_F16})
    _FLOATS = tuple(_DTYPES)


def _stream(device=None):
    """The current stream's handle, without the Stream object around it (3 us of a small call)."""
    import torch
    return torch._C._cuda_getCurrentRawStream(
        torch.cuda.current_device() if device is None else device)


class Layer:
    """One MoE layer over a device arena held in a torch uint8 tensor (marshalling only)."""

    def __init__(self, arena_tensor, hidden: int, ffn: int, n_experts: int, shared: bool,
                 descs, max_tokens: int, k: int, flags: int = 0):
        import torch
        self.arena_tensor = arena_tensor
        self.hidden, self.ffn, self.n_experts, self.k = hidden, ffn, n_experts, k
        self.flags = flags
        self.handle = arena_create(arena_tensor.data_ptr(), arena_tensor.numel(), hidden, ffn,
                                   n_experts, n_experts if shared else -1, descs)
        self.ws_bytes = workspace_size(self.handle, max_tokens, k, flags)
        self.ws = torch.zeros(self.ws_bytes, dtype=torch.uint8, device=arena_tensor.device)

    def forward(self, x, logits, out=None, flags=None):
        import torch
        T = x.shape[0]
        if out is None:
            out = torch.empty_like(x)
        forward(self.handle, x.data_ptr(), logits.data_ptr(), T, self.k, out.data_ptr(),
                self.ws.data_ptr(), self.ws_bytes, self.flags if flags is None else flags,
                _stream())
        return out

    def views(self, T: int, flags=None) -> dict:
        return ws_views(self.handle, self.ws.data_ptr(), T, self.k,
                        self.flags if flags is None else flags)

    def status(self, clear: bool = True) -> int:
        return read_status(self.views(1)["status"], _stream(), clear)

    def close(self):
        if self.handle:
            arena_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _contiguous(t, name: str, shape, dtype, device: int):
    """t, checked: contiguous, on the CUDA device with this index, of the shape and type asked for
    (a type or a tuple of types)."""
    if t.get_device() != device or not t.is_cuda:
        raise ValueError(f"{name}: a tensor on CUDA device {device} is needed")
    if t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: shape {tuple(t.shape)}, not a contiguous {tuple(shape)}")
    if t.dtype is not dtype and not (isinstance(dtype, tuple) and t.dtype in dtype):
        raise ValueError(f"{name}: type {t.dtype}")
    return t


class ScaledExperts:
    """The experts of one layer in e4m3 with 128 x 128 block scales, held in torch tensors, and
    the workspace for up to max_tokens tokens (marshalling only).

    Everything is on the CUDA device that is current when the layer is made, and its calls are made
    with that device current.  Its calls share one workspace: they follow one another on a stream (graphs of them too); what
    runs at the same time on another stream is an object of its own.  No gradients.

    gate, up [n][ffn][hidden] and down [n][hidden][ffn] (uint8 or float8_e4m3fn), scales fp32
    [n][ceil(rows / 128)][ceil(cols / 128)], n = experts (+ 1 with `shared`)."""

    def __init__(self, gate, gate_scale, up, up_scale, down, down_scale, max_tokens: int, k: int,
                 shared: bool = False, rule: RouteRule | None = None):
        import torch
        _fill_dtypes()
        n, f, h = gate.shape
        fb, hb = -(-f // 128), -(-h // 128)
        codes, f32, dev = (torch.uint8, torch.float8_e4m3fn), torch.float32, torch.cuda.current_device()
        self.device = dev
        self.tensors = (_contiguous(gate, "gate", (n, f, h), codes, dev),
                        _contiguous(up, "up", (n, f, h), codes, dev),
                        _contiguous(down, "down", (n, h, f), codes, dev),
                        _contiguous(gate_scale, "gate_scale", (n, fb, hb), f32, dev),
                        _contiguous(up_scale, "up_scale", (n, fb, hb), f32, dev),
                        _contiguous(down_scale, "down_scale", (n, hb, fb), f32, dev))
        self.hidden, self.ffn, self.n_experts, self.k = h, f, n - int(shared), k
        self.rule = RouteRule() if rule is None else rule
        self.weights = ScaledWeights(h, f, n - int(shared), int(shared),
                                     *(t.data_ptr() for t in self.tensors))
        self.max_tokens = max_tokens
        self.ws_bytes = scaled_experts_workspace_size(self.weights, max_tokens, k)
        self.ws = torch.empty(self.ws_bytes, dtype=torch.uint8, device=gate.device)
        self.route_bytes = route_workspace_size(max_tokens, self.n_experts, k)
        self.route_ws = torch.empty(self.route_bytes, dtype=torch.uint8, device=gate.device)
        self.status_word = torch.zeros(1, dtype=torch.int32, device=gate.device)
        self._ws, self._status = self.ws.data_ptr(), self.status_word.data_ptr()

    def _current(self) -> int:
        """The layer's device, which has to be the current one."""
        import torch
        if torch.cuda.current_device() != self.device:
            raise ValueError(f"CUDA device {torch.cuda.current_device()} is current, the layer is on "
                             f"{self.device}")
        return self.device

    def route(self, logits):
        """(ids, w, offsets, perm, inv_perm) of fp32 logits [T][experts] by the layer's rule."""
        import torch
        T, E, k, dev = logits.shape[0], self.n_experts, self.k, self._current()
        _contiguous(logits, "logits", (T, E), torch.float32, dev)
        if self.rule.bias is not None:
            _contiguous(self.rule.bias, "the rule's bias", (E,), torch.float32, dev)
        new = lambda *s: torch.empty(s, dtype=torch.int32, device=logits.device)  # noqa: E731
        ids, counts, offsets, perm, inv = new(T, k), new(E), new(E + 1), new(T * k), new(T * k)
        w = torch.empty((T, k), dtype=torch.float32, device=logits.device)
        route_scored(logits.data_ptr(), T, E, k, self.rule, ids.data_ptr(), w.data_ptr(),
                     counts.data_ptr(), offsets.data_ptr(), perm.data_ptr(), inv.data_ptr(),
                     self.status_word.data_ptr(), self.route_ws.data_ptr(), self.route_bytes,
                     _stream(dev))
        return ids, w, offsets, perm, inv

    def forward(self, x, ids, w, offsets, perm, inv_perm, gate=None, out=None):
        """The experts' combined output [T][hidden] for tokens routed by route() or route_topk (perm,
        the inverse of inv_perm, is not read)."""
        import torch
        T, k, E, dev = x.shape[0], self.k, self.n_experts, self._current()
        i32, f32, rows = torch.int32, torch.float32, (T, self.hidden)
        _contiguous(x, "x", rows, _FLOATS, dev)
        _contiguous(ids, "ids", (T, k), i32, dev)
        _contiguous(w, "w", (T, k), f32, dev)
        _contiguous(offsets, "offsets", (E + 1,), i32, dev)
        _contiguous(inv_perm, "inv_perm", (T * k,), i32, dev)
        if gate is not None:
            _contiguous(gate, "gate", (T,), f32, dev)
        if out is None:
            out = torch.empty_like(x)
        else:
            _contiguous(out, "out", rows, _FLOATS, dev)
        scaled_experts(self.weights, x.data_ptr(), dtype_of(x), T, k, ids.data_ptr(),
                       w.data_ptr(), offsets.data_ptr(), inv_perm.data_ptr(),
                       None if gate is None else gate.data_ptr(), out.data_ptr(), dtype_of(out),
                       self._status, self._ws, self.ws_bytes, _stream(dev))
        return out

    def __call__(self, x, logits, gate=None, out=None):
        """route(logits), then forward."""
        return self.forward(x, *self.route(logits), gate=gate, out=out)

    def status(self, clear: bool = True) -> int:
        return read_status(self.status_word.data_ptr(), _stream(self._current()), clear)
