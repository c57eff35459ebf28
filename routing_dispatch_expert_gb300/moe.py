"""Python binding of libmoe_gb300.so (include/moe.h): argument marshalling only.

Every step of the layer runs in the library's CUDA kernels; this module converts torch tensors to
device pointers, passes the current CUDA stream, and raises ``MoeError`` on a non-zero status.
There is no fallback: if the library is not built, loading it raises.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import os
import threading
import warnings

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
SO_PATH = os.path.join(_PKG, "_build", "libmoe_gb300.so")

MOE_OK, MOE_ERR_INVALID, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_CUDA, MOE_ERR_DEVICE = 0, -1, -2, -3, -4, -5
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
DTYPES = {"bf16": 0, "fp8": 1, "nvfp4": 2, "mxfp4": 3}
MOE_DTYPE_BF16, MOE_DTYPE_FP8_BLOCK128, MOE_DTYPE_NVFP4, MOE_DTYPE_MXFP4 = 0, 1, 2, 3
MOE_TYPE_F32, MOE_TYPE_BF16, MOE_TYPE_F16 = 0, 1, 2
ELEMENT_TYPES = {torch.float32: MOE_TYPE_F32, torch.bfloat16: MOE_TYPE_BF16, torch.float16: MOE_TYPE_F16}
FP4_FORMATS = {"nvfp4": 0, "mxfp4": 1}
FP4_BLOCK = {"nvfp4": 16, "mxfp4": 32}
MOE_LOGITS_GIVEN = 1
MOE_STATUS_BAD_EXPERT_INDEX, MOE_STATUS_WAIT_TIMEOUT = 1, 2


class MoeError(RuntimeError):
    def __init__(self, code: int, message: str):
        super().__init__(f"[{code}] {message}")
        self.code = code


class MoePlacement(ctypes.Structure):
    _fields_ = [("n_slots", ctypes.c_int32), ("max_replicas", ctypes.c_int32), ("slot_expert", ctypes.c_void_p),
                ("slot_replica", ctypes.c_void_p), ("replicas", ctypes.c_void_p), ("replica_slot", ctypes.c_void_p)]


class MoeConfig(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("h", ctypes.c_int32), ("E", ctypes.c_int32), ("k", ctypes.c_int32),
                ("I", ctypes.c_int32), ("I_shared", ctypes.c_int32), ("n_group", ctypes.c_int32),
                ("topk_group", ctypes.c_int32), ("score", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("routed_scale", ctypes.c_float), ("dtype", ctypes.c_int32), ("capacity_factor", ctypes.c_float),
                ("placement", ctypes.POINTER(MoePlacement))]


class MoeWeightsStruct(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("w_router", "bias", "w_gu", "s_gu", "w_d", "s_d", "w_gu_shared",
                                               "s_gu_shared", "w_d_shared", "s_d_shared", "g_gu", "g_d",
                                               "g_gu_shared", "g_d_shared")]


class MoeWsLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("logits", "topk_idx", "topk_w", "counts", "offsets", "inv_pos",
                                               "row_token", "row_weight", "xd", "xd_scales", "hbuf", "h_scales", "yd",
                                               "router_w3", "scratch", "total")]


class MoeFp4Activations(ctypes.Structure):
    _fields_ = [("g_x", ctypes.c_void_p), ("g_h", ctypes.c_void_p)]


_lock = threading.Lock()
_lib = None


def load():
    """Load the CUDA library (built by ``routing_dispatch_expert_gb300.build``)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(SO_PATH):
                raise ImportError(f"libmoe_gb300.so is not built ({SO_PATH}); run routing_dispatch_expert_gb300.build")
            L = ctypes.CDLL(SO_PATH)
            vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
            cfgp = ctypes.POINTER(MoeConfig)
            wp = ctypes.POINTER(MoeWeightsStruct)
            actp = ctypes.POINTER(MoeFp4Activations)
            sig = {
                "moe_workspace_size": [cfgp, ctypes.POINTER(sz)],
                "moe_workspace_layout": [cfgp, ctypes.POINTER(MoeWsLayout)],
                "moe_route": [cfgp, vp, wp, vp, i32, vp, vp, vp, sz, vp],
                "moe_dispatch": [cfgp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
                "moe_dispatch_noalloc": [cfgp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp],
                "moe_expert_ffn": [cfgp, wp, vp, vp, vp, vp, vp, vp, sz, vp],
                "moe_combine": [cfgp, vp, vp, vp, vp],
                "moe_forward": [cfgp, vp, wp, vp, vp, sz, vp],
                "moe_quantize_weights_fp8": [vp, i64, i64, i64, vp, vp, vp],
                "moe_quantize_weights_nvfp4": [vp, i64, i64, i64, vp, vp, vp, vp],
                "moe_device_status": [cfgp, vp, ctypes.POINTER(ctypes.c_int32), vp],
                "moe_selftest_wait_timeout": [cfgp, vp, sz, i64, vp],
                "moe_graph_create": [cfgp, vp, wp, vp, vp, sz, vp, ctypes.POINTER(vp)],
                "moe_graph_launch": [vp, vp],
                "moe_graph_destroy": [vp],
                "moe_eplb_plan": [vp, i32, i32, i32, vp, vp, vp, vp, vp],
                "moe_balance": [cfgp, vp, vp, vp],
                "moe_quantize_fp4": [vp, i32, i64, i64, i64, i32, vp, vp, vp, vp],
                "moe_dequantize_fp4": [vp, vp, i64, i64, i32, vp, i32, vp, vp],
                "moe_matmul_fp4": [vp, vp, vp, vp, vp, vp, i64, i64, i64, i32, i32, vp, i64, vp, vp],
                "moe_matmul_fp4_status": [ctypes.POINTER(ctypes.c_int32), vp],
                "moe_dispatch_fp4": [cfgp, actp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
                "moe_expert_ffn_fp4": [cfgp, wp, actp, vp, vp, vp, vp, vp, vp, sz, vp],
                "moe_forward_fp4": [cfgp, vp, wp, actp, vp, vp, sz, vp],
                "moe_balance_loss_workspace_size": [cfgp, i32, ctypes.POINTER(sz)],
                "moe_balance_loss": [cfgp, vp, i32, vp, vp, i32, vp, ctypes.c_float, vp, vp, vp, vp, vp, sz, vp],
                "moe_balance_loss_backward": [cfgp, vp, i32, vp, vp, vp, i32, vp, ctypes.c_float, vp, vp, vp],
                "moe_rms_norm": [vp, i32, i64, i64, i64, vp, i32, i64, vp, i32, ctypes.c_float, vp, vp, vp, vp, vp],
                "moe_rms_norm_backward_workspace_size": [i64, i64, ctypes.POINTER(sz)],
                "moe_rms_norm_backward": [vp, i32, i64, i64, vp, i32, i64, vp, vp, i32, ctypes.c_float, vp, vp, vp, vp, sz,
                                          vp],
                "moe_sort_tokens_workspace_size": [cfgp, ctypes.POINTER(sz)],
                "moe_sort_tokens": [cfgp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp],
                "moe_permute": [cfgp, vp, i32, i64, i64, vp, vp, vp, vp, vp, vp],
                "moe_unpermute": [cfgp, vp, i32, i64, vp, vp, vp, vp, vp],
                "moe_unpermute_backward": [cfgp, vp, vp, i32, i64, vp, vp, vp, vp, vp, vp],
                "moe_route_backward": [cfgp, vp, i32, vp, vp, vp, vp],
            }
            for name, args in sig.items():
                f = getattr(L, name)
                f.argtypes = args
                f.restype = i32
            L.moe_last_error.argtypes = []
            L.moe_last_error.restype = ctypes.c_char_p
            L.moe_launch_count.argtypes = []
            L.moe_launch_count.restype = ctypes.c_uint64
            _load_calls()
            _lib = L
    return _lib


class _NoCalls:
    """In the place of csrc/calls.cpp where it is not built: takes no call, so that each goes through its steps here."""

    def __getattr__(self, name):
        return lambda *args: None


_calls = None  # csrc/calls.cpp, once the library is loaded


def _load_calls():
    """The module as it is built for this torch and Python. The library's calls do not need it: those that it makes are made
    here then, at two to three times the host time."""
    global _calls
    from .build import calls_path

    path = calls_path()
    try:
        spec = importlib.util.spec_from_file_location("_calls", path)
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.bind(MoeConfig, MoeError)
        _calls = module
    except ImportError as e:
        warnings.warn(f"csrc/calls.cpp is not built for this torch and Python, small calls take longer ({e}); run "
                      "routing_dispatch_expert_gb300.build")
        _calls = _NoCalls()


def _check(rc: int):
    if rc != MOE_OK:
        raise MoeError(rc, load().moe_last_error().decode())


def _memory(t):
    """Address of a tensor. One without memory of its own (a wrapper's, say) is refused: it has the address of its offset, and
    without one would be taken for a tensor that was not given."""
    p = t.data_ptr()
    if p < 1 << 40 and t.numel() and p <= t.storage_offset() * t.element_size():  # no offset is past 2^40 bytes
        raise ValueError("a tensor has no memory of its own")
    return p


def _ptr(t):
    return None if t is None else ctypes.c_void_p(_memory(t))


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def make_config(T, h, E, k, I, I_shared=0, n_group=1, topk_group=1, score="softmax", renorm=False, routed_scale=1.0,
                dtype="bf16", capacity_factor=0.0, placement: "Placement | None" = None) -> MoeConfig:
    cfg = MoeConfig(T, h, E, k, I, I_shared, n_group, topk_group,
                    MOE_SCORE_SOFTMAX if score == "softmax" else MOE_SCORE_SIGMOID, int(bool(renorm)),
                    float(routed_scale), DTYPES[dtype],
                    float(capacity_factor), None if placement is None else ctypes.pointer(placement.struct))
    cfg._placement = placement  # keep the tables alive as long as the config
    return cfg


def eplb_plan(load, n_cards: int, n_redundant: int) -> dict:
    """moe_eplb_plan on the host: numpy arrays replicas [E], slot_expert / slot_replica [E + R],
    replica_slot [E, R + 1], card_load [n_cards]."""
    import numpy as np

    load = np.ascontiguousarray(load, dtype=np.int64)
    E = load.size
    S = E + n_redundant
    out = dict(replicas=np.empty(E, np.int32), slot_expert=np.empty(S, np.int32), slot_replica=np.empty(S, np.int32),
               replica_slot=np.empty((E, n_redundant + 1), np.int32), card_load=np.empty(n_cards, np.float64))
    p = lambda a: ctypes.c_void_p(a.ctypes.data)  # noqa: E731
    _check(load_lib_eplb()(p(load), E, n_cards, n_redundant, p(out["replicas"]), p(out["slot_expert"]),
                           p(out["slot_replica"]), p(out["replica_slot"]), p(out["card_load"])))
    return out


def load_lib_eplb():
    return load().moe_eplb_plan


class Placement:
    """Device copy of an EPLB plan (see eplb_plan) and its C struct, for make_config(placement=...)."""

    def __init__(self, plan: dict, device="cuda"):
        self.tables = {k: torch.from_numpy(plan[k]).to(device) for k in ("slot_expert", "slot_replica", "replicas",
                                                                          "replica_slot")}
        self.n_slots = int(plan["slot_expert"].size)
        self.struct = MoePlacement(self.n_slots, int(plan["replica_slot"].shape[1]),
                                   self.tables["slot_expert"].data_ptr(), self.tables["slot_replica"].data_ptr(),
                                   self.tables["replicas"].data_ptr(), self.tables["replica_slot"].data_ptr())


class Weights:
    """Device tensors of one layer and their C struct. bf16 expert weights for dtype 'bf16'; for
    'fp8' pass e4m3 codes (torch.uint8) and fp32 128x128 scales (see quantize_weights_fp8); for
    'nvfp4' pass codes, e4m3 block scales and fp32 matrix scales (see quantize_weights_nvfp4); for 'mxfp4'
    codes and e8m0 block scales (see quantize_fp4), without matrix scales."""

    def __init__(self, w_router, bias=None, w_gu=None, w_d=None, w_gu_shared=None, w_d_shared=None, s_gu=None,
                 s_d=None, s_gu_shared=None, s_d_shared=None, g_gu=None, g_d=None, g_gu_shared=None,
                 g_d_shared=None):
        self.tensors = dict(w_router=w_router, bias=bias, w_gu=w_gu, s_gu=s_gu, w_d=w_d, s_d=s_d,
                            w_gu_shared=w_gu_shared, s_gu_shared=s_gu_shared, w_d_shared=w_d_shared,
                            s_d_shared=s_d_shared, g_gu=g_gu, g_d=g_d, g_gu_shared=g_gu_shared,
                            g_d_shared=g_d_shared)
        self.struct = MoeWeightsStruct(**{n: _address(t) for n, t in self.tensors.items()})


def workspace_size(cfg: MoeConfig) -> int:
    n = ctypes.c_size_t()
    _check(load().moe_workspace_size(ctypes.byref(cfg), ctypes.byref(n)))
    return n.value


def workspace_layout(cfg: MoeConfig) -> dict:
    l = MoeWsLayout()
    _check(load().moe_workspace_layout(ctypes.byref(cfg), ctypes.byref(l)))
    return {n: getattr(l, n) for n, _ in MoeWsLayout._fields_}


def alloc_workspace(cfg: MoeConfig, device="cuda") -> torch.Tensor:
    return torch.empty(workspace_size(cfg), dtype=torch.uint8, device=device)


def ws_view(ws: torch.Tensor, cfg: MoeConfig, name: str, dtype, shape) -> torch.Tensor:
    """A typed view of one intermediate inside a moe_forward workspace."""
    off = workspace_layout(cfg)[name]
    n = 1
    for s in shape:
        n *= s
    nbytes = n * torch.empty((), dtype=dtype).element_size()
    return ws[off:off + nbytes].view(dtype).view(*shape)


def route(cfg, x, weights: Weights | None, topk_idx, topk_w, logits=None, logits_given=False, ws=None):
    _check(load().moe_route(ctypes.byref(cfg), _ptr(x), None if weights is None else ctypes.byref(weights.struct),
                            _ptr(logits), MOE_LOGITS_GIVEN if logits_given else 0, _ptr(topk_idx), _ptr(topk_w),
                            _ptr(ws), 0 if ws is None else ws.numel(), _stream()))


def dispatch(cfg, x, topk_idx, topk_w, counts, offsets, inv_pos, row_token, row_weight, xd, xd_scales, ws):
    _check(load().moe_dispatch(ctypes.byref(cfg), _ptr(x), _ptr(topk_idx), _ptr(topk_w), _ptr(counts), _ptr(offsets),
                               _ptr(inv_pos), _ptr(row_token), _ptr(row_weight), _ptr(xd), _ptr(xd_scales), _ptr(ws),
                               ws.numel(), _stream()))


def dispatch_noalloc(cfg, x, topk_idx, topk_w, counts, offsets, inv_pos, row_token, row_weight, xd, xd_scales):
    """moe_dispatch without a workspace, for callers that cannot allocate device memory (scratch is a
    static array inside the library; concurrent calls race; see include/moe.h)."""
    _check(load().moe_dispatch_noalloc(ctypes.byref(cfg), _ptr(x), _ptr(topk_idx), _ptr(topk_w), _ptr(counts),
                                       _ptr(offsets), _ptr(inv_pos), _ptr(row_token), _ptr(row_weight), _ptr(xd),
                                       _ptr(xd_scales), _stream()))


def expert_ffn(cfg, weights: Weights, xd, xd_scales, offsets, row_weight, yd, ws):
    _check(load().moe_expert_ffn(ctypes.byref(cfg), ctypes.byref(weights.struct), _ptr(xd), _ptr(xd_scales),
                                 _ptr(offsets), _ptr(row_weight), _ptr(yd), _ptr(ws), ws.numel(), _stream()))


def combine(cfg, yd, inv_pos, y):
    _check(load().moe_combine(ctypes.byref(cfg), _ptr(yd), _ptr(inv_pos), _ptr(y), _stream()))


def forward(cfg, x, weights: Weights, y, ws):
    _check(load().moe_forward(ctypes.byref(cfg), _ptr(x), ctypes.byref(weights.struct), _ptr(y), _ptr(ws), ws.numel(),
                              _stream()))


def quantize_weights_fp8(w: torch.Tensor):
    """Static 128x128 quantisation of bf16 weights [..., rows, cols] -> (e4m3 codes uint8, fp32 scales)."""
    rows, cols = w.shape[-2], w.shape[-1]
    batch = w.numel() // (rows * cols)
    q = torch.empty(w.shape, dtype=torch.uint8, device=w.device)
    s = torch.empty(tuple(w.shape[:-2]) + (rows // 128, cols // 128), dtype=torch.float32, device=w.device)
    _check(load().moe_quantize_weights_fp8(_ptr(w), batch, rows, cols, _ptr(q), _ptr(s), _stream()))
    return q, s


def quantize_weights_nvfp4(w: torch.Tensor):
    """NVFP4 quantisation of bf16 weights [..., rows, cols] -> (codes uint8 [..., rows, cols/2], e4m3 block
    scales uint8 [..., rows, cols/16], fp32 matrix scales [...])."""
    rows, cols = w.shape[-2], w.shape[-1]
    batch = w.numel() // (rows * cols)
    lead = tuple(w.shape[:-2])
    q = torch.empty(lead + (rows, cols // 2), dtype=torch.uint8, device=w.device)
    s = torch.empty(lead + (rows, cols // 16), dtype=torch.uint8, device=w.device)
    g = torch.empty(lead if lead else (1,), dtype=torch.float32, device=w.device)
    _check(load().moe_quantize_weights_nvfp4(_ptr(w), batch, rows, cols, _ptr(q), _ptr(s), _ptr(g), _stream()))
    return q, s, g


# The small calls of a decode or training step are bound by the host, so the entry points below that check their tensors
# do so in one expression (_like) and look for the words of a refusal (_need) only when that fails, take the stream's
# handle without making a Stream object, and pass addresses as plain ints: 24 -> 8.5 us for a quantise call. The steps of
# the 4-bit layer take addresses as they are, like those of the other layers.
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream
_u8, _i32, _f32 = torch.uint8, torch.int32, torch.float32
_forward_ad = torch.autograd.forward_ad


def _like(t, dtype, shape):
    """Whether t is a contiguous CUDA tensor of this dtype and shape."""
    return (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.is_cuda)


def _need(t, name, dtypes, shape, contiguous=True):
    """ValueError that says why t is not a CUDA tensor of one of these dtypes and of this shape (None: any size);
    returns where it is one."""
    dtypes = dtypes if isinstance(dtypes, tuple) else (dtypes,)
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, not {t.dtype}")
    if t.dim() != len(shape) or any(n is not None and n != m for n, m in zip(shape, t.shape)):
        raise ValueError(f"{name} must have shape {shape}, not {tuple(t.shape)}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _no_tangents(*tensors):
    """Refuses a tensor with a tangent of forward mode: no call of the library takes a derivative that way, and an output
    without one would stand for a derivative of zero."""
    if getattr(_forward_ad, "_current_level", 0) < 0:  # no level is open
        return
    for t in tensors:
        if isinstance(t, torch.Tensor) and _forward_ad.unpack_dual(t).tangent is not None:
            raise NotImplementedError("there is no forward-mode derivative of this call")


def _plain(*tensors):
    """Refuses what a kernel would not see of the tensors among these: a tangent, or that there is no memory."""
    _no_tangents(*tensors)
    for t in tensors:
        if isinstance(t, torch.Tensor):
            _memory(t)


def _fp4_format(fmt):
    if fmt not in FP4_FORMATS:
        raise ValueError(f"unknown 4-bit format {fmt!r}: 'nvfp4' or 'mxfp4'")
    return FP4_FORMATS[fmt]


def _fp4_matrix(q, s, fmt, name):
    """(rows, cols) of a 4-bit matrix."""
    if not (isinstance(q, torch.Tensor) and q.dim() == 2 and _like(q, _u8, q.shape)):
        _need(q, name + " codes", _u8, (None, None))
    rows, half = q.shape
    cols = 2 * half
    if not _like(s, _u8, (rows, cols // FP4_BLOCK[fmt])):
        _need(s, name + " scales", _u8, (rows, cols // FP4_BLOCK[fmt]))
    return rows, cols


def _fp4_scale(g, name):
    """Address of an fp32 [1] scale, or None."""
    if g is None:
        return None
    if not _like(g, _f32, (1,)):
        _need(g, name, _f32, (1,))
    return _memory(g)


def quantize_fp4(x: torch.Tensor, fmt: str = "nvfp4", g: torch.Tensor | None = None, q=None, s=None):
    """Rows [rows, cols] (fp32, bf16 or fp16; cols a multiple of 32; the rows may be strided) to microscaled 4
    bits: (codes uint8 [rows, cols/2], scales uint8 [rows, cols/16] for 'nvfp4', [rows, cols/32] for 'mxfp4').
    g: fp32 [1], the NVFP4 scale of the matrix (moe_quantize_fp4 in include/moe.h), None = 1."""
    f = _fp4_format(fmt)
    if not (isinstance(x, torch.Tensor) and x.dim() == 2 and x.is_cuda and x.dtype in ELEMENT_TYPES):
        _need(x, "x", tuple(ELEMENT_TYPES), (None, None), contiguous=False)
    rows, cols = x.shape
    ldx, one = x.stride()
    if one != 1 and cols > 1:
        raise ValueError("the elements of a row of x must be contiguous")
    n = cols // FP4_BLOCK[fmt]
    if q is None:
        q = torch.empty(rows, cols // 2, dtype=_u8, device=x.device)
    elif not _like(q, _u8, (rows, cols // 2)):
        _need(q, "q", _u8, (rows, cols // 2))
    if s is None:
        s = torch.empty(rows, n, dtype=_u8, device=x.device)
    elif not _like(s, _u8, (rows, n)):
        _need(s, "s", _u8, (rows, n))
    _check((_lib or load()).moe_quantize_fp4(_memory(x), ELEMENT_TYPES[x.dtype], rows, cols, ldx if rows > 1 else cols,
                                             f, _fp4_scale(g, "g"), _memory(q), _memory(s),
                                             _raw_stream(_current_device())))
    return q, s


def dequantize_fp4(q: torch.Tensor, s: torch.Tensor, fmt: str = "nvfp4", g: torch.Tensor | None = None,
                   dtype=torch.float32, y=None) -> torch.Tensor:
    """The values [rows, cols] that 4-bit rows stand for, rounded once to dtype (or to y's)."""
    f = _fp4_format(fmt)
    rows, cols = _fp4_matrix(q, s, fmt, "4-bit")
    if y is None:
        y = torch.empty(rows, cols, dtype=dtype, device=q.device)
    if y.dtype not in ELEMENT_TYPES or not _like(y, y.dtype, (rows, cols)):
        _need(y, "y", tuple(ELEMENT_TYPES), (rows, cols))
    _check((_lib or load()).moe_dequantize_fp4(_memory(q), _memory(s), rows, cols, f, _fp4_scale(g, "g"),
                                               ELEMENT_TYPES[y.dtype], _memory(y), _raw_stream(_current_device())))
    return y


def matmul_fp4(aq, a_s, bq, b_s, fmt: str = "nvfp4", ga=None, gb=None, dtype=torch.bfloat16, y=None,
               status=None) -> torch.Tensor:
    """y [M, N] = A B^T of 4-bit matrices A [M, K] and B [N, K] (codes, scales, NVFP4 matrix scales fp32 [1] or
    None = 1), fp32 accumulation, rounded once to bf16 or fp32. y may have strided rows. status: int32 [1] that
    MOE_STATUS_WAIT_TIMEOUT is added to if a wait of the kernel gives up; None: matmul_fp4_status() reports it."""
    f = _fp4_format(fmt)
    M, K = _fp4_matrix(aq, a_s, fmt, "A")
    N, kb = _fp4_matrix(bq, b_s, fmt, "B")
    if K != kb:
        raise ValueError(f"A has rows of {K} elements, B of {kb}")
    ldy = N
    if y is None:
        y = torch.empty(M, N, dtype=dtype, device=aq.device)
        if dtype is not torch.bfloat16 and dtype is not _f32:
            raise ValueError(f"y must be bf16 or fp32, not {dtype}")
    else:
        _need(y, "y", (torch.bfloat16, _f32), (M, N), contiguous=False)
        if M > 1:
            ldy = y.stride(0)
        if N > 1 and y.stride(1) != 1:
            raise ValueError("the elements of a row of y must be contiguous")
    if status is not None:
        _need(status, "status", _i32, (1,))
    _check((_lib or load()).moe_matmul_fp4(_memory(aq), _memory(a_s), _fp4_scale(ga, "ga"), _memory(bq),
                                           _memory(b_s), _fp4_scale(gb, "gb"), M, N, K, f, ELEMENT_TYPES[y.dtype],
                                           _memory(y), ldy, _address(status),
                                           _raw_stream(_current_device())))
    return y


def matmul_fp4_status() -> int:
    """MOE_STATUS_* bits of the matmul_fp4 calls without a status of their own since the last read, once the current
    stream has come this far; 0: every wait ended. Reading clears them."""
    v = ctypes.c_int32()
    rc = load().moe_matmul_fp4_status(ctypes.byref(v), _stream())
    if rc not in (MOE_OK, MOE_ERR_DEVICE):
        _check(rc)
    return v.value


class Fp4Activations:
    """Scales of a layer's 4-bit rows (fp32 [1] each, None = 1): g_x of the rows that enter the gate/up product,
    g_h of the SwiGLU product; usually the largest magnitude seen in calibration / 2688. NVFP4 only."""

    def __init__(self, g_x: torch.Tensor | None = None, g_h: torch.Tensor | None = None):
        self.tensors = (g_x, g_h)
        self.struct = MoeFp4Activations(_fp4_scale(g_x, "g_x"), _fp4_scale(g_h, "g_h"))


def _act(act: Fp4Activations | None):
    return None if act is None else ctypes.byref(act.struct)


def _address(t):
    return None if t is None else _memory(t)


def dispatch_fp4(cfg, act: Fp4Activations | None, x, topk_idx, topk_w, counts, offsets, inv_pos, row_token, row_weight,
                 xq, xs, ws):
    """moe_dispatch_fp4: dispatch with the rows quantised to the 4 bits of cfg's weights."""
    _check((_lib or load()).moe_dispatch_fp4(ctypes.byref(cfg), _act(act), _address(x), _address(topk_idx),
                                             _address(topk_w), _address(counts), _address(offsets), _address(inv_pos),
                                             _address(row_token), _address(row_weight), _address(xq), _address(xs),
                                             _address(ws), ws.numel(), _raw_stream(_current_device())))


def expert_ffn_fp4(cfg, weights: Weights, act: Fp4Activations | None, xq, xs, offsets, row_weight, yd, ws):
    """moe_expert_ffn_fp4: the experts on 4-bit rows."""
    _check((_lib or load()).moe_expert_ffn_fp4(ctypes.byref(cfg), ctypes.byref(weights.struct), _act(act), _address(xq),
                                               _address(xs), _address(offsets), _address(row_weight), _address(yd),
                                               _address(ws), ws.numel(), _raw_stream(_current_device())))


def forward_fp4(cfg, x, weights: Weights, act: Fp4Activations | None, y, ws):
    """moe_forward_fp4: the whole layer with 4-bit rows and 4-bit weights (dtype 'nvfp4' or 'mxfp4')."""
    _check((_lib or load()).moe_forward_fp4(ctypes.byref(cfg), _address(x), ctypes.byref(weights.struct), _act(act),
                                            _address(y), _address(ws), ws.numel(), _raw_stream(_current_device())))


def balance_loss_workspace(cfg: MoeConfig, n_seq: int = 1, device="cuda") -> torch.Tensor:
    n = ctypes.c_size_t()
    _check(load().moe_balance_loss_workspace_size(ctypes.byref(cfg), n_seq, ctypes.byref(n)))
    return torch.empty(n.value, dtype=torch.uint8, device=device)


def _balance_inputs(cfg, logits, seq_offsets, token_mask):
    """(n_seq, type of the logits, addresses of seq_offsets and token_mask) after the checks of both directions."""
    if not (_like(logits, _f32, (cfg.T, cfg.E)) or _like(logits, torch.bfloat16, (cfg.T, cfg.E))):
        _need(logits, "logits", (_f32, torch.bfloat16), (cfg.T, cfg.E))
    mask = offsets = None
    if token_mask is not None:
        if not (_like(token_mask, _u8, (cfg.T,)) or _like(token_mask, torch.bool, (cfg.T,))):
            _need(token_mask, "token_mask", (_u8, torch.bool), (cfg.T,))
        mask = _memory(token_mask)
    n_seq = 1
    if seq_offsets is not None:
        if not (isinstance(seq_offsets, torch.Tensor) and _like(seq_offsets, _i32, (seq_offsets.numel(),))):
            _need(seq_offsets, "seq_offsets", _i32, (None,))
        n_seq = seq_offsets.shape[0] - 1
        if n_seq < 1:
            raise ValueError("seq_offsets must hold the begin of each sequence and the end of the last")
        offsets = _memory(seq_offsets)
    return n_seq, ELEMENT_TYPES[logits.dtype], offsets, mask


def _balance_loss(logits, cfg, topk_idx, alpha, seq_offsets, token_mask, ws):
    """(loss, counts, mean_prob, tokens)."""
    _no_tangents(logits)
    S, kind, offsets, mask = _balance_inputs(cfg, logits, seq_offsets, token_mask)
    if not _like(topk_idx, _i32, (cfg.T, cfg.k)):
        _need(topk_idx, "topk_idx", _i32, (cfg.T, cfg.k))
    dev = logits.device
    if ws is None:
        ws = balance_loss_workspace(cfg, S, dev)
    elif not _like(ws, _u8, (ws.numel(),)):
        _need(ws, "ws", _u8, (None,))
    loss = torch.empty(S, dtype=_f32, device=dev)
    counts = torch.empty(S, cfg.E, dtype=_i32, device=dev)
    mean = torch.empty(S, cfg.E, dtype=_f32, device=dev)
    tokens = torch.empty(S, dtype=_i32, device=dev)
    _check((_lib or load()).moe_balance_loss(ctypes.byref(cfg), _memory(logits), kind, _memory(topk_idx), offsets, S,
                                             mask, alpha, loss.data_ptr(), _memory(counts), mean.data_ptr(),
                                             _memory(tokens), _memory(ws), ws.numel(),
                                             _raw_stream(_current_device())))
    return loss, counts, mean, tokens


class _BalanceLoss(torch.autograd.Function):
    """The loss as a node of autograd, whose gradient is moe_balance_loss_backward."""

    @staticmethod
    def forward(ctx, logits, cfg, topk_idx, alpha, seq_offsets, token_mask, ws):
        loss, counts, mean, tokens = _balance_loss(logits, cfg, topk_idx, alpha, seq_offsets, token_mask, ws)
        ctx.mark_non_differentiable(counts, mean, tokens)
        ctx.save_for_backward(logits, counts, tokens, seq_offsets, token_mask)
        ctx.cfg, ctx.alpha = cfg, alpha
        return loss, counts, mean, tokens

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dloss, *_):
        logits, counts, tokens, seq_offsets, token_mask = ctx.saved_tensors
        if not dloss.is_contiguous() or dloss.data_ptr() % 16:  # an expanded sum's gradient, a slice of another tensor
            dloss = dloss.clone(memory_format=torch.contiguous_format)
        d = balance_loss_backward(ctx.cfg, logits, counts, tokens, ctx.alpha, dloss, seq_offsets, token_mask)
        return d, None, None, None, None, None, None


def balance_loss(cfg, logits, topk_idx, alpha: float, seq_offsets=None, token_mask=None, ws=None) -> dict:
    """The router's load-balance loss (moe_balance_loss in include/moe.h) of logits [T, E] (fp32 or bf16) and the
    chosen experts topk_idx [T, k]: loss [S], counts [S, E], mean_prob [S, E] and tokens [S] of S sequences
    (seq_offsets int32 [S + 1]; None: one of all tokens). token_mask [T]: 0 = padding. ws: balance_loss_workspace.

    The loss is differentiable once with respect to logits that require a gradient, by balance_loss_backward; counts,
    mean_prob and tokens carry no gradient. (As for any operation: a backward pass that is captured into a CUDA graph
    must not share leaves with an eager graph that is still alive.)"""
    run = _balance_loss
    if getattr(logits, "requires_grad", False) and torch.is_grad_enabled():
        run = _BalanceLoss.apply
    loss, counts, mean, tokens = run(logits, cfg, topk_idx, alpha, seq_offsets, token_mask, ws)
    return {"loss": loss, "counts": counts, "mean_prob": mean, "tokens": tokens}


def balance_loss_backward(cfg, logits, counts, tokens, alpha: float, dloss, seq_offsets=None, token_mask=None,
                          dlogits=None) -> torch.Tensor:
    """Gradient of balance_loss with respect to logits (of their dtype), from its counts and tokens and the
    gradients dloss [S] of its losses: what backward() of the loss calls, for use without autograd. The gradient is
    not itself differentiable."""
    S, kind, offsets, mask = _balance_inputs(cfg, logits, seq_offsets, token_mask)
    if not (_like(counts, _i32, (S, cfg.E)) and _like(tokens, _i32, (S,)) and _like(dloss, _f32, (S,))):
        _need(counts, "counts", _i32, (S, cfg.E))
        _need(tokens, "tokens", _i32, (S,))
        _need(dloss, "dloss", _f32, (S,))
    if dlogits is None:
        dlogits = torch.empty_like(logits)
    else:
        _need(dlogits, "dlogits", logits.dtype, (cfg.T, cfg.E))
    _check((_lib or load()).moe_balance_loss_backward(ctypes.byref(cfg), _memory(logits), kind, _memory(counts),
                                                      _memory(tokens), offsets, S, mask, alpha, _memory(dloss),
                                                      _memory(dlogits), _raw_stream(_current_device())))
    return dlogits


# ------------------------------------------------------------------------------------------
# around the experts: the norm in front, rows sorted by expert and back, and the gradients
# ------------------------------------------------------------------------------------------
# On small tensors the calls below are bound by the host, so each is first made as a whole by csrc/calls.cpp. What that
# does not take (it returns None) goes through the steps here, which find the words of a refusal.
def _new(shape, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda")


def _native():
    if _calls is None:
        load()
    return _calls


def _here(a, b=None, c=None, d=None, e=None):
    """Raw handle of the current stream; the tensors have to be on its device."""
    dev = _current_device()
    if (a.get_device() != dev or (b is not None and b.get_device() != dev) or (c is not None and c.get_device() != dev)
            or (d is not None and d.get_device() != dev) or (e is not None and e.get_device() != dev)):
        raise ValueError(f"tensors must be on the current device, cuda:{dev}")
    return _raw_stream(dev)


def _gradient(t):
    """A gradient that autograd hands over, as the library reads it: contiguous, on 16 bytes."""
    if t.is_contiguous() and t.data_ptr() % 16 == 0:
        return t
    return t.clone(memory_format=torch.contiguous_format)


def _kept(cfg):
    """A copy of a configuration for a backward pass, which the caller may change meanwhile (T, for the next batch)."""
    copy = MoeConfig.from_buffer_copy(cfg)
    copy._placement = getattr(cfg, "_placement", None)
    return copy


def _wants_gradient(a, b=None, c=None):
    return (getattr(a, "requires_grad", False) or getattr(b, "requires_grad", False)
            or getattr(c, "requires_grad", False)) and torch.is_grad_enabled()


def _row_matrix(t, name, dtypes, shape=(None, None)):
    """Elements from row to row of a matrix whose rows may be strided."""
    if not (isinstance(t, torch.Tensor) and t.dim() == 2 and t.is_cuda and t.dtype in dtypes
            and (shape[0] is None or t.shape == shape)):
        _need(t, name, tuple(dtypes), shape, contiguous=False)
    ld, one = t.stride()
    if one != 1 and t.shape[1] > 1:
        raise ValueError(f"the elements of a row of {name} must be contiguous")
    return ld if t.shape[0] > 1 else t.shape[1]


def _norm_weight(weight, dtype, cols):
    """(address, type) of the norm's weight."""
    if weight is None:
        return None, ELEMENT_TYPES[dtype]
    if not (_like(weight, dtype, (cols,)) or _like(weight, _f32, (cols,))):
        _need(weight, "weight", (dtype, _f32), (cols,))
    return weight.data_ptr(), ELEMENT_TYPES[weight.dtype]


def _rms_norm(x, weight, residual, eps, fp8, with_y):
    """(y, total, q, s), None where not wanted."""
    out = (_calls or _native()).rms_norm(x, weight, residual, eps, fp8, with_y)
    if out is not None:
        return out
    _plain(x, weight, residual)
    ldx = _row_matrix(x, "x", ELEMENT_TYPES)
    shape, dtype = x.shape, x.dtype
    rows, cols = shape
    w, w_type = _norm_weight(weight, dtype, cols)
    y = total = q = s = r = to = None
    r_type = ldr = 0
    if residual is not None:
        if not (_like(residual, dtype, shape) or _like(residual, _f32, shape)):
            ldr = _row_matrix(residual, "residual", (dtype, _f32), shape)
            total = _new((rows, cols), residual.dtype)
        else:
            ldr, total = cols, _new((rows, cols), residual.dtype)
        r, r_type, to = residual.data_ptr(), ELEMENT_TYPES[residual.dtype], total.data_ptr()
    if with_y:
        y = _new((rows, cols), dtype)
    if fp8:
        q = _new((rows, cols), _u8)
        n = (cols + 127) // 128
        s = _new((rows, n), _f32)
    rc = (_lib or load()).moe_rms_norm(x.data_ptr(), ELEMENT_TYPES[dtype], rows, cols, ldx, r, r_type, ldr, w, w_type, eps,
                                       y.data_ptr() if with_y else None, to, q.data_ptr() if fp8 else None,
                                       s.data_ptr() if fp8 else None, _here(x, weight, residual))
    if rc:
        _check(rc)
    return y, total, q, s


class _RmsNorm(torch.autograd.Function):
    """The norm as a node of autograd, whose gradient is moe_rms_norm_backward."""

    @staticmethod
    def forward(ctx, x, weight, residual, eps, fp8, with_y):
        y, total, q, s = _rms_norm(x, weight, residual, eps, fp8, with_y)
        ctx.set_materialize_grads(False)
        ctx.mark_non_differentiable(*(t for t in (q, s) if t is not None))
        ctx.save_for_backward(x if total is None else total, weight)
        ctx.eps, ctx.types = eps, (x.dtype, None if residual is None else residual.dtype)
        return y, total, q, s

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dtotal, *_):
        total, weight = ctx.saved_tensors
        kind, other = ctx.types
        if dy is None:  # only the total was used: it is the sum
            return (None if dtotal is None else dtotal.to(kind), None, dtotal, None, None, None)
        dx, dresidual, dweight = rms_norm_backward(_gradient(dy), total, weight, ctx.eps,
                                                   None if dtotal is None else _gradient(dtotal),
                                                   weight_gradient=ctx.needs_input_grad[1])
        return dx, dweight, None if other is None else dresidual, None, None, None


def rms_norm(x, weight=None, residual=None, eps: float = 1e-6):
    """Root-mean-square norm (moe_rms_norm in include/moe.h) of x [rows, cols] (fp32, bf16 or fp16; the rows may be
    strided), or of x + residual (of x's type or fp32), times weight [cols] (x's type or fp32; None: ones): y of x's type,
    and with a residual (y, total), total = x + residual of the residual's type.

    Differentiable once with respect to x, residual and weight. (As for any operation: a backward pass that is captured
    into a CUDA graph must not share leaves with an eager graph that is still alive.)"""
    run = _RmsNorm.apply if _wants_gradient(x, weight, residual) else _rms_norm
    y, total, _, _ = run(x, weight, residual, eps, False, True)
    return y if residual is None else (y, total)


def rms_norm_fp8(x, weight=None, residual=None, eps: float = 1e-6, with_y: bool = False) -> dict:
    """rms_norm with an output in 8 bits: q uint8 [rows, cols] (e4m3 codes) and s fp32 [rows, ceil(cols / 128)], the rows of
    an FP8 layer; total with a residual, and y of x's type with_y (for a router). y and total are differentiable, codes and
    scales are not."""
    run = _RmsNorm.apply if _wants_gradient(x, weight, residual) else _rms_norm
    out = dict(zip(("y", "total", "q", "s"), run(x, weight, residual, eps, True, with_y)))
    return {name: t for name, t in out.items() if t is not None}


def rms_norm_backward(dy, total, weight=None, eps: float = 1e-6, dtotal=None, weight_gradient: bool = True, ws=None):
    """Gradient of rms_norm (moe_rms_norm_backward): (dx of dy's type, dresidual of total's type, dweight of weight's type or
    None) from dy, the total that was normalised (x without a residual) and the gradient dtotal that reaches the total
    from elsewhere. dresidual is dx itself where the types are the same. ws: rms_norm_backward_workspace."""
    out = (_calls or _native()).rms_norm_backward(dy, total, weight, eps, dtotal, weight_gradient, ws)
    if out is not None:
        return out
    _plain(dy, total, weight, dtotal, ws)
    if not (isinstance(dy, torch.Tensor) and dy.dim() == 2 and dy.dtype in ELEMENT_TYPES and dy.is_cuda
            and dy.is_contiguous()):
        _need(dy, "dy", tuple(ELEMENT_TYPES), (None, None))
    shape, kind = dy.shape, dy.dtype
    rows, cols = shape
    ldt = _row_matrix(total, "total", (kind, _f32), shape)
    of = total.dtype
    if dtotal is not None and not _like(dtotal, of, shape):
        _need(dtotal, "dtotal", of, shape)
    w, w_type = _norm_weight(weight, kind, cols)
    dx = _new((rows, cols), kind)
    dresidual, dweight = dx, None
    if of is not kind:
        dresidual = _new((rows, cols), of)
    if weight is not None and weight_gradient:
        dweight = _new((cols,), weight.dtype)
        if ws is None:
            ws = _new((_rms_norm_backward_bytes(rows, cols),), _u8)
        elif not _like(ws, _u8, (ws.numel(),)):
            _need(ws, "ws", _u8, (None,))
    rc = (_lib or load()).moe_rms_norm_backward(
        dy.data_ptr(), ELEMENT_TYPES[kind], rows, cols, total.data_ptr(), ELEMENT_TYPES[of], ldt,
        None if dtotal is None else dtotal.data_ptr(), w, w_type, eps, dx.data_ptr(),
        None if dresidual is dx else dresidual.data_ptr(), None if dweight is None else dweight.data_ptr(),
        None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(), _here(dy, total, dtotal, weight, ws))
    if rc:
        _check(rc)
    return dx, dresidual, dweight


@functools.lru_cache(maxsize=256)
def _rms_norm_backward_bytes(rows, cols):
    n = ctypes.c_size_t()
    _check((_lib or load()).moe_rms_norm_backward_workspace_size(rows, cols, ctypes.byref(n)))
    return n.value


def rms_norm_backward_workspace(rows: int, cols: int, device="cuda") -> torch.Tensor:
    return torch.empty(_rms_norm_backward_bytes(rows, cols), dtype=_u8, device=device)


@functools.lru_cache(maxsize=256)
def _sort_tokens_bytes(T, E, k):
    n = ctypes.c_size_t()
    _check((_lib or load()).moe_sort_tokens_workspace_size(ctypes.byref(make_config(T, 256, E, k, 256)), ctypes.byref(n)))
    return n.value


def sort_tokens_workspace(cfg: MoeConfig, device="cuda") -> torch.Tensor:
    return torch.empty(_sort_tokens_bytes(cfg.T, cfg.E, cfg.k), dtype=_u8, device=device)


def _groups(cfg):
    return cfg.placement.contents.n_slots if cfg.placement else cfg.E


def sort_tokens(cfg, topk_idx, topk_w=None, ws=None) -> dict:
    """The assignments of topk_idx int32 [T, k] sorted by expert (moe_sort_tokens): counts, offsets, inv_pos [T, k], row_token
    [T k], and row_weight [T k] with topk_w fp32 [T, k]. Entries outside [0, E) are no assignment. ws:
    sort_tokens_workspace. row_weight carries no gradient: weights that require one are refused (they are applied, and get
    theirs, in unpermute)."""
    if getattr(topk_w, "requires_grad", False) and torch.is_grad_enabled():
        raise ValueError("row_weight carries no gradient: pass topk_w.detach(), and topk_w itself to unpermute")
    out = (_calls or _native()).sort_tokens(cfg, topk_idx, topk_w, ws)
    if out is not None:
        counts, offsets, inv_pos, row_token, row_weight = out
        out = {"counts": counts, "offsets": offsets, "inv_pos": inv_pos, "row_token": row_token}
        if row_weight is not None:
            out["row_weight"] = row_weight
        return out
    _plain(topk_idx, topk_w, ws)
    T, k = cfg.T, cfg.k
    shape = (T, k)
    if not _like(topk_idx, _i32, shape):
        _need(topk_idx, "topk_idx", _i32, shape)
    if topk_w is not None and not _like(topk_w, _f32, shape):
        _need(topk_w, "topk_w", _f32, shape)
    n = _groups(cfg)
    if ws is None:
        size = _sort_tokens_bytes(T, cfg.E, k)
        if size:
            ws = _new((size,), _u8)
    elif not _like(ws, _u8, (ws.numel(),)):
        _need(ws, "ws", _u8, (None,))
    counts, offsets = _new((n,), _i32), _new((n + 1,), _i32)
    inv_pos, row_token = _new(shape, _i32), _new((T * k,), _i32)
    out = {"counts": counts, "offsets": offsets, "inv_pos": inv_pos, "row_token": row_token}
    w = row_weight = None
    if topk_w is not None:
        out["row_weight"] = row_weight = _new((T * k,), _f32)
        w, row_weight = topk_w.data_ptr(), row_weight.data_ptr()
    rc = (_lib or load()).moe_sort_tokens(
        ctypes.byref(cfg), topk_idx.data_ptr(), w, counts.data_ptr(), offsets.data_ptr(), inv_pos.data_ptr(),
        row_token.data_ptr(), row_weight, None if ws is None else ws.data_ptr(), 0 if ws is None else ws.numel(),
        _here(topk_idx, topk_w, ws))
    if rc:
        _check(rc)
    return out


def _positions(cfg, shape, inv_pos, offsets=None):
    if not _like(inv_pos, _i32, shape):
        _need(inv_pos, "inv_pos", _i32, shape)
    if offsets is not None and not _like(offsets, _i32, (_groups(cfg) + 1,)):
        _need(offsets, "offsets", _i32, (_groups(cfg) + 1,))


def _route_weights_of(weights, shape):
    """Address of the route weights, or None."""
    if weights is None:
        return None
    if not _like(weights, _f32, shape):
        _need(weights, "weights", _f32, shape)
    return weights.data_ptr()


_COPIED = (torch.bfloat16, _f32, torch.float16, _u8)


def _permute(x, cfg, inv_pos, offsets, scales):
    out = (_calls or _native()).permute(cfg, x, inv_pos, offsets, scales)
    if out is not None:
        return out
    _plain(x, inv_pos, offsets, scales)
    T, k = cfg.T, cfg.k
    _positions(cfg, (T, k), inv_pos, offsets)
    ldx = _row_matrix(x, "x", _COPIED if scales is None else (_u8,))
    rows, cols = x.shape
    if rows != T:
        _need(x, "x", x.dtype, (T, cols), contiguous=False)
    xd = _new((T * k, cols), x.dtype)
    xd_scales = of = to = None
    if scales is not None:
        n = (cols + 127) // 128
        if not _like(scales, _f32, (T, n)):
            _need(scales, "scales", _f32, (T, n))
        xd_scales = _new((T * k, n), _f32)
        of, to = scales.data_ptr(), xd_scales.data_ptr()
    rc = (_lib or load()).moe_permute(ctypes.byref(cfg), x.data_ptr(), x.element_size(), cols, ldx, of, inv_pos.data_ptr(),
                                      offsets.data_ptr(), xd.data_ptr(), to, _here(x, inv_pos, offsets, scales))
    if rc:
        _check(rc)
    return xd if scales is None else (xd, xd_scales)


class _Permute(torch.autograd.Function):
    """Rows sorted by expert as a node of autograd, whose gradient is moe_unpermute without weights."""

    @staticmethod
    def forward(ctx, x, cfg, inv_pos, offsets):
        ctx.cfg = _kept(cfg)
        ctx.save_for_backward(inv_pos)
        return _permute(x, cfg, inv_pos, offsets, None)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dxd):
        return _unpermute(_gradient(dxd), None, None, ctx.cfg, ctx.saved_tensors[0]), None, None, None


def permute(cfg, x, inv_pos, offsets, scales=None):
    """Rows of x [T, cols] (fp32, bf16, fp16 or uint8; the rows may be strided) into expert order (moe_permute): xd [T k, cols], with
    inv_pos and offsets of sort_tokens. Rows past the last one held are zero. With scales fp32 [T, ceil(cols / 128)], x
    holds e4m3 codes (uint8) and (xd, xd_scales) are returned. Differentiable once with respect to x (not 8-bit)."""
    if scales is None and _wants_gradient(x):
        return _Permute.apply(x, cfg, inv_pos, offsets)
    return _permute(x, cfg, inv_pos, offsets, scales)


def _unpermute(yd, weights, base, cfg, inv_pos):
    y = (_calls or _native()).unpermute(cfg, yd, inv_pos, weights, base)
    if y is not None:
        return y
    _plain(yd, inv_pos, weights, base)
    T, k = cfg.T, cfg.k
    shape = (T, k)
    _positions(cfg, shape, inv_pos)
    w = _route_weights_of(weights, shape)
    if not (isinstance(yd, torch.Tensor) and yd.dim() == 2 and yd.dtype in ELEMENT_TYPES and yd.is_cuda
            and yd.is_contiguous() and yd.shape[0] == T * k):
        _need(yd, "yd", tuple(ELEMENT_TYPES), (T * k, None))
    dtype, cols = yd.dtype, yd.shape[1]
    b = None
    if base is None:
        y = _new((T, cols), dtype)
    else:
        if not _like(base, dtype, (T, cols)):
            _need(base, "base", dtype, (T, cols))
        y, b = _new((T, cols), dtype), base.data_ptr()
    rc = (_lib or load()).moe_unpermute(ctypes.byref(cfg), yd.data_ptr(), ELEMENT_TYPES[dtype], cols, inv_pos.data_ptr(), w, b,
                                        y.data_ptr(), _here(yd, inv_pos, weights, base))
    if rc:
        _check(rc)
    return y


class _Unpermute(torch.autograd.Function):
    """Rows back in token order as a node of autograd, whose gradient is moe_unpermute_backward."""

    @staticmethod
    def forward(ctx, yd, weights, base, cfg, inv_pos, offsets):
        ctx.cfg = _kept(cfg)
        ctx.save_for_backward(yd if weights is not None and weights.requires_grad else None, weights, inv_pos, offsets)
        return _unpermute(yd, weights, base, cfg, inv_pos)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        yd, weights, inv_pos, offsets = ctx.saved_tensors
        dyd = dw = None
        if ctx.needs_input_grad[0] or ctx.needs_input_grad[1]:
            dyd, dw = unpermute_backward(ctx.cfg, _gradient(dy), yd, inv_pos, offsets, weights)
        return dyd, dw, dy if ctx.needs_input_grad[2] else None, None, None, None


def unpermute(cfg, yd, inv_pos, weights=None, base=None, offsets=None):
    """Rows yd [T k, cols] (fp32, bf16 or fp16) back in token order, added up (moe_unpermute): y[t] = base[t] + sum over the
    slots of weights[t, j] yd[inv_pos[t, j]]; weights fp32 [T, k] (None: ones), base [T, cols] of yd's type or None.
    Differentiable once with respect to yd, weights and base; that takes the offsets of sort_tokens too."""
    if _wants_gradient(yd, weights, base):
        if offsets is None:
            raise ValueError("the gradient of unpermute needs offsets")
        _positions(cfg, (cfg.T, cfg.k), inv_pos, offsets)
        return _Unpermute.apply(yd, weights, base, cfg, inv_pos, offsets)
    return _unpermute(yd, weights, base, cfg, inv_pos)


def unpermute_backward(cfg, dy, yd, inv_pos, offsets, weights=None):
    """Gradient of unpermute (moe_unpermute_backward): (dyd [T k, cols] of dy's type, zero in the rows past the last one held;
    dweights fp32 [T, k], None where yd is None) from dy [T, cols]."""
    out = (_calls or _native()).unpermute_backward(cfg, dy, yd, inv_pos, offsets, weights)
    if out is not None:
        return out
    _plain(dy, yd, inv_pos, offsets, weights)
    T, k = cfg.T, cfg.k
    shape = (T, k)
    _positions(cfg, shape, inv_pos, offsets)
    w = _route_weights_of(weights, shape)
    if not (isinstance(dy, torch.Tensor) and dy.dim() == 2 and dy.dtype in ELEMENT_TYPES and dy.is_cuda
            and dy.is_contiguous() and dy.shape[0] == T):
        _need(dy, "dy", tuple(ELEMENT_TYPES), (T, None))
    cols, kind = dy.shape[1], dy.dtype
    dw = of = to = None
    if yd is None:
        dyd = _new((T * k, cols), kind)
    else:
        if not _like(yd, kind, (T * k, cols)):
            _need(yd, "yd", kind, (T * k, cols))
        dyd, dw = _new((T * k, cols), kind), _new(shape, _f32)
        of, to = yd.data_ptr(), dw.data_ptr()
    rc = (_lib or load()).moe_unpermute_backward(ctypes.byref(cfg), dy.data_ptr(), of, ELEMENT_TYPES[kind], cols,
                                                 inv_pos.data_ptr(), offsets.data_ptr(), w, dyd.data_ptr(), to,
                                                 _here(dy, yd, inv_pos, offsets, weights))
    if rc:
        _check(rc)
    return dyd, dw


def _route_weights(logits, cfg, bias):
    """(topk_idx, topk_w)."""
    _plain(logits, bias)
    if not _like(logits, _f32, (cfg.T, cfg.E)):
        _need(logits, "logits", _f32, (cfg.T, cfg.E))
    if bias is not None and not _like(bias, _f32, (cfg.E,)):
        _need(bias, "bias", _f32, (cfg.E,))
    idx = torch.empty(cfg.T, cfg.k, dtype=_i32, device=logits.device)
    w = torch.empty(cfg.T, cfg.k, dtype=_f32, device=logits.device)
    struct = MoeWeightsStruct(bias=_address(bias))
    _check((_lib or load()).moe_route(ctypes.byref(cfg), None, ctypes.byref(struct), logits.data_ptr(), MOE_LOGITS_GIVEN,
                                      idx.data_ptr(), w.data_ptr(), None, 0, _here(logits, bias)))
    return idx, w


class _RouteWeights(torch.autograd.Function):
    """The route weights as a node of autograd, whose gradient is moe_route_backward."""

    @staticmethod
    def forward(ctx, logits, cfg, bias):
        idx, w = _route_weights(logits, cfg, bias)
        ctx.cfg = _kept(cfg)
        ctx.mark_non_differentiable(idx)
        ctx.save_for_backward(logits, idx)
        return idx, w

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, _, dw):
        logits, idx = ctx.saved_tensors
        return route_backward(ctx.cfg, logits, idx, _gradient(dw)), None, None


def route_weights(cfg, logits, bias=None):
    """(topk_idx int32 [T, k], topk_w fp32 [T, k]) of the router's logits fp32 [T, E] (moe_route with the logits given; bias
    fp32 [E], sigmoid scoring only). The weights are differentiable once with respect to the logits, by route_backward; the
    selection and its bias carry no gradient."""
    run = _RouteWeights.apply if _wants_gradient(logits) else _route_weights
    return run(logits, cfg, bias)


def route_backward(cfg, logits, topk_idx, dtopk_w, dlogits=None) -> torch.Tensor:
    """Gradient of the route weights with respect to the logits [T, E] (fp32 or bf16), of their dtype
    (moe_route_backward), from the chosen experts topk_idx int32 [T, k] and the weights' gradient dtopk_w fp32 [T, k]."""
    if dlogits is None:
        out = (_calls or _native()).route_backward(cfg, logits, topk_idx, dtopk_w)
        if out is not None:
            return out
    _plain(logits, topk_idx, dtopk_w, dlogits)
    T, E, k = cfg.T, cfg.E, cfg.k
    if not (_like(logits, _f32, (T, E)) or _like(logits, torch.bfloat16, (T, E))):
        _need(logits, "logits", (_f32, torch.bfloat16), (T, E))
    if not (_like(topk_idx, _i32, (T, k)) and _like(dtopk_w, _f32, (T, k))):
        _need(topk_idx, "topk_idx", _i32, (T, k))
        _need(dtopk_w, "dtopk_w", _f32, (T, k))
    if dlogits is None:
        dlogits = _new((T, E), logits.dtype)
    elif not _like(dlogits, logits.dtype, (T, E)):
        _need(dlogits, "dlogits", logits.dtype, (T, E))
    rc = (_lib or load()).moe_route_backward(ctypes.byref(cfg), logits.data_ptr(), ELEMENT_TYPES[logits.dtype],
                                             topk_idx.data_ptr(), dtopk_w.data_ptr(), dlogits.data_ptr(),
                                             _here(logits, topk_idx, dtopk_w, dlogits))
    if rc:
        _check(rc)
    return dlogits


def launch_count() -> int:
    """Kernels the library has launched in this process so far."""
    return int(load().moe_launch_count())


def device_status(cfg, ws) -> int:
    v = ctypes.c_int32()
    rc = load().moe_device_status(ctypes.byref(cfg), _ptr(ws), ctypes.byref(v), _stream())
    if rc not in (MOE_OK, MOE_ERR_DEVICE):
        _check(rc)
    return v.value


def selftest_wait_timeout(cfg, ws, limit_cycles: int) -> None:
    """Enqueue the failure-detection self-test (moe_selftest_wait_timeout): a bounded wait that nothing
    completes records MOE_STATUS_WAIT_TIMEOUT in the workspace's status word (ws None: in the word of
    matmul_fp4_status)."""
    _check(load().moe_selftest_wait_timeout(ctypes.byref(cfg), _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                            int(limit_cycles), _stream()))


def balance(cfg, ws) -> dict:
    """Load balance of the last step, computed by the library (moe_balance) on the device from the
    counts in its workspace and read back (one small copy): busiest expert's rows, busiest / mean
    (inference guide 6.4, section 5.1: the step waits for the busiest expert), experts with rows, kept
    rows, and the assignments a capacity limit dropped; plus the per-expert counts themselves (per
    physical slot under a placement)."""
    S = cfg.placement.contents.n_slots if cfg.placement else cfg.E
    stats = torch.zeros(8, dtype=torch.int32, device=ws.device)
    _check(load().moe_balance(ctypes.byref(cfg), _ptr(ws), _ptr(stats), _stream()))
    st = stats.cpu()
    counts = ws_view(ws, cfg, "counts", torch.int32, (S,)).cpu()
    return {"counts": counts.tolist(), "max_rows": int(st[0]), "active": int(st[1]), "kept": int(st[2]),
            "dropped": int(st[3]), "max_over_mean": float(st[4:5].view(torch.float32)[0])}


class MoeLayer:
    """Convenience wrapper: a config, its weights and a workspace; ``layer(x)`` runs moe_forward, or
    moe_forward_fp4 (4-bit rows and weights) with fp4_activations."""

    def __init__(self, cfg: MoeConfig, weights: Weights, device="cuda", fp4_activations: Fp4Activations | None = None):
        self.cfg = cfg
        self.weights = weights
        self.fp4_activations = fp4_activations
        self.ws = alloc_workspace(cfg, device)
        # a fresh workspace holds arbitrary bits in its status word; read-and-clear it once
        device_status(cfg, self.ws)

    def __call__(self, x: torch.Tensor, y: torch.Tensor | None = None) -> torch.Tensor:
        if y is None:
            y = torch.empty_like(x)
        if self.fp4_activations is not None:
            forward_fp4(self.cfg, x, self.weights, self.fp4_activations, y, self.ws)
        else:
            forward(self.cfg, x, self.weights, y, self.ws)
        return y


class Graph:
    """moe_forward captured as one CUDA graph (moe_graph_create); launch() recomputes y from x."""

    def __init__(self, cfg, x, weights: Weights, y, ws, stream=None):
        self.stream = stream if stream is not None else torch.cuda.current_stream()
        if self.stream.cuda_stream == 0:
            raise ValueError("capture needs a created CUDA stream, not the legacy default stream")
        self._keep = (cfg, x, weights, y, ws)
        h = ctypes.c_void_p()
        _check(load().moe_graph_create(ctypes.byref(cfg), _ptr(x), ctypes.byref(weights.struct), _ptr(y), _ptr(ws),
                                       ws.numel(), ctypes.c_void_p(self.stream.cuda_stream), ctypes.byref(h)))
        self._h = h

    def launch(self):
        _check(load().moe_graph_launch(self._h, ctypes.c_void_p(self.stream.cuda_stream)))

    def __del__(self):
        h = getattr(self, "_h", None)
        if h is not None and h.value:
            load().moe_graph_destroy(h)


class GraphedMoeLayer:
    """One CUDA graph per padded batch size (the nearest captured size at or above the batch). The graphs
    share static x / y buffers and one workspace sized for the largest batch; padding rows are computed
    and dropped (every token's output depends only on its own row)."""

    def __init__(self, make_cfg, weights: Weights, sizes, h, device="cuda", stream=None):
        self.sizes = sorted(set(int(t) for t in sizes))
        self.weights = weights
        self.stream = stream if stream is not None else torch.cuda.Stream(device=device)
        t_max = self.sizes[-1]
        self.x = torch.zeros(t_max, h, dtype=torch.bfloat16, device=device)
        self.y = torch.zeros(t_max, h, dtype=torch.bfloat16, device=device)
        self.ws = alloc_workspace(make_cfg(t_max), device)
        self.graphs = {}
        with torch.cuda.stream(self.stream):
            device_status(make_cfg(t_max), self.ws)
            for t in self.sizes:
                cfg = make_cfg(t)
                self.graphs[t] = Graph(cfg, self.x[:t], weights, self.y[:t], self.ws, self.stream)
        self.stream.synchronize()

    def padded_size(self, T: int) -> int:
        for t in self.sizes:
            if t >= T:
                return t
        raise ValueError(f"batch of {T} tokens exceeds the largest captured size {self.sizes[-1]}")

    def __call__(self, x: torch.Tensor) -> torch.Tensor:
        T = x.shape[0]
        t = self.padded_size(T)
        self.stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(self.stream):
            self.x[:T].copy_(x)
            self.graphs[t].launch()
            out = self.y[:T].clone()
        torch.cuda.current_stream().wait_stream(self.stream)
        return out
