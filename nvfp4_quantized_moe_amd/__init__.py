"""Python binding of libnvfp4moe.so — NVFP4 MoE expert FFN on MI355X (gfx950).

Argument marshalling only: every step runs in the library's HIP kernels;
torch provides device memory and the current stream. The functions carry the
names of the C entry points declared in include/nvfp4moe.h.

No call takes part in autograd: outputs come back without a history, also from
tensors that require a gradient. Gradients are calls of their own
(moe_gate_backward, moe_block_norm_backward, moe_layer_norm_backward, and for a
linear layer mxfp4_gemm on codes along the other axis), for a user's autograd
function to call; the expert layer and the dense expert have none.

Importing this module loads the built library and fails loudly when it is
missing; there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os

import torch

__all__ = [
    "lib", "LIB_PATH", "NVFP4Error", "EPI_BF16", "EPI_SILU_MUL", "EPI_SILU_MUL_DUAL", "WS_REGIONS", "nvfp4_quantize",
    "nvfp4_quantize_ws_bytes", "nvfp4_quantize_noalloc", "moe_route_slots", "moe_route_ws_bytes", "nvfp4_tile_table_len",
    "nvfp4_grouped_gemm", "moe_weighted_scatter", "nvfp4_fold_scales", "nvfp4_packed_bytes",
    "nvfp4_pack_weights", "nvfp4_moe_forward", "nvfp4_quantize_static", "nvfp4_grouped_gemm_silu_nvfp4",
    "nvfp4_moe_forward_static", "calibrate_static_gs", "nvfp4_moe_forward_stage_events", "STAGES",
    "nvfp4_moe_ws_bytes", "nvfp4_moe_ws_layout", "nvfp4_moe_tile_m", "MoEWeights", "prepare_weights",
    "ws_view", "SCORE_SOFTMAX", "SCORE_SIGMOID", "SCORE_SQRT_SOFTPLUS", "moe_gate_topk", "moe_balance_loss",
    "moe_balance_loss_ws_bytes", "moe_gate_backward", "moe_block_norm", "moe_block_norm_backward",
    "moe_block_norm_backward_ws_bytes", "int8_quantize_rows", "int8_gemm", "int8_gemm_ws_bytes", "int8_ffn_forward",
    "int8_ffn_ws_bytes",
    "Int8FFNWeights", "prepare_int8_weights", "MX_ROWS", "MX_COLUMNS", "MX_BOTH", "MX_SCALE_FLOOR", "MX_SCALE_CEIL",
    "mxfp4_padded", "mxfp4_quantize", "mxfp4_dequantize", "mxfp4_gemm", "mxfp4_gemm_ws_bytes",
    "nvfp4_moe_forward_few", "nvfp4_moe_few_ws_bytes", "nvfp4_moe_few_max_tokens", "moe_layer_norm",
    "moe_layer_norm_backward", "moe_layer_norm_backward_ws_bytes",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libnvfp4moe.so")
if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run `python __graft_entry__.py` (build()) first")
lib = ctypes.CDLL(LIB_PATH)
try:
    from . import _native  # the calls of the operators around the expert FFN (csrc/binding.cpp)
except ImportError as e:
    raise ImportError(f"the native calls are not built ({e}); run `python __graft_entry__.py` (build()) first") from e

EPI_BF16, EPI_SILU_MUL, EPI_SILU_MUL_DUAL = 0, 1, 2
SCORE_SOFTMAX, SCORE_SIGMOID, SCORE_SQRT_SOFTPLUS = 0, 1, 2
MX_ROWS, MX_COLUMNS, MX_BOTH = 1, 2, 3
MX_SCALE_FLOOR, MX_SCALE_CEIL = 0, 1
WS_REGIONS = ["x_q", "x_sf", "scalars", "counts", "offsets", "slot_token", "slot_expert", "slot_weight",
              "token_slot", "tiles", "route_scratch", "h", "h_q", "h_sf", "y", "quant_scratch", "end"]

_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_f32 = ctypes.c_float


class _Weights(ctypes.Structure):
    _fields_ = [("num_local", _i32), ("hidden", _i32), ("inter", _i32),
                ("w1", _vp), ("w1_gs", _vp), ("w2", _vp), ("w2_gs", _vp), ("w1_dual_gs", _i32)]


def _sig(name, res, *args):
    f = getattr(lib, name)
    f.restype = res
    f.argtypes = list(args)
    return f


_status_string = _sig("nvfp4_status_string", ctypes.c_char_p, ctypes.c_int)
_version = _sig("nvfp4moe_version", ctypes.c_int)
_quantize_ws = _sig("nvfp4_quantize_ws_bytes", _sz, _i64, _i64, _i64)
_quantize = _sig("nvfp4_quantize", ctypes.c_int, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _sz, _vp)
_quantize_noalloc = _sig("nvfp4_quantize_noalloc", ctypes.c_int, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp)
_quantize_static = _sig("nvfp4_quantize_static", ctypes.c_int, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp)
_route_ws = _sig("moe_route_ws_bytes", _sz, _i32, _i32, _i32)
_tile_len = _sig("nvfp4_tile_table_len", _i64, _i64, _i32, _i32)
_route = _sig("moe_route_slots", ctypes.c_int, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
              _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp)
_gemm = _sig("nvfp4_grouped_gemm", ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
             _i32, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp)
_gemm_nvfp4 = _sig("nvfp4_grouped_gemm_silu_nvfp4", ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp,
                   _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp)
_packed_bytes = _sig("nvfp4_packed_bytes", _i64, _i64, _i64, _i64)
_pack = _sig("nvfp4_pack_weights", ctypes.c_int, _vp, _vp, _i64, _i64, _i64, _vp, _vp)
_scatter = _sig("moe_weighted_scatter", ctypes.c_int, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp)
_fold = _sig("nvfp4_fold_scales", ctypes.c_int, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp)
_moe_ws_layout = _sig("nvfp4_moe_ws_layout", _sz, _i32, _i32, _i32, _i32, _i32, _i32,
                      ctypes.POINTER(_sz))
_moe_ws = _sig("nvfp4_moe_ws_bytes", _sz, _i32, _i32, _i32, _i32, _i32)
_moe_tile_m = _sig("nvfp4_moe_tile_m", _i32, _i32, _i32, _i32)
_forward = _sig("nvfp4_moe_forward", ctypes.c_int, ctypes.POINTER(_Weights), _vp, _i32, _vp, _vp,
                _i32, _i32, _vp, _vp, _sz, _vp)
_forward_stages = _sig("nvfp4_moe_forward_stage_events", ctypes.c_int, ctypes.POINTER(_Weights), _vp, _i32, _vp,
                       _vp, _i32, _i32, _vp, _vp, _sz, ctypes.POINTER(_vp), _vp)
_forward_static = _sig("nvfp4_moe_forward_static", ctypes.c_int, ctypes.POINTER(_Weights), _vp, _i32, _vp, _vp,
                       _i32, _i32, _vp, _vp, _vp, _sz, _vp)
# the C entry points behind _native, which checks their arguments and calls them itself; declared here for callers
# who bring pointers of their own
_gate_topk = _sig("moe_gate_topk", ctypes.c_int, _vp, _i32, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i32, _f32,
                  _vp, _vp, _vp)
_balance_ws = _sig("moe_balance_loss_ws_bytes", _sz, _i32, _i32, _i32)
_balance = _sig("moe_balance_loss", ctypes.c_int, _vp, _i32, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32,
                _vp, _vp, _vp, _vp, _sz, _vp)
_gate_backward = _sig("moe_gate_backward", ctypes.c_int, _vp, _i32, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _f32,
                      _vp, _vp, _vp, _vp, _vp, _i32, _vp, _vp)
_block_norm = _sig("moe_block_norm", ctypes.c_int, _vp, _i32, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _i32, _f32, _f32,
                   _vp, _vp, _vp, _vp, _vp, _vp)
_block_norm_ws = _sig("moe_block_norm_backward_ws_bytes", _sz, _i32, _i32)
_block_norm_backward = _sig("moe_block_norm_backward", ctypes.c_int, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i32,
                            _vp, _vp, _vp, _i32, _f32, _f32, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp)
_int8_rows = _sig("int8_quantize_rows", ctypes.c_int, _vp, _i32, _i32, _i32, _vp, _vp, _vp)
_int8_gemm_ws = _sig("int8_gemm_ws_bytes", _sz, _i32, _i32, _i32)
_int8_gemm = _sig("int8_gemm", ctypes.c_int, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _sz, _vp)
_int8_ffn_ws = _sig("int8_ffn_ws_bytes", _sz, _i32, _i32, _i32)
_int8_ffn = _sig("int8_ffn_forward", ctypes.c_int, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp, _sz, _vp)
_mx_padded = _sig("mxfp4_padded", _i32, _i32)
_mx_quantize = _sig("mxfp4_quantize", ctypes.c_int, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp)
_mx_dequantize = _sig("mxfp4_dequantize", ctypes.c_int, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp)
_mx_gemm_ws = _sig("mxfp4_gemm_ws_bytes", _sz, _i32, _i32, _i32)
_mx_gemm = _sig("mxfp4_gemm", ctypes.c_int, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _i32, _vp, _vp, _sz, _vp)
_few_max = _sig("nvfp4_moe_few_max_tokens", _i32)
_few_ws = _sig("nvfp4_moe_few_ws_bytes", _sz, _i32, _i32, _i32, _i32, _i32)
_few = _sig("nvfp4_moe_forward_few", ctypes.c_int, ctypes.POINTER(_Weights), _vp, _i32, _vp, _vp, _i32, _i32, _vp, _vp,
            _vp, _sz, _vp)
_layer_norm = _sig("moe_layer_norm", ctypes.c_int, _vp, _i32, _vp, _i32, _i32, _i32, _vp, _vp, _f32, _f32, _vp, _vp, _i32,
                   _vp, _vp, _vp)
_layer_norm_ws = _sig("moe_layer_norm_backward_ws_bytes", _sz, _i32, _i32)
_layer_norm_backward = _sig("moe_layer_norm_backward", ctypes.c_int, _vp, _i32, _vp, _vp, _i32, _i32, _i32, _vp, _f32,
                            _f32, _vp, _vp, _vp, _vp, _vp, _sz, _vp)


class NVFP4Error(RuntimeError):
    def __init__(self, status: int, call: str):
        super().__init__(f"{call}: status {status} ({_status_string(status).decode()})")
        self.status = status


def _check(status: int, call: str):
    if status != 0:
        raise NVFP4Error(status, call)


def _ptr(t):
    return None if t is None else t.data_ptr()


# The current stream and device as plain integers: the objects of torch.cuda
# take longer to make (3 us a stream) than the smallest kernels here to run.
_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _stream():
    return _raw_stream(_current_device())


_native.set_up(_current_device, _raw_stream, NVFP4Error)


def _dev(t, dtype, name):
    """t must be a contiguous tensor of dtype on the current device (the
    device whose current stream the call is issued on)."""
    if not (t.is_cuda and t.dtype is dtype and t.is_contiguous()):
        raise ValueError(f"{name}: expected a contiguous CUDA {dtype} tensor, got {t.dtype} on {t.device}")
    if t.get_device() != _current_device():
        raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{_current_device()}")
    return t


def _buf(t, dtype, numel, name):
    """A caller-provided buffer (or None): as _dev, holding at least numel
    elements, since the library sees only its address."""
    if t is None:
        return None
    _dev(t, dtype, name)
    if t.numel() < numel:
        raise ValueError(f"{name}: needs at least {numel} elements, got {t.numel()}")
    return t


def _shape(t, shape, name):
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def version() -> int:
    return _version()


def _alloc_ws(nbytes, device):
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


# ---------------------------------------------------------------------- quantize

def nvfp4_quantize_ws_bytes(B, M, K) -> int:
    return int(_quantize_ws(B, M, K))


def nvfp4_quantize(x, amax_in=None, q=None, sf=None, gs=None, ws=None):
    """x: BF16 [M, K] or [B, M, K] -> (q uint8 [..., K/2], sf uint8 [..., K/16], gs float32 [B])."""
    _dev(x, torch.bfloat16, "x")
    if x.dim() not in (2, 3):
        raise ValueError(f"x: expected [M, K] or [B, M, K], got shape {tuple(x.shape)}")
    batched = x.dim() == 3
    B, M, K = (x.shape if batched else (1, *x.shape))
    dev = x.device
    q = torch.empty((B, M, K // 2), dtype=torch.uint8, device=dev) if q is None else _buf(q, torch.uint8, B * M * K // 2, "q")
    sf = (torch.empty((B, M, K // 16), dtype=torch.uint8, device=dev) if sf is None
          else _buf(sf, torch.uint8, B * M * K // 16, "sf"))
    gs = torch.empty((B,), dtype=torch.float32, device=dev) if gs is None else _buf(gs, torch.float32, B, "gs")
    ws = _alloc_ws(nvfp4_quantize_ws_bytes(B, M, K), dev) if ws is None else _buf(ws, torch.uint8, 0, "ws")
    _buf(amax_in, torch.float32, B, "amax_in")
    _check(_quantize(_ptr(x), B, M, K, _ptr(amax_in), _ptr(q), _ptr(sf), _ptr(gs), _ptr(ws),
                     ws.numel(), _stream()), "nvfp4_quantize")
    if not batched:
        return q[0], sf[0], gs
    return q, sf, gs


def nvfp4_quantize_noalloc(x, q, sf, gs, amax_in=None):
    """nvfp4_quantize into caller-provided q, sf, gs without a workspace: the
    library keeps the amax partials in its own device array (at most 128
    tensors; calls that overlap on one device race). Allocates nothing."""
    _dev(x, torch.bfloat16, "x")
    if x.dim() not in (2, 3):
        raise ValueError(f"x: expected [M, K] or [B, M, K], got shape {tuple(x.shape)}")
    B, M, K = (x.shape if x.dim() == 3 else (1, *x.shape))
    _buf(q, torch.uint8, B * M * K // 2, "q")
    _buf(sf, torch.uint8, B * M * K // 16, "sf")
    _buf(gs, torch.float32, B, "gs")
    _buf(amax_in, torch.float32, B, "amax_in")
    _check(_quantize_noalloc(_ptr(x), B, M, K, _ptr(amax_in), _ptr(q), _ptr(sf), _ptr(gs), _stream()),
           "nvfp4_quantize_noalloc")


def nvfp4_quantize_static(x, gs, q=None, sf=None):
    """x: BF16 [M, K] or [B, M, K] quantized with the fixed global scales gs
    (float32 [B], device) -> (q uint8 [..., K/2], sf uint8 [..., K/16])."""
    _dev(x, torch.bfloat16, "x")
    if x.dim() not in (2, 3):
        raise ValueError(f"x: expected [M, K] or [B, M, K], got shape {tuple(x.shape)}")
    batched = x.dim() == 3
    B, M, K = (x.shape if batched else (1, *x.shape))
    _buf(gs, torch.float32, B, "gs")
    dev = x.device
    q = torch.empty((B, M, K // 2), dtype=torch.uint8, device=dev) if q is None else _buf(q, torch.uint8, B * M * K // 2, "q")
    sf = (torch.empty((B, M, K // 16), dtype=torch.uint8, device=dev) if sf is None
          else _buf(sf, torch.uint8, B * M * K // 16, "sf"))
    _check(_quantize_static(_ptr(x), B, M, K, _ptr(gs), _ptr(q), _ptr(sf), _stream()), "nvfp4_quantize_static")
    if not batched:
        return q[0], sf[0]
    return q, sf


# ------------------------------------------------------------------------- route

def moe_route_ws_bytes(T, k, num_local) -> int:
    return int(_route_ws(T, k, num_local))


def nvfp4_tile_table_len(cap, num_local, tile_m) -> int:
    return int(_tile_len(cap, num_local, tile_m))


def moe_route_slots(topk_ids, topk_w, expert_start, num_local, tile_m):
    _dev(topk_ids, torch.int32, "topk_ids")
    _dev(topk_w, torch.float32, "topk_w")
    T, k = topk_ids.shape
    _shape(topk_w, (T, k), "topk_w")
    dev = topk_ids.device
    cap = T * k
    i32 = dict(dtype=torch.int32, device=dev)
    out = dict(
        counts=torch.empty(num_local, **i32), offsets=torch.empty(num_local + 1, **i32),
        slot_token=torch.empty(cap, **i32), slot_expert=torch.empty(cap, **i32),
        slot_weight=torch.empty(cap, dtype=torch.float32, device=dev), token_slot=torch.empty(cap, **i32),
        tile_table=torch.empty(nvfp4_tile_table_len(cap, num_local, tile_m), **i32),
    )
    ws = _alloc_ws(moe_route_ws_bytes(T, k, num_local), dev)
    _check(_route(_ptr(topk_ids), _ptr(topk_w), T, k, expert_start, num_local, tile_m,
                  _ptr(out["counts"]), _ptr(out["offsets"]), _ptr(out["slot_token"]), _ptr(out["slot_expert"]),
                  _ptr(out["slot_weight"]), _ptr(out["token_slot"]), _ptr(out["tile_table"]),
                  _ptr(ws), ws.numel(), _stream()), "moe_route_slots")
    return out


# -------------------------------------------------------------------------- gate

def moe_gate_topk(logits, k, score=SCORE_SOFTMAX, bias=None, token_mask=None, n_group=1, topk_group=1,
                  renormalize=True, scale=1.0, topk_ids=None, topk_w=None):
    """Router logits BF16 or float32 [T, E] -> (topk_ids int32 [T, k], topk_w float32 [T, k]), as moe_route_slots
    and nvfp4_moe_forward take them. bias: float32 [E], added to the scores for the choice alone; token_mask: uint8
    [T], 0 for padding (ids -1, weights 0); n_group / topk_group: choose within the best groups of experts."""
    return _native.gate_topk(logits, k, score, bias, token_mask, n_group, topk_group, renormalize, scale, topk_ids, topk_w)


def moe_balance_loss_ws_bytes(T, E, B) -> int:
    return int(_balance_ws(T, E, B))


def moe_balance_loss(logits, topk_ids, score=SCORE_SOFTMAX, token_mask=None, cu_seqlens=None, loss=None, counts=None,
                     tokens=None, ws=None):
    """Balance loss and mean squared log-sum of the logits over the gate's choices -> (loss float32 [2], counts
    int32 [B, E], tokens int32 [B + 2]); counts and tokens are what moe_gate_backward takes. cu_seqlens: int32
    [B + 1] sequence bounds (None: all tokens are one sequence)."""
    return _native.balance_loss(logits, topk_ids, score, token_mask, cu_seqlens, loss, counts, tokens, ws)


def moe_gate_backward(logits, topk_ids, score=SCORE_SOFTMAX, renormalize=True, scale=1.0, token_mask=None,
                      d_topk_w=None, d_loss=None, counts=None, tokens=None, cu_seqlens=None, d_logits=None):
    """Gradient of the logits (their type and shape): through the weights when d_topk_w (float32 [T, k]) is given
    (score, renormalize and scale as in moe_gate_topk), of the losses when d_loss (float32 [2]) is given (counts
    and tokens from moe_balance_loss, the same cu_seqlens), or the sum of both."""
    return _native.gate_backward(logits, topk_ids, score, renormalize, scale, token_mask, d_topk_w, d_loss, counts, tokens,
                                 cu_seqlens, d_logits)


# ------------------------------------------------------------ norms of the block

def moe_block_norm(x, residual, w_pre=None, w_post=None, gate=None, scale=1.0, eps=1e-6, gs=None, residual_out=None,
                   y=None, y_q=None, y_sf=None):
    """The residual update behind a block and the norm in front of the next: n = rms_norm(x) * w_post (or x),
    residual_out = residual + scale * gate * n, y = rms_norm(residual_out) * w_pre -> (residual_out, y), y None
    without w_pre. x, residual: BF16 or float32 [T, H] (residual None: zeros, of x's type); w_pre, w_post: float32
    [H]; gate: float32 [H] or [T, 1]. With gs (float32 [1], device) also y as NVFP4 with that fixed global scale:
    (residual_out, y, y_q, y_sf)."""
    return _native.block_norm(x, residual, w_pre, w_post, gate, scale, eps, gs, residual_out, y, y_q, y_sf)


def moe_block_norm_backward_ws_bytes(T, H) -> int:
    return int(_block_norm_ws(T, H))


_NORM_GRADIENTS = ("d_x", "d_residual", "d_w_pre", "d_w_post", "d_gate")


def moe_block_norm_backward(d_y, d_residual_out, x, residual_out, w_pre=None, w_post=None, gate=None, scale=1.0,
                            eps=1e-6, d_x=None, d_residual=None, d_w_pre=None, d_w_post=None, d_gate=None, ws=None):
    """Gradients of moe_block_norm from d_y (None without w_pre) and d_residual_out (None: zeros), with the x and the
    residual_out of the forward call -> dict of d_x, d_residual, d_w_pre, d_w_post, d_gate (None where there is no
    such input)."""
    return dict(zip(_NORM_GRADIENTS, _native.block_norm_backward(
        d_y, d_residual_out, x, residual_out, w_pre, w_post, gate, scale, eps, d_x, d_residual, d_w_pre, d_w_post, d_gate,
        ws)))


def moe_layer_norm(x, residual=None, w=None, b=None, scale=1.0, eps=1e-5, mx_rule=None, residual_out=None, y=None,
                   y_q=None, y_scale=None):
    """Layer norm behind the residual update: residual_out = residual + scale * x, y = (residual_out - mean) *
    rsqrt(var + eps) * w + b -> (residual_out, y). x: BF16 or float32 [T, H], residual of either type (None: x itself
    is normalized and comes back in its place); w, b: float32 [H] or None. With mx_rule (MX_SCALE_FLOOR or
    MX_SCALE_CEIL) also y as MXFP4: (residual_out, y, y_q, y_scale), for mxfp4_gemm."""
    return _native.layer_norm(x, residual, w, b, scale, eps, mx_rule, residual_out, y, y_q, y_scale)


def moe_layer_norm_backward_ws_bytes(T, H) -> int:
    return int(_layer_norm_ws(T, H))


_LAYER_NORM_GRADIENTS = ("d_x", "d_residual", "d_w", "d_b")


def moe_layer_norm_backward(d_y, d_residual_out, residual_out, w=None, b=None, scale=1.0, eps=1e-5, residual=True,
                            d_x=None, d_residual=None, d_w=None, d_b=None, ws=None):
    """Gradients of moe_layer_norm from d_y and d_residual_out (None: zeros), with the residual_out of the forward call
    -> dict of d_x, d_residual, d_w, d_b (None where there is no such input). residual False: the forward call had no
    residual, and residual_out is the x it normalized."""
    return dict(zip(_LAYER_NORM_GRADIENTS, _native.layer_norm_backward(
        d_y, d_residual_out, residual_out, w, b, scale, eps, residual, d_x, d_residual, d_w, d_b, ws)))


# ------------------------------------------------------------------ grouped GEMM

def nvfp4_packed_bytes(B, N, K) -> int:
    return int(_packed_bytes(B, N, K))


def nvfp4_pack_weights(q, sf, out=None):
    """Row-major NVFP4 matrices q uint8 [B, N, K/2], sf uint8 [B, N, K/16] ->
    packed uint8 [B, N/32, K/128, 2304] in the grouped GEMM's operand order."""
    _dev(q, torch.uint8, "q")
    _dev(sf, torch.uint8, "sf")
    B, N, Kh = q.shape
    K = Kh * 2
    if tuple(sf.shape) != (B, N, K // 16):
        raise ValueError(f"sf shape {tuple(sf.shape)} does not match q {tuple(q.shape)}")
    if N % 32 or K % 128:
        raise ValueError(f"packing needs N % 32 == 0 and K % 128 == 0, got N={N}, K={K}")
    out = (torch.empty((B, N // 32, K // 128, 2304), dtype=torch.uint8, device=q.device) if out is None
           else _buf(out, torch.uint8, B * N * K // 32 * 18, "out"))
    _check(_pack(_ptr(q), _ptr(sf), B, N, K, _ptr(out), _stream()), "nvfp4_pack_weights")
    return out


def _check_gemm_operands(a_q, a_sf, a_row_index, a_gs, b_gs, offsets, tile_table, rows_cap, tile_m, L, K, n_b_gs):
    _dev(a_q, torch.uint8, "a_q")
    _dev(a_sf, torch.uint8, "a_sf")
    if a_q.dim() != 2 or a_q.shape[1] != K // 2 or tuple(a_sf.shape) != (a_q.shape[0], K // 16):
        raise ValueError(f"a_q {tuple(a_q.shape)} / a_sf {tuple(a_sf.shape)}: expected [rows, {K // 2}] / "
                         f"[rows, {K // 16}]")
    # rows read: slot s, or a_row_index[s], for the slots below offsets[L] (device data, at most rows_cap); with
    # a row index the indices' range is the caller's contract, without one every slot row must exist
    if a_row_index is None and a_q.shape[0] < rows_cap:
        raise ValueError(f"a_q: {a_q.shape[0]} rows, but slots up to rows_cap = {rows_cap} read their own row")
    _buf(a_row_index, torch.int32, 0, "a_row_index")
    _buf(a_gs, torch.float32, 1, "a_gs")
    _buf(b_gs, torch.float32, n_b_gs, "b_gs")
    _buf(offsets, torch.int32, L + 1, "offsets")
    _buf(tile_table, torch.int32, nvfp4_tile_table_len(rows_cap, L, tile_m), "tile_table")


def _packed_dims(b_packed, name="b_packed"):
    """(L, N, K) of packed weights uint8 [L, N/32, K/128, 2304]."""
    _dev(b_packed, torch.uint8, name)
    if b_packed.dim() != 4 or b_packed.shape[3] != 2304:
        raise ValueError(f"{name}: expected packed weights [L, N/32, K/128, 2304], got {tuple(b_packed.shape)}")
    L, n32, k128, _ = b_packed.shape
    return L, n32 * 32, k128 * 128


def nvfp4_grouped_gemm(a_q, a_sf, a_row_index, a_gs, b_packed, b_gs, offsets, tile_table, rows_cap,
                       tile_m, epilogue=EPI_BF16, d=None, amax_out=None):
    """b_packed: uint8 [L, N/32, K/128, 2304] from nvfp4_pack_weights. A rows:
    a_row_index[s] for slot s when given (device indices < a_q's row count,
    the caller's contract), else s (a_q then needs rows_cap rows)."""
    L, N, K = _packed_dims(b_packed)
    dev = b_packed.device
    n_out = N // 2 if epilogue in (EPI_SILU_MUL, EPI_SILU_MUL_DUAL) else N
    _check_gemm_operands(a_q, a_sf, a_row_index, a_gs, b_gs, offsets, tile_table, rows_cap, tile_m, L, K,
                         2 * L if epilogue == EPI_SILU_MUL_DUAL else L)
    d = (torch.empty((rows_cap, n_out), dtype=torch.bfloat16, device=dev) if d is None
         else _buf(d, torch.bfloat16, rows_cap * n_out, "d"))
    _buf(amax_out, torch.float32, 1, "amax_out")
    _check(_gemm(_ptr(a_q), _ptr(a_sf), _ptr(a_row_index), _ptr(a_gs), _ptr(b_packed), _ptr(b_gs),
                 _ptr(offsets), _ptr(tile_table), L, rows_cap, N, K, tile_m, epilogue, _ptr(d), _ptr(amax_out),
                 _stream()), "nvfp4_grouped_gemm")
    return d


def nvfp4_grouped_gemm_silu_nvfp4(a_q, a_sf, a_row_index, a_gs, b_packed, b_gs, offsets, tile_table, rows_cap,
                                  tile_m, out_gs, d_q=None, d_sf=None):
    """L1 with the SiLU*up epilogue writing h as NVFP4 with the fixed global
    scale out_gs [1]: returns (h_q uint8 [rows_cap, N/4], h_sf uint8 [rows_cap, N/32]).
    b_gs [L] (folded W1) or [L, 2] (gate and up global scales)."""
    L, N, K = _packed_dims(b_packed)
    dev = b_packed.device
    dual = 1 if b_gs.dim() == 2 else 0
    _check_gemm_operands(a_q, a_sf, a_row_index, a_gs, b_gs, offsets, tile_table, rows_cap, tile_m, L, K,
                         2 * L if dual else L)
    _buf(out_gs, torch.float32, 1, "out_gs")
    d_q = (torch.empty((rows_cap, N // 4), dtype=torch.uint8, device=dev) if d_q is None
           else _buf(d_q, torch.uint8, rows_cap * (N // 4), "d_q"))
    d_sf = (torch.empty((rows_cap, N // 32), dtype=torch.uint8, device=dev) if d_sf is None
            else _buf(d_sf, torch.uint8, rows_cap * (N // 32), "d_sf"))
    _check(_gemm_nvfp4(_ptr(a_q), _ptr(a_sf), _ptr(a_row_index), _ptr(a_gs), _ptr(b_packed), _ptr(b_gs), dual,
                       _ptr(offsets), _ptr(tile_table), L, rows_cap, N, K, tile_m, _ptr(out_gs), _ptr(d_q),
                       _ptr(d_sf), _stream()), "nvfp4_grouped_gemm_silu_nvfp4")
    return d_q, d_sf


def moe_weighted_scatter(y, token_slot, topk_w, out=None):
    """out[t] = sum over j of topk_w[t, j] * y[token_slot[t*k + j]] (slots >= 0),
    y BF16 [rows, H] with every slot index < rows (the caller's contract)."""
    _dev(y, torch.bfloat16, "y")
    _dev(topk_w, torch.float32, "topk_w")
    T, k = topk_w.shape
    H = y.shape[1]
    _buf(token_slot, torch.int32, T * k, "token_slot")
    out = (torch.empty((T, H), dtype=torch.bfloat16, device=y.device) if out is None
           else _buf(out, torch.bfloat16, T * H, "out"))
    _check(_scatter(_ptr(y), _ptr(token_slot), _ptr(topk_w), T, k, H, _ptr(out), _stream()),
           "moe_weighted_scatter")
    return out


def nvfp4_fold_scales(w1_sf, gs_gate, gs_up, gs1=None):
    """In place on w1_sf [L, 2I, K/16]; returns gs1 [L]."""
    _dev(w1_sf, torch.uint8, "w1_sf")
    L, two_i, k16 = w1_sf.shape
    _buf(gs_gate, torch.float32, L, "gs_gate")
    _buf(gs_up, torch.float32, L, "gs_up")
    gs1 = torch.empty(L, dtype=torch.float32, device=w1_sf.device) if gs1 is None else _buf(gs1, torch.float32, L, "gs1")
    _check(_fold(_ptr(w1_sf), _ptr(gs_gate), _ptr(gs_up), _ptr(gs1), L, two_i // 2, k16 * 16, _stream()),
           "nvfp4_fold_scales")
    return gs1


# -------------------------------------------------------- 8-bit integer products

def int8_quantize_rows(x, q=None, scale=None):
    """x BF16 or float32 [M, K] -> (q int8 [M, K], scale float32 [M] = row amax * (1 / 127))."""
    return _native.quantize_rows(x, q, scale)


def int8_gemm_ws_bytes(M, N, K) -> int:
    return int(_int8_gemm_ws(M, N, K))


def int8_gemm(a_q, a_scale, b_q, b_scale, epilogue=EPI_BF16, add=None, d=None, ws=None):
    """a_q int8 [M, K], a_scale float32 [M], b_q int8 [N, K], b_scale float32 [N] -> BF16 [M, N] (EPI_BF16), or
    [M, N / 2] of silu(gate) * up with the gate rows of b_q first (EPI_SILU_MUL); add: BF16 of that shape."""
    return _native.gemm(a_q, a_scale, b_q, b_scale, epilogue, add, d, ws)


def _matrix(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name}: expected 2 dimensions, got shape {tuple(t.shape)}")
    return t.shape


class Int8FFNWeights:
    """Device weights of a dense expert: w1_q int8 [2I, H] (gate rows, then up rows) with w1_scale float32 [2I], and
    w2_q int8 [H, I] with w2_scale float32 [H]."""

    def __init__(self, w1_q, w1_scale, w2_q, w2_scale):
        _dev(w1_q, torch.int8, "w1_q")
        _dev(w2_q, torch.int8, "w2_q")
        two_i, self.hidden = _matrix(w1_q, "w1_q")
        self.inter = two_i // 2
        _shape(w2_q, (self.hidden, self.inter), "w2_q")
        if two_i % 2:
            raise ValueError(f"w1_q: an even number of rows (gate and up), got {two_i}")
        for scale, rows, name in ((w1_scale, two_i, "w1_scale"), (w2_scale, self.hidden, "w2_scale")):
            _shape(_dev(scale, torch.float32, name), (rows,), name)
        self.w1_q, self.w1_scale, self.w2_q, self.w2_scale = w1_q, w1_scale, w2_q, w2_scale


def prepare_int8_weights(w_gate, w_up, w_down) -> Int8FFNWeights:
    """Offline: BF16 or float32 w_gate, w_up [I, H] and w_down [H, I], quantized per output channel."""
    w1_q, w1_scale = int8_quantize_rows(torch.cat([w_gate, w_up], dim=0).contiguous())
    w2_q, w2_scale = int8_quantize_rows(w_down.contiguous())
    return Int8FFNWeights(w1_q, w1_scale, w2_q, w2_scale)


def int8_ffn_ws_bytes(T, hidden, inter) -> int:
    return int(_int8_ffn_ws(T, hidden, inter))


def int8_ffn_forward(weights: Int8FFNWeights, x, add=None, out=None, ws=None):
    """Dense expert FFN of x BF16 [T, H] in 8-bit integers -> BF16 [T, H], plus add (BF16 [T, H], such as the routed
    experts' output; may be out) when given."""
    w = weights
    return _native.ffn(w.w1_q, w.w1_scale, w.w2_q, w.w2_scale, x, add, out, ws)


# ------------------------------------------- microscaled 4-bit floats (MXFP4)

def mxfp4_padded(n) -> int:
    """Columns that a matrix of n columns is padded to: whole groups of 128."""
    p = int(_mx_padded(n))
    if p < 0:
        raise ValueError(f"n: expected 0 to 262144, got {n}")
    return p


def mxfp4_quantize(x, direction=MX_ROWS, rule=MX_SCALE_FLOOR, q=None, scale=None, q_t=None, scale_t=None):
    """x BF16 or float32 [M, K] -> MXFP4 along its rows (MX_ROWS: q uint8 [M, Kp/2], scale uint8 [Kp/128, M, 4]), along
    its columns (MX_COLUMNS: q_t [K, Mp/2], scale_t [Mp/128, K, 4], the transposed matrix) or both (MX_BOTH: all
    four), Kp = mxfp4_padded(K). rule: MX_SCALE_FLOOR (the largest values of a block may saturate) or MX_SCALE_CEIL
    (none does). Scales in rows, [M, Kp/32], are scale.permute(1, 0, 2).reshape(M, -1)."""
    return _native.mx_quantize(x, direction, rule, q, scale, q_t, scale_t)


def _mx_type(dtype):
    if dtype is torch.bfloat16:
        return 0
    if dtype is torch.float32:
        return 1
    raise ValueError(f"dtype: expected torch.bfloat16 or torch.float32, got {dtype}")


def mxfp4_dequantize(q, scale, dtype=torch.bfloat16, cols=None, out=None):
    """The values of MXFP4 codes, [R, cols] (None: all the padded columns), BF16 (exact) or float32."""
    return _native.mx_dequantize(q, scale, _mx_type(dtype), cols, out)


def mxfp4_gemm_ws_bytes(M, N, K) -> int:
    return int(_mx_gemm_ws(M, N, K))


def mxfp4_gemm(a_q, a_scale, b_q, b_scale, epilogue=EPI_BF16, add=None, dtype=torch.bfloat16, d=None, ws=None):
    """The product A B^T of MXFP4 matrices [M, K] and [N, K], as mxfp4_quantize makes them -> [M, N] (EPI_BF16) of
    dtype, or BF16 [M, N / 2] of silu(gate) * up with the gate rows of b_q first (EPI_SILU_MUL); add: of that type
    and shape (such as a residual, or a weight's gradient so far), may be d."""
    return _native.mx_gemm(a_q, a_scale, b_q, b_scale, epilogue, add, _mx_type(dtype), d, ws)


# --------------------------------------------------------------------- the layer

def nvfp4_moe_ws_layout(T, k, hidden, inter, num_local) -> dict:
    offs = (_sz * len(WS_REGIONS))()
    tile_m = nvfp4_moe_tile_m(T, k, num_local)
    _moe_ws_layout(T, k, hidden, inter, num_local, tile_m, offs)
    return {name: int(offs[i]) for i, name in enumerate(WS_REGIONS)}


def nvfp4_moe_ws_bytes(T, k, hidden, inter, num_local) -> int:
    return int(_moe_ws(T, k, hidden, inter, num_local))


def nvfp4_moe_tile_m(T, k, num_local) -> int:
    return int(_moe_tile_m(T, k, num_local))


def ws_view(ws, layout, region, dtype, shape):
    """A typed view of one workspace region (for reading intermediates)."""
    off = layout[region]
    n = 1
    for s in shape:
        n *= s
    nbytes = n * torch.empty((), dtype=dtype).element_size()
    return ws[off:off + nbytes].view(dtype).view(*shape)


class MoEWeights:
    """Device NVFP4 layer weights for one rank (L local experts): packed W1
    (gate rows then up rows) and packed W2. W1's gate/up scales are either
    folded to one global scale per expert (w1_gs [L]) or kept per half
    (w1_gs [L, 2] = gs_gate, gs_up). With keep_unpacked, prepare_weights also
    keeps the row-major forms (w1_q, w1_sf, w2_q, w2_sf) for inspection."""

    def __init__(self, w1, w1_gs, w2, w2_gs):
        self.w1, self.w1_gs, self.w2, self.w2_gs = w1, w1_gs, w2, w2_gs
        self.dual_gs = w1_gs.dim() == 2
        self.num_local, two_i, self.hidden = _packed_dims(w1, "w1")
        self.inter = two_i // 2
        if _packed_dims(w2, "w2") != (self.num_local, self.hidden, self.inter):
            raise ValueError(f"packed W2 shape {tuple(w2.shape)} does not match W1 {tuple(w1.shape)}")
        _dev(w1_gs, torch.float32, "w1_gs")
        _dev(w2_gs, torch.float32, "w2_gs")
        if tuple(w1_gs.shape) not in ((self.num_local,), (self.num_local, 2)):
            raise ValueError(f"w1_gs shape {tuple(w1_gs.shape)}: expected [L] or [L, 2]")
        if tuple(w2_gs.shape) != (self.num_local,):
            raise ValueError(f"w2_gs shape {tuple(w2_gs.shape)}: expected [L] = [{self.num_local}]")
        self._c = _Weights(self.num_local, self.hidden, self.inter, w1.data_ptr(), w1_gs.data_ptr(),
                           w2.data_ptr(), w2_gs.data_ptr(), 1 if self.dual_gs else 0)


def prepare_weights(w_gate, w_up, w_down, keep_unpacked=False, fold=True) -> MoEWeights:
    """Offline weight preparation on the GPU: quantize each (expert, projection)
    with its own global scale, fold the gate/up scale ratio (or, with
    fold=False, keep both halves' scales and global scales), and pack both
    matrices for the grouped GEMM.

    w_gate, w_up: BF16 [L, I, H]; w_down: BF16 [L, H, I].
    """
    L, I, H = w_gate.shape
    gate_up = torch.cat([w_gate, w_up], dim=1).contiguous()          # [L, 2I, H]: tensor b = 2e + p
    q1, sf1, gs_pair = nvfp4_quantize(gate_up.view(2 * L, I, H))
    del gate_up
    w1_q = q1.view(L, 2 * I, H // 2)
    w1_sf = sf1.view(L, 2 * I, H // 16)
    gs_pair = gs_pair.view(L, 2)
    gs_gate, gs_up = gs_pair[:, 0].contiguous(), gs_pair[:, 1].contiguous()
    w1_gs = nvfp4_fold_scales(w1_sf, gs_gate, gs_up) if fold else gs_pair.contiguous()
    w2_q, w2_sf, w2_gs = nvfp4_quantize(w_down.contiguous())
    w = MoEWeights(nvfp4_pack_weights(w1_q, w1_sf), w1_gs, nvfp4_pack_weights(w2_q, w2_sf), w2_gs)
    w.gs_gate, w.gs_up = gs_gate, gs_up
    if keep_unpacked:
        w.w1_q, w.w1_sf, w.w2_q, w.w2_sf = w1_q, w1_sf, w2_q, w2_sf
    return w


def _check_layer_inputs(weights, x, topk_w, T, k):
    _shape(x, (T, weights.hidden), "x")
    _shape(topk_w, (T, k), "topk_w")
    for name in ("w1", "w1_gs", "w2", "w2_gs"):
        _dev(getattr(weights, name), getattr(weights, name).dtype, f"weights.{name}")


def _layer_buffers(weights, x, topk_ids, topk_w, out, ws):
    _dev(x, torch.bfloat16, "x")
    _dev(topk_ids, torch.int32, "topk_ids")
    _dev(topk_w, torch.float32, "topk_w")
    T, k = topk_ids.shape
    H = weights.hidden
    _check_layer_inputs(weights, x, topk_w, T, k)
    dev = x.device
    out = torch.empty((T, H), dtype=torch.bfloat16, device=dev) if out is None else _buf(out, torch.bfloat16, T * H, "out")
    need = nvfp4_moe_ws_bytes(T, k, H, weights.inter, weights.num_local)
    ws = _alloc_ws(need, dev) if ws is None else _buf(ws, torch.uint8, 0, "ws")
    return T, k, out, ws


def nvfp4_moe_forward(weights: MoEWeights, x, topk_ids, topk_w, expert_start, out=None, ws=None):
    """One rank's partial output BF16 [T, H] of the expert FFN."""
    T, k, out, ws = _layer_buffers(weights, x, topk_ids, topk_w, out, ws)
    _check(_forward(ctypes.byref(weights._c), _ptr(x), T, _ptr(topk_ids), _ptr(topk_w), k, expert_start,
                    _ptr(out), _ptr(ws), ws.numel(), _stream()), "nvfp4_moe_forward")
    return out


# stages between the events of nvfp4_moe_forward_stage_events (NVFP4_STAGE_* order)
STAGES = ["a1_amax_route", "a2_quantize_x", "a3_route", "a4_a5_l1_gemm", "a6_quantize_h", "a7_l2_gemm",
          "a8_scatter"]


def nvfp4_moe_forward_stage_events(weights: MoEWeights, x, topk_ids, topk_w, expert_start, events, out=None,
                                   ws=None):
    """nvfp4_moe_forward with events recorded between its launches: events is
    a list of len(STAGES) + 1 torch.cuda.Event (timing enabled, each recorded
    once beforehand so that it exists) or None (no record there); events[i]
    to events[i + 1] spans stage STAGES[i] of this call."""
    if len(events) != len(STAGES) + 1:
        raise ValueError(f"events: expected {len(STAGES) + 1} entries, got {len(events)}")
    handles = (_vp * len(events))()
    for i, e in enumerate(events):
        if e is not None:
            if not e.cuda_event:
                raise ValueError(f"events[{i}]: not created yet (record it once first)")
            handles[i] = e.cuda_event
    T, k, out, ws = _layer_buffers(weights, x, topk_ids, topk_w, out, ws)
    _check(_forward_stages(ctypes.byref(weights._c), _ptr(x), T, _ptr(topk_ids), _ptr(topk_w), k, expert_start,
                           _ptr(out), _ptr(ws), ws.numel(), handles, _stream()), "nvfp4_moe_forward_stage_events")
    return out


def nvfp4_moe_forward_static(weights: MoEWeights, x, topk_ids, topk_w, expert_start, gs, out=None, ws=None):
    """The layer with fixed global scales gs = float32 [2] (gs_x, gs_h) on the
    device, e.g. from calibrate_static_gs; no amax passes, h quantized in L1."""
    _dev(gs, torch.float32, "gs")
    if gs.numel() != 2:
        raise ValueError(f"gs: expected 2 values (gs_x, gs_h), got {gs.numel()}")
    T, k, out, ws = _layer_buffers(weights, x, topk_ids, topk_w, out, ws)
    _check(_forward_static(ctypes.byref(weights._c), _ptr(x), T, _ptr(topk_ids), _ptr(topk_w), k, expert_start,
                           _ptr(gs), _ptr(out), _ptr(ws), ws.numel(), _stream()), "nvfp4_moe_forward_static")
    return out


def calibrate_static_gs(weights: MoEWeights, x, topk_ids, topk_w, expert_start):
    """Global scales (gs_x, gs_h) that nvfp4_moe_forward measures on a
    calibration batch, as a device float32 [2] for nvfp4_moe_forward_static."""
    T, k = topk_ids.shape
    ws = _alloc_ws(nvfp4_moe_ws_bytes(T, k, weights.hidden, weights.inter, weights.num_local), x.device)
    nvfp4_moe_forward(weights, x, topk_ids, topk_w, expert_start, ws=ws)
    lay = nvfp4_moe_ws_layout(T, k, weights.hidden, weights.inter, weights.num_local)
    sc = ws_view(ws, lay, "scalars", torch.float32, (4,))
    return torch.stack([sc[0], sc[2]]).contiguous()


def nvfp4_moe_few_max_tokens() -> int:
    return int(_few_max())


def nvfp4_moe_few_ws_bytes(T, k, hidden, inter, num_local) -> int:
    return int(_few_ws(T, k, hidden, inter, num_local))


def nvfp4_moe_forward_few(weights: MoEWeights, x, topk_ids, topk_w, expert_start, add=None, out=None, ws=None):
    """One rank's partial output BF16 [T, H] of the expert FFN for at most 64 tokens, in two launches (three for narrow
    layers) on the same weights, with BF16 activations (nvfp4_moe_forward quantizes them), plus add (BF16 [T, H], such
    as the dense expert's output; may be out) when given."""
    w = weights
    return _native.moe_few(w.w1, w.w1_gs, w.w2, w.w2_gs, x, topk_ids, topk_w, expert_start, add, out, ws)
