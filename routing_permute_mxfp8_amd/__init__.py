"""Python binding of the MI355X MoE-layer hot path (libmoe_mx.so, C ABI in include/moe_mx.h).

Argument marshalling only: outputs and workspaces are allocated with torch on the
tensors' device, pointers and the current HIP stream are passed to the library,
and every step of the computation runs in the library's HIP kernels. If the
library has not been built (python -m routing_permute_mxfp8_amd.build, or
__graft_entry__.build()) the calls raise; there is no fallback path.

Byte conventions: FP8 codes and E8M0 scales are returned as torch.uint8 tensors
(view them as torch.float8_e4m3fn / float8_e5m2 / float8_e8m0fnu if wanted);
inputs may be uint8 or the matching float8 dtype.
"""

from __future__ import annotations

import ctypes
import functools
import os

import torch

from .build import lib_path

__all__ = [
    "MoeError", "load", "QUANT_NONE", "QUANT_E5M2", "QUANT_E4M3", "QUANT_MXFP4", "FP8_E5M2", "FP8_E4M3",
    "mx_scale_cols", "token_permute_out_rows", "mx_quantize", "init_routing", "init_routing_noalloc", "token_permute",
    "mega_moe", "mega_moe_workspace_bytes", "gmm1_swiglu_quant", "gmm2_combine", "combine_finalize",
    "pack_weights", "WEIGHTS_ND", "WEIGHTS_PACKED", "DTYPE_FP8_E5M2", "DTYPE_FP8_E4M3", "DTYPE_FP4_E2M1",
    "gate_topk", "balance_loss", "gate_backward", "GATE_SOFTMAX", "GATE_SIGMOID",
    "mxfp4_matmul",
]

QUANT_NONE, QUANT_E5M2, QUANT_E4M3, QUANT_MXFP4 = -1, 2, 3, 9
FP8_E5M2, FP8_E4M3 = 23, 24
WEIGHTS_ND, WEIGHTS_PACKED = 0, 1
GATE_SOFTMAX, GATE_SIGMOID = 0, 1   # scores of the router's logits
_DT = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2, torch.int32: 3, torch.int64: 4}
# x dtypes of MX codes for init_routing's pass-through (one FP8 code a byte, two FP4 codes a byte)
DTYPE_FP8_E5M2, DTYPE_FP8_E4M3, DTYPE_FP4_E2M1 = 5, 6, 7
_STATUS = {0: "OK", 1: "INVALID_ARG", 2: "SHAPE", 3: "DTYPE", 4: "UNSUPPORTED", 5: "WORKSPACE", 6: "HIP"}


class MoeError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{_STATUS.get(status, status)}: {message}")
        self.status = status


class MegaArgs(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p), ("num_tokens", ctypes.c_int64), ("hidden", ctypes.c_int64),
        ("topk_ids", ctypes.c_void_p), ("topk", ctypes.c_int64),
        ("topk_weights", ctypes.c_void_p), ("topk_weights_dtype", ctypes.c_int),
        ("num_experts", ctypes.c_int64), ("inter", ctypes.c_int64),
        ("w1", ctypes.c_void_p), ("w1_scales", ctypes.c_void_p),
        ("w2", ctypes.c_void_p), ("w2_scales", ctypes.c_void_p),
        ("num_shared", ctypes.c_int64),
        ("shared_w1", ctypes.c_void_p), ("shared_w1_scales", ctypes.c_void_p),
        ("shared_w2", ctypes.c_void_p), ("shared_w2_scales", ctypes.c_void_p),
        ("quant_out_dtype", ctypes.c_int), ("activation", ctypes.c_int), ("weight_format", ctypes.c_int),
        ("y", ctypes.c_void_p), ("expert_token_nums", ctypes.c_void_p),
        ("xq", ctypes.c_void_p), ("sx", ctypes.c_void_p), ("h1", ctypes.c_void_p),
        ("aq", ctypes.c_void_p), ("sa", ctypes.c_void_p), ("o", ctypes.c_void_p),
        ("sorted_row_idx", ctypes.c_void_p),
        ("stage_events", ctypes.POINTER(ctypes.c_void_p)),
        ("num_activation_params", ctypes.c_int), ("activation_params", ctypes.c_float * 3),
        ("weight_dtype", ctypes.c_int), ("shared_weight_dtype", ctypes.c_int),
        ("x_is_quantized", ctypes.c_int), ("x_scales", ctypes.c_void_p),
        ("combine_comm_mode", ctypes.c_int),
    ]

MEGA_STAGE_EVENTS = 7
# activation kinds of mega_moe (MegaMoE "Activation function formulas")
ACT_SWIGLU, ACT_SWIGLUSTEP, ACT_SWIGLUOAI, ACT_SITUGLU, ACT_GELU = 0, 1, 2, 3, 4
FP4_E2M1 = 296   # MXFP4 weights (A8W4-FP)
MEGA_STAGES = ["routing", "permute_quant", "gmm1_swiglu_quant", "gmm2", "shared_experts", "combine"]


_lib = None

_I64, _INT, _VP, _SZ = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
_SIGS = {
    "moe_last_error": ([], ctypes.c_char_p),
    "moe_version": ([], _INT),
    "moe_mx_scale_cols": ([_I64], _I64),
    "moe_token_permute_out_rows": ([_I64, _I64], _I64),
    "moe_mx_quantize": ([_VP, _INT, _I64, _I64, _INT, _VP, _VP, _VP], _INT),
    "moe_mx_packed_scale_bytes": ([_I64, _I64, _I64], _I64),
    "moe_mx_pack_weights": ([_VP, _VP, _I64, _I64, _I64, _VP, _VP, _VP], _INT),
    "moe_mx_pack_weights_fp4": ([_VP, _VP, _I64, _I64, _I64, _VP, _VP, _VP], _INT),
    "moe_init_routing_workspace_size": ([_I64, _I64, _I64, ctypes.POINTER(_SZ)], _INT),
    "moe_init_routing": ([_VP, _INT, _VP, _I64, _I64, _VP, _I64, _I64, _I64, _I64, _INT, _INT, _INT,
                          _VP, _VP, _VP, _VP, _VP, _VP, _SZ, _VP], _INT),
    "moe_init_routing_noalloc": ([_VP, _INT, _VP, _I64, _I64, _VP, _I64, _I64, _I64, _I64, _INT, _INT, _INT,
                                  _VP, _VP, _VP, _VP, _VP, _VP], _INT),
    "moe_token_permute_workspace_size": ([_I64, _I64, ctypes.POINTER(_SZ)], _INT),
    "moe_token_permute": ([_VP, _INT, _I64, _I64, _VP, _INT, _I64, _I64, _I64, _INT, _INT,
                           _VP, _VP, _VP, _VP, _SZ, _VP], _INT),
    "mega_moe_workspace_size": ([ctypes.POINTER(MegaArgs), ctypes.POINTER(_SZ)], _INT),
    "mega_moe": ([ctypes.POINTER(MegaArgs), _VP, _SZ, _VP], _INT),
    "moe_gmm_workspace_size": ([_I64, _I64, _I64, _I64, ctypes.POINTER(_SZ)], _INT),
    "moe_gmm1_swiglu_quant": ([_VP, _VP, _I64, _I64, _I64, _VP, _I64, _VP, _VP, _INT, _INT, _VP, _VP, _VP,
                               _VP, _SZ, _VP], _INT),
    "moe_gmm2_combine": ([_VP, _VP, _I64, _I64, _I64, _VP, _I64, _VP, _VP, _INT, _INT, _VP, _VP, _I64, _VP,
                          _VP, _VP, _SZ, _VP], _INT),
    "moe_combine_finalize": ([_VP, _I64, _I64, _VP, _VP], _INT),
    "moe_gate_topk": ([_VP, _INT, _I64, _I64, _I64, _INT, _VP, _I64, _I64, _INT, ctypes.c_float, _VP, _VP, _VP], _INT),
    "moe_balance_loss_workspace_size": ([_I64, _I64, _I64, ctypes.POINTER(_SZ)], _INT),
    "moe_balance_loss": ([_VP, _INT, _I64, _I64, _VP, _I64, _INT, _VP, _I64, _VP, ctypes.c_float, _VP, _VP, _VP,
                          _VP, _SZ, _VP], _INT),
    "moe_gate_backward": ([_VP, _INT, _I64, _I64, _VP, _I64, _INT, _INT, ctypes.c_float, _VP, _VP, _VP, _VP, _I64,
                           _VP, _VP, _VP], _INT),
    "moe_mxfp4_matmul_workspace_size": ([_I64, _I64, _I64, _I64, _INT, _INT, ctypes.POINTER(_SZ)], _INT),
    "moe_mxfp4_matmul": ([_VP, _INT, _VP, _I64, _VP, _I64, _VP, _VP, _I64, _I64, _INT, _VP, _INT, _VP, _SZ, _VP], _INT),
    "moe_probe_stream": ([_INT, _VP, _VP, _I64, _VP], _INT),
    "moe_probe_mfma": ([_INT, _VP, ctypes.POINTER(_I64), ctypes.POINTER(ctypes.c_double), _VP], _INT),
}


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libmoe_mx.so (built in-tree); raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or lib_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built: run routing_permute_mxfp8_amd/build.py "
                           "(the HIP library is required; there is no fallback)")
    lib = ctypes.CDLL(path)
    for name, (args, res) in _SIGS.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def _check(status: int):
    if status != 0:
        raise MoeError(status, _lib.moe_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _u8(t):
    if t is None:
        return None
    return t if t.dtype == torch.uint8 else t.view(torch.uint8)


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _workspace(nbytes: int, device):
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def _need_gpu(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("tensors must be on the GPU")
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors must be contiguous")


def mx_scale_cols(cols: int) -> int:
    return int(load().moe_mx_scale_cols(cols))


def token_permute_out_rows(flat: int, num_out_tokens) -> int:
    return int(load().moe_token_permute_out_rows(flat, 0 if num_out_tokens is None else int(num_out_tokens)))


def mx_quantize(x: torch.Tensor, quant_mode: int = QUANT_E4M3):
    """MX-quantize the rows of a 2-D bf16/fp16/fp32 tensor: (codes uint8 [R, C] ([R, C/2] packed
    for QUANT_MXFP4), scales uint8 [R, AlignUp(C/32, 2)])."""
    lib = load()
    _need_gpu(x)
    rows, cols = x.shape
    codes = torch.empty((rows, cols // 2 if quant_mode == QUANT_MXFP4 else cols), dtype=torch.uint8, device=x.device)
    scales = torch.empty((rows, mx_scale_cols(cols)), dtype=torch.uint8, device=x.device)
    _check(lib.moe_mx_quantize(_ptr(x), _DT[x.dtype], rows, cols, quant_mode, _ptr(codes), _ptr(scales),
                               _stream(x.device)))
    return codes, scales


def pack_weights(codes, scales, fp4: bool = False):
    """MX weights [G, N, K] codes + [G, N, K/32] scales (the pages' layout) -> the library's
    MFMA-native packed layout: (codes uint8 [G, N, K] in packed order, scales uint8 1-D).
    fp4: MXFP4 codes [G, N, K/2] (two a byte; K = 2 * the last dimension)."""
    lib = load()
    codes, scales = _u8(codes), _u8(scales)
    _need_gpu(codes, scales)
    g, n, kb = codes.shape
    k = 2 * kb if fp4 else kb
    pc = torch.empty_like(codes)
    ps = torch.empty((int(lib.moe_mx_packed_scale_bytes(g, n, k)),), dtype=torch.uint8, device=codes.device)
    fn = lib.moe_mx_pack_weights_fp4 if fp4 else lib.moe_mx_pack_weights
    _check(fn(_ptr(codes), _ptr(scales), g, n, k, _ptr(pc), _ptr(ps), _stream(codes.device)))
    return pc, ps


def init_routing_noalloc(x, expert_idx, expert_num: int, active_range=None, quant_mode: int = QUANT_NONE,
                         row_idx_type: int = 1, expert_tokens_num_type: int = 1):
    """init_routing through moe_init_routing_noalloc: the library takes no workspace (its
    scratch is a static per-GPU array of 8 MiB; larger calls raise MoeError). The outputs
    are allocated here, as for init_routing; the same results."""
    lib = load()
    _need_gpu(x, expert_idx)
    if expert_idx.dtype != torch.int32 or expert_idx.dim() != 2 or expert_idx.shape[0] != x.shape[0]:
        raise ValueError("expert_idx must be int32 [N, K] with N = x.shape[0]")
    n, h = x.shape
    k = expert_idx.shape[1]
    s, e = (0, expert_num) if active_range is None else active_range
    ex, idx, tok, sc, avail = _routing_outputs(x, n, h, k, expert_num, s, e, quant_mode, expert_tokens_num_type)
    _check(lib.moe_init_routing_noalloc(_ptr(x), _DT[x.dtype], None, n, h, _ptr(expert_idx), k, expert_num, s, e,
                                        quant_mode, row_idx_type, expert_tokens_num_type, _ptr(ex), _ptr(idx),
                                        _ptr(tok), _ptr(sc), _ptr(avail), _stream(x.device)))
    return ex, idx, tok, sc, avail


def _routing_outputs(x, n, h, k, expert_num, s, e, quant_mode, expert_tokens_num_type):
    flat = n * k
    mx = quant_mode != QUANT_NONE
    dev = x.device
    ex = torch.empty((flat, h // 2 if quant_mode == QUANT_MXFP4 else h), dtype=torch.uint8 if mx else x.dtype,
                     device=dev)
    idx = torch.empty((flat,), dtype=torch.int32, device=dev)
    if expert_tokens_num_type == 2:   # key_value: (expert, count) rows
        tok = torch.empty((expert_num, 2), dtype=torch.int64, device=dev)
    else:
        tok = torch.empty((max(e - s, 0),), dtype=torch.int64, device=dev)
    sc = torch.empty((flat, mx_scale_cols(h)), dtype=torch.uint8, device=dev) if mx else None
    avail = torch.empty((1,), dtype=torch.int64, device=dev)
    return ex, idx, tok, sc, avail


def init_routing(x, expert_idx, expert_num: int, active_range=None, quant_mode: int = QUANT_NONE,
                 row_idx_type: int = 1, expert_tokens_num_type: int = 1, x_codes: int | None = None, scale=None):
    """MoeInitRoutingV3 (dropless). Returns (expanded_x, expanded_row_idx, expert_tokens,
    expanded_scale or None, available_idx_num) with expanded_x of shape [N*K, H].

    x_codes: DTYPE_FP8_E5M2 / DTYPE_FP8_E4M3 / DTYPE_FP4_E2M1 when x holds MX codes (uint8
    [N, H], or [N, H/2] for FP4, H the logical hidden size): the rows are gathered as they
    are (quant_mode -1), with their E8M0 scales [N, mx_scale_cols(H)] when scale is given."""
    lib = load()
    _need_gpu(x, expert_idx)
    if expert_idx.dtype != torch.int32 or expert_idx.dim() != 2 or expert_idx.shape[0] != x.shape[0]:
        raise ValueError(f"expert_idx must be int32 [N, K] with N = x.shape[0] (got {expert_idx.dtype} "
                         f"{tuple(expert_idx.shape)})")
    n, h = x.shape
    if x_codes is not None:
        return _init_routing_codes(lib, x, expert_idx, expert_num, active_range, row_idx_type,
                                   expert_tokens_num_type, x_codes, scale)
    k = expert_idx.shape[1]
    s, e = (0, expert_num) if active_range is None else active_range
    dev = x.device
    ex, idx, tok, sc, avail = _routing_outputs(x, n, h, k, expert_num, s, e, quant_mode, expert_tokens_num_type)
    nbytes = ctypes.c_size_t()
    _check(lib.moe_init_routing_workspace_size(n, k, expert_num, ctypes.byref(nbytes)))
    ws = _workspace(nbytes.value, dev)
    _check(lib.moe_init_routing(_ptr(x), _DT[x.dtype], None, n, h, _ptr(expert_idx), k, expert_num, s, e, quant_mode,
                                row_idx_type, expert_tokens_num_type, _ptr(ex), _ptr(idx), _ptr(tok), _ptr(sc),
                                _ptr(avail), _ptr(ws), ws.numel(), _stream(dev)))
    return ex, idx, tok, sc, avail


def _init_routing_codes(lib, x, expert_idx, expert_num, active_range, row_idx_type, expert_tokens_num_type,
                        x_codes, scale):
    n, row_bytes = x.shape
    h = 2 * row_bytes if x_codes == DTYPE_FP4_E2M1 else row_bytes
    k = expert_idx.shape[1]
    s, e = (0, expert_num) if active_range is None else active_range
    flat = n * k
    dev = x.device
    ex = torch.empty((flat, row_bytes), dtype=torch.uint8, device=dev)
    idx = torch.empty((flat,), dtype=torch.int32, device=dev)
    if expert_tokens_num_type == 2:
        tok = torch.empty((expert_num, 2), dtype=torch.int64, device=dev)
    else:
        tok = torch.empty((max(e - s, 0),), dtype=torch.int64, device=dev)
    sc = None
    if scale is not None:
        _need_gpu(scale)
        scale = _u8(scale)
        if tuple(scale.shape) != (n, mx_scale_cols(h)):
            raise ValueError(f"scale must be [N, {mx_scale_cols(h)}] E8M0 bytes")
        sc = torch.empty((flat, mx_scale_cols(h)), dtype=torch.uint8, device=dev)
    avail = torch.empty((1,), dtype=torch.int64, device=dev)
    nbytes = ctypes.c_size_t()
    _check(lib.moe_init_routing_workspace_size(n, k, expert_num, ctypes.byref(nbytes)))
    ws = _workspace(nbytes.value, dev)
    _check(lib.moe_init_routing(_ptr(_u8(x)), x_codes, _ptr(scale), n, h, _ptr(expert_idx), k, expert_num, s, e,
                                QUANT_NONE, row_idx_type, expert_tokens_num_type, _ptr(ex), _ptr(idx), _ptr(tok),
                                _ptr(sc), _ptr(avail), _ptr(ws), ws.numel(), _stream(dev)))
    return ex, idx, tok, sc, avail


def token_permute(tokens, indices, num_out_tokens=None, padded_mode: bool = False, quant_mode: int = QUANT_NONE,
                  *, num_experts: int):
    """moe_token_permute: (permuted_tokens [M, H], sorted_indices int32 [F], expanded_scale or empty).

    num_experts is the exclusive bound of the index values (the counting sort's bucket count)."""
    lib = load()
    _need_gpu(tokens, indices)
    n, h = tokens.shape
    topk = 1 if indices.dim() == 1 else indices.shape[1]
    flat = indices.numel()
    m = token_permute_out_rows(flat, num_out_tokens)
    mx = quant_mode != QUANT_NONE
    dev = tokens.device
    out = torch.empty((m, h // 2 if quant_mode == QUANT_MXFP4 else h), dtype=torch.uint8 if mx else tokens.dtype,
                      device=dev)
    srt = torch.empty((flat,), dtype=torch.int32, device=dev)
    sc = (torch.empty((m, mx_scale_cols(h)), dtype=torch.uint8, device=dev) if mx
          else torch.empty((0,), dtype=torch.float32, device=dev))
    nbytes = ctypes.c_size_t()
    _check(lib.moe_token_permute_workspace_size(flat, num_experts, ctypes.byref(nbytes)))
    ws = _workspace(nbytes.value, dev)
    _check(lib.moe_token_permute(_ptr(tokens), _DT[tokens.dtype], n, h, _ptr(indices), _DT[indices.dtype], topk,
                                 num_experts, 0 if num_out_tokens is None else int(num_out_tokens),
                                 int(bool(padded_mode)), quant_mode, _ptr(out), _ptr(srt),
                                 _ptr(sc) if mx else None, _ptr(ws), ws.numel(), _stream(dev)))
    return out, srt, sc


def _check_layer_dtypes(x, topk_ids, topk_weights, x_scales=None):
    """The C side reads int32 ids, fp32/bf16 gate weights and bf16 x (uint8 codes with
    x_scales): anything else would be misread, so it is rejected here."""
    if topk_ids.dtype != torch.int32:
        raise ValueError(f"topk_ids must be int32 (got {topk_ids.dtype}); convert e.g. torch.topk's int64 ids")
    if topk_weights.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"topk_weights must be float32 or bfloat16 (got {topk_weights.dtype})")
    if x_scales is None:
        if x.dtype != torch.bfloat16:
            raise ValueError(f"x must be bfloat16 (got {x.dtype})")
    elif x.dtype not in (torch.uint8, torch.float8_e4m3fn, torch.float8_e5m2):
        raise ValueError(f"pre-quantized x must hold FP8 codes (uint8 or float8), got {x.dtype}")
    if topk_ids.dim() != 2 or topk_ids.shape != topk_weights.shape or topk_ids.shape[0] != x.shape[0]:
        raise ValueError("topk_ids and topk_weights must both be [N, K] with N = x.shape[0]")


def _mega_struct(x, topk_ids, topk_weights, w1, w1_scales, w2, w2_scales, shared, quant_out_dtype, y, etn,
                 debug, weight_format=WEIGHTS_ND, activation=ACT_SWIGLU, activation_params=(), weight_dtype=0,
                 shared_weight_dtype=0, x_scales=None, combine_comm_mode=0):
    n, h = x.shape
    k = topk_ids.shape[1]
    e, two_i, _ = w1.shape
    a = MegaArgs()
    a.x, a.num_tokens, a.hidden = _ptr(x), n, h
    a.topk_ids, a.topk = _ptr(topk_ids), k
    a.topk_weights, a.topk_weights_dtype = _ptr(topk_weights), _DT[topk_weights.dtype]
    a.num_experts, a.inter = e, two_i // 2
    a.w1, a.w1_scales, a.w2, a.w2_scales = _ptr(_u8(w1)), _ptr(_u8(w1_scales)), _ptr(_u8(w2)), _ptr(_u8(w2_scales))
    if shared is not None:
        sw1, ss1, sw2, ss2 = shared
        a.num_shared = sw1.shape[0]
        a.shared_w1, a.shared_w1_scales = _ptr(_u8(sw1)), _ptr(_u8(ss1))
        a.shared_w2, a.shared_w2_scales = _ptr(_u8(sw2)), _ptr(_u8(ss2))
    a.quant_out_dtype, a.activation, a.weight_format = quant_out_dtype, activation, weight_format
    if len(activation_params) > 3:
        raise ValueError("activation_params holds at most 3 values")
    a.num_activation_params = len(activation_params)
    a.weight_dtype, a.shared_weight_dtype = weight_dtype, shared_weight_dtype
    if x_scales is not None:   # pre-quantized pass-through: x holds FP8 codes
        a.x_is_quantized, a.x_scales = 1, _ptr(_u8(x_scales))
    a.combine_comm_mode = combine_comm_mode
    for j, v in enumerate(activation_params):
        a.activation_params[j] = float(v)
    a.y, a.expert_token_nums = _ptr(y), _ptr(etn)
    for name in ("xq", "sx", "h1", "aq", "sa", "o", "sorted_row_idx"):
        setattr(a, name, _ptr(debug.get(name)) if debug else None)
    return a


def mega_moe(x, topk_ids, topk_weights, w1, w1_scales, w2, w2_scales, shared=None,
             quant_out_dtype: int = FP8_E4M3, debug: bool = False, workspace=None, stage_events=None,
             weight_format: int = WEIGHTS_ND, activation: int = ACT_SWIGLU, activation_params=(),
             weight_dtype: int = 0, shared_weight_dtype: int = 0, x_scales=None, combine_comm_mode: int = 0):
    """The MX MoE layer. Returns (y bf16 [N, H], expert_token_nums int32 [E]) and, with
    debug=True, a dict of the stage intermediates (xq, sx, h1, aq, sa, o, sorted_row_idx).

    shared: None or (shared_w1, shared_w1_scales, shared_w2, shared_w2_scales) stacked
    over the shared experts. workspace: optional preallocated uint8 device tensor.
    weight_format: WEIGHTS_ND (the pages' layout) or WEIGHTS_PACKED (w1/w2 and the
    shared weights as returned by pack_weights; the code tensors keep their [E, N, K] shape).
    stage_events: optional list of MEGA_STAGE_EVENTS torch.cuda.Event(enable_timing=True) or
    None entries, recorded by the library on the stream at the boundaries of MEGA_STAGES
    (a None entry is skipped; each record costs a few microseconds of GPU time).
    activation / activation_params: ACT_* and its parameter list as in the C header (gelu
    makes A, and w2's input width, 2 * inter).
    weight_dtype: 0 or the activations' FP8 type (FP8 weights), or FP4_E2M1 (MXFP4 codes
    two a byte, e.g. from mx_quantize(..., QUANT_MXFP4); pack_weights(..., fp4=True)).
    shared_weight_dtype: 0 = the same as weight_dtype, else one of the values above
    (e.g. FP8_E4M3 for FP8 shared experts beside MXFP4 routed experts).
    x_scales: pre-quantized pass-through: x holds FP8 codes of quant_out_dtype (uint8
    [N, H], e.g. from mx_quantize) and x_scales their E8M0 scales [N, H/32].
    combine_comm_mode: 0 (each expert output row rounded to bf16 before the weighted sum,
    MegaMoE's default) or 1 (a token's expert outputs summed in fp32, rounded once)."""
    lib = load()
    _need_gpu(x, topk_ids, topk_weights, w1, w1_scales, w2, w2_scales)
    _check_layer_dtypes(x, topk_ids, topk_weights, x_scales)
    if x_scales is not None and x_scales.shape[1] != x.shape[1] // 32:
        x_scales = x_scales[:, :x.shape[1] // 32].contiguous()   # drop the AlignUp(.., 2) padding column
    n, h = x.shape
    k = topk_ids.shape[1]
    e, two_i, _ = w1.shape
    inter = two_i // 2
    aw = two_i if activation == ACT_GELU else inter   # width of A
    dev = x.device
    y = torch.empty((n, h), dtype=torch.bfloat16, device=dev)
    etn = torch.empty((e,), dtype=torch.int32, device=dev)
    dbg = None
    if debug:
        f = n * k
        dbg = dict(xq=torch.empty((f, h), dtype=torch.uint8, device=dev),
                   sx=torch.empty((f, h // 32), dtype=torch.uint8, device=dev),
                   h1=torch.empty((f, 2 * inter), dtype=torch.float32, device=dev),
                   aq=torch.empty((f, aw), dtype=torch.uint8, device=dev),
                   sa=torch.empty((f, aw // 32), dtype=torch.uint8, device=dev),
                   o=torch.empty((f, h), dtype=torch.float32, device=dev),
                   sorted_row_idx=torch.empty((f,), dtype=torch.int32, device=dev))
    a = _mega_struct(x, topk_ids, topk_weights, w1, w1_scales, w2, w2_scales, shared, quant_out_dtype, y, etn, dbg,
                     weight_format, activation, activation_params, weight_dtype, shared_weight_dtype, x_scales,
                     combine_comm_mode)
    if stage_events is not None:
        if len(stage_events) != MEGA_STAGE_EVENTS:
            raise ValueError(f"stage_events needs {MEGA_STAGE_EVENTS} entries (events or None)")
        for ev in stage_events:
            if ev is not None and not ev.cuda_event:
                ev.record()   # torch creates the HIP event at its first record
        handles = (ctypes.c_void_p * MEGA_STAGE_EVENTS)(*[ev.cuda_event if ev is not None else None
                                                          for ev in stage_events])
        a.stage_events = ctypes.cast(handles, ctypes.POINTER(ctypes.c_void_p))
    nbytes = ctypes.c_size_t()
    _check(lib.mega_moe_workspace_size(ctypes.byref(a), ctypes.byref(nbytes)))
    ws = workspace if workspace is not None and workspace.numel() >= nbytes.value else _workspace(nbytes.value, dev)
    _check(lib.mega_moe(ctypes.byref(a), _ptr(ws), ws.numel(), _stream(dev)))
    if debug:
        return y, etn, dbg
    return y, etn


def mega_moe_workspace_bytes(x, topk_ids, topk_weights, w1, w1_scales, w2, w2_scales, shared=None,
                             quant_out_dtype: int = FP8_E4M3, weight_format: int = WEIGHTS_ND,
                             activation: int = ACT_SWIGLU, activation_params=(), weight_dtype: int = 0,
                             shared_weight_dtype: int = 0, combine_comm_mode: int = 0) -> int:
    lib = load()
    _check_layer_dtypes(x, topk_ids, topk_weights)
    a = _mega_struct(x, topk_ids, topk_weights, w1, w1_scales, w2, w2_scales, shared, quant_out_dtype, x, x, None,
                     weight_format, activation, activation_params, weight_dtype, shared_weight_dtype,
                     combine_comm_mode=combine_comm_mode)
    nbytes = ctypes.c_size_t()
    _check(lib.mega_moe_workspace_size(ctypes.byref(a), ctypes.byref(nbytes)))
    return nbytes.value


def gmm1_swiglu_quant(xq, sx, group_offsets, w1, w1_scales, quant_out_dtype: int = FP8_E4M3, want_h1: bool = False,
                      weight_format: int = WEIGHTS_ND):
    """Stage 2 on given operands: (aq uint8 [rows, I], sa uint8 [rows, I/32], h1 fp32 [rows, 2I] or None)."""
    lib = load()
    xq, sx, w1, w1_scales = _u8(xq), _u8(sx), _u8(w1), _u8(w1_scales)
    _need_gpu(xq, sx, group_offsets, w1, w1_scales)
    rows, h = xq.shape
    g, two_i, _ = w1.shape
    inter = two_i // 2
    dev = xq.device
    aq = torch.empty((rows, inter), dtype=torch.uint8, device=dev)
    sa = torch.empty((rows, inter // 32), dtype=torch.uint8, device=dev)
    h1 = torch.empty((rows, two_i), dtype=torch.float32, device=dev) if want_h1 else None
    nbytes = ctypes.c_size_t()
    _check(lib.moe_gmm_workspace_size(rows, g, h, inter, ctypes.byref(nbytes)))
    ws = _workspace(nbytes.value, dev)
    _check(lib.moe_gmm1_swiglu_quant(_ptr(xq), _ptr(sx), rows, h, inter, _ptr(group_offsets), g, _ptr(w1),
                                     _ptr(w1_scales), weight_format, quant_out_dtype, _ptr(aq), _ptr(sa), _ptr(h1),
                                     _ptr(ws), ws.numel(), _stream(dev)))
    return aq, sa, h1


def gmm2_combine(aq, sa, group_offsets, w2, w2_scales, row_token, row_weight, y_accum,
                 quant_out_dtype: int = FP8_E4M3, want_o: bool = False, weight_format: int = WEIGHTS_ND):
    """Stages 3-4 on given operands: y_accum[row_token[r]] += row_weight[r] * O[r]; returns O (fp32) or None."""
    lib = load()
    aq, sa, w2, w2_scales = _u8(aq), _u8(sa), _u8(w2), _u8(w2_scales)
    _need_gpu(aq, sa, group_offsets, w2, w2_scales, row_token, row_weight, y_accum)
    rows, inter = aq.shape
    g, h, _ = w2.shape
    dev = aq.device
    o = torch.empty((rows, h), dtype=torch.float32, device=dev) if want_o else None
    nbytes = ctypes.c_size_t()
    _check(lib.moe_gmm_workspace_size(rows, g, h, inter, ctypes.byref(nbytes)))
    ws = _workspace(nbytes.value, dev)
    _check(lib.moe_gmm2_combine(_ptr(aq), _ptr(sa), rows, inter, h, _ptr(group_offsets), g, _ptr(w2),
                                _ptr(w2_scales), weight_format, quant_out_dtype, _ptr(row_token), _ptr(row_weight),
                                y_accum.shape[0], _ptr(y_accum), _ptr(o), _ptr(ws), ws.numel(), _stream(dev)))
    return o


def combine_finalize(y_accum):
    """bf16 (round to nearest even) of an fp32 accumulation buffer."""
    lib = load()
    _need_gpu(y_accum)
    n, h = y_accum.shape
    y = torch.empty((n, h), dtype=torch.bfloat16, device=y_accum.device)
    _check(lib.moe_combine_finalize(_ptr(y_accum), n, h, _ptr(y), _stream(y_accum.device)))
    return y


class _on:
    """The tensors' device as the current one while a call is made on it (a no-op, without
    the cost of torch's device context, where it is current already)."""

    __slots__ = ("want", "was")

    def __init__(self, index: int):
        self.want, self.was = index, torch.cuda.current_device()

    def __enter__(self):
        if self.want != self.was:
            torch.cuda.set_device(self.want)

    def __exit__(self, *exc):
        if self.want != self.was:
            torch.cuda.set_device(self.was)
        return False


def _device_of(first, **others):
    """The index of the GPU that holds `first` and every other given tensor, all contiguous."""
    if not first.is_cuda:
        raise ValueError("tensors must be on the GPU")
    if not first.is_contiguous():
        raise ValueError("tensors must be contiguous")
    for name, t in others.items():
        if t is not None:
            if t.device != first.device:
                raise ValueError(f"{name} is on {t.device}, not on {first.device}")
            if not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous")
    return first.device.index


@functools.lru_cache(maxsize=4096)
def _sized(query: str, *sizes) -> int:
    """A workspace size, which depends on the sizes alone."""
    nbytes = ctypes.c_size_t()
    _check(getattr(load(), query)(*sizes, ctypes.byref(nbytes)))
    return nbytes.value


def _raw(t):
    return None if t is None else t.data_ptr()


def _raw_stream(index: int):
    return torch._C._cuda_getCurrentRawStream(index)


def _gate_logits(logits, topk_ids=None):
    if logits.dim() != 2 or logits.dtype not in (torch.float32, torch.float16, torch.bfloat16):
        raise ValueError(f"logits must be float32, float16 or bfloat16 [rows, experts] (got {logits.dtype} "
                         f"{tuple(logits.shape)})")
    if topk_ids is not None and (topk_ids.dtype != torch.int32 or topk_ids.dim() != 2
                                 or topk_ids.shape[0] != logits.shape[0]):
        raise ValueError(f"topk_ids must be int32 [rows, k] with the logits' rows (got {topk_ids.dtype} "
                         f"{tuple(topk_ids.shape)})")
    return logits.shape


def _gate_seqs(rows, seq_offsets, row_mask):
    """The number of sequences, after the checks of their offsets and of the row mask."""
    if row_mask is not None and (row_mask.dtype not in (torch.uint8, torch.bool) or tuple(row_mask.shape) != (rows,)):
        raise ValueError(f"row_mask must be uint8 or bool [rows] (got {row_mask.dtype} {tuple(row_mask.shape)})")
    if seq_offsets is None:
        return 1
    if seq_offsets.dtype != torch.int32 or seq_offsets.dim() != 1 or seq_offsets.numel() < 2:
        raise ValueError(f"seq_offsets must be int32 [sequences + 1] (got {seq_offsets.dtype} "
                         f"{tuple(seq_offsets.shape)})")
    return seq_offsets.numel() - 1


def gate_topk(logits, k: int, *, scoring: int = GATE_SOFTMAX, bias=None, num_groups: int = 1, topk_groups: int = 1,
              renormalize: bool = True, scale: float = 1.0):
    """The router's choice: (topk_ids int32 [N, K], topk_weights fp32 [N, K]) of logits [N, E]
    (fp32, fp16 or bf16), as init_routing and mega_moe take them.

    scoring: GATE_SOFTMAX (over all E) or GATE_SIGMOID. bias: fp32 [E] added to the scores for
    the choice only (NaN counts as -inf: chosen last). num_groups / topk_groups: only the
    topk_groups best of num_groups equal groups of neighbouring experts (by the sum of their two
    best ranks) take part. The ids come in descending order of rank, ties by the lowest index.
    renormalize: the weights of a row sum to `scale` (else they are scale * score). A logit of
    -inf or NaN takes its expert out (score 0, chosen last). The weights carry no autograd
    history: gate_backward gives the logits' gradient."""
    lib = load()
    n, e = _gate_logits(logits)
    index = _device_of(logits, bias=bias)
    if bias is not None and (bias.dtype != torch.float32 or tuple(bias.shape) != (e,)):
        raise ValueError(f"bias must be float32 [{e}] (got {bias.dtype} {tuple(bias.shape)})")
    dev = logits.device
    with _on(index):
        ids = torch.empty((n, max(k, 0)), dtype=torch.int32, device=dev)
        w = torch.empty((n, max(k, 0)), dtype=torch.float32, device=dev)
        _check(lib.moe_gate_topk(logits.data_ptr(), _DT[logits.dtype], n, e, k, scoring, _raw(bias), num_groups,
                                 topk_groups, int(bool(renormalize)), scale, ids.data_ptr(), w.data_ptr(),
                                 _raw_stream(index)))
    return ids, w


def balance_loss(logits, topk_ids, *, scoring: int = GATE_SOFTMAX, seq_offsets=None, row_mask=None,
                 alpha: float = 1.0):
    """The load-balance loss of a router's rows: (loss fp32 [1], counts int32 [B, E], coef fp32
    [B, E]) of logits [N, E] and the ids gate_topk chose.

    loss = alpha * mean over the sequences with a counted row of sum_e f_e P_e, f_e = E times
    the share of the sequence's choices that went to expert e, P_e = the mean score of e
    (sigmoid scores divided by their sum). seq_offsets: int32 [B + 1] (None: all rows are one
    sequence); row_mask: uint8 or bool [N], rows with 0 do not count. counts: the choices of
    each expert. coef: the derivative of the loss by the scores of a counted row, for
    gate_backward."""
    lib = load()
    n, e = _gate_logits(logits, topk_ids)
    seqs = _gate_seqs(n, seq_offsets, row_mask)
    index = _device_of(logits, topk_ids=topk_ids, seq_offsets=seq_offsets, row_mask=row_mask)
    dev = logits.device
    nbytes = _sized("moe_balance_loss_workspace_size", n, e, seqs)
    with _on(index):
        loss = torch.empty((1,), dtype=torch.float32, device=dev)
        counts = torch.empty((seqs, e), dtype=torch.int32, device=dev)
        coef = torch.empty((seqs, e), dtype=torch.float32, device=dev)
        ws = _workspace(nbytes, dev)
        _check(lib.moe_balance_loss(logits.data_ptr(), _DT[logits.dtype], n, e, topk_ids.data_ptr(), topk_ids.shape[1],
                                    scoring, _raw(seq_offsets), seqs, _raw(row_mask), alpha, loss.data_ptr(),
                                    counts.data_ptr(), coef.data_ptr(), ws.data_ptr(), ws.numel(), _raw_stream(index)))
    return loss, counts, coef


def gate_backward(logits, topk_ids, grad_weights=None, *, scoring: int = GATE_SOFTMAX, renormalize: bool = True,
                  scale: float = 1.0, grad_loss=None, coef=None, seq_offsets=None, row_mask=None):
    """The logits' gradient ([N, E], the logits' type) in one pass: of gate_topk's weights, given
    grad_weights fp32 [N, K] (scoring, renormalize and scale as in that call; the choice is held
    fixed), and of balance_loss's loss, given grad_loss fp32 [1] with that call's coef,
    seq_offsets and row_mask (the counts are held fixed). Either may be None."""
    lib = load()
    n, e = _gate_logits(logits, topk_ids)
    seqs = _gate_seqs(n, seq_offsets, row_mask)
    k = topk_ids.shape[1]
    if grad_weights is not None and (grad_weights.dtype != torch.float32 or tuple(grad_weights.shape) != (n, k)):
        raise ValueError(f"grad_weights must be float32 [{n}, {k}] (got {grad_weights.dtype} "
                         f"{tuple(grad_weights.shape)})")
    if grad_loss is not None and (grad_loss.dtype != torch.float32 or grad_loss.numel() != 1):
        raise ValueError("grad_loss must be one float32 value")
    if coef is not None and (coef.dtype != torch.float32 or tuple(coef.shape) != (seqs, e)):
        raise ValueError(f"coef must be float32 [{seqs}, {e}] (got {coef.dtype} {tuple(coef.shape)})")
    index = _device_of(logits, topk_ids=topk_ids, grad_weights=grad_weights, grad_loss=grad_loss, coef=coef,
                       seq_offsets=seq_offsets, row_mask=row_mask)
    with _on(index):
        grad = torch.empty_like(logits)
        _check(lib.moe_gate_backward(logits.data_ptr(), _DT[logits.dtype], n, e, topk_ids.data_ptr(), k, scoring,
                                     int(bool(renormalize)), scale, _raw(grad_weights), _raw(grad_loss), _raw(coef),
                                     _raw(seq_offsets), seqs, _raw(row_mask), grad.data_ptr(), _raw_stream(index)))
    return grad


def mxfp4_matmul(x, w, w_scales, *, x_scales=None, group_offsets=None, out_dtype=torch.bfloat16,
                 weight_format: int = WEIGHTS_ND, out=None, workspace=None):
    """MXFP4 x MXFP4 product: out [R, N] (bf16 or fp32), out[r] = DQ(x[r]) DQ(w[g])^T for the
    rows r of group g.

    x: bf16, fp16 or fp32 [R, K], quantised in the call as mx_quantize(x, QUANT_MXFP4) would, or
    its MXFP4 codes uint8 [R, K/2] with x_scales uint8 [R, K/32] (from mx_quantize, init_routing
    or token_permute in mode QUANT_MXFP4). w, w_scales: codes uint8 [G, N, K/2] and scales
    [G, N, K/32], or both from pack_weights(..., fp4=True) with weight_format=WEIGHTS_PACKED;
    without group_offsets (one group) w may be [N, K/2]. group_offsets: int32 [G + 1], the rows
    of group g are [off[g], off[g + 1]); rows outside all groups are left as they were in `out`
    (uninitialised when out is None). workspace: optional preallocated uint8 device tensor."""
    lib = load()
    if x.dim() != 2 or (x_scales is None) != (x.dtype in (torch.float32, torch.float16, torch.bfloat16)):
        raise ValueError(f"x must be float32, float16 or bfloat16 [rows, k], or uint8 codes [rows, k/2] with x_scales "
                         f"(got {x.dtype} {tuple(x.shape)}, x_scales {'missing' if x_scales is None else 'given'})")
    if x_scales is not None and x.dtype != torch.uint8:
        raise ValueError(f"MXFP4 codes must be uint8 (got {x.dtype})")
    w, w_scales, x_scales = _u8(w), _u8(w_scales), _u8(x_scales)
    if w.dim() == 2 and group_offsets is None:
        w = w.unsqueeze(0)
    if w.dim() != 3:
        raise ValueError(f"w must be [groups, n, k/2] (got {tuple(w.shape)})")
    rows, k = x.shape if x_scales is None else (x.shape[0], 2 * x.shape[1])
    g, n, kb = w.shape
    if 2 * kb != k:
        raise ValueError(f"x has k = {k}, w has k = {2 * kb}")
    want = lib.moe_mx_packed_scale_bytes(g, n, k) if weight_format == WEIGHTS_PACKED else g * n * (k // 32)
    if w_scales.numel() != want:
        raise ValueError(f"w_scales must hold {want} bytes (got {tuple(w_scales.shape)})")
    if x_scales is not None and tuple(x_scales.shape) != (rows, k // 32):
        raise ValueError(f"x_scales must be [{rows}, {k // 32}] (got {tuple(x_scales.shape)})")
    if group_offsets is None:
        if g != 1:
            raise ValueError(f"{g} groups need group_offsets")
    elif group_offsets.dtype != torch.int32 or tuple(group_offsets.shape) != (g + 1,):
        raise ValueError(f"group_offsets must be int32 [{g + 1}] (got {group_offsets.dtype} "
                         f"{tuple(group_offsets.shape)})")
    if out is None:
        if out_dtype not in (torch.bfloat16, torch.float32):
            raise ValueError(f"out_dtype must be bfloat16 or float32 (got {out_dtype})")
    elif out.dtype not in (torch.bfloat16, torch.float32) or tuple(out.shape) != (rows, n):
        raise ValueError(f"out must be bfloat16 or float32 [{rows}, {n}] (got {out.dtype} {tuple(out.shape)})")
    if workspace is not None and workspace.dtype != torch.uint8:
        raise ValueError(f"workspace must be uint8 (got {workspace.dtype})")
    index = _device_of(x, w=w, w_scales=w_scales, x_scales=x_scales, group_offsets=group_offsets, out=out,
                       workspace=workspace)
    xd = DTYPE_FP4_E2M1 if x_scales is not None else _DT[x.dtype]
    nbytes = _sized("moe_mxfp4_matmul_workspace_size", rows, g, n, k, xd, weight_format)
    with _on(index):
        if out is None:
            out = torch.empty((rows, n), dtype=out_dtype, device=x.device)
        ws = workspace
        if nbytes and (ws is None or ws.numel() < nbytes):
            ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
        _check(lib.moe_mxfp4_matmul(x.data_ptr(), xd, _raw(x_scales), rows, _raw(group_offsets), g, w.data_ptr(),
                                    w_scales.data_ptr(), n, k, weight_format, out.data_ptr(), _DT[out.dtype], _raw(ws),
                                    0 if ws is None else ws.numel(), _raw_stream(index)))
    return out


def probe_stream(src, dst=None, copy: bool = False, fill_caches: bool = False):
    """One launch of the library's streaming kernel: read src (uint8 device tensor, a
    multiple of 16 bytes), or copy it to dst, with non-temporal accesses; with
    fill_caches a read with plain loads (to evict other data from the caches). Returns
    None; time it with events."""
    lib = load()
    _need_gpu(src)
    if copy and (dst is None or dst.numel() < src.numel()):
        raise ValueError("probe_stream: copy needs a dst at least as large as src")
    if dst is None:
        dst = torch.empty(16, dtype=torch.uint8, device=src.device)
    mode = 1 if copy else (2 if fill_caches else 0)
    _check(lib.moe_probe_stream(mode, _ptr(src), _ptr(dst), src.numel(), _stream(src.device)))


def probe_mfma(iters: int, out=None, device="cuda"):
    """One launch of the library's MFMA loop; returns (out tensor, flops of the launch)."""
    lib = load()
    n = ctypes.c_int64()
    fl = ctypes.c_double()
    _check(lib.moe_probe_mfma(iters, None, ctypes.byref(n), ctypes.byref(fl), None))
    if out is None or out.numel() < n.value:
        out = torch.empty(n.value, dtype=torch.float32, device=device)
    _check(lib.moe_probe_mfma(iters, _ptr(out), None, None, _stream(out.device)))
    return out, fl.value
