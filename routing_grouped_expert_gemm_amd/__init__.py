"""Python binding of libmok (include/mok.h): argument marshalling only.

Every step of the MoE-layer forward runs in the library's HIP kernels; PyTorch supplies
device memory and the current HIP stream. Importing this module loads libmok.so and fails
loudly (ImportError) if it has not been built: there is no fallback of any kind.

Entry points carry the C names: mok_route, mok_topk, mok_dispatch_plan,
mok_dispatch_plan_workspace_bytes, mok_moe_workspace_bytes, mok_moe_forward,
mok_quantize_mxfp8, mok_quantize_mxfp8_f32, mok_quantize_mxfp4_f32, mok_get_device_error,
mok_status_string, mok_version. Around the layer: mok_topk_scored, mok_route_scored and
mok_topk_scored_backward (routing by scores), mok_gated_norm and mok_gated_norm_backward, mok_quantize_int4,
mok_w4_gemm and MoeW4Layer (mok_moe_w4_forward: the experts on 4-bit weights).
"""
from __future__ import annotations

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmok.so")   # always the in-tree build

MOK_OK, MOK_EINVAL, MOK_EUNSUPPORTED, MOK_EWORKSPACE, MOK_EHIP = range(5)
MOK_FP32, MOK_BF16, MOK_MXFP8, MOK_MXFP4 = 0, 1, 2, 3
MOK_FLAG_NO_RING, MOK_FLAG_STAGE_LOOP = 1, 2
(MOK_STAGE_ROUTE, MOK_STAGE_PLAN, MOK_STAGE_QUANT, MOK_STAGE_UP, MOK_STAGE_DOWN, MOK_STAGE_COMBINE,
 MOK_STAGE_GATHER) = range(7)
MOK_N_STAGES = 7
(MOK_REGION_WORKLIST, MOK_REGION_H, MOK_REGION_H_SCALES, MOK_REGION_A_CODES, MOK_REGION_A_SCALES,
 MOK_REGION_WG_CODES, MOK_REGION_WG_SCALES, MOK_REGION_WU_CODES, MOK_REGION_WU_SCALES,
 MOK_REGION_WD_CODES, MOK_REGION_WD_SCALES, MOK_REGION_SG_CODES, MOK_REGION_SG_SCALES,
 MOK_REGION_SU_CODES, MOK_REGION_SU_SCALES, MOK_REGION_SD_CODES, MOK_REGION_SD_SCALES) = range(17)
MOK_DEVERR_OVERFLOW, MOK_DEVERR_WAIT = 1, 2
MOK_SCORE_SOFTMAX, MOK_SCORE_SIGMOID = 0, 1

EXPORTS = ["mok_status_string", "mok_version", "mok_route", "mok_topk",
           "mok_dispatch_plan_workspace_bytes", "mok_dispatch_plan", "mok_dispatch_plan_noalloc",
           "mok_moe_workspace_bytes",
           "mok_moe_forward", "mok_moe_workspace_region", "mok_moe_backward",
           "mok_moe_backward_workspace_bytes", "mok_moe_backward_error", "mok_pull_gather",
           "mok_push_dispatch", "mok_quantize_mxfp8", "mok_quantize_mxfp4",
           "mok_quantize_mxfp8_f32", "mok_quantize_mxfp4_f32", "mok_get_device_error",
           "mok_balance_loss_workspace_bytes", "mok_balance_loss", "mok_balance_loss_backward",
           "mok_rmsnorm", "mok_rmsnorm_backward_workspace_bytes", "mok_rmsnorm_backward",
           "mok_route_backward_workspace_bytes", "mok_route_backward",
           "mok_mx_gemm_workspace_bytes", "mok_mx_gemm",
           "mok_topk_scored", "mok_route_scored", "mok_topk_scored_backward",
           "mok_gated_norm", "mok_gated_norm_backward_workspace_bytes", "mok_gated_norm_backward",
           "mok_quantize_int4", "mok_w4_gemm", "mok_moe_w4_workspace_bytes", "mok_moe_w4_forward"]


class MokError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {status_string(status)}")
        self.status = status


if not os.path.exists(LIB_PATH):
    raise ImportError(f"libmok.so is not built ({LIB_PATH}); run "
                      "`python routing_grouped_expert_gemm_amd/_build.py` or __graft_entry__.build()")

_lib = ctypes.CDLL(LIB_PATH)
_P, _I64, _I32, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t


class MoeArgs(ctypes.Structure):
    """Mirror of struct mok_moe_args."""
    _fields_ = [
        ("dtype", _I32), ("d", _I32), ("E", _I32), ("k", _I32), ("I", _I32),
        ("e0", _I32), ("E_l", _I32), ("tokens_per_rank", _I32),
        ("T_pool", _I64), ("own_begin", _I64), ("T_own", _I32),
        ("n_shared", _I32), ("I_shared", _I32), ("minibatch_rows", _I32), ("ring_rows", _I32),
        ("flags", ctypes.c_uint32),
        ("x", _P), ("w_router", _P), ("topk_idx_in", _P), ("topk_w_in", _P),
        ("w_gate", _P), ("w_up", _P), ("w_down", _P),
        ("ws_gate", _P), ("ws_up", _P), ("ws_down", _P),
        ("workspace", _P), ("workspace_bytes", _SZ),
        ("y_slots", _P), ("y_shared", _P), ("y", _P),
        ("logits_out", _P), ("topk_idx_out", _P), ("topk_w_out", _P),
        ("counts_out", _P), ("offsets_out", _P), ("rank_counts_out", _P), ("route_ids_out", _P),
        ("stage_events", _P),
    ]


class BwdArgs(ctypes.Structure):
    """Mirror of struct mok_moe_bwd_args."""
    _fields_ = [
        ("dtype", _I32), ("d", _I32), ("E", _I32), ("k", _I32), ("I", _I32), ("e0", _I32),
        ("E_l", _I32), ("tokens_per_rank", _I32), ("T_pool", _I64), ("own_begin", _I64),
        ("T_own", _I32), ("n_shared", _I32), ("I_shared", _I32), ("route_rows_cap", _I64),
        ("x", _P), ("topk_idx", _P), ("topk_w", _P), ("w_gate", _P), ("w_up", _P),
        ("w_down", _P), ("ws_gate", _P), ("ws_up", _P), ("ws_down", _P),
        ("dy", _P), ("dy_slots", _P), ("dy_shared", _P),
        ("workspace", _P), ("workspace_bytes", _SZ),
        ("dx_slots", _P), ("dx_shared", _P), ("dx", _P), ("dtopk_w", _P),
        ("dw_gate", _P), ("dw_up", _P), ("dw_down", _P),
        ("dws_gate", _P), ("dws_up", _P), ("dws_down", _P),
    ]


class MoeW4Args(ctypes.Structure):
    """Mirror of struct mok_moe_w4_args."""
    _fields_ = [
        ("T", _I64), ("d", _I32), ("I", _I32), ("E", _I32), ("k", _I32), ("e0", _I32),
        ("E_l", _I32), ("group", _I32), ("x", _P), ("topk_idx", _P), ("topk_w", _P),
        ("gate_codes", _P), ("up_codes", _P), ("down_codes", _P),
        ("gate_scales", _P), ("up_scales", _P), ("down_scales", _P),
        ("gate_zeros", _P), ("up_zeros", _P), ("down_zeros", _P),
        ("y_in", _P), ("y", _P), ("workspace", _P), ("workspace_bytes", _SZ),
    ]


_lib.mok_status_string.argtypes = [ctypes.c_int]
_lib.mok_status_string.restype = ctypes.c_char_p
_lib.mok_version.argtypes = []
_lib.mok_version.restype = ctypes.c_char_p
_lib.mok_route.argtypes = [_P, _P, _I64, _I32, _I32, _I32, _I32, _P, _P, _P, _P]
_lib.mok_topk.argtypes = [_P, _I64, _I32, _I32, _P, _P, _P]
_lib.mok_dispatch_plan_workspace_bytes.argtypes = [_I64, _I32, _I32, ctypes.POINTER(_SZ)]
_lib.mok_dispatch_plan.argtypes = [_P, _I64, _I32, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P,
                                   _SZ, _P]
_lib.mok_dispatch_plan_noalloc.argtypes = [_P, _I64, _I32, _I32, _I32, _I32, _I32, _P, _P, _P,
                                           _P, _P]
_lib.mok_moe_workspace_bytes.argtypes = [ctypes.POINTER(MoeArgs), ctypes.POINTER(_SZ)]
_lib.mok_moe_forward.argtypes = [ctypes.POINTER(MoeArgs), _P]
_lib.mok_moe_workspace_region.argtypes = [ctypes.POINTER(MoeArgs), _I32, ctypes.POINTER(_SZ),
                                          ctypes.POINTER(_SZ), ctypes.POINTER(_I64)]
_lib.mok_moe_backward_workspace_bytes.argtypes = [ctypes.POINTER(BwdArgs), ctypes.POINTER(_SZ)]
_lib.mok_moe_backward.argtypes = [ctypes.POINTER(BwdArgs), _P]
_lib.mok_moe_backward_error.argtypes = [_P, ctypes.POINTER(BwdArgs), ctypes.POINTER(ctypes.c_uint32),
                                        _P]
_lib.mok_quantize_mxfp8.argtypes = [_P, _I64, _I32, _P, _P, _P]
_lib.mok_quantize_mxfp4.argtypes = [_P, _I64, _I32, _P, _P, _P]
_lib.mok_quantize_mxfp8_f32.argtypes = [_P, _I64, _I32, _P, _P, _P]
_lib.mok_quantize_mxfp4_f32.argtypes = [_P, _I64, _I32, _P, _P, _P]
_lib.mok_pull_gather.argtypes = [_P, _I64, _I32, _I32, _I32, _P, _P, _I32, _P, _P]
_lib.mok_push_dispatch.argtypes = [_P, _I64, _I32, _I32, _I32, _P, _I32, _I32, _I64, _P, _P, _P,
                                   _P]
_F32 = ctypes.c_float
_lib.mok_balance_loss_workspace_bytes.argtypes = [_I64, _I32, _I32, ctypes.POINTER(_SZ)]
_lib.mok_balance_loss.argtypes = [_P, _P, _I64, _I32, _I32, _P, _I32, _F32, _P, _P, _P, _P, _SZ, _P]
_lib.mok_balance_loss_backward.argtypes = [_P, _P, _I64, _I32, _I32, _P, _I32, _F32, _P, _P, _P]
_lib.mok_rmsnorm.argtypes = [_P, _P, _P, _I64, _I32, _I32, _F32, _P, _P, _P, _P, _P, _P]
_lib.mok_rmsnorm_backward_workspace_bytes.argtypes = [_I64, _I32, ctypes.POINTER(_SZ)]
_lib.mok_rmsnorm_backward.argtypes = [_P, _P, _P, _P, _P, _I64, _I32, _I32, _P, _P, _P, _SZ, _P]
_lib.mok_route_backward_workspace_bytes.argtypes = [_I64, _I32, _I32, _I32, ctypes.POINTER(_SZ)]
_lib.mok_route_backward.argtypes = [_P] * 7 + [_I64] + [_I32] * 4 + [_P, _P, _P, _SZ, _P]
_lib.mok_mx_gemm_workspace_bytes.argtypes = [_I64, _I64, _I32, ctypes.POINTER(_SZ)]
_lib.mok_mx_gemm.argtypes = [_P, _P, _I32, _P, _P, _I32, _I64, _I64, _I32, _I32, _P, _P, _SZ, _P]
_RULE = [_I32, _P, _I32, _I32, _I32, _I32, _F32]     # score, bias, groups, renorm, scale
_lib.mok_topk_scored.argtypes = [_P, _I64, _I32, _I32] + _RULE + [_P, _P, _P]
_lib.mok_route_scored.argtypes = [_P, _P, _I64] + [_I32] * 4 + _RULE + [_P] * 4
_lib.mok_topk_scored_backward.argtypes = [_P] * 4 + [_I64] + [_I32] * 4 + [_F32, _P, _P]
_lib.mok_gated_norm.argtypes = ([_P, _P, _P, _I32, _P, _P, _I64, _I32, _I32] + [_F32] * 3 + [_P] * 5)
_lib.mok_gated_norm_backward_workspace_bytes.argtypes = [_I64, _I32, ctypes.POINTER(_SZ)]
_lib.mok_gated_norm_backward.argtypes = ([_P] * 6 + [_I32] + [_P] * 3 + [_I64, _I32, _I32, _F32, _F32]
                                         + [_P] * 6 + [_SZ, _P])
_lib.mok_quantize_int4.argtypes = [_P, _I64, _I32, _I32, _P, _P, _P, _P]
_lib.mok_w4_gemm.argtypes = [_P] * 4 + [_I64, _I64, _I32, _I32, _I32, _P, _P]
_lib.mok_moe_w4_workspace_bytes.argtypes = [ctypes.POINTER(MoeW4Args), ctypes.POINTER(_SZ)]
_lib.mok_moe_w4_forward.argtypes = [ctypes.POINTER(MoeW4Args), _P]
_lib.mok_get_device_error.argtypes = [_P, ctypes.POINTER(ctypes.c_uint32), _P]
for _n in EXPORTS:
    if _n not in ("mok_status_string", "mok_version"):
        getattr(_lib, _n).restype = ctypes.c_int


def status_string(status: int) -> str:
    return _lib.mok_status_string(status).decode()


def version() -> str:
    return _lib.mok_version().decode()


def _check(fn: str, status: int) -> None:
    if status != MOK_OK:
        raise MokError(fn, status)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream=None, dev=None):
    if stream is not None:
        return getattr(stream, "cuda_stream", stream)
    import torch
    if dev is None:
        dev = torch.cuda.current_device()
    # the current stream's handle (building the Stream object around it costs 2.7 us a call)
    return torch._C._cuda_getCurrentRawStream(dev)


# ------------------------------------------------------------------------ entry points

def mok_route(x, w_router, k: int, logits, topk_idx, topk_w, stream=None) -> None:
    """Router projection + top-k + weights (x [T,d] and w_router [E,d]: float32 or bf16)."""
    import torch
    T, d = x.shape
    E = w_router.shape[0]
    io = MOK_FP32 if x.dtype == torch.float32 else MOK_BF16
    _check("mok_route", _lib.mok_route(_ptr(x), _ptr(w_router), T, d, E, k, io, _ptr(logits),
                                       _ptr(topk_idx), _ptr(topk_w), _stream(stream)))


def mok_topk(logits, k: int, topk_idx, topk_w, stream=None) -> None:
    T, E = logits.shape
    _check("mok_topk", _lib.mok_topk(_ptr(logits), T, E, k, _ptr(topk_idx), _ptr(topk_w),
                                     _stream(stream)))


def mok_dispatch_plan_workspace_bytes(T_pool: int, k: int, E_l: int) -> int:
    out = _SZ(0)
    _check("mok_dispatch_plan_workspace_bytes",
           _lib.mok_dispatch_plan_workspace_bytes(T_pool, k, E_l, ctypes.byref(out)))
    return out.value


def mok_dispatch_plan(topk_idx, E: int, e0: int, E_l: int, tokens_per_rank: int, counts, offsets,
                      rank_counts, route_ids, ws, stream=None) -> None:
    T, k = topk_idx.shape
    _check("mok_dispatch_plan",
           _lib.mok_dispatch_plan(_ptr(topk_idx), T, k, E, e0, E_l, tokens_per_rank, _ptr(counts),
                                  _ptr(offsets), _ptr(rank_counts), _ptr(route_ids), _ptr(ws),
                                  ws.numel() * ws.element_size(), _stream(stream)))


def mok_dispatch_plan_noalloc(topk_idx, E: int, e0: int, E_l: int, tokens_per_rank: int, counts,
                              offsets, rank_counts, route_ids, stream=None) -> None:
    """mok_dispatch_plan with the library's fixed device scratch (no workspace argument)."""
    T, k = topk_idx.shape
    _check("mok_dispatch_plan_noalloc",
           _lib.mok_dispatch_plan_noalloc(_ptr(topk_idx), T, k, E, e0, E_l, tokens_per_rank,
                                          _ptr(counts), _ptr(offsets), _ptr(rank_counts),
                                          _ptr(route_ids), _stream(stream)))


def mok_moe_workspace_bytes(args: MoeArgs) -> int:
    out = _SZ(0)
    _check("mok_moe_workspace_bytes", _lib.mok_moe_workspace_bytes(ctypes.byref(args),
                                                                   ctypes.byref(out)))
    return out.value


def mok_moe_forward(args: MoeArgs, stream=None) -> None:
    _check("mok_moe_forward", _lib.mok_moe_forward(ctypes.byref(args), _stream(stream)))


def mok_moe_workspace_region(args: MoeArgs, region: int):
    """(byte offset, bytes, rows R) of an intermediate inside the forward's workspace."""
    off, n, rows = _SZ(0), _SZ(0), _I64(0)
    _check("mok_moe_workspace_region",
           _lib.mok_moe_workspace_region(ctypes.byref(args), region, ctypes.byref(off),
                                         ctypes.byref(n), ctypes.byref(rows)))
    return off.value, n.value, rows.value


def _io(x):
    import torch
    return MOK_FP32 if x.dtype == torch.float32 else MOK_BF16


def mok_pull_gather(x, k: int, route_ids, offsets, buf, stream=None) -> None:
    """buf[i] = x[route_ids[i] // k] for the plan's rows (E_l = offsets.numel() - 1)."""
    T, d = x.shape
    _check("mok_pull_gather", _lib.mok_pull_gather(_ptr(x), T, d, k, _io(x), _ptr(route_ids),
                                                   _ptr(offsets), offsets.numel() - 1,
                                                   _ptr(buf), _stream(stream)))


def mok_push_dispatch(x, topk_idx, e0: int, fill, buf, src_route, stream=None) -> None:
    """Atomic-slot push of every local route's row into buf [E_l, capacity, d]."""
    T, d = x.shape
    k = topk_idx.shape[1]
    E_l, cap = buf.shape[0], buf.shape[1]
    _check("mok_push_dispatch",
           _lib.mok_push_dispatch(_ptr(x), T, d, k, _io(x), _ptr(topk_idx), e0, E_l, cap,
                                  _ptr(fill), _ptr(buf), _ptr(src_route), _stream(stream)))


def mok_quantize_mxfp8(src_bf16, codes, scales, stream=None) -> None:
    rows, K = src_bf16.shape
    _check("mok_quantize_mxfp8", _lib.mok_quantize_mxfp8(_ptr(src_bf16), rows, K, _ptr(codes),
                                                         _ptr(scales), _stream(stream)))


def mok_quantize_mxfp4(src_bf16, codes, scales, stream=None) -> None:
    """MXFP4 along rows: codes [rows, K/2] (two E2M1 codes a byte), scales [rows, K/32]."""
    rows, K = src_bf16.shape
    _check("mok_quantize_mxfp4", _lib.mok_quantize_mxfp4(_ptr(src_bf16), rows, K, _ptr(codes),
                                                         _ptr(scales), _stream(stream)))


def mok_quantize_mxfp8_f32(src_f32, codes, scales, stream=None) -> None:
    """MXFP8 of float32 rows: codes [rows, K], scales [rows, K/32]."""
    rows, K = src_f32.shape
    _check("mok_quantize_mxfp8_f32", _lib.mok_quantize_mxfp8_f32(
        _ptr(src_f32), rows, K, _ptr(codes), _ptr(scales), _stream(stream)))


def mok_quantize_mxfp4_f32(src_f32, codes, scales, stream=None) -> None:
    """MXFP4 of float32 rows: codes [rows, K/2], scales [rows, K/32]."""
    rows, K = src_f32.shape
    _check("mok_quantize_mxfp4_f32", _lib.mok_quantize_mxfp4_f32(
        _ptr(src_f32), rows, K, _ptr(codes), _ptr(scales), _stream(stream)))


def mok_get_device_error(workspace, stream=None) -> int:
    err = ctypes.c_uint32(0)
    _check("mok_get_device_error", _lib.mok_get_device_error(_ptr(workspace), ctypes.byref(err),
                                                             _stream(stream)))
    return err.value


# ------------------------------------------------------- operators around the layer
#
# These check what they marshal: a tensor of another type or shape, a strided one, or one on
# another device than the first raises MokError (MOK_EINVAL) before anything is enqueued. The work
# goes to the tensors' own device: its current stream, or `stream`, which must belong to it.

def _refuse(fn: str):
    raise MokError(fn, MOK_EINVAL)


def _arg(fn: str, t, dtype, shape, dev: int):
    """Pointer of t (None: NULL): contiguous, of this dtype and shape, on GPU dev."""
    if t is None:
        return None
    if (t.dtype is dtype and t.shape == shape and t.get_device() == dev >= 0
            and t.is_contiguous()):
        return t.data_ptr()
    _refuse(fn)


def _scratch(fn: str, ws, dev: int):
    """(pointer, bytes) of a workspace tensor of any dtype."""
    if ws is None:
        return None, 0
    if ws.get_device() != dev or not ws.is_contiguous():
        _refuse(fn)
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _enqueue(fn: str, dev: int, f, args, stream) -> None:
    """f(*args, stream) with GPU dev current."""
    import torch
    if torch.cuda.current_device() == dev:
        status = f(*args, _stream(stream, dev))
    else:
        with torch.cuda.device(dev):
            status = f(*args, _stream(stream, dev))
    if status != MOK_OK:
        raise MokError(fn, status)


def _io_of(fn: str, t) -> int:
    import torch
    if t.dtype is torch.bfloat16:
        return MOK_BF16
    if t.dtype is not torch.float32:
        _refuse(fn)
    return MOK_FP32


def mok_balance_loss_workspace_bytes(T: int, E: int, n_seq: int = 1) -> int:
    out = _SZ(0)
    _check("mok_balance_loss_workspace_bytes",
           _lib.mok_balance_loss_workspace_bytes(T, E, n_seq, ctypes.byref(out)))
    return out.value


def mok_balance_loss(logits, topk_idx, alpha: float, loss, counts, mean_prob, ws, *,
                     seq_offsets=None, stream=None) -> None:
    """Balance loss of logits [T, E] float32 and picks [T, k] int32: loss [1], counts [S, E] int32
    and mean probabilities [S, E] float32 of the S packed sequences of seq_offsets [S + 1] int32
    (None: one sequence). ws: mok_balance_loss_workspace_bytes(T, E, S) bytes."""
    import torch
    fn, f32, i32 = "mok_balance_loss", torch.float32, torch.int32
    if logits.dim() != 2 or topk_idx.dim() != 2 or (seq_offsets is not None
                                                    and seq_offsets.dim() != 1):
        _refuse(fn)
    (T, E), k, dev = logits.shape, topk_idx.shape[1], logits.get_device()
    S = 1 if seq_offsets is None else seq_offsets.shape[0] - 1
    _enqueue(fn, dev, _lib.mok_balance_loss,
             (_arg(fn, logits, f32, (T, E), dev), _arg(fn, topk_idx, i32, (T, k), dev), T, E, k,
              _arg(fn, seq_offsets, i32, (S + 1,), dev), S, alpha, _arg(fn, loss, f32, (1,), dev),
              _arg(fn, counts, i32, (S, E), dev), _arg(fn, mean_prob, f32, (S, E), dev),
              *_scratch(fn, ws, dev)), stream)


def mok_balance_loss_backward(logits, counts, k: int, alpha: float, dloss, dlogits, *,
                              seq_offsets=None, stream=None) -> None:
    """Gradient of mok_balance_loss for the logits: dlogits [T, E] float32 (overwritten), with the
    forward's counts and the upstream gradient dloss [1] (both on the device)."""
    import torch
    fn, f32, i32 = "mok_balance_loss_backward", torch.float32, torch.int32
    if logits.dim() != 2 or (seq_offsets is not None and seq_offsets.dim() != 1):
        _refuse(fn)
    (T, E), dev = logits.shape, logits.get_device()
    S = 1 if seq_offsets is None else seq_offsets.shape[0] - 1
    _enqueue(fn, dev, _lib.mok_balance_loss_backward,
             (_arg(fn, logits, f32, (T, E), dev), _arg(fn, counts, i32, (S, E), dev), T, E, k,
              _arg(fn, seq_offsets, i32, (S + 1,), dev), S, alpha, _arg(fn, dloss, f32, (1,), dev),
              _arg(fn, dlogits, f32, (T, E), dev)), stream)


def mok_rmsnorm(x, weight, eps: float, *, residual=None, h=None, rstd=None, y=None, codes=None,
                scales=None, stream=None) -> None:
    """h = x + residual, y = h / rms(h) * weight for rows x [T, d] float32 or bf16. Outputs, those
    that are given: h, y [T, d], rstd [T] float32, y in MXFP8 as codes [T, d] and scales
    [T, d / 32] uint8."""
    import torch
    fn, u8 = "mok_rmsnorm", torch.uint8
    if x.dim() != 2:
        _refuse(fn)
    (T, d), t, dev, io = x.shape, x.dtype, x.get_device(), _io_of(fn, x)
    rows = (T, d)
    _enqueue(fn, dev, _lib.mok_rmsnorm,
             (_arg(fn, x, t, rows, dev), _arg(fn, residual, t, rows, dev),
              _arg(fn, weight, t, (d,), dev), T, d, io, eps, _arg(fn, h, t, rows, dev),
              _arg(fn, rstd, torch.float32, (T,), dev), _arg(fn, y, t, rows, dev),
              _arg(fn, codes, u8, rows, dev), _arg(fn, scales, u8, (T, d // 32), dev)), stream)


def mok_rmsnorm_backward_workspace_bytes(T: int, d: int) -> int:
    out = _SZ(0)
    _check("mok_rmsnorm_backward_workspace_bytes",
           _lib.mok_rmsnorm_backward_workspace_bytes(T, d, ctypes.byref(out)))
    return out.value


def mok_rmsnorm_backward(dy, h, rstd, weight, dx, dweight=None, ws=None, *, dh=None,
                         stream=None) -> None:
    """Backward of mok_rmsnorm: dx [T, d] (the gradient of x and of residual; dh: what reaches h
    from the residual stream) and dweight [d] float32 (with ws of
    mok_rmsnorm_backward_workspace_bytes(T, d) bytes)."""
    import torch
    fn, f32 = "mok_rmsnorm_backward", torch.float32
    if dy.dim() != 2:
        _refuse(fn)
    (T, d), t, dev, io = dy.shape, dy.dtype, dy.get_device(), _io_of(fn, dy)
    rows = (T, d)
    _enqueue(fn, dev, _lib.mok_rmsnorm_backward,
             (_arg(fn, dy, t, rows, dev), _arg(fn, h, t, rows, dev), _arg(fn, rstd, f32, (T,), dev),
              _arg(fn, weight, t, (d,), dev), _arg(fn, dh, t, rows, dev), T, d, io,
              _arg(fn, dx, t, rows, dev), _arg(fn, dweight, f32, (d,), dev),
              *_scratch(fn, ws, dev)), stream)


def mok_route_backward_workspace_bytes(T: int, d: int, E: int, dtype) -> int:
    import torch
    out = _SZ(0)
    io = {torch.float32: MOK_FP32, torch.bfloat16: MOK_BF16}.get(dtype, -1)
    _check("mok_route_backward_workspace_bytes",
           _lib.mok_route_backward_workspace_bytes(T, d, E, io, ctypes.byref(out)))
    return out.value


def mok_route_backward(x, w_router, topk_idx, topk_w, dtopk_w, dx=None, dw_router=None, ws=None, *,
                       dlogits=None, dx_in=None, stream=None) -> None:
    """Gradients through mok_route with the picks held fixed: dx [T, d] (dx_in added) and
    dw_router [E, d] float32 (with ws of mok_route_backward_workspace_bytes(T, d, E, x.dtype)
    bytes), from dtopk_w [T, k] and, where given, dlogits [T, E]; with topk_idx, topk_w and dtopk_w
    None from dlogits alone."""
    import torch
    fn, f32 = "mok_route_backward", torch.float32
    if x.dim() != 2 or w_router.dim() != 2 or (topk_idx is not None and topk_idx.dim() != 2):
        _refuse(fn)
    (T, d), E, k = x.shape, w_router.shape[0], 1 if topk_idx is None else topk_idx.shape[1]
    t, dev, io = x.dtype, x.get_device(), _io_of(fn, x)
    _enqueue(fn, dev, _lib.mok_route_backward,
             (_arg(fn, x, t, (T, d), dev), _arg(fn, w_router, t, (E, d), dev),
              _arg(fn, topk_idx, torch.int32, (T, k), dev), _arg(fn, topk_w, f32, (T, k), dev),
              _arg(fn, dtopk_w, f32, (T, k), dev), _arg(fn, dlogits, f32, (T, E), dev),
              _arg(fn, dx_in, t, (T, d), dev), T, d, E, k, io, _arg(fn, dx, t, (T, d), dev),
              _arg(fn, dw_router, f32, (E, d), dev), *_scratch(fn, ws, dev)), stream)


def mok_mx_gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    out = _SZ(0)
    _check("mok_mx_gemm_workspace_bytes",
           _lib.mok_mx_gemm_workspace_bytes(M, N, K, ctypes.byref(out)))
    return out.value


def mok_mx_gemm(a_codes, a_scales, b_codes, b_scales, c, ws=None, *, stream=None) -> None:
    """c [M, N] (bf16 or float32) = A B^T of quantised rows: codes [rows, K] (MXFP8) or
    [rows, K / 2] (MXFP4) and scales [rows, K / 32], all uint8, as
    mok_quantize_mxfp8 / mok_quantize_mxfp4 write them; the format of each operand is
    read from its shapes. ws: mok_mx_gemm_workspace_bytes(M, N, K) bytes."""
    import torch
    fn, u8 = "mok_mx_gemm", torch.uint8
    if a_scales.dim() != 2 or b_scales.dim() != 2 or a_codes.dim() != 2 or b_codes.dim() != 2:
        _refuse(fn)
    (M, nb), N, dev = a_scales.shape, b_scales.shape[0], a_codes.get_device()
    K, ca, cb = 32 * nb, a_codes.shape[1], b_codes.shape[1]
    out = {torch.bfloat16: MOK_BF16, torch.float32: MOK_FP32}.get(c.dtype)
    if out is None or ca not in (K, K // 2) or cb not in (K, K // 2):
        _refuse(fn)
    _enqueue(fn, dev, _lib.mok_mx_gemm,
             (_arg(fn, a_codes, u8, (M, ca), dev), _arg(fn, a_scales, u8, (M, nb), dev),
              MOK_MXFP8 if ca == K else MOK_MXFP4, _arg(fn, b_codes, u8, (N, cb), dev),
              _arg(fn, b_scales, u8, (N, nb), dev), MOK_MXFP8 if cb == K else MOK_MXFP4, M, N, K,
              out, _arg(fn, c, c.dtype, (M, N), dev), *_scratch(fn, ws, dev)), stream)


def _score_of(fn: str, score: str) -> int:
    if score == "sigmoid":
        return MOK_SCORE_SIGMOID
    if score != "softmax":
        _refuse(fn)
    return MOK_SCORE_SOFTMAX


def mok_topk_scored(logits, k: int, topk_idx, topk_w, *, score: str = "sigmoid", bias=None,
                    n_groups: int = 1, topk_groups: int = 1, group_top: int = 2,
                    renorm: bool = True, scale: float = 1.0, stream=None) -> None:
    """The k experts of each row of logits [T, E] float32 by their scores ("sigmoid" or "softmax")
    plus bias [E] float32, out of the topk_groups best of n_groups groups: topk_idx [T, k] int32 and
    topk_w [T, k] float32 (scores, renormalised over the picks if renorm, times scale)."""
    import torch
    fn, f32 = "mok_topk_scored", torch.float32
    if logits.dim() != 2:
        _refuse(fn)
    (T, E), dev = logits.shape, logits.get_device()
    _enqueue(fn, dev, _lib.mok_topk_scored,
             (_arg(fn, logits, f32, (T, E), dev), T, E, k, _score_of(fn, score),
              _arg(fn, bias, f32, (E,), dev), n_groups, topk_groups, group_top, renorm, scale,
              _arg(fn, topk_idx, torch.int32, (T, k), dev), _arg(fn, topk_w, f32, (T, k), dev)),
             stream)


def mok_route_scored(x, w_router, k: int, logits, topk_idx, topk_w, *, score: str = "sigmoid",
                     bias=None, n_groups: int = 1, topk_groups: int = 1, group_top: int = 2,
                     renorm: bool = True, scale: float = 1.0, stream=None) -> None:
    """Router projection of x [T, d] and w_router [E, d] (float32 or bf16), as mok_route's, into
    logits [T, E] float32, then the choice of mok_topk_scored."""
    import torch
    fn, f32 = "mok_route_scored", torch.float32
    if x.dim() != 2 or w_router.dim() != 2:
        _refuse(fn)
    (T, d), E, t, dev, io = x.shape, w_router.shape[0], x.dtype, x.get_device(), _io_of(fn, x)
    _enqueue(fn, dev, _lib.mok_route_scored,
             (_arg(fn, x, t, (T, d), dev), _arg(fn, w_router, t, (E, d), dev), T, d, E, k, io,
              _score_of(fn, score), _arg(fn, bias, f32, (E,), dev), n_groups, topk_groups, group_top,
              renorm, scale, _arg(fn, logits, f32, (T, E), dev),
              _arg(fn, topk_idx, torch.int32, (T, k), dev), _arg(fn, topk_w, f32, (T, k), dev)),
             stream)


def mok_topk_scored_backward(logits, topk_idx, dtopk_w, dlogits, *, score: str = "sigmoid",
                             renorm: bool = True, scale: float = 1.0, dlogits_in=None,
                             stream=None) -> None:
    """Gradient of mok_topk_scored's weights for the logits with the picks held fixed: dlogits
    [T, E] float32 (overwritten; dlogits_in, which may be the same tensor, added) from dtopk_w
    [T, k] float32."""
    import torch
    fn, f32 = "mok_topk_scored_backward", torch.float32
    if logits.dim() != 2 or topk_idx.dim() != 2:
        _refuse(fn)
    (T, E), k, dev = logits.shape, topk_idx.shape[1], logits.get_device()
    _enqueue(fn, dev, _lib.mok_topk_scored_backward,
             (_arg(fn, logits, f32, (T, E), dev), _arg(fn, topk_idx, torch.int32, (T, k), dev),
              _arg(fn, dtopk_w, f32, (T, k), dev), _arg(fn, dlogits_in, f32, (T, E), dev), T, E, k,
              _score_of(fn, score), renorm, scale, _arg(fn, dlogits, f32, (T, E), dev)), stream)


def _gate_shape(fn: str, gate, rows):
    """(gate_per_row, shape) of a gate [d] for all rows or [T, d] of its own for each."""
    if gate is not None and gate.dim() == 2:
        return 1, rows
    return 0, rows[1:]


def mok_gated_norm(y, residual, eps: float, h, *, w_post=None, gate=None, w_pre=None, n=None,
                   rstd_y=None, rstd_h=None, alpha: float = 1.0, beta: float = 1.0,
                   stream=None) -> None:
    """h = alpha residual + beta gate norm(y) w_post and n = norm(h) w_pre, for rows y [T, d] float32
    or bf16; gate [d] or [T, d]; w_post None: y itself, gate None: 1, w_pre None: no n. rstd_y,
    rstd_h [T] float32: for the backward."""
    import torch
    fn, f32 = "mok_gated_norm", torch.float32
    if y.dim() != 2:
        _refuse(fn)
    rows, t, dev, io = tuple(y.shape), y.dtype, y.get_device(), _io_of(fn, y)
    (T, d), (per, shape) = rows, _gate_shape(fn, gate, rows)
    _enqueue(fn, dev, _lib.mok_gated_norm,
             (_arg(fn, y, t, rows, dev), _arg(fn, w_post, t, (d,), dev),
              _arg(fn, gate, t, shape, dev), per, _arg(fn, residual, t, rows, dev),
              _arg(fn, w_pre, t, (d,), dev), T, d, io, eps, alpha, beta,
              _arg(fn, h, t, rows, dev), _arg(fn, n, t, rows, dev), _arg(fn, rstd_y, f32, (T,), dev),
              _arg(fn, rstd_h, f32, (T,), dev)), stream)


def mok_gated_norm_backward_workspace_bytes(T: int, d: int) -> int:
    out = _SZ(0)
    _check("mok_gated_norm_backward_workspace_bytes",
           _lib.mok_gated_norm_backward_workspace_bytes(T, d, ctypes.byref(out)))
    return out.value


def mok_gated_norm_backward(dh, y, dres=None, dy=None, ws=None, *, dn=None, h=None, gate=None,
                            w_post=None, w_pre=None, rstd_y=None, rstd_h=None, dgate=None,
                            dw_post=None, dw_pre=None, alpha: float = 1.0, beta: float = 1.0,
                            stream=None) -> None:
    """Backward of mok_gated_norm from dh (None: nothing reaches h but through n) and dn: dres, dy
    [T, d], dgate ([T, d] in the rows' type for such a gate, [d] float32 for one of all rows), dw_post
    and dw_pre [d] float32, those that are given; ws: mok_gated_norm_backward_workspace_bytes(T, d)
    bytes where a sum over the rows is wanted."""
    import torch
    fn, f32 = "mok_gated_norm_backward", torch.float32
    if y.dim() != 2:
        _refuse(fn)
    rows, t, dev, io = tuple(y.shape), y.dtype, y.get_device(), _io_of(fn, y)
    (T, d), (per, shape) = rows, _gate_shape(fn, gate, rows)
    _enqueue(fn, dev, _lib.mok_gated_norm_backward,
             (_arg(fn, dh, t, rows, dev), _arg(fn, dn, t, rows, dev), _arg(fn, y, t, rows, dev),
              _arg(fn, h, t, rows, dev), _arg(fn, w_post, t, (d,), dev),
              _arg(fn, gate, t, shape, dev), per, _arg(fn, w_pre, t, (d,), dev),
              _arg(fn, rstd_y, f32, (T,), dev), _arg(fn, rstd_h, f32, (T,), dev), T, d, io, alpha, beta,
              _arg(fn, dres, t, rows, dev), _arg(fn, dy, t, rows, dev),
              _arg(fn, dgate, t if per else f32, shape, dev), _arg(fn, dw_post, f32, (d,), dev),
              _arg(fn, dw_pre, f32, (d,), dev), *_scratch(fn, ws, dev)), stream)


def _w4_args(fn: str, codes, scales, zeros, lead, dev: int):
    """(N, K, group, three pointers) of a 4-bit weight: codes lead + [N, K / 2] uint8, scales lead +
    [N, K / group] bf16 and, unless None, zeros uint8 of the scales' shape."""
    import torch
    n = len(lead)
    if codes.dim() != n + 2 or scales.dim() != n + 2 or scales.shape[-1] < 1:
        _refuse(fn)
    N, K, ng = codes.shape[-2], 2 * codes.shape[-1], scales.shape[-1]
    shape = (*lead, N, ng)
    return (N, K, K // ng if K % ng == 0 else -1, _arg(fn, codes, torch.uint8, (*lead, N, K // 2), dev),
            _arg(fn, scales, torch.bfloat16, shape, dev), _arg(fn, zeros, torch.uint8, shape, dev))


def mok_quantize_int4(src_bf16, codes, scales, zeros=None, stream=None) -> None:
    """4-bit codes [rows, K / 2] uint8 of rows [rows, K] bf16, two a byte, with scales
    [rows, K / group] bf16 and, if given, zero points uint8 of the same shape; the group (32, 64 or
    128) is read from the shapes."""
    import torch
    fn = "mok_quantize_int4"
    if src_bf16.dim() != 2:
        _refuse(fn)
    (rows, K), dev = src_bf16.shape, src_bf16.get_device()
    N, K4, g, c, s, z = _w4_args(fn, codes, scales, zeros, (), dev)
    if (N, K4) != (rows, K):
        _refuse(fn)
    _enqueue(fn, dev, _lib.mok_quantize_int4,
             (_arg(fn, src_bf16, torch.bfloat16, (rows, K), dev), rows, K, g, c, s, z), stream)


def mok_w4_gemm(x, codes, scales, out, *, zeros=None, stream=None) -> None:
    """out [M, N] (bf16 or float32) = x W^T for x [M, K] bf16 and a weight of 4-bit codes
    [N, K / 2] uint8 with scales [N, K / group] bf16 and zeros (None: 8)."""
    import torch
    fn = "mok_w4_gemm"
    io = {torch.bfloat16: MOK_BF16, torch.float32: MOK_FP32}.get(out.dtype)
    if x.dim() != 2 or io is None:
        _refuse(fn)
    M, dev = x.shape[0], x.get_device()
    N, K, g, c, s, z = _w4_args(fn, codes, scales, zeros, (), dev)
    _enqueue(fn, dev, _lib.mok_w4_gemm,
             (_arg(fn, x, torch.bfloat16, (M, K), dev), c, s, z, M, N, K, g, io,
              _arg(fn, out, out.dtype, (M, N), dev)), stream)


def mok_moe_w4_workspace_bytes(args: MoeW4Args) -> int:
    out = _SZ(0)
    _check("mok_moe_w4_workspace_bytes",
           _lib.mok_moe_w4_workspace_bytes(ctypes.byref(args), ctypes.byref(out)))
    return out.value


def mok_moe_w4_forward(args: MoeW4Args, stream=None) -> None:
    _check("mok_moe_w4_forward", _lib.mok_moe_w4_forward(ctypes.byref(args), _stream(stream)))


# ------------------------------------------------------------------------ layer helper

_DT = {"fp32": MOK_FP32, "bf16": MOK_BF16, "mxfp8": MOK_MXFP8, "mxfp4": MOK_MXFP4}


class MoeLayer:
    """Holds the argument struct, the workspace and the outputs of one layer configuration.

    Shapes follow mok_moe_args. `forward()` enqueues one mok_moe_forward on the current stream.
    """

    def __init__(self, *, dtype: str, d: int, E: int, k: int, I: int, e0: int, E_l: int,
                 tokens_per_rank: int, T_pool: int, own_begin: int, T_own: int, n_shared: int,
                 I_shared: int, minibatch_rows: int, ring_rows: int, x, w_gate, w_up, w_down,
                 ws_gate=None, ws_up=None, ws_down=None, w_router=None, topk_idx=None,
                 topk_w=None, flags: int = 0, keep_intermediates: bool = False, device="cuda"):
        import torch
        self._keep = [x, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, w_router, topk_idx, topk_w]
        odt = torch.float32 if dtype == "fp32" else torch.bfloat16
        a = MoeArgs()
        a.dtype, a.d, a.E, a.k, a.I = _DT[dtype], d, E, k, I
        a.e0, a.E_l, a.tokens_per_rank = e0, E_l, tokens_per_rank
        a.T_pool, a.own_begin, a.T_own = T_pool, own_begin, T_own
        a.n_shared, a.I_shared = n_shared, I_shared
        a.minibatch_rows, a.ring_rows, a.flags = minibatch_rows, ring_rows, flags
        a.x, a.w_router = _ptr(x), _ptr(w_router)
        a.topk_idx_in, a.topk_w_in = _ptr(topk_idx), _ptr(topk_w)
        a.w_gate, a.w_up, a.w_down = _ptr(w_gate), _ptr(w_up), _ptr(w_down)
        a.ws_gate, a.ws_up, a.ws_down = _ptr(ws_gate), _ptr(ws_up), _ptr(ws_down)
        self.y_slots = torch.empty((T_pool * k, d), dtype=odt, device=device)
        # at least one row, so that a share with no own tokens still passes a valid pointer
        ysh = torch.empty((max(1, T_own), d), dtype=odt, device=device) if n_shared else None
        self.y_shared = ysh[:T_own] if n_shared else None
        self.y = torch.empty((T_pool, d), dtype=odt, device=device) if E_l == E else None
        a.y_slots, a.y_shared, a.y = _ptr(self.y_slots), _ptr(ysh), _ptr(self.y)
        self._keep.append(ysh)
        self.inter = {}
        if keep_intermediates:
            i32 = dict(dtype=torch.int32, device=device)
            if w_router is not None:
                self.inter["logits"] = torch.empty((T_pool, E), dtype=torch.float32, device=device)
                self.inter["topk_idx"] = torch.empty((T_pool, k), **i32)
                self.inter["topk_w"] = torch.empty((T_pool, k), dtype=torch.float32, device=device)
                a.logits_out = _ptr(self.inter["logits"])
                a.topk_idx_out = _ptr(self.inter["topk_idx"])
                a.topk_w_out = _ptr(self.inter["topk_w"])
            self.inter["counts"] = torch.empty(E_l, **i32)
            self.inter["offsets"] = torch.empty(E_l + 1, **i32)
            self.inter["rank_counts"] = torch.empty((E_l, T_pool // tokens_per_rank), **i32)
            self.inter["route_ids"] = torch.empty(max(1, T_pool * min(k, E_l)), **i32)
            a.counts_out = _ptr(self.inter["counts"])
            a.offsets_out = _ptr(self.inter["offsets"])
            a.rank_counts_out = _ptr(self.inter["rank_counts"])
            a.route_ids_out = _ptr(self.inter["route_ids"])
        nbytes = mok_moe_workspace_bytes(a)
        self.workspace = torch.empty(max(1, nbytes), dtype=torch.uint8, device=device)
        a.workspace, a.workspace_bytes = _ptr(self.workspace), nbytes
        self.args = a

    def forward(self, stream=None) -> None:
        mok_moe_forward(self.args, stream)

    def device_error(self, stream=None) -> int:
        return mok_get_device_error(self.workspace, stream)

    def region(self, region: int):
        """(uint8 view of the workspace bytes of an intermediate, rows R); see
        mok_moe_workspace_region. Read it after the forward has finished."""
        off, n, rows = mok_moe_workspace_region(self.args, region)
        return self.workspace[off:off + n], rows


class MoeBackward:
    """Argument struct, workspace and outputs of one backward configuration (mok_moe_backward).

    Whole layer: pass dy [T_pool, d]. Share: dy_slots [T_pool*k, d] and dy_shared [T_own, d].
    Outputs: dx_slots, dx_shared, dx (whole layer), dtopk_w, dw_* and dws_* (float32). A share's
    dtopk_w is zero at the routes of other experts, so that mok_route_backward gives its part of the
    gradients: the shares' parts add up to the layer's."""

    def __init__(self, *, d: int, E: int, k: int, I: int, e0: int, E_l: int,
                 tokens_per_rank: int, T_pool: int, own_begin: int, T_own: int, n_shared: int,
                 I_shared: int, x, topk_idx, topk_w, w_gate, w_up, w_down, ws_gate=None,
                 ws_up=None, ws_down=None, dy=None, dy_slots=None, dy_shared=None,
                 route_rows_cap: int = 0, device="cuda"):
        import torch
        self._keep = [x, topk_idx, topk_w, w_gate, w_up, w_down, ws_gate, ws_up, ws_down, dy,
                      dy_slots, dy_shared]
        a = BwdArgs()
        a.dtype, a.d, a.E, a.k, a.I, a.e0, a.E_l = MOK_BF16, d, E, k, I, e0, E_l
        a.tokens_per_rank, a.T_pool, a.own_begin, a.T_own = tokens_per_rank, T_pool, own_begin, T_own
        a.n_shared, a.I_shared, a.route_rows_cap = n_shared, I_shared, route_rows_cap
        a.x, a.topk_idx, a.topk_w = _ptr(x), _ptr(topk_idx), _ptr(topk_w)
        a.w_gate, a.w_up, a.w_down = _ptr(w_gate), _ptr(w_up), _ptr(w_down)
        a.ws_gate, a.ws_up, a.ws_down = _ptr(ws_gate), _ptr(ws_up), _ptr(ws_down)
        a.dy, a.dy_slots, a.dy_shared = _ptr(dy), _ptr(dy_slots), _ptr(dy_shared)
        bf, f32 = dict(dtype=torch.bfloat16, device=device), dict(dtype=torch.float32, device=device)
        self.dx_slots = torch.empty((T_pool * k, d), **bf)
        sh = n_shared > 0 and T_own > 0
        self.dx_shared = torch.empty((T_own, d), **bf) if sh else None
        self.dx = torch.empty((T_pool, d), **bf) if E_l == E else None
        self.dtopk_w = torch.empty((T_pool, k), **f32)
        self.dw_gate = torch.empty((E_l, I, d), **f32)
        self.dw_up = torch.empty((E_l, I, d), **f32)
        self.dw_down = torch.empty((E_l, d, I), **f32)
        if n_shared:
            self.dws_gate = torch.empty((n_shared, I_shared, d), **f32)
            self.dws_up = torch.empty((n_shared, I_shared, d), **f32)
            self.dws_down = torch.empty((n_shared, d, I_shared), **f32)
        else:
            self.dws_gate = self.dws_up = self.dws_down = None
        a.dx_slots, a.dx_shared, a.dx = _ptr(self.dx_slots), _ptr(self.dx_shared), _ptr(self.dx)
        a.dtopk_w = _ptr(self.dtopk_w)
        a.dw_gate, a.dw_up, a.dw_down = _ptr(self.dw_gate), _ptr(self.dw_up), _ptr(self.dw_down)
        a.dws_gate, a.dws_up, a.dws_down = (_ptr(self.dws_gate), _ptr(self.dws_up),
                                            _ptr(self.dws_down))
        n = _SZ(0)
        _check("mok_moe_backward_workspace_bytes",
               _lib.mok_moe_backward_workspace_bytes(ctypes.byref(a), ctypes.byref(n)))
        self.workspace = torch.empty(max(1, n.value), dtype=torch.uint8, device=device)
        a.workspace, a.workspace_bytes = _ptr(self.workspace), n.value
        self.args = a

    def backward(self, stream=None) -> None:
        if self.args.E_l < self.args.E:        # the call writes dtopk_w at its local routes only
            import torch
            with torch.cuda.stream(stream if stream is None
                                   else torch.cuda.ExternalStream(_stream(stream))):
                self.dtopk_w.zero_()
        _check("mok_moe_backward", _lib.mok_moe_backward(ctypes.byref(self.args), _stream(stream)))

    def device_error(self, stream=None) -> int:
        err = ctypes.c_uint32(0)
        _check("mok_moe_backward_error",
               _lib.mok_moe_backward_error(_ptr(self.workspace), ctypes.byref(self.args),
                                           ctypes.byref(err), _stream(stream)))
        return err.value


class MoeW4Layer:
    """The routed experts on 4-bit weights (mok_moe_w4_forward): holds the weights of the local
    experts [e0, e0 + E_l) and a workspace for up to max_tokens tokens a call.

    gate, up, down: (codes, scales, zeros or None), codes [E_l, I, d / 2] ([E_l, d, I / 2] for down)
    uint8, scales [E_l, I, d / group] ([E_l, d, I / group]) bf16, zeros uint8 like the scales. Calls
    share the workspace: they must be ordered on one stream (captured graphs of a layer too)."""

    def __init__(self, gate, up, down, *, E: int, k: int, e0: int = 0, max_tokens: int):
        import torch
        fn = "MoeW4Layer"
        if gate[0].dim() != 3:
            _refuse(fn)
        E_l, dev = gate[0].shape[0], gate[0].get_device()
        a = MoeW4Args()
        for name, w in (("gate", gate), ("up", up), ("down", down)):
            N, K, g, c, s, z = _w4_args(fn, *w, (E_l,), dev)
            if name == "gate":
                a.I, a.d, a.group = N, K, g
            if ((a.d, a.I) if name == "down" else (a.I, a.d)) != (N, K) or g != a.group:
                _refuse(fn)
            setattr(a, name + "_codes", c)
            setattr(a, name + "_scales", s)
            setattr(a, name + "_zeros", z)
        a.E, a.k, a.e0, a.E_l, a.T = E, k, e0, E_l, max_tokens
        self._keep, self._dev, self.max_tokens = (gate, up, down), dev, max_tokens
        n = mok_moe_w4_workspace_bytes(a)
        self.workspace = torch.empty(n, dtype=torch.uint8, device=gate[0].device)
        a.workspace, a.workspace_bytes = _ptr(self.workspace), n
        self.args = a

    def forward(self, x, topk_idx, topk_w, y, *, y_in=None, stream=None) -> None:
        """y [T, d] bf16 = y_in + the local experts' weighted FFNs of x [T, d] bf16, T <= max_tokens;
        topk_idx [T, k] int32, topk_w [T, k] float32. y may be x or y_in."""
        import torch
        fn, a, dev, bf = "mok_moe_w4_forward", self.args, self._dev, torch.bfloat16
        T = x.shape[0]
        if T > self.max_tokens:
            _refuse(fn)
        a.T, rows, picks = T, (T, a.d), (T, a.k)
        a.x, a.y, a.y_in = _arg(fn, x, bf, rows, dev), _arg(fn, y, bf, rows, dev), _arg(fn, y_in, bf, rows, dev)
        a.topk_idx = _arg(fn, topk_idx, torch.int32, picks, dev)
        a.topk_w = _arg(fn, topk_w, torch.float32, picks, dev)
        _enqueue(fn, dev, _lib.mok_moe_w4_forward, (ctypes.byref(a),), stream)
