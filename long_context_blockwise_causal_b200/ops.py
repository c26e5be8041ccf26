"""ctypes binding of liblwm_blockattn.so (argument marshalling only).

Every step of the attention path runs in the library's CUDA kernels; this
module turns torch tensors into device pointers, sizes and the current
stream, and turns status codes into exceptions. It never computes
anything itself and has no fallback: without the built library (or on a
tensor that is not on a CUDA device) it raises.
"""

from __future__ import annotations

import ctypes
import functools
import os
from typing import NamedTuple

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)),
                         "liblwm_blockattn.so")
_lib = None

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA, \
    ERR_TIMEOUT, ERR_PRECONDITION = range(7)
DTYPE_BF16, DTYPE_FP32 = 0, 1
QK_BF16, QK_BF16X3 = 0, 1
ROPE_INTERLEAVED, ROPE_HALF = 0, 1
KV8_E4M3, KV8_INT8 = 0, 1
TILE_EMPTY, TILE_PARTIAL, TILE_FULL = 0, 1, 2
BLOCK = 128
HEAD_DIM = 128

_vp = ctypes.c_void_p
_i = ctypes.c_int
_sz = ctypes.c_size_t
_d = ctypes.c_double

_SIGS = {
    "lwm_blockattn_fwd_workspace_size": (_sz, [_i] * 9),
    "lwm_blockattn_bwd_workspace_size": (_sz, [_i] * 9),
    "lwm_blockattn_fwd": (_i, [_vp, _vp, _vp, _vp, _vp, _d, _i, _i, _i,
                               _i, _i, _i, _i, _i, _i, _i, _vp, _vp, _vp,
                               _sz, _vp]),
    "lwm_blockattn_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _d,
                               _i, _i, _i, _i, _i, _i, _i, _i, _i, _i, _vp,
                               _vp, _vp, _vp, _sz, _vp]),
    "lwm_blockattn_classify": (_i, [_vp, _i, _i, _i, _i, _vp, _vp, _vp,
                                    _vp]),
    "lwm_blockattn_rope_table": (_i, [_d, _i, _i, _vp, _vp]),
    "lwm_blockattn_visibility": (_i, [_vp, _vp, _i, _i, _i, _i, _i, _i, _i]
                                 + [_vp] * 13),
    "lwm_blockattn_check_inputs": (_i, [_vp, _vp, _i, _i, _i,
                                        ctypes.POINTER(_i), _vp]),
    "lwm_blockattn_last_status": (_i, [_vp]),
    "lwm_status_string": (ctypes.c_char_p, [_i]),
    "lwm_blockattn_version": (_i, []),
    "lwm_blockattn_kernel_launches": (ctypes.c_uint64, []),
    "lwm_blockattn_selftest_wait_timeout": (_i, [ctypes.c_uint64, _vp]),
    "lwm_blockattn_rope_apply": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i,
                                      _i, _vp, _vp]),
    "lwm_blockattn_decode_workspace_size": (_sz, [_i, _i, _i, _i]),
    "lwm_blockattn_decode": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i, _i,
                                  _i, _i, _i, _i, _i, _vp, _vp, _vp, _sz,
                                  _vp]),
    "lwm_blockattn_fwd_noalloc": (_i, [_vp, _vp, _vp, _vp, _vp, _d, _i, _i,
                                       _i, _i, _i, _i, _i, _i, _i, _i, _vp,
                                       _vp, _vp]),
    "lwm_blockattn_fwd_block_workspace_size": (_sz, [_i] * 6),
    "lwm_blockattn_fwd_block": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i,
                                     _d, _i, _vp, _i, _i, _i, _i, _i, _i,
                                     _vp, _vp, _vp, _sz, _vp]),
    "lwm_blockattn_merge": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i,
                                 _vp]),
    "lwm_blockattn_bwd_delta": (_i, [_vp, _vp, _i, _i, _i, _i, _i, _vp,
                                     _vp]),
    "lwm_blockattn_bwd_block_workspace_size": (_sz, [_i] * 5),
    "lwm_blockattn_bwd_block": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                                     _i, _i, _i, _i, _i, _i, _i, _vp, _vp,
                                     _vp, _vp, _sz, _vp]),
    "lwm_blockattn_grad_finish": (_i, [_vp, _vp, _vp, _i, _i, _i, _i, _i, _i,
                                       _i, _vp, _vp]),
    "lwm_kv8_write": (_i, [_vp] * 6 + [_i] * 9 + [_vp] * 6),
    "lwm_kv8_read": (_i, [_vp] * 6 + [_i] * 7 + [_vp] * 3),
    "lwm_kv8_select": (_i, [_vp] * 7 + [_i] * 11 + [_vp] * 3),
    "lwm_kv8_decode_workspace_size": (_sz, [_i] * 6),
    "lwm_kv8_decode": (_i, [_vp] * 9 + [_i, _vp] + [_i] * 9
                       + [_vp, _vp, _vp, _sz, _vp]),
    "lwm_blockffn_workspace_size": (_sz, [_i, _i]),
    "lwm_blockffn_fwd": (_i, [_vp, _vp, _vp, _vp, _i, _i, _i, _i, _i, _vp,
                              _vp, _sz, _vp]),
    "lwm_blockffn_bwd_workspace_size": (_sz, [_i, _i]),
    "lwm_blockffn_bwd": (_i, [_vp, _vp, _vp, _vp, _vp, _i, _i, _i, _i, _i,
                              _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
}


class LwmError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)} ({status})")


def lib() -> ctypes.CDLL:
    """Load the shared library once; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"{_LIB_PATH} is missing; build it with "
                "`python -m long_context_blockwise_causal_b200.build`")
        L = ctypes.CDLL(_LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _lib = L
    return _lib


def exported_symbols():
    return list(_SIGS)


def status_string(status: int) -> str:
    return lib().lwm_status_string(int(status)).decode()


def _check(status: int, where: str):
    if status != OK:
        raise LwmError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code_of(dtype) -> int:
    if dtype == torch.bfloat16:
        return DTYPE_BF16
    if dtype == torch.float32:
        return DTYPE_FP32
    raise TypeError(f"unsupported dtype {dtype}")


def _dtype_code(t: torch.Tensor) -> int:
    return _dtype_code_of(t.dtype)


def _qk_code(qk_precision) -> int:
    if qk_precision in (QK_BF16, "bf16"):
        return QK_BF16
    if qk_precision in (QK_BF16X3, "bf16x3"):
        return QK_BF16X3
    raise ValueError(f"qk_precision {qk_precision!r}")


def _layout_code(rope_layout) -> int:
    if rope_layout in (ROPE_INTERLEAVED, "interleaved"):
        return ROPE_INTERLEAVED
    if rope_layout in (ROPE_HALF, "half", "rotate_half"):
        return ROPE_HALF
    raise ValueError(f"rope_layout {rope_layout!r}")


def _expect(where, name, t, shape, dtype=None):
    """Shapes and dtypes are checked here, before any pointer reaches the
    library: the C calls take sizes from q (or x) and trust every other
    buffer to match them."""
    if t is None:
        return
    if tuple(t.shape) != tuple(shape) or (dtype is not None
                                          and t.dtype != dtype):
        raise LwmError(ERR_INVALID_ARG,
                       f"{where}: {name} is {tuple(t.shape)} {t.dtype}, "
                       f"expected {tuple(shape)}"
                       + ("" if dtype is None else f" {dtype}"))


def _expect_dims(where, name, t, dims):
    if t.dim() != dims:
        raise LwmError(ERR_INVALID_ARG,
                       f"{where}: {name} must have {dims} dimensions")


def _same_device(where, *ts):
    devs = {t.device for t in ts if t is not None}
    if len(devs) > 1:
        raise LwmError(ERR_INVALID_ARG, f"{where}: tensors on {sorted(map(str, devs))}")


def _check_attn(where, q, k, v, segment_ids, positions, lse=None,
                like_q=()):
    """q, k, v (and like_q) [B,N,H,D] of one dtype; ids and positions
    [B,N] int32; lse [B,H,N] fp32."""
    _expect_dims(where, "q", q, 4)
    B, N, H, _ = q.shape
    for name, t in (("k", k), ("v", v)) + tuple(like_q):
        _expect(where, name, t, q.shape, q.dtype)
    _expect(where, "segment_ids", segment_ids, (B, N), torch.int32)
    _expect(where, "positions", positions, (B, N), torch.int32)
    _expect(where, "lse", lse, (B, H, N), torch.float32)
    _same_device(where, q, k, v, segment_ids, positions, lse,
                 *(t for _, t in like_q))


def _need_cuda(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous CUDA tensors")


def fwd_workspace_size(B, N, H, max_pos, dtype=torch.bfloat16,
                       qk_precision="bf16", D=HEAD_DIM, block_q=BLOCK,
                       block_k=BLOCK) -> int:
    return int(lib().lwm_blockattn_fwd_workspace_size(
        B, N, H, D, block_q, block_k, max_pos, _dtype_code_of(dtype),
        _qk_code(qk_precision)))


def bwd_workspace_size(B, N, H, max_pos, dtype=torch.bfloat16,
                       qk_precision="bf16", D=HEAD_DIM, block_q=BLOCK,
                       block_k=BLOCK) -> int:
    return int(lib().lwm_blockattn_bwd_workspace_size(
        B, N, H, D, block_q, block_k, max_pos, _dtype_code_of(dtype),
        _qk_code(qk_precision)))


def _workspace(nbytes, device, workspace):
    if workspace is None:
        return torch.empty(max(nbytes, 1), dtype=torch.uint8, device=device)
    if workspace.numel() * workspace.element_size() < nbytes:
        raise LwmError(ERR_WORKSPACE, "workspace")
    return workspace


def fwd(q, k, v, segment_ids, positions, theta, max_pos=None,
        qk_precision="bf16", out=None, lse=None, workspace=None,
        stream=None, block_q=BLOCK, block_k=BLOCK, rope_layout="interleaved"):
    """Forward pass. Returns (out [B,N,H,D] in q's dtype, lse [B,H,N] fp32).
    ``rope_layout``: "interleaved" pairs (2k, 2k+1) or "half" (k, k+D/2),
    the rotate-half layout of Hugging Face Llama checkpoints."""
    _check_attn("fwd", q, k, v, segment_ids, positions, lse,
                like_q=(("out", out),))
    _need_cuda(q, k, v, segment_ids, positions, out, lse, workspace)
    B, N, H, D = q.shape
    if max_pos is None:
        max_pos = int(positions.max().item()) + 1 if positions.numel() else 1
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    ws = _workspace(fwd_workspace_size(B, N, H, max_pos, q.dtype,
                                       qk_precision, D, block_q, block_k),
                    q.device, workspace)
    st = lib().lwm_blockattn_fwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(segment_ids), _ptr(positions),
        float(theta), block_q, block_k, int(max_pos), B, N, H, D,
        _dtype_code(q), _qk_code(qk_precision), _layout_code(rope_layout),
        _ptr(out), _ptr(lse), _ptr(ws), ws.numel(), _stream(stream))
    _check(st, "lwm_blockattn_fwd")
    return out, lse


def fwd_noalloc(q, k, v, segment_ids, positions, theta, max_pos,
                qk_precision="bf16", out=None, lse=None, stream=None,
                block_q=BLOCK, block_k=BLOCK, rope_layout="interleaved"):
    """Forward through lwm_blockattn_fwd_noalloc: the library's own fixed
    scratch array replaces the workspace (see the header for its limits).
    ``out``/``lse`` are allocated here only if the caller passes none."""
    _check_attn("fwd_noalloc", q, k, v, segment_ids, positions, lse,
                like_q=(("out", out),))
    _need_cuda(q, k, v, segment_ids, positions, out, lse)
    B, N, H, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    # the library uses the scratch array of the current device: make it the
    # tensors' device (and take that device's stream by default)
    with torch.cuda.device(q.device):
        st = lib().lwm_blockattn_fwd_noalloc(
            _ptr(q), _ptr(k), _ptr(v), _ptr(segment_ids), _ptr(positions),
            float(theta), block_q, block_k, int(max_pos), B, N, H, D,
            _dtype_code(q), _qk_code(qk_precision),
            _layout_code(rope_layout), _ptr(out), _ptr(lse),
            _stream(stream))
    _check(st, "lwm_blockattn_fwd_noalloc")
    return out, lse


def bwd(q, k, v, out, dout, lse, segment_ids, positions, theta,
        max_pos=None, qk_precision="bf16", dq=None, dk=None, dv=None,
        workspace=None, stream=None, block_q=BLOCK, block_k=BLOCK,
        rope_layout="interleaved"):
    """Backward pass. Returns (dq, dk, dv) in q's dtype (dq, dk in the
    layout q and k came in)."""
    _check_attn("bwd", q, k, v, segment_ids, positions, lse,
                like_q=(("out", out), ("dout", dout), ("dq", dq), ("dk", dk),
                        ("dv", dv)))
    _need_cuda(q, k, v, out, dout, lse, segment_ids, positions, dq, dk, dv,
               workspace)
    B, N, H, D = q.shape
    if max_pos is None:
        max_pos = int(positions.max().item()) + 1 if positions.numel() else 1
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    ws = _workspace(bwd_workspace_size(B, N, H, max_pos, q.dtype,
                                       qk_precision, D, block_q, block_k),
                    q.device, workspace)
    st = lib().lwm_blockattn_bwd(
        _ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse),
        _ptr(segment_ids), _ptr(positions), float(theta), block_q, block_k,
        int(max_pos), B, N, H, D, _dtype_code(q), _qk_code(qk_precision),
        _layout_code(rope_layout), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(ws),
        ws.numel(), _stream(stream))
    _check(st, "lwm_blockattn_bwd")
    return dq, dk, dv


def fwd_block_workspace_size(B, Nq, Nk, H, max_pos, D=HEAD_DIM) -> int:
    return int(lib().lwm_blockattn_fwd_block_workspace_size(
        B, Nq, Nk, H, D, max_pos))


def fwd_block(q, k_rot, v, seg_q, pos_q, seg_k, q_off, k_off, theta,
              max_pos, out=None, lse=None, workspace=None, stream=None,
              rope_layout="interleaved", table=None):
    """Partial forward of query rows [q_off, q_off+Nq) against the rotated
    key / value rows [k_off, k_off+Nk) of the same packed sequence (one step
    of a ring). Returns (out [B,Nq,H,D] bf16, lse [B,H,Nq] fp32); rows that
    see no key get (0, -inf). k_rot and v have q's heads: those of a grouped
    cache are repeated by the caller."""
    w = "fwd_block"
    _expect_dims(w, "q", q, 4)
    _expect_dims(w, "k_rot", k_rot, 4)
    B, Nq, H, D = q.shape
    Nk = k_rot.shape[1]
    for name, t, shape in (("q", q, q.shape), ("k_rot", k_rot, (B, Nk, H, D)),
                           ("v", v, (B, Nk, H, D)), ("out", out, q.shape)):
        _expect(w, name, t, shape, torch.bfloat16)
    for name, t, shape in (("seg_q", seg_q, (B, Nq)), ("pos_q", pos_q, (B, Nq)),
                           ("seg_k", seg_k, (B, Nk))):
        _expect(w, name, t, shape, torch.int32)
    _expect(w, "lse", lse, (B, H, Nq), torch.float32)
    if table is not None:
        _expect_dims(w, "table", table, 3)
        _expect(w, "table", table, (table.shape[0], D // 2, 2), torch.float32)
    _same_device(w, q, k_rot, v, seg_q, pos_q, seg_k, out, lse, workspace,
                 table)
    _need_cuda(q, k_rot, v, seg_q, pos_q, seg_k, out, lse, workspace, table)
    if table is not None and table.shape[0] < max_pos:
        raise ValueError("rope table shorter than max_pos")
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((B, H, Nq), dtype=torch.float32, device=q.device)
    ws = _workspace(fwd_block_workspace_size(B, Nq, Nk, H, max_pos, D),
                    q.device, workspace)
    st = lib().lwm_blockattn_fwd_block(
        _ptr(q), _ptr(k_rot), _ptr(v), _ptr(seg_q), _ptr(pos_q), _ptr(seg_k),
        int(q_off), int(k_off), float(theta), int(max_pos), _ptr(table), B,
        Nq, Nk, H, D, _layout_code(rope_layout), _ptr(out), _ptr(lse),
        _ptr(ws), ws.numel(), _stream(stream))
    _check(st, "lwm_blockattn_fwd_block")
    return out, lse


def merge(out, lse, out_part, lse_part, stream=None):
    """In place: fold the partial (out_part, lse_part) over another key set
    into (out, lse) with the log-sum-exp rule. Returns (out, lse)."""
    _need_cuda(out, lse, out_part, lse_part)
    B, N, H, D = out.shape
    st = lib().lwm_blockattn_merge(_ptr(out), _ptr(lse), _ptr(out_part),
                                   _ptr(lse_part), B, N, H, D,
                                   _dtype_code(out), _stream(stream))
    _check(st, "lwm_blockattn_merge")
    return out, lse


def bwd_delta(out, dout, delta=None, stream=None):
    """D = rowsum(dout * out) as fp32 [B,H,N]."""
    _need_cuda(out, dout, delta)
    B, N, H, D = out.shape
    if delta is None:
        delta = torch.empty((B, H, N), dtype=torch.float32, device=out.device)
    st = lib().lwm_blockattn_bwd_delta(_ptr(out), _ptr(dout), B, N, H, D,
                                       _dtype_code(out), _ptr(delta),
                                       _stream(stream))
    _check(st, "lwm_blockattn_bwd_delta")
    return delta


def bwd_block_workspace_size(B, Nq, Nk, H, D=HEAD_DIM) -> int:
    return int(lib().lwm_blockattn_bwd_block_workspace_size(B, Nq, Nk, H, D))


def bwd_block(q_rot, k_rot, v, dout, lse, delta, seg_q, seg_k, q_off, k_off,
              dq_acc, dk_acc, dv_acc, workspace=None, stream=None):
    """Partial backward of a query chunk against a key chunk: adds into the
    fp32 accumulators dq_acc [B,Nq,H,D], dk_acc and dv_acc [B,Nk,H,D]
    (rotated frame, no 1/sqrt(D); finish them with grad_finish)."""
    _need_cuda(q_rot, k_rot, v, dout, lse, delta, seg_q, seg_k, dq_acc,
               dk_acc, dv_acc, workspace)
    B, Nq, H, D = q_rot.shape
    Nk = k_rot.shape[1]
    ws = _workspace(bwd_block_workspace_size(B, Nq, Nk, H, D), q_rot.device,
                    workspace)
    st = lib().lwm_blockattn_bwd_block(
        _ptr(q_rot), _ptr(k_rot), _ptr(v), _ptr(dout), _ptr(lse),
        _ptr(delta), _ptr(seg_q), _ptr(seg_k), int(q_off), int(k_off), B, Nq,
        Nk, H, D, _ptr(dq_acc), _ptr(dk_acc), _ptr(dv_acc), _ptr(ws),
        ws.numel(), _stream(stream))
    _check(st, "lwm_blockattn_bwd_block")
    return dq_acc, dk_acc, dv_acc


def grad_finish(acc, positions=None, table=None, out=None, stream=None,
                rope_layout="interleaved"):
    """bf16 gradient from an fp32 accumulator: R(-pos) acc / sqrt(D) when
    positions are given (dq, dk), else acc (dv)."""
    _need_cuda(acc, positions, table, out)
    B, N, H, D = acc.shape
    if out is None:
        out = torch.empty(acc.shape, dtype=torch.bfloat16, device=acc.device)
    st = lib().lwm_blockattn_grad_finish(
        _ptr(acc), _ptr(positions), _ptr(table),
        0 if table is None else table.shape[0], B, N, H, D, DTYPE_BF16,
        _layout_code(rope_layout), _ptr(out), _stream(stream))
    _check(st, "lwm_blockattn_grad_finish")
    return out


def _check_ffn(where, x, w_gate, w_up, w_down, like_x=(), grads=()):
    """x (and like_x) [T, Dm]; Wg, Wu [F, Dm] and Wd [Dm, F] of x's dtype;
    grads: (name, tensor, shape) in fp32."""
    _expect_dims(where, "x", x, 2)
    _expect_dims(where, "w_gate", w_gate, 2)
    T, Dm = x.shape
    F = w_gate.shape[0]
    _expect(where, "w_gate", w_gate, (F, Dm), x.dtype)
    _expect(where, "w_up", w_up, (F, Dm), x.dtype)
    _expect(where, "w_down", w_down, (Dm, F), x.dtype)
    for name, t in like_x:
        _expect(where, name, t, (T, Dm), x.dtype)
    for name, t, shape in grads:
        _expect(where, name, t, shape, torch.float32)
    _same_device(where, x, w_gate, w_up, w_down, *(t for _, t in like_x),
                 *(t for _, t, _ in grads))


def ffn_workspace_size(chunk, F) -> int:
    return int(lib().lwm_blockffn_workspace_size(chunk, F))


def ffn_fwd(x, w_gate, w_up, w_down, chunk=8192, y=None, workspace=None,
            stream=None):
    """Blockwise SwiGLU MLP: y = (silu(x Wg^T) * (x Wu^T)) Wd^T, `chunk`
    tokens at a time. x [T, Dm]; Wg, Wu [F, Dm]; Wd [Dm, F]; bf16."""
    _check_ffn("ffn_fwd", x, w_gate, w_up, w_down, like_x=(("y", y),))
    _need_cuda(x, w_gate, w_up, w_down, y, workspace)
    T, Dm = x.shape
    F = w_gate.shape[0]
    y = torch.empty_like(x) if y is None else y
    c = max(1, min(int(chunk), T))
    ws = _workspace(ffn_workspace_size(c, F), x.device, workspace)
    st = lib().lwm_blockffn_fwd(
        _ptr(x), _ptr(w_gate), _ptr(w_up), _ptr(w_down), T, Dm, F, int(chunk),
        _dtype_code(x), _ptr(y), _ptr(ws), ws.numel(), _stream(stream))
    _check(st, "lwm_blockffn_fwd")
    return y


def ffn_bwd_workspace_size(chunk, F) -> int:
    return int(lib().lwm_blockffn_bwd_workspace_size(chunk, F))


def ffn_bwd(x, w_gate, w_up, w_down, dy, chunk=8192, dx=None, dw_gate=None,
            dw_up=None, dw_down=None, workspace=None, stream=None):
    """Backward of ffn_fwd: returns (dx bf16 [T, Dm], dWg, dWu fp32 [F, Dm],
    dWd fp32 [Dm, F]); h and g are recomputed chunk by chunk."""
    if x.dim() == 2 and w_gate.dim() == 2:
        Fg, Dmx = w_gate.shape[0], x.shape[1]
        _check_ffn("ffn_bwd", x, w_gate, w_up, w_down,
                   like_x=(("dy", dy), ("dx", dx)),
                   grads=(("dw_gate", dw_gate, (Fg, Dmx)),
                          ("dw_up", dw_up, (Fg, Dmx)),
                          ("dw_down", dw_down, (Dmx, Fg))))
    else:
        _check_ffn("ffn_bwd", x, w_gate, w_up, w_down)
    _need_cuda(x, w_gate, w_up, w_down, dy, dx, dw_gate, dw_up, dw_down,
               workspace)
    T, Dm = x.shape
    F = w_gate.shape[0]
    dev = x.device
    dx = torch.empty_like(x) if dx is None else dx
    f32 = dict(dtype=torch.float32, device=dev)
    dw_gate = torch.empty((F, Dm), **f32) if dw_gate is None else dw_gate
    dw_up = torch.empty((F, Dm), **f32) if dw_up is None else dw_up
    dw_down = torch.empty((Dm, F), **f32) if dw_down is None else dw_down
    c = max(1, min(int(chunk), T))
    ws = _workspace(ffn_bwd_workspace_size(c, F), dev, workspace)
    st = lib().lwm_blockffn_bwd(
        _ptr(x), _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(dy), T, Dm, F,
        int(chunk), _dtype_code(x), _ptr(dx), _ptr(dw_gate), _ptr(dw_up),
        _ptr(dw_down), _ptr(ws), ws.numel(), _stream(stream))
    _check(st, "lwm_blockffn_bwd")
    return dx, dw_gate, dw_up, dw_down


def classify(segment_ids, block_q=BLOCK, block_k=BLOCK, with_class=True,
             stream=None):
    """Returns kv_lo, kv_hi [B,Tq] int32 and tile_class [B,Tq,Tk] uint8."""
    _need_cuda(segment_ids)
    B, N = segment_ids.shape
    tq = -(-N // block_q)
    tk = -(-N // block_k)
    dev = segment_ids.device
    lo = torch.empty((B, tq), dtype=torch.int32, device=dev)
    hi = torch.empty((B, tq), dtype=torch.int32, device=dev)
    cls = torch.empty((B, tq, tk), dtype=torch.uint8, device=dev) \
        if with_class else None
    st = lib().lwm_blockattn_classify(_ptr(segment_ids), B, N, block_q,
                                      block_k, _ptr(lo), _ptr(hi), _ptr(cls),
                                      _stream(stream))
    _check(st, "lwm_blockattn_classify")
    return lo, hi, cls


VISIBILITY_QUERY_VIEW = ("row_lo", "row_hi", "kv_lo", "kv_hi", "lo_max",
                         "hi_min")
VISIBILITY_KEY_VIEW = ("col_lo", "col_hi", "q_lo", "q_hi", "klo_max",
                       "khi_min")


def visibility(seg_q, seg_k=None, q_off=0, k_off=0, query_view=True,
               key_view=True, block_q=BLOCK, block_k=BLOCK, stream=None):
    """The metadata the attention kernels classify tiles with (see
    lwm_blockattn_visibility). seg_q [B,Nq] int32 ids of queries
    [q_off, q_off+Nq); seg_k [B,Nk] of keys [k_off, k_off+Nk) (default:
    seg_q, self-attention). Returns a dict of int32 tensors: per query row
    and per query block (query view), per key and per key block (key
    view)."""
    seg_k = seg_q if seg_k is None else seg_k
    _need_cuda(seg_q, seg_k)
    _expect_dims("visibility", "seg_q", seg_q, 2)
    _expect_dims("visibility", "seg_k", seg_k, 2)
    B, Nq = seg_q.shape
    Nk = seg_k.shape[1]
    _expect("visibility", "seg_q", seg_q, (B, Nq), torch.int32)
    _expect("visibility", "seg_k", seg_k, (B, Nk), torch.int32)
    _same_device("visibility", seg_q, seg_k)
    dev = seg_q.device
    tq, tk = -(-Nq // block_q), -(-Nk // block_k)
    shapes = dict(zip(VISIBILITY_QUERY_VIEW,
                      [(B, Nq)] * 2 + [(B, tq)] * 4))
    shapes.update(zip(VISIBILITY_KEY_VIEW, [(B, Nk)] * 2 + [(B, tk)] * 4))
    want = (VISIBILITY_QUERY_VIEW if query_view else ()) + \
        (VISIBILITY_KEY_VIEW if key_view else ())
    res = {n: torch.empty(shapes[n], dtype=torch.int32, device=dev)
           for n in want}
    ptrs = [_ptr(res.get(n)) for n in VISIBILITY_QUERY_VIEW +
            VISIBILITY_KEY_VIEW]
    st = lib().lwm_blockattn_visibility(_ptr(seg_q), _ptr(seg_k), B, Nq, Nk,
                                        int(q_off), int(k_off), block_q,
                                        block_k, *ptrs, _stream(stream))
    _check(st, "lwm_blockattn_visibility")
    return res


def rope_table(theta, max_pos, D=HEAD_DIM, device="cuda", stream=None):
    """The fp32 (cos, sin) table [max_pos, D/2, 2] the kernels use."""
    t = torch.empty((max_pos, D // 2, 2), dtype=torch.float32, device=device)
    st = lib().lwm_blockattn_rope_table(float(theta), D, max_pos, _ptr(t),
                                        _stream(stream))
    _check(st, "lwm_blockattn_rope_table")
    return t


def rope_apply(x, positions, table, stream=None, out=None,
               rope_layout="interleaved"):
    """R(pos) x (bf16 [B,N,H,D]) with a table from rope_table(), pairs as
    ``rope_layout`` says (the output keeps that layout)."""
    _need_cuda(x, positions, table, out)
    B, N, H, D = x.shape
    out = torch.empty_like(x) if out is None else out
    st = lib().lwm_blockattn_rope_apply(
        _ptr(x), _ptr(positions), _ptr(table), table.shape[0], B, N, H, D,
        _dtype_code(x), _layout_code(rope_layout), _ptr(out), _stream(stream))
    _check(st, "lwm_blockattn_rope_apply")
    return out


def decode_workspace_size(B, H, L, D=HEAD_DIM) -> int:
    return int(lib().lwm_blockattn_decode_workspace_size(B, H, D, L))


def decode(q, k_rot, v, kv_start, kv_len, q_pos, table, out=None, lse=None,
           workspace=None, stream=None, rope_layout="interleaved"):
    """One query token per (b, h) [B,H,D] against a cache of rotated keys
    and values [B,L,H,D]; returns (out [B,H,D], lse [B,H])."""
    _expect_dims("decode", "q", q, 3)
    _expect_dims("decode", "k_rot", k_rot, 4)
    _expect_dims("decode", "table", table, 3)
    Bq, Hq, Dq = q.shape
    kshape = (Bq, k_rot.shape[1], Hq, Dq)
    _expect("decode", "k_rot", k_rot, kshape, q.dtype)
    _expect("decode", "v", v, kshape, q.dtype)
    for name, t in (("kv_start", kv_start), ("kv_len", kv_len),
                    ("q_pos", q_pos)):
        _expect("decode", name, t, (Bq,), torch.int32)
    _expect("decode", "table", table, (table.shape[0], Dq // 2, 2),
            torch.float32)
    _expect("decode", "out", out, q.shape, q.dtype)
    _expect("decode", "lse", lse, (Bq, Hq), torch.float32)
    _same_device("decode", q, k_rot, v, kv_start, kv_len, q_pos, table, out,
                 lse)
    _need_cuda(q, k_rot, v, kv_start, kv_len, q_pos, table, out, lse,
               workspace)
    B, H, D = q.shape
    L = k_rot.shape[1]
    out = torch.empty_like(q) if out is None else out
    if lse is None:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    ws = _workspace(decode_workspace_size(B, H, L, D), q.device, workspace)
    st = lib().lwm_blockattn_decode(
        _ptr(q), _ptr(k_rot), _ptr(v), _ptr(kv_start), _ptr(kv_len),
        _ptr(q_pos), _ptr(table), table.shape[0], B, L, H, D, _dtype_code(q),
        _layout_code(rope_layout), _ptr(out), _ptr(lse), _ptr(ws), ws.numel(),
        _stream(stream))
    _check(st, "lwm_blockattn_decode")
    return out, lse


class Kv8Cache(NamedTuple):
    """An 8-bit KV cache: the caller's tensors, as the header lays them out.
    k, v [B,H,L,D] torch.float8_e4m3fn or torch.int8; k_scale, v_scale
    [B,H,ceil(L/128)] fp32; k_bounds [B,H,ceil(L/128),2,D] int8."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor
    k_bounds: torch.Tensor


_KV8_TYPES = {torch.float8_e4m3fn: KV8_E4M3, torch.int8: KV8_INT8}


def kv8_cache(B, L, H, dtype=torch.float8_e4m3fn, D=HEAD_DIM,
              device="cuda") -> Kv8Cache:
    """An empty (zeroed) cache of L slots and H heads per row."""
    if dtype not in _KV8_TYPES:
        raise TypeError(f"unsupported cache dtype {dtype}")
    n = -(-L // BLOCK)
    z = lambda shape, dt: torch.zeros(shape, dtype=dt, device=device)
    return Kv8Cache(z((B, H, L, D), dtype), z((B, H, L, D), dtype),
                    z((B, H, n), torch.float32), z((B, H, n), torch.float32),
                    z((B, H, n, 2, D), torch.int8))


def _kv8_sizes(where, cache):
    """(B, H, L, D, type code) of a cache whose k and v have them."""
    k = cache.k
    code = _KV8_TYPES.get(k.dtype)
    if code is None:
        raise LwmError(ERR_INVALID_ARG, f"{where}: cache.k is {k.dtype}")
    shape = k.shape
    if len(shape) != 4:
        _expect_dims(where, "cache.k", k, 4)
    B, H, L, D = shape
    return B, H, L, D, code


# Counts beyond a C int are refused: ctypes would pass on their low 32 bits.
_C_INT = 1 << 31


def _kv8_group(where, q, H):
    """Query heads of q [B,Hq,D], a multiple of the cache's H heads."""
    shape = q.shape
    if len(shape) != 3:
        _expect_dims(where, "q", q, 3)
    Hq = shape[1]
    if H and Hq % H:
        raise LwmError(ERR_INVALID_ARG,
                       f"{where}: {Hq} query heads over {H} cache heads")
    return Hq


def _kv8_ready(where, cache, sizes, table, tensors):
    """Shapes, types and placement of every tensor of a call, before any
    pointer reaches the library: the cache's, the table's and those of
    `tensors` (name, tensor or None, shape, dtype). Returns the device. These
    calls are short, so the usual case is one pass that finds nothing."""
    B, H, L, D = sizes
    k, v, ks, vs, kb = cache
    n = (L + BLOCK - 1) // BLOCK
    scales, dev = (B, H, n), k.get_device()
    every = (("cache.v", v, k.shape, k.dtype),
             ("cache.k_scale", ks, scales, torch.float32),
             ("cache.v_scale", vs, scales, torch.float32),
             ("cache.k_bounds", kb, (B, H, n, 2, D), torch.int8), *tensors)
    if table is not None:
        _expect_dims(where, "table", table, 3)
        every += (("table", table, (table.shape[0], D // 2, 2),
                   torch.float32),)
    for _, t, shape, dtype in every:
        if t is not None and (t.dtype is not dtype or t.shape != shape
                              or t.get_device() != dev
                              or not t.is_contiguous()):
            break
    else:
        if dev >= 0 and k.is_contiguous():
            return dev
    for name, t, shape, dtype in every:
        _expect(where, name, t, shape, dtype)
    everything = (k, *(t for _, t, _, _ in every))
    _same_device(where, *everything)
    _need_cuda(*everything)
    return dev


def _kv8_stream(where, cache, stream):
    """The context of a call on a stream that the caller names."""
    if stream.device != cache.k.device:
        raise LwmError(ERR_INVALID_ARG, f"{where}: the cache is on "
                       f"{cache.k.device}, the stream on {stream.device}")
    return torch.cuda.stream(stream)


def _kv8_call(name, call, dev, args):
    """call(*args, stream) with the tensors' device current, on that device's
    current stream."""
    # (the current stream's handle, without building a Stream object, which
    # would be 1.2 us of a 12 us call)
    handle = torch._C._cuda_getCurrentRawStream(dev)
    if torch.cuda.current_device() == dev:
        st = call(*args, handle)
    else:
        with torch.cuda.device(dev):
            st = call(*args, handle)
    if st != OK:
        raise LwmError(st, name)


def kv8_write(cache, k, v, positions, start, table, n_new=None,
              rope_layout="interleaved", stream=None):
    """Rotate and quantise k, v [B,T,H,D] bf16 into the cache at slots
    start[b] + t (in place; see the header for the block scales). ``n_new``
    [B]: new tokens of a padded row. Returns the cache."""
    if stream is not None:
        with _kv8_stream("kv8_write", cache, stream):
            return kv8_write(cache, k, v, positions, start, table, n_new,
                             rope_layout)
    w = "kv8_write"
    B, H, L, D, code = _kv8_sizes(w, cache)
    _expect_dims(w, "k", k, 4)
    T = k.shape[1]
    new = (B, T, H, D)
    dev = _kv8_ready(
        w, cache, (B, H, L, D), table,
        (("start", start, (B,), torch.int32),
         ("n_new", n_new, (B,), torch.int32),
         ("k", k, new, torch.bfloat16), ("v", v, new, torch.bfloat16),
         ("positions", positions, (B, T), torch.int32)))
    _kv8_call("lwm_kv8_write", lib().lwm_kv8_write, dev, (
        k.data_ptr(), v.data_ptr(), positions.data_ptr(), start.data_ptr(),
        None if n_new is None else n_new.data_ptr(), table.data_ptr(),
        table.shape[0], B, T, L, H, D, DTYPE_BF16, code,
        _layout_code(rope_layout), cache.k.data_ptr(), cache.v.data_ptr(),
        cache.k_scale.data_ptr(), cache.v_scale.data_ptr(),
        cache.k_bounds.data_ptr()))
    return cache


def kv8_read(cache, start, T, kv_len=None, k_rot=None, v=None, stream=None):
    """Slots start[b] .. start[b] + T - 1 of the cache as (k_rot, v) bf16
    [B,T,H,D], zeros outside [0, min(kv_len[b], L)); the layout fwd_block
    takes rotated keys and values in, where the queries have as many heads as
    the cache. Those of a grouped cache are repeated first, head i of the
    queries being given head i // (Hq // H):
    ``k_rot.repeat_interleave(Hq // H, 2)``."""
    if stream is not None:
        with _kv8_stream("kv8_read", cache, stream):
            return kv8_read(cache, start, T, kv_len, k_rot, v)
    w = "kv8_read"
    B, H, L, D, code = _kv8_sizes(w, cache)
    T = int(T)
    if not 0 <= T < _C_INT:
        raise LwmError(ERR_INVALID_ARG, f"{w}: T is {T}")
    shape = (B, T, H, D)
    dev = _kv8_ready(w, cache, (B, H, L, D), None,
                     (("start", start, (B,), torch.int32),
                      ("kv_len", kv_len, (B,), torch.int32),
                      ("k_rot", k_rot, shape, torch.bfloat16),
                      ("v", v, shape, torch.bfloat16)))
    if k_rot is None:
        k_rot = torch.empty(shape, dtype=torch.bfloat16, device=cache.k.device)
    if v is None:
        v = torch.empty_like(k_rot)
    _kv8_call("lwm_kv8_read", lib().lwm_kv8_read, dev, (
        cache.k.data_ptr(), cache.v.data_ptr(), cache.k_scale.data_ptr(),
        cache.v_scale.data_ptr(), start.data_ptr(),
        None if kv_len is None else kv_len.data_ptr(), B, T, L, H, D,
        DTYPE_BF16, code, k_rot.data_ptr(), v.data_ptr()))
    return k_rot, v


def kv8_select(q, cache, kv_start, kv_len, q_pos, table, n_select, n_sink=1,
               n_recent=1, blocks=None, scores=None,
               rope_layout="interleaved", stream=None):
    """The ``n_select`` blocks of 128 slots per (row, cache head) whose key
    bounds admit the largest scores for q [B,Hq,D]: (blocks int32, scores
    fp32) [B,H,n_select], ascending, (-1, -inf) behind a short list. The
    first ``n_sink`` and last ``n_recent`` visible blocks are always in.
    Scores are comparable within a call; times 448/127 (e4m3) or 1 (int8) and
    1/sqrt(D) they are in the units of lse (see the header)."""
    if stream is not None:
        with _kv8_stream("kv8_select", cache, stream):
            return kv8_select(q, cache, kv_start, kv_len, q_pos, table,
                              n_select, n_sink, n_recent, blocks, scores,
                              rope_layout)
    w = "kv8_select"
    B, H, L, D, _ = _kv8_sizes(w, cache)
    Hq = _kv8_group(w, q, H)
    K, n_sink, n_recent = int(n_select), int(n_sink), int(n_recent)
    if not (1 <= K < _C_INT and 0 <= n_sink < _C_INT
            and 0 <= n_recent < _C_INT):
        raise LwmError(ERR_INVALID_ARG, f"{w}: {K} blocks, the first "
                       f"{n_sink} and the last {n_recent} always")
    lists = (B, H, K)
    dev = _kv8_ready(
        w, cache, (B, H, L, D), table,
        (("kv_start", kv_start, (B,), torch.int32),
         ("kv_len", kv_len, (B,), torch.int32),
         ("q_pos", q_pos, (B,), torch.int32),
         ("q", q, (B, Hq, D), torch.bfloat16),
         ("blocks", blocks, lists, torch.int32),
         ("scores", scores, lists, torch.float32)))
    if blocks is None:
        blocks = kv_len.new_empty(lists)
    if scores is None:
        scores = cache.k_scale.new_empty(lists)
    _kv8_call("lwm_kv8_select", lib().lwm_kv8_select, dev, (
        q.data_ptr(), cache.k_bounds.data_ptr(), cache.k_scale.data_ptr(),
        kv_start.data_ptr(), kv_len.data_ptr(), q_pos.data_ptr(),
        table.data_ptr(), table.shape[0], B, L, Hq, H, D, DTYPE_BF16,
        _layout_code(rope_layout), K, n_sink, n_recent,
        blocks.data_ptr(), scores.data_ptr()))
    return blocks, scores


def kv8_decode_workspace_size(B, L, Hq, H, n_blocks=None, D=HEAD_DIM) -> int:
    sizes = (B, L, Hq, H, D, -1 if n_blocks is None else n_blocks)
    if not all(-_C_INT <= n < _C_INT for n in sizes):
        return 0                            # as any size the library refuses
    return int(lib().lwm_kv8_decode_workspace_size(*sizes))


@functools.lru_cache(maxsize=1024)
def _kv8_decode_bytes(dev, B, L, Hq, H, D, n_blocks):
    """The workspace's size on a device, of the sizes alone."""
    with torch.cuda.device(dev):
        return max(1, int(lib().lwm_kv8_decode_workspace_size(
            B, L, Hq, H, D, n_blocks)))


def kv8_decode(q, cache, kv_start, kv_len, q_pos, table, blocks=None,
               out=None, lse=None, workspace=None,
               rope_layout="interleaved", stream=None):
    """One query token per (row, head), q [B,Hq,D], against slots
    [kv_start[b], kv_len[b]) of an 8-bit cache, or only those of ``blocks``
    [B,H,n] (a list of kv8_select, strictly ascending). Query head i reads
    cache head i // (Hq // H). Returns (out [B,Hq,D], lse [B,Hq])."""
    if stream is not None:
        with _kv8_stream("kv8_decode", cache, stream):
            return kv8_decode(q, cache, kv_start, kv_len, q_pos, table,
                              blocks, out, lse, workspace, rope_layout)
    w = "kv8_decode"
    B, H, L, D, code = _kv8_sizes(w, cache)
    Hq = _kv8_group(w, q, H)
    K = -1
    if blocks is not None:
        _expect_dims(w, "blocks", blocks, 3)
        K = blocks.shape[2]
    dev = _kv8_ready(
        w, cache, (B, H, L, D), table,
        (("kv_start", kv_start, (B,), torch.int32),
         ("kv_len", kv_len, (B,), torch.int32),
         ("q_pos", q_pos, (B,), torch.int32),
         ("q", q, (B, Hq, D), torch.bfloat16),
         ("blocks", blocks, (B, H, K), torch.int32),
         ("out", out, (B, Hq, D), torch.bfloat16),
         ("lse", lse, (B, Hq), torch.float32),
         ("workspace", workspace, getattr(workspace, "shape", None),
          getattr(workspace, "dtype", None))))
    if workspace is None:                                      # int8: bytes
        workspace = cache.k_bounds.new_empty(
            _kv8_decode_bytes(dev, B, L, Hq, H, D, K))
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = cache.k_scale.new_empty((B, Hq))
    _kv8_call("lwm_kv8_decode", lib().lwm_kv8_decode, dev, (
        q.data_ptr(), cache.k.data_ptr(), cache.v.data_ptr(),
        cache.k_scale.data_ptr(), cache.v_scale.data_ptr(),
        kv_start.data_ptr(), kv_len.data_ptr(), q_pos.data_ptr(),
        None if blocks is None else blocks.data_ptr(), K, table.data_ptr(),
        table.shape[0], B, L, Hq, H, D, DTYPE_BF16, code,
        _layout_code(rope_layout), out.data_ptr(), lse.data_ptr(),
        workspace.data_ptr(), workspace.numel() * workspace.element_size()))
    return out, lse


def check_inputs(segment_ids, positions, max_pos, stream=None):
    """(ok, 1 + largest position). Synchronous."""
    _need_cuda(segment_ids, positions)
    B, N = segment_ids.shape
    mp = ctypes.c_int(0)
    st = lib().lwm_blockattn_check_inputs(_ptr(segment_ids), _ptr(positions),
                                          B, N, int(max_pos),
                                          ctypes.byref(mp), _stream(stream))
    if st not in (OK, ERR_PRECONDITION):
        _check(st, "lwm_blockattn_check_inputs")
    return st == OK, mp.value


def kernel_launches() -> int:
    """Kernels the library has launched in this process so far."""
    return int(lib().lwm_blockattn_kernel_launches())


def selftest_wait_timeout(limit_ns=20_000_000, stream=None):
    """Launch the bounded-wait self-test kernel (see the header)."""
    _check(lib().lwm_blockattn_selftest_wait_timeout(int(limit_ns),
                                                     _stream(stream)),
           "lwm_blockattn_selftest_wait_timeout")


def last_status(stream=None) -> int:
    return int(lib().lwm_blockattn_last_status(_stream(stream)))
