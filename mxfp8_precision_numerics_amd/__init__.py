"""FP8 / MXFP8 training numerics on MI355X (gfx950).

The functions below take torch tensors (PyTorch supplies device memory and the current HIP stream), allocate the
outputs, and call the C ABI of libmxq.so with raw pointers. All arithmetic happens in the library's gfx950 kernels.

  mx_quantize            MXFP8 row/column quantization (E4M3 payload, E8M0 scale per 32 values)
  pertensor_quantize     per-tensor current/delayed scaling to E4M3 or E5M2 (+ transposed copy)
  scaled_gemm            C = A B^T with FP8 operands (per-tensor or MX block scales), fp32 accumulate, bf16 out
  grouped_scaled_gemm    the MX GEMM over ragged expert row groups (and a strided-B form for the routed dgrad)
  grouped_wgrad_mx       the routed Wgrad: one MX contraction per expert over its token rows
  fp8_adam_step          precision-decoupled FP8 AdamW step (fp32 master, E4M3 m + scale, fp16 v, bf16 copy)
  swiglu_mx_quantize(_oriented), swiglu_backward_mx_quantize, route_weighted_mx_quantize
                         the routed MLP's fused elementwise + MX quantize steps (forward and backward)
  rmsnorm_mx_quantize, rmsnorm_backward_mx_checkpoint
                         RMSNorm with the residual's addition and an MXFP8 output, and its backward from an 8-bit
                         checkpoint of its input
  swiglu_mx_quantize_checkpoint, swiglu_backward_mx_checkpoint
                         SwiGLU + MX quantize with an 8-bit checkpoint of its input, and its backward from it
  moe_mx_few_tokens      the routed experts of up to 64 tokens, from router logits to the weighted sum
  int8_quantize_tokens   8-bit integers with one scale for each row (a token, or an output channel of a weight)
  int8_scaled_gemm, int8_grouped_gemm
                         C = A B^T of int8 operands with a scale for each token and output channel, optionally with SwiGLU
                         in the same pass; dense, or over ragged expert groups of any number of rows
  qk_norm_rope, qk_norm_rope_backward
                         RMSNorm of every query and key head with the rotation by position (on several axes) in one pass
"""
from __future__ import annotations

import ctypes as C
import functools
from typing import NamedTuple, Optional

import torch

from . import _lib
from ._lib import E4M3, E5M2, FLOOR, MX_BLOCK32, PER_TENSOR, RCEIL, AdamHParams, MXQError  # noqa: F401

__all__ = ["mx_quantize", "mx_quantize_ranged", "pertensor_quantize", "scaled_gemm", "scaled_gemm_ranged", "grouped_scaled_gemm", "fp8_adam_step",
           "swiglu_mx_quantize", "swiglu_mx_quantize_oriented", "swiglu_backward_mx_quantize", "route_weighted_mx_quantize",
           "grouped_scaled_gemm_strided", "grouped_wgrad_mx",
           "rmsnorm_mx_quantize", "rmsnorm_backward_mx_checkpoint", "swiglu_mx_quantize_checkpoint",
           "swiglu_backward_mx_checkpoint", "moe_mx_few_tokens", "RMSNormOut",
           "int8_quantize_tokens", "int8_scaled_gemm", "int8_grouped_gemm", "Int8Tensor",
           "qk_norm_rope", "qk_norm_rope_backward", "QKNormGrads",
           "workspace_bytes", "MXTensor", "AdamHParams", "MXQError", "E4M3", "E5M2", "RCEIL", "FLOOR",
           "PER_TENSOR", "MX_BLOCK32"]


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else C.c_void_p(t.data_ptr())


def _stream(device) -> C.c_void_p:
    return C.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _dev(t: torch.Tensor, dtype, name: str):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


class MXTensor(NamedTuple):
    """One MXFP8 tensor in both orientations: qdata and E8M0 scales travel together (either pair may be None)."""
    q_row: Optional[torch.Tensor]   # [rows][cols] uint8, blocks of 32 along each row
    s_row: Optional[torch.Tensor]   # [rows][cols/32] uint8
    q_col: Optional[torch.Tensor]   # [cols][rows] uint8, blocks of 32 down each column, stored transposed
    s_col: Optional[torch.Tensor]   # [cols][rows/32] uint8


def workspace_bytes(op: str, n: int) -> int:
    return int(_lib.load().mxq_workspace_bytes(op.encode(), int(n)))


def mx_quantize(x: torch.Tensor, rowwise: bool = True, colwise: bool = True, rule: int = RCEIL,
                out: Optional[MXTensor] = None) -> MXTensor:
    _dev(x, torch.bfloat16, "x")
    rows, cols = x.shape
    if out is None:
        dev = x.device
        e = lambda *s: torch.empty(s, dtype=torch.uint8, device=dev)  # noqa: E731
        out = MXTensor(e(rows, cols) if rowwise else None, e(rows, cols // 32) if rowwise else None,
                       e(cols, rows) if colwise else None, e(cols, rows // 32) if colwise else None)
    st = _lib.load().mxq_quantize(_ptr(x), rows, cols, _ptr(out.q_row), _ptr(out.s_row), _ptr(out.q_col),
                                  _ptr(out.s_col), rule, _stream(x.device))
    _lib.check("mxq_quantize", st)
    return out


def mx_quantize_ranged(x: torch.Tensor, rowwise: bool = True, colwise: bool = True, rule: int = RCEIL,
                       out: Optional[MXTensor] = None, words: Optional[torch.Tensor] = None):
    """mx_quantize plus each orientation's range word (int32 device scalars: 1 if a 64-value window is wide).
    Returns (MXTensor, words) with words = int32[2]: [row orientation, column orientation]."""
    _dev(x, torch.bfloat16, "x")
    rows, cols = x.shape
    dev = x.device
    if out is None:
        e = lambda *s: torch.empty(s, dtype=torch.uint8, device=dev)  # noqa: E731
        out = MXTensor(e(rows, cols) if rowwise else None, e(rows, cols // 32) if rowwise else None,
                       e(cols, rows) if colwise else None, e(cols, rows // 32) if colwise else None)
    if words is None:
        words = torch.zeros(2, dtype=torch.int32, device=dev)
    st = _lib.load().mxq_quantize_ranged(_ptr(x), rows, cols, _ptr(out.q_row), _ptr(out.s_row), _ptr(out.q_col),
                                         _ptr(out.s_col), rule,
                                         C.c_void_p(words.data_ptr()) if out.q_row is not None else None,
                                         C.c_void_p(words.data_ptr() + 4) if out.q_col is not None else None,
                                         _stream(dev))
    _lib.check("mxq_quantize_ranged", st)
    return out, words


def scaled_gemm_ranged(a_q: torch.Tensor, a_s: torch.Tensor, a_wide: torch.Tensor, b_q: torch.Tensor,
                       b_s: torch.Tensor, b_wide: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """MX C = A B^T (bf16) with the instruction picked on the device from the operands' range words (int32 device
    scalars, e.g. words[0:1] / words[1:2] of mx_quantize_ranged)."""
    _dev(a_q, torch.uint8, "a_q"); _dev(b_q, torch.uint8, "b_q")
    M, K = a_q.shape
    N = b_q.shape[0]
    if b_q.shape[1] != K:
        raise ValueError("a_q and b_q must share K")
    if not (a_wide.is_cuda and b_wide.is_cuda and a_wide.dtype == torch.int32 and b_wide.dtype == torch.int32):
        raise ValueError("range words must be int32 device tensors")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a_q.device)
    st = _lib.load().scaled_gemm_ranged(_ptr(a_q), _ptr(a_s), C.c_void_p(a_wide.data_ptr()), _ptr(b_q), _ptr(b_s),
                                        C.c_void_p(b_wide.data_ptr()), M, N, K, _ptr(out), out.stride(0),
                                        _stream(a_q.device))
    _lib.check("scaled_gemm_ranged", st)
    return out


def swiglu_mx_quantize(c: torch.Tensor, rule: int = RCEIL, out: Optional[MXTensor] = None) -> MXTensor:
    """c: bf16 [rows][2F] (gate | up) -> MXFP8 row orientation of silu(gate) * up: MXTensor(q_row, s_row, None, None)."""
    _dev(c, torch.bfloat16, "c")
    rows, f2 = c.shape
    F = f2 // 2
    if out is None:
        out = MXTensor(torch.empty((rows, F), dtype=torch.uint8, device=c.device),
                       torch.empty((rows, F // 32), dtype=torch.uint8, device=c.device), None, None)
    st = _lib.load().swiglu_mx_quantize(_ptr(c), rows, F, _ptr(out.q_row), _ptr(out.s_row), rule, _stream(c.device))
    _lib.check("swiglu_mx_quantize", st)
    return out


def _mx_out(rows: int, cols: int, rowwise: bool, colwise: bool, dev) -> MXTensor:
    e = lambda *s: torch.empty(s, dtype=torch.uint8, device=dev)  # noqa: E731
    return MXTensor(e(rows, cols) if rowwise else None, e(rows, cols // 32) if rowwise else None,
                    e(cols, rows) if colwise else None, e(cols, rows // 32) if colwise else None)


def swiglu_mx_quantize_oriented(c: torch.Tensor, rowwise: bool = True, colwise: bool = True, rule: int = RCEIL,
                                out: Optional[MXTensor] = None) -> MXTensor:
    """c: bf16 [rows][2F] (gate | up) -> MXFP8 of silu(gate) * up [rows][F] in the requested orientations (the
    column one is the down projection's Wgrad operand)."""
    _dev(c, torch.bfloat16, "c")
    rows, f2 = c.shape
    F = f2 // 2
    if out is None:
        out = _mx_out(rows, F, rowwise, colwise, c.device)
    st = _lib.load().swiglu_mx_quantize_oriented(_ptr(c), rows, F, _ptr(out.q_row), _ptr(out.s_row), _ptr(out.q_col),
                                                 _ptr(out.s_col), rule, _stream(c.device))
    _lib.check("swiglu_mx_quantize_oriented", st)
    return out


def route_weighted_mx_quantize(dy: torch.Tensor, route_w: torch.Tensor, rowwise: bool = True, colwise: bool = True,
                               rule: int = RCEIL, out: Optional[MXTensor] = None) -> MXTensor:
    """dy: bf16 [rows][cols] (routed rows in expert order), route_w: float32[rows] -> MXFP8 of route_w[r] * dy[r][c]
    in the requested orientations (the down projection's dgrad and Wgrad operands)."""
    _dev(dy, torch.bfloat16, "dy"); _dev(route_w, torch.float32, "route_w")
    rows, cols = dy.shape
    if route_w.numel() != rows:
        raise ValueError("route_w must hold one weight per row of dy")
    if out is None:
        out = _mx_out(rows, cols, rowwise, colwise, dy.device)
    st = _lib.load().route_weighted_mx_quantize(_ptr(dy), _ptr(route_w), rows, cols, _ptr(out.q_row),
                                                _ptr(out.s_row), _ptr(out.q_col), _ptr(out.s_col), rule,
                                                _stream(dy.device))
    _lib.check("route_weighted_mx_quantize", st)
    return out


def swiglu_backward_mx_quantize(c: torch.Tensor, dh: torch.Tensor, rowwise: bool = True, colwise: bool = True,
                                rule: int = RCEIL, out: Optional[MXTensor] = None) -> MXTensor:
    """c: bf16 [rows][2F] (gate | up, the forward up/gate GEMM output), dh: bf16 [rows][F] (gradient of
    silu(gate) * up) -> MXFP8 of (d_gate | d_up) [rows][2F] in the requested orientations."""
    _dev(c, torch.bfloat16, "c"); _dev(dh, torch.bfloat16, "dh")
    rows, f2 = c.shape
    F = f2 // 2
    if tuple(dh.shape) != (rows, F) or f2 != 2 * F:
        raise ValueError("dh must be [rows][F] for c of shape [rows][2F]")
    if out is None:
        out = _mx_out(rows, f2, rowwise, colwise, c.device)
    st = _lib.load().swiglu_backward_mx_quantize(_ptr(c), _ptr(dh), rows, F, _ptr(out.q_row), _ptr(out.s_row),
                                                 _ptr(out.q_col), _ptr(out.s_col), rule, _stream(c.device))
    _lib.check("swiglu_backward_mx_quantize", st)
    return out


class PerTensorFP8(NamedTuple):
    q: Optional[torch.Tensor]       # [rows][cols] uint8
    q_t: Optional[torch.Tensor]     # [cols][rows] uint8
    amax: torch.Tensor              # float32[1] on the device
    scale: torch.Tensor             # float32[1] on the device (q ~ x * scale)


def _pt_out(x: torch.Tensor, want_q: bool, want_qt: bool, out: Optional[PerTensorFP8]):
    """Output buffers of a per-tensor cast: `out` checked against x's shape (its q / q_t, either may be None, decide
    which orientations are written), else new ones."""
    rows, cols = x.shape
    dev = x.device
    if out is None:
        return (torch.empty((rows, cols), dtype=torch.uint8, device=dev) if want_q else None,
                torch.empty((cols, rows), dtype=torch.uint8, device=dev) if want_qt else None,
                torch.empty(1, dtype=torch.float32, device=dev), torch.empty(1, dtype=torch.float32, device=dev))
    for t, shape, dt, name in ((out.q, (rows, cols), torch.uint8, "out.q"), (out.q_t, (cols, rows), torch.uint8, "out.q_t"),
                               (out.amax, (1,), torch.float32, "out.amax"), (out.scale, (1,), torch.float32, "out.scale")):
        if t is None and name in ("out.q", "out.q_t"):
            continue
        if t is None or tuple(t.shape) != shape or t.dtype != dt or t.device != dev or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous {dt} tensor of shape {shape} on {dev}")
    return out.q, out.q_t, out.amax, out.scale


def pertensor_quantize(x: torch.Tensor, fmt: int = E4M3, margin: float = 1.0, scale_in: Optional[torch.Tensor] = None,
                       want_q: bool = True, want_qt: bool = True, workspace: Optional[torch.Tensor] = None,
                       out: Optional[PerTensorFP8] = None) -> PerTensorFP8:
    """Per-tensor FP8 cast of x (bf16 [rows][cols]) to q and its transpose q_t. `out` reuses caller buffers."""
    _dev(x, torch.bfloat16, "x")
    rows, cols = x.shape
    dev = x.device
    q, qt, amax, scale = _pt_out(x, want_q, want_qt, out)
    nbytes = workspace_bytes("pertensor", rows * cols)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    if scale_in is not None:
        _dev(scale_in, torch.float32, "scale_in")
    st = _lib.load().fp8_quantize_pertensor(_ptr(x), rows, cols, fmt, C.c_float(margin), _ptr(scale_in), _ptr(amax),
                                            _ptr(scale), _ptr(q), _ptr(qt), _ptr(workspace), workspace.numel(),
                                            _stream(dev))
    _lib.check("fp8_quantize_pertensor", st)
    return PerTensorFP8(q, qt, amax, scale)


def pertensor_quantize_delayed(x: torch.Tensor, amax_history: torch.Tensor, hist_pos: torch.Tensor, fmt: int = E4M3,
                               margin: float = 1.0, want_q: bool = True, want_qt: bool = True,
                               workspace: Optional[torch.Tensor] = None,
                               out: Optional[PerTensorFP8] = None) -> PerTensorFP8:
    """Delayed-scaling cast: scale from the amax history (float32[H], updated in place with this call's amax at
    hist_pos, an int32[1] that advances). `out` reuses caller buffers."""
    _dev(x, torch.bfloat16, "x"); _dev(amax_history, torch.float32, "amax_history"); _dev(hist_pos, torch.int32, "hist_pos")
    rows, cols = x.shape
    dev = x.device
    q, qt, amax, scale = _pt_out(x, want_q, want_qt, out)
    if workspace is None:
        workspace = torch.empty(workspace_bytes("pertensor_delayed", rows * cols), dtype=torch.uint8, device=dev)
    st = _lib.load().fp8_quantize_pertensor_delayed(_ptr(x), rows, cols, fmt, C.c_float(margin), _ptr(amax_history),
                                                    _ptr(hist_pos), amax_history.numel(), _ptr(amax), _ptr(scale),
                                                    _ptr(q), _ptr(qt), _ptr(workspace), workspace.numel(), _stream(dev))
    _lib.check("fp8_quantize_pertensor_delayed", st)
    return PerTensorFP8(q, qt, amax, scale)


def scaled_gemm(a_q: torch.Tensor, a_scale: torch.Tensor, b_q: torch.Tensor, b_scale: torch.Tensor,
                scaling: int = MX_BLOCK32, a_fmt: int = E4M3, b_fmt: int = E4M3,
                out: Optional[torch.Tensor] = None, exact: bool = False, path: str = "checked") -> torch.Tensor:
    """C[M][N] = A[M][K] B[N][K]^T in bf16. MX: scales are E8M0 grids [M][K/32], [N][K/32]; per-tensor: float32[1].
    path "checked" calls scaled_gemm (the FP8 instruction where a device-side range check allows it, else the exact
    path), "exact" (or exact=True) scaled_gemm_exact, "fp8" scaled_gemm_fp8 (FP8 instruction at every K, bound not
    guaranteed)."""
    _dev(a_q, torch.uint8, "a_q"); _dev(b_q, torch.uint8, "b_q")
    M, K = a_q.shape
    N = b_q.shape[0]
    if b_q.shape[1] != K:
        raise ValueError("a_q and b_q must share K")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a_q.device)
    ldc = out.stride(0)
    if exact:
        path = "exact"
    name = {"checked": "scaled_gemm", "exact": "scaled_gemm_exact", "fp8": "scaled_gemm_fp8"}[path]
    st = getattr(_lib.load(), name)(_ptr(a_q), _ptr(a_scale), a_fmt, _ptr(b_q), _ptr(b_scale), b_fmt, M, N, K,
                                    scaling, _ptr(out), ldc, _stream(a_q.device))
    _lib.check(name, st)
    return out


def grouped_scaled_gemm(a_q: torch.Tensor, a_s: torch.Tensor, offsets: torch.Tensor, b_q: torch.Tensor,
                        b_s: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    _dev(a_q, torch.uint8, "a_q"); _dev(b_q, torch.uint8, "b_q"); _dev(offsets, torch.int64, "offsets")
    total, K = a_q.shape
    G, N, Kb = b_q.shape
    if Kb != K or offsets.numel() != G + 1:
        raise ValueError("shape mismatch")
    if out is None:
        out = torch.empty((total, N), dtype=torch.bfloat16, device=a_q.device)
    st = _lib.load().grouped_scaled_gemm(_ptr(a_q), _ptr(a_s), _ptr(offsets), G, total, _ptr(b_q), _ptr(b_s), N, K,
                                         _ptr(out), _stream(a_q.device))
    _lib.check("grouped_scaled_gemm", st)
    return out


def grouped_scaled_gemm_strided(a_q: torch.Tensor, a_s: torch.Tensor, offsets: torch.Tensor, b_q: torch.Tensor,
                                b_s: torch.Tensor, G: int, N: int, K: int, ldb: int, b_group_stride: int, ldbs: int,
                                bs_group_stride: int, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The grouped MX GEMM with expert g's B row n at b_q[g * b_group_stride + n * ldb] (K bytes) and its scales at
    b_s[g * bs_group_stride + n * ldbs] (K/32 bytes): e.g. a column-orientation weight cache read in place."""
    _dev(a_q, torch.uint8, "a_q"); _dev(b_q, torch.uint8, "b_q"); _dev(offsets, torch.int64, "offsets")
    _dev(a_s, torch.uint8, "a_s"); _dev(b_s, torch.uint8, "b_s")
    total, Ka = a_q.shape
    if Ka != K or offsets.numel() != G + 1:
        raise ValueError("shape mismatch")
    last = (G - 1) * b_group_stride + (N - 1) * ldb + K
    last_s = (G - 1) * bs_group_stride + (N - 1) * ldbs + K // 32
    if b_q.numel() < last or b_s.numel() < last_s:
        raise ValueError("b_q / b_s do not hold every expert's rows at the given strides")
    if out is None:
        out = torch.empty((total, N), dtype=torch.bfloat16, device=a_q.device)
    elif out.dtype != torch.bfloat16 or out.shape[0] != total or out.shape[1] < N or out.stride(1) != 1:
        raise ValueError("out must be bf16 [total_rows][>= N] with unit column stride")
    st = _lib.load().grouped_scaled_gemm_strided(_ptr(a_q), _ptr(a_s), _ptr(offsets), G, total, _ptr(b_q), _ptr(b_s),
                                                 ldb, b_group_stride, ldbs, bs_group_stride, N, K, _ptr(out),
                                                 out.stride(0), _stream(a_q.device))
    _lib.check("grouped_scaled_gemm_strided", st)
    return out


def grouped_wgrad_mx(a_q: torch.Tensor, a_s: torch.Tensor, b_q: torch.Tensor, b_s: torch.Tensor,
                     offsets: torch.Tensor, out: Optional[torch.Tensor] = None,
                     accumulate: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Per-expert contraction over token ranges: C_g = A[:, off_g:off_g+1] B[:, off_g:off_g+1]^T for column-
    orientation operands a_q [M][Kt], b_q [N][Kt]. Returns bf16 [G][M][N], or adds into `accumulate` (float32
    [G][M][N]) and returns it."""
    _dev(a_q, torch.uint8, "a_q"); _dev(b_q, torch.uint8, "b_q"); _dev(offsets, torch.int64, "offsets")
    _dev(a_s, torch.uint8, "a_s"); _dev(b_s, torch.uint8, "b_s")
    M, Kt = a_q.shape
    N = b_q.shape[0]
    G = offsets.numel() - 1
    if b_q.shape[1] != Kt or tuple(a_s.shape) != (M, Kt // 32) or tuple(b_s.shape) != (N, Kt // 32):
        raise ValueError("shape mismatch")
    if accumulate is not None:
        _dev(accumulate, torch.float32, "accumulate")
        if tuple(accumulate.shape) != (G, M, N):
            raise ValueError("accumulate must be float32 [G][M][N]")
        c_bf16, c_f32, res = None, accumulate, accumulate
    else:
        if out is None:
            out = torch.empty((G, M, N), dtype=torch.bfloat16, device=a_q.device)
        _dev(out, torch.bfloat16, "out")
        if tuple(out.shape) != (G, M, N):
            raise ValueError("out must be bf16 [G][M][N]")
        c_bf16, c_f32, res = out, None, out
    st = _lib.load().grouped_wgrad_mx(_ptr(a_q), _ptr(a_s), _ptr(b_q), _ptr(b_s), _ptr(offsets), G, M, N, Kt,
                                      _ptr(c_bf16), _ptr(c_f32), _stream(a_q.device))
    _lib.check("grouped_wgrad_mx", st)
    return res


def fp8_adam_step(master: torch.Tensor, grad: torch.Tensor, m_q: torch.Tensor, m_scale: torch.Tensor,
                  v: torch.Tensor, w: Optional[torch.Tensor], hp: AdamHParams,
                  workspace: Optional[torch.Tensor] = None) -> None:
    """In place on master, m_q, m_scale, v; writes w (bf16 copy) when given."""
    _dev(master, torch.float32, "master"); _dev(grad, torch.bfloat16, "grad"); _dev(m_q, torch.uint8, "m_q")
    _dev(m_scale, torch.float32, "m_scale"); _dev(v, torch.float16, "v")
    n = master.numel()
    if workspace is None:
        workspace = torch.empty(workspace_bytes("adam", n), dtype=torch.uint8, device=master.device)
    st = _lib.load().fp8_adam_step(_ptr(master), _ptr(grad), _ptr(m_q), _ptr(m_scale), _ptr(v), _ptr(w), n,
                                   C.byref(hp), _ptr(workspace), workspace.numel(), _stream(master.device))
    _lib.check("fp8_adam_step", st)


def fp8_adam_step_delayed(master: torch.Tensor, grad: torch.Tensor, m_q: torch.Tensor, m_scale: torch.Tensor,
                          v: torch.Tensor, w: Optional[torch.Tensor], hp: AdamHParams, m_history: torch.Tensor,
                          hist_pos: torch.Tensor, workspace: Optional[torch.Tensor] = None) -> None:
    """fp8_adam_step with the first-moment scale from the amax history (one pass over the state)."""
    _dev(master, torch.float32, "master"); _dev(grad, torch.bfloat16, "grad"); _dev(m_q, torch.uint8, "m_q")
    _dev(m_scale, torch.float32, "m_scale"); _dev(v, torch.float16, "v")
    _dev(m_history, torch.float32, "m_history"); _dev(hist_pos, torch.int32, "hist_pos")
    n = master.numel()
    if workspace is None:
        workspace = torch.empty(workspace_bytes("adam_delayed", n), dtype=torch.uint8, device=master.device)
    st = _lib.load().fp8_adam_step_delayed(_ptr(master), _ptr(grad), _ptr(m_q), _ptr(m_scale), _ptr(v), _ptr(w), n,
                                           C.byref(hp), _ptr(m_history), _ptr(hist_pos), m_history.numel(),
                                           _ptr(workspace), workspace.numel(), _stream(master.device))
    _lib.check("fp8_adam_step_delayed", st)


def fp8_adam_step_mx_cache(master: torch.Tensor, grad: torch.Tensor, m_q: torch.Tensor, m_scale: torch.Tensor,
                           v: torch.Tensor, w: Optional[torch.Tensor], hp: AdamHParams, rows: int, cols: int,
                           rowwise: bool = True, colwise: bool = True, rule: int = RCEIL,
                           out: Optional[MXTensor] = None, workspace: Optional[torch.Tensor] = None) -> MXTensor:
    """fp8_adam_step on a [rows][cols] weight that also rebuilds its MXFP8 caches from the updated fp32 master."""
    _dev(master, torch.float32, "master"); _dev(grad, torch.bfloat16, "grad"); _dev(m_q, torch.uint8, "m_q")
    _dev(m_scale, torch.float32, "m_scale"); _dev(v, torch.float16, "v")
    dev = master.device
    if out is None:
        e = lambda *s: torch.empty(s, dtype=torch.uint8, device=dev)  # noqa: E731
        out = MXTensor(e(rows, cols) if rowwise else None, e(rows, cols // 32) if rowwise else None,
                       e(cols, rows) if colwise else None, e(cols, rows // 32) if colwise else None)
    if workspace is None:
        workspace = torch.empty(workspace_bytes("adam", rows * cols), dtype=torch.uint8, device=dev)
    st = _lib.load().fp8_adam_step_mx_cache(_ptr(master), _ptr(grad), _ptr(m_q), _ptr(m_scale), _ptr(v), _ptr(w),
                                            rows, cols, _ptr(out.q_row), _ptr(out.s_row), _ptr(out.q_col),
                                            _ptr(out.s_col), rule, C.byref(hp), _ptr(workspace), workspace.numel(),
                                            _stream(dev))
    _lib.check("fp8_adam_step_mx_cache", st)
    return out


class AutoScaled(NamedTuple):
    q: torch.Tensor                 # uint8 codes
    scale: torch.Tensor             # float32[1]: the mu these codes carry
    overflow: torch.Tensor          # int64[1]: codes at the maximum magnitude


def fp8_autoscale_cast(g: torch.Tensor, mu: torch.Tensor, fmt: int = E4M3,
                       workspace: Optional[torch.Tensor] = None, out: Optional[AutoScaled] = None) -> AutoScaled:
    """q = FP8(mu * g); mu (float32[1], device) is updated in place for the next step. `out` reuses caller buffers
    (q uint8 of g's shape, scale float32[1], overflow int64[1])."""
    _dev(g, torch.bfloat16, "g"); _dev(mu, torch.float32, "mu")
    dev = g.device
    n = g.numel()
    if out is None:
        q = torch.empty(g.shape, dtype=torch.uint8, device=dev)
        scale = torch.empty(1, dtype=torch.float32, device=dev)
        overflow = torch.empty(1, dtype=torch.int64, device=dev)
    else:
        q, scale, overflow = out.q, out.scale, out.overflow
        for t, shape, dt, name in ((q, tuple(g.shape), torch.uint8, "out.q"), (scale, (1,), torch.float32, "out.scale"),
                                   (overflow, (1,), torch.int64, "out.overflow")):
            if tuple(t.shape) != shape or t.dtype != dt or t.device != dev or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous {dt} tensor of shape {shape} on {dev}")
    if workspace is None:
        workspace = torch.empty(workspace_bytes("autoscale", n), dtype=torch.uint8, device=dev)
    st = _lib.load().fp8_autoscale_cast(_ptr(g), n, fmt, _ptr(mu), _ptr(q), _ptr(scale), _ptr(overflow),
                                        _ptr(workspace), workspace.numel(), _stream(dev))
    _lib.check("fp8_autoscale_cast", st)
    return AutoScaled(q, scale, overflow)


def fp8_requantize_shared(q: torch.Tensor, fmt_in: int, scale_in: torch.Tensor, gathered_scales: torch.Tensor,
                          fmt_out: int = E4M3, out: Optional[torch.Tensor] = None):
    """Returns (q_out, shared scale s_g, sum scale N * s_g), all on the device."""
    _dev(q, torch.uint8, "q"); _dev(scale_in, torch.float32, "scale_in")
    _dev(gathered_scales, torch.float32, "gathered_scales")
    dev = q.device
    if out is None:
        out = torch.empty_like(q)
    else:
        _dev(out, torch.uint8, "out")
        if out.numel() != q.numel():
            raise ValueError("out must hold as many codes as q")
    sg = torch.empty(1, dtype=torch.float32, device=dev)
    ssum = torch.empty(1, dtype=torch.float32, device=dev)
    st = _lib.load().fp8_requantize_shared(_ptr(q), q.numel(), fmt_in, _ptr(scale_in), _ptr(gathered_scales),
                                           gathered_scales.numel(), fmt_out, _ptr(out), _ptr(sg), _ptr(ssum),
                                           _stream(dev))
    _lib.check("fp8_requantize_shared", st)
    return out, sg, ssum


class RMSNormOut(NamedTuple):
    mx: MXTensor                        # MXFP8 of the normalized values, in the requested orientations
    sum: Optional[torch.Tensor]         # bf16 [rows][cols]: x + residual (None without a residual)
    rstd: torch.Tensor                  # float32[rows]
    checkpoint: Optional[MXTensor]      # MXFP8 row orientation of the norm's input (q_col and s_col None)


# The calls below also serve single tokens, where the host's own time is what counts: addresses go to ctypes as plain
# integers, the current stream is read without making a stream object, and a buffer is checked once. A call that
# allocates its four outputs takes 12.3 us, of which the launch is 3.0, against 15.4 with the helpers above.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _here(dev: torch.device) -> int:
    """The current stream of `dev`, as an address."""
    if _raw_stream is not None and dev.index is not None:
        return _raw_stream(dev.index)
    return torch.cuda.current_stream(dev).cuda_stream


def _at(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _expect(t: Optional[torch.Tensor], shape, dtype, dev, name: str):
    """A buffer of exactly this shape (a tuple), type and device, contiguous."""
    if t is None or t.shape != shape or t.dtype is not dtype or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {shape} on {dev}")


def _scratch(t: torch.Tensor, dev) -> int:
    """The bytes of a caller's workspace, which lies on the inputs' device and may be of any type. (Its length is the
    library's to check.)"""
    if t.device != dev or not t.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    return t.numel() * t.element_size()


def _mx_rows(rows: int, cols: int, dev) -> MXTensor:
    """A new MXFP8 tensor in the row orientation."""
    return MXTensor(torch.empty((rows, cols), dtype=torch.uint8, device=dev),
                    torch.empty((rows, cols // 32), dtype=torch.uint8, device=dev), None, None)


def _expect_mx(mx: MXTensor, rows: int, cols: int, dev, name: str):
    """The pairs of mx that are there hold an MXFP8 [rows][cols]."""
    for q, s, a, b, o in ((mx.q_row, mx.s_row, rows, cols, "row"), (mx.q_col, mx.s_col, cols, rows, "col")):
        if q is None and s is None:
            continue
        _expect(q, (a, b), torch.uint8, dev, f"{name}.q_{o}")
        _expect(s, (a, b // 32), torch.uint8, dev, f"{name}.s_{o}")


def rmsnorm_mx_quantize(x: torch.Tensor, gamma: torch.Tensor, eps: float, residual: Optional[torch.Tensor] = None,
                        rowwise: bool = True, colwise: bool = True, checkpoint: bool = True, rule: int = RCEIL,
                        out: Optional[RMSNormOut] = None) -> RMSNormOut:
    """RMSNorm of x (+ residual), bf16 [rows][cols], with gamma float32[cols], straight into MXFP8 of y = h rstd gamma
    in the requested orientations, plus h = bf16(x + residual) when a residual is given, rstd, and the 8-bit checkpoint
    of h that rmsnorm_backward_mx_checkpoint reads. `out` reuses caller buffers (out.sum may be x or residual)."""
    _dev(x, torch.bfloat16, "x")
    if x.dim() != 2:
        raise ValueError("x must be [rows][cols]")
    rows, cols = x.shape
    dev = x.device
    _expect(gamma, (cols,), torch.float32, dev, "gamma")
    if residual is not None:
        _expect(residual, (rows, cols), torch.bfloat16, dev, "residual")
    if out is None:
        out = RMSNormOut(_mx_rows(rows, cols, dev) if rowwise and not colwise else
                         _mx_out(rows, cols, rowwise, colwise, dev), None if residual is None else torch.empty_like(x),
                         torch.empty(rows, dtype=torch.float32, device=dev),
                         _mx_rows(rows, cols, dev) if checkpoint else None)
    else:
        _expect_mx(out.mx, rows, cols, dev, "out.mx")
        _expect(out.rstd, (rows,), torch.float32, dev, "out.rstd")
        if residual is not None:
            _expect(out.sum, (rows, cols), torch.bfloat16, dev, "out.sum")
        elif out.sum is not None:
            out = out._replace(sum=None)                          # nothing is written there
        if out.checkpoint is not None:
            _expect_mx(out.checkpoint, rows, cols, dev, "out.checkpoint")
    ck = out.checkpoint if out.checkpoint is not None else MXTensor(None, None, None, None)
    st = _lib.load().rmsnorm_mx_quantize(_at(x), _at(residual), _at(gamma), rows, cols, eps,
                                         _at(out.sum) if residual is not None else None, _at(out.rstd),
                                         _at(out.mx.q_row), _at(out.mx.s_row), _at(out.mx.q_col),
                                         _at(out.mx.s_col), _at(ck.q_row), _at(ck.s_row), rule, _here(dev))
    _lib.check("rmsnorm_mx_quantize", st)
    return out


def rmsnorm_backward_mx_checkpoint(dy: torch.Tensor, checkpoint: MXTensor, rstd: torch.Tensor, gamma: torch.Tensor,
                                   residual_grad: Optional[torch.Tensor] = None, want_dgamma: bool = True,
                                   accumulate: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                                   workspace: Optional[torch.Tensor] = None):
    """(dx, dgamma) of the norm from its 8-bit checkpoint (row orientation) and rstd. dx (bf16) includes residual_grad,
    the gradient arriving on the residual stream. dgamma is a new float32[cols], or is added into `accumulate`; None
    with want_dgamma=False. `out` may be dy or residual_grad."""
    _dev(dy, torch.bfloat16, "dy")
    if dy.dim() != 2:
        raise ValueError("dy must be [rows][cols]")
    rows, cols = dy.shape
    dev = dy.device
    _expect(checkpoint.q_row, (rows, cols), torch.uint8, dev, "checkpoint.q_row")
    _expect(checkpoint.s_row, (rows, cols // 32), torch.uint8, dev, "checkpoint.s_row")
    _expect(rstd, (rows,), torch.float32, dev, "rstd")
    _expect(gamma, (cols,), torch.float32, dev, "gamma")
    if residual_grad is not None:
        _expect(residual_grad, (rows, cols), torch.bfloat16, dev, "residual_grad")
    if out is None:
        out = torch.empty_like(dy)
    else:
        _expect(out, (rows, cols), torch.bfloat16, dev, "out")
    dgamma = accumulate
    if accumulate is not None:
        _expect(accumulate, (cols,), torch.float32, dev, "accumulate")
    elif want_dgamma:
        dgamma = torch.empty(cols, dtype=torch.float32, device=dev)
    if dgamma is not None and workspace is None:
        workspace = torch.empty(workspace_bytes("rmsnorm_backward", cols), dtype=torch.uint8, device=dev)
    st = _lib.load().rmsnorm_backward_mx_checkpoint(
        _at(dy), _at(residual_grad), _at(checkpoint.q_row), _at(checkpoint.s_row), _at(rstd), _at(gamma), rows,
        cols, _at(out), _at(dgamma), 1 if accumulate is not None else 0, _at(workspace),
        0 if workspace is None else _scratch(workspace, dev), _here(dev))
    _lib.check("rmsnorm_backward_mx_checkpoint", st)
    return out, dgamma


def swiglu_mx_quantize_checkpoint(c: torch.Tensor, rule: int = RCEIL, out=None):
    """c: bf16 [rows][2F] (gate | up) -> (MXFP8 row orientation of silu(gate) * up, MXFP8 row orientation of c): the
    down projection's operand and the checkpoint that swiglu_backward_mx_checkpoint reads. `out` reuses a pair of
    MXTensors."""
    _dev(c, torch.bfloat16, "c")
    rows, f2 = c.shape
    F = f2 // 2
    if f2 != 2 * F:
        raise ValueError("c must be [rows][2F]")
    if out is None:
        out = (_mx_rows(rows, F, c.device), _mx_rows(rows, f2, c.device))
    else:
        _expect_mx(out[0], rows, F, c.device, "out[0]")
        _expect_mx(out[1], rows, f2, c.device, "out[1]")
    h, ck = out
    st = _lib.load().swiglu_mx_quantize_checkpoint(_at(c), rows, F, _at(h.q_row), _at(h.s_row), _at(ck.q_row),
                                                   _at(ck.s_row), rule, _here(c.device))
    _lib.check("swiglu_mx_quantize_checkpoint", st)
    return h, ck


def swiglu_backward_mx_checkpoint(checkpoint: MXTensor, dh: torch.Tensor, rowwise: bool = True, colwise: bool = True,
                                  hidden: bool = True, rule: int = RCEIL, out=None):
    """checkpoint: swiglu_mx_quantize_checkpoint's MXFP8 of c [rows][2F]; dh: bf16 [rows][F] -> (MXFP8 of
    (d_gate | d_up) [rows][2F] in the requested orientations, MXFP8 of silu(gate) * up [rows][F] in the column
    orientation: the down projection's Wgrad operand, or None with hidden=False). `out` reuses such a pair."""
    _dev(dh, torch.bfloat16, "dh")
    rows, F = dh.shape
    dev = dh.device
    _expect(checkpoint.q_row, (rows, 2 * F), torch.uint8, dev, "checkpoint.q_row")
    _expect(checkpoint.s_row, (rows, 2 * F // 32), torch.uint8, dev, "checkpoint.s_row")
    if out is None:
        out = (_mx_out(rows, 2 * F, rowwise, colwise, dev), _mx_out(rows, F, False, True, dev) if hidden else None)
    else:
        _expect_mx(out[0], rows, 2 * F, dev, "out[0]")
        if out[1] is not None:
            _expect_mx(out[1], rows, F, dev, "out[1]")
    dc, h = out
    st = _lib.load().swiglu_backward_mx_checkpoint(
        _at(checkpoint.q_row), _at(checkpoint.s_row), _at(dh), rows, F, _at(dc.q_row), _at(dc.s_row),
        _at(dc.q_col), _at(dc.s_col), None if h is None else _at(h.q_col), None if h is None else _at(h.s_col),
        rule, _here(dev))
    _lib.check("swiglu_backward_mx_checkpoint", st)
    return dc, h


def moe_few_tokens_workspace_bytes(tokens: int, experts: int, topk: int, D: int, F: int) -> int:
    return int(_lib.load().moe_mx_few_tokens_workspace_bytes(int(tokens), int(experts), int(topk), int(D), int(F)))


def moe_mx_few_tokens(x_q: torch.Tensor, x_s: torch.Tensor, logits: torch.Tensor, topk: int, w_up_q: torch.Tensor,
                      w_up_s: torch.Tensor, w_down_q: torch.Tensor, w_down_s: torch.Tensor, normalize: bool = True,
                      out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The routed experts of up to 64 tokens: x MXFP8 [tokens][D], logits float32 [tokens][experts], w_up MXFP8
    [experts][2F][D] (gate rows, then up rows), w_down MXFP8 [experts][D][F] (row orientation) -> bf16 [tokens][D], the
    softmax-weighted sum over each token's topk experts (weights over the chosen experts, or with normalize=False over
    all)."""
    _dev(x_q, torch.uint8, "x_q")
    if x_q.dim() != 2 or logits.dim() != 2 or w_up_q.dim() != 3:
        raise ValueError("x_q must be [tokens][D], logits [tokens][experts], w_up_q [experts][2F][D]")
    T, D = x_q.shape
    E, F = logits.shape[1], w_up_q.shape[1] // 2
    dev = x_q.device
    _expect(x_s, (T, D // 32), torch.uint8, dev, "x_s")
    _expect(logits, (T, E), torch.float32, dev, "logits")
    _expect(w_up_q, (E, 2 * F, D), torch.uint8, dev, "w_up_q")
    _expect(w_up_s, (E, 2 * F, D // 32), torch.uint8, dev, "w_up_s")
    _expect(w_down_q, (E, D, F), torch.uint8, dev, "w_down_q")
    _expect(w_down_s, (E, D, F // 32), torch.uint8, dev, "w_down_s")
    if out is None:
        out = torch.empty((T, D), dtype=torch.bfloat16, device=dev)
    else:
        _expect(out, (T, D), torch.bfloat16, dev, "out")
    if workspace is None:
        workspace = torch.empty(moe_few_tokens_workspace_bytes(T, E, topk, D, F), dtype=torch.uint8, device=dev)
    st = _lib.load().moe_mx_few_tokens(_at(x_q), _at(x_s), _at(logits), T, E, topk, 1 if normalize else 0,
                                       _at(w_up_q), _at(w_up_s), _at(w_down_q), _at(w_down_s), D, F, _at(out),
                                       _at(workspace), _scratch(workspace, dev), _here(dev))
    _lib.check("moe_mx_few_tokens", st)
    return out


class Int8Tensor(NamedTuple):
    """Codes and the scale of each row (a token, or an output channel): x ~ q * scale[:, None]."""
    q: torch.Tensor                     # int8 [rows][cols]
    scale: torch.Tensor                 # float32[rows]


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _checked(dev: torch.device, name: str, *args):
    """Calls the library with `dev` as the current device, on its current stream."""
    fn = getattr(_lib.load(), name)
    if dev.index == _current_device():
        st = fn(*args, _here(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _here(dev))
    if st:
        _lib.check(name, st)


def int8_quantize_tokens(x: torch.Tensor, out: Optional[Int8Tensor] = None) -> Int8Tensor:
    """x: bf16 [rows][cols] -> int8 codes and one scale for each row: the operands of int8_scaled_gemm, from activations
    (a row is a token) or from a weight [N][K] (a row is an output channel). `out` reuses caller buffers."""
    _dev(x, torch.bfloat16, "x")
    if x.dim() != 2:
        raise ValueError("x must be [rows][cols]")
    rows, cols = x.shape
    dev = x.device
    if out is None:
        out = Int8Tensor(x.new_empty((rows, cols), dtype=torch.int8), x.new_empty(rows, dtype=torch.float32))
    else:
        _expect(out.q, (rows, cols), torch.int8, dev, "out.q")
        _expect(out.scale, (rows,), torch.float32, dev, "out.scale")
    _checked(dev, "int8_quantize_tokens", x.data_ptr(), rows, cols, out.q.data_ptr(), out.scale.data_ptr())
    if cols == 0:                                                  # the library writes nothing; rows without values are zero
        out.scale.zero_()
    return out


def _rows_out(out: torch.Tensor, rows: int, cols: int, dev) -> torch.Tensor:
    """The caller's bf16 [rows][cols], whose rows may be further apart."""
    if out.dtype is not torch.bfloat16 or out.shape != (rows, cols) or out.device != dev or \
            (rows and cols and (out.stride(1) != 1 and cols > 1 or out.stride(0) < cols and rows > 1)):
        raise ValueError(f"out must be a bf16 tensor of shape {(rows, cols)} on {dev} with contiguous rows")
    return out


def int8_scaled_gemm(a_q: torch.Tensor, a_scale: torch.Tensor, b_q: torch.Tensor, b_scale: torch.Tensor,
                     swiglu: bool = False, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """bf16 C[M][N] = (A[M][K] B[N][K]^T) a_scale[m] b_scale[n], the sum exact. With swiglu, B holds the N/2 gate rows,
    then the N/2 up rows, and the result is silu(gate) * up [M][N/2]. `out` may be rows of a wider tensor."""
    _dev(a_q, torch.int8, "a_q")
    if a_q.dim() != 2 or b_q.dim() != 2:
        raise ValueError("a_q must be [M][K], b_q [N][K]")
    M, K = a_q.shape
    N = b_q.shape[0]
    dev = a_q.device
    _expect(b_q, (N, K), torch.int8, dev, "b_q")
    _expect(a_scale, (M,), torch.float32, dev, "a_scale")
    _expect(b_scale, (N,), torch.float32, dev, "b_scale")
    cols = N // 2 if swiglu else N
    out = a_q.new_empty((M, cols), dtype=torch.bfloat16) if out is None else _rows_out(out, M, cols, dev)
    _checked(dev, "int8_scaled_gemm", a_q.data_ptr(), a_scale.data_ptr(), b_q.data_ptr(), b_scale.data_ptr(), M, N, K,
             1 if swiglu else 0, out.data_ptr(), out.stride(0) if M > 1 else max(cols, 1))
    return out


def int8_grouped_gemm(a_q: torch.Tensor, a_scale: torch.Tensor, offsets: torch.Tensor, b_q: torch.Tensor,
                      b_scale: torch.Tensor, swiglu: bool = False, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """int8_scaled_gemm over expert groups of any number of rows: rows [offsets[g], offsets[g + 1]) (int64[G + 1], on the
    device) of a_q [rows][K] times b_q [G][N][K]^T with b_scale [G][N]. Rows outside every group are not written."""
    _dev(a_q, torch.int8, "a_q")
    if a_q.dim() != 2 or b_q.dim() != 3:
        raise ValueError("a_q must be [rows][K], b_q [G][N][K]")
    rows, K = a_q.shape
    G, N = b_q.shape[:2]
    dev = a_q.device
    _expect(b_q, (G, N, K), torch.int8, dev, "b_q")
    _expect(offsets, (G + 1,), torch.int64, dev, "offsets")
    _expect(a_scale, (rows,), torch.float32, dev, "a_scale")
    _expect(b_scale, (G, N), torch.float32, dev, "b_scale")
    cols = N // 2 if swiglu else N
    out = a_q.new_empty((rows, cols), dtype=torch.bfloat16) if out is None else _rows_out(out, rows, cols, dev)
    _checked(dev, "int8_grouped_gemm", a_q.data_ptr(), a_scale.data_ptr(), offsets.data_ptr(), G, rows, b_q.data_ptr(),
             b_scale.data_ptr(), N, K, 1 if swiglu else 0, out.data_ptr(), out.stride(0) if rows > 1 else max(cols, 1))
    return out


@functools.lru_cache(maxsize=None)
def _qk_workspace(head_dim: int) -> int:
    return workspace_bytes("qk_norm_backward", head_dim)


class QKNormGrads(NamedTuple):
    dqk: torch.Tensor                   # bf16 [tokens][(heads_q + heads_k) * head_dim], or the caller's wider rows
    dgamma_q: Optional[torch.Tensor]    # float32[head_dim] (None without a norm, or when not wanted)
    dgamma_k: Optional[torch.Tensor]


def _expect_rotation(tokens: int, positions: torch.Tensor, inv_freq: torch.Tensor, pair_axis, gamma_q, gamma_k,
                     head_dim: int, dev):
    """Checks what qk_norm_rope and its backward share; returns (axes, rot, pair_axis as bytes)."""
    axes = 1 if positions.dim() == 1 else positions.shape[0]
    _expect(positions, (tokens,) if positions.dim() == 1 else (axes, tokens), torch.int64, dev, "positions")
    pairs = inv_freq.numel()
    _expect(inv_freq, (pairs,), torch.float32, dev, "inv_freq")
    if (gamma_q is None) != (gamma_k is None):
        raise ValueError("gamma_q and gamma_k go together")
    if gamma_q is not None:
        _expect(gamma_q, (head_dim,), torch.float32, dev, "gamma_q")
        _expect(gamma_k, (head_dim,), torch.float32, dev, "gamma_k")
    if pair_axis is not None:
        if len(pair_axis) != pairs:
            raise ValueError("pair_axis must name one axis for each of inv_freq's pairs")
        # an array would hand bytes() its memory; of a list it takes whole numbers only
        pair_axis = bytes(pair_axis if isinstance(pair_axis, (bytes, list, tuple)) else list(pair_axis))
    return axes, 2 * pairs, pair_axis


def _expect_heads(t: torch.Tensor, tokens: int, heads: int, head_dim: int, dev, name: str):
    """A view [tokens][heads][head_dim] of any token and head stride."""
    if t.dtype is not torch.bfloat16 or t.shape != (tokens, heads, head_dim) or t.device != dev or t.stride(2) != 1:
        raise ValueError(f"{name} must be a bf16 view of shape {(tokens, heads, head_dim)} on {dev} with contiguous heads")


def _expect_rows(t: torch.Tensor, tokens: int, width: int, dev, name: str):
    """bf16 rows of at least `width` values."""
    if t.dtype is not torch.bfloat16 or t.dim() != 2 or t.shape[0] != tokens or t.shape[1] < width or t.device != dev or \
            t.stride(1) != 1:
        raise ValueError(f"{name} must be bf16 [{tokens}][>= {width}] on {dev} with contiguous rows")


def qk_norm_rope(qkv: torch.Tensor, heads_q: int, heads_k: int, head_dim: int, positions: torch.Tensor,
                 inv_freq: torch.Tensor, gamma_q: Optional[torch.Tensor] = None, gamma_k: Optional[torch.Tensor] = None,
                 eps: float = 1e-6, pair_axis=None, interleaved: bool = False, out=None):
    """RMSNorm of every query and key head (without gammas: none) and the rotation by position, from a QKV projection's
    output: qkv bf16 [tokens][>= (heads_q + heads_k) * head_dim], query heads first, then key heads. positions int64
    [tokens] or [axes][tokens]; inv_freq float32[pairs], turning the first 2 * pairs values of a head; pair_axis names the
    axis of each pair (a sequence of whole numbers; None: axis 0), e.g. [0] * 16 + [1] * 24 + [2] * 24 for time, height and
    width; interleaved pairs neighbours instead of halves. Returns (q, k), bf16 [tokens][heads][head_dim]; `out` is such a
    pair of views of any token and head strides (rows of a cache, head-major tensors, or qkv's own heads)."""
    width = (heads_q + heads_k) * head_dim
    if not qkv.is_cuda or qkv.dim() != 2:
        raise ValueError("qkv must be a device tensor [tokens][>= heads * head_dim]")
    tokens, dev = qkv.shape[0], qkv.device
    _expect_rows(qkv, tokens, width, dev, "qkv")
    axes, rot, pair_axis = _expect_rotation(tokens, positions, inv_freq, pair_axis, gamma_q, gamma_k, head_dim, dev)
    if out is None:
        q, k = qkv.new_empty((tokens, heads_q, head_dim)), qkv.new_empty((tokens, heads_k, head_dim))
    else:
        q, k = out
        _expect_heads(q, tokens, heads_q, head_dim, dev, "out[0]")
        _expect_heads(k, tokens, heads_k, head_dim, dev, "out[1]")
    qt, qh, _ = q.stride()
    kt, kh, _ = k.stride()
    _checked(dev, "qk_norm_rope", qkv.data_ptr(), qkv.stride(0), tokens, heads_q, heads_k, head_dim, _at(gamma_q),
             _at(gamma_k), eps, positions.data_ptr(), axes, inv_freq.data_ptr(), rot, pair_axis, 1 if interleaved else 0,
             q.data_ptr(), qt, qh, k.data_ptr(), kt, kh)
    return q, k


def qk_norm_rope_backward(dq: torch.Tensor, dk: torch.Tensor, qkv: Optional[torch.Tensor], positions: torch.Tensor,
                          inv_freq: torch.Tensor, gamma_q: Optional[torch.Tensor] = None,
                          gamma_k: Optional[torch.Tensor] = None, eps: float = 1e-6, pair_axis=None,
                          interleaved: bool = False, want_dgamma: bool = True, accumulate=None,
                          out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> QKNormGrads:
    """Gradients of qk_norm_rope: dq and dk bf16 [tokens][heads][head_dim] (views of any token and head strides), qkv its
    input (None without a norm). dqk is bf16 [tokens][(heads_q + heads_k) * head_dim]; `out` may hold wider rows, whose
    further columns are left as they were, or be qkv itself. dgamma_q and dgamma_k are new float32[head_dim], or are added
    into the pair `accumulate` (two buffers, also for a shared gamma); None without a norm or with want_dgamma=False."""
    if not dq.is_cuda or dq.dim() != 3 or dk.dim() != 3:
        raise ValueError("dq and dk must be device tensors [tokens][heads][head_dim]")
    tokens, heads_q, head_dim = dq.shape
    heads_k, dev = dk.shape[1], dq.device
    width = (heads_q + heads_k) * head_dim
    _expect_heads(dq, tokens, heads_q, head_dim, dev, "dq")
    _expect_heads(dk, tokens, heads_k, head_dim, dev, "dk")
    axes, rot, pair_axis = _expect_rotation(tokens, positions, inv_freq, pair_axis, gamma_q, gamma_k, head_dim, dev)
    if gamma_q is None:
        qkv, ld = None, width
    else:
        if qkv is None:
            raise ValueError("qkv is needed with a norm")
        _expect_rows(qkv, tokens, width, dev, "qkv")
        ld = qkv.stride(0)
    if out is None:
        out = dq.new_empty((tokens, width))
    else:
        _expect_rows(out, tokens, width, dev, "out")
    gq = gk = None
    if gamma_q is not None and want_dgamma and accumulate is not None:
        gq, gk = accumulate
        _expect(gq, (head_dim,), torch.float32, dev, "accumulate[0]")
        _expect(gk, (head_dim,), torch.float32, dev, "accumulate[1]")
    elif gamma_q is not None and want_dgamma:
        gq, gk = gamma_q.new_empty(head_dim), gamma_q.new_empty(head_dim)
    if gq is not None and workspace is None:
        workspace = gamma_q.new_empty(_qk_workspace(head_dim) // 4)
    qt, qh, _ = dq.stride()
    kt, kh, _ = dk.stride()
    _checked(dev, "qk_norm_rope_backward", dq.data_ptr(), qt, qh, dk.data_ptr(), kt, kh, _at(qkv), ld, tokens, heads_q,
             heads_k, head_dim, _at(gamma_q), _at(gamma_k), eps, positions.data_ptr(), axes, inv_freq.data_ptr(), rot,
             pair_axis, 1 if interleaved else 0, out.data_ptr(), out.stride(0), _at(gq), _at(gk),
             1 if accumulate is not None else 0, _at(workspace), 0 if workspace is None else _scratch(workspace, dev))
    return QKNormGrads(out, gq, gk)
