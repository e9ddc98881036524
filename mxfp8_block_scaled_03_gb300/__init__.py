"""mxfp8_block_scaled_03_gb300 -- MXFP8 expert-MLP forward for GB300 (sm_103a).

Thin Python binding over the C ABI in ``include/mxfp8moe.h`` (library
``_build/libmxfp8moe.so``).  The functions keep the C names and only marshal arguments:
torch tensors supply device pointers and the current CUDA stream; every step of the computation
runs in the library's CUDA kernels.  There is no CPU fallback: if the library is missing, calls
raise ``RuntimeError``.

Operations (page "Efficient MoE training for biological foundation models", Key technical
approaches, items 1-3):
  mxfp8_quantize     bf16 -> E4M3 codes + E8M0 scale bytes, row-wise and/or column-wise blocks
                     of 32.
  grouped_mlp_fwd    GroupedLinear(split_sizes) -> ScaledSwiGLU -> MXFP8 requant ->
                     GroupedLinear, in one call.
  moe_permute / grouped_mlp_fwd_tokens / moe_combine
                     the MoE layer around it: device sort of the router's choices by expert,
                     the forward gathering token rows itself, and the per-token sum of outputs.
  moe_decode_fwd, nvfp4_moe_decode_fwd, mxfp8_matvec, nvfp4_matvec
                     the whole layer, and a linear, for a few tokens (decode steps), from the
                     same weights.
  residual_norm_fwd / residual_norm_bwd
                     the norms behind and before a block with its gate and the scaled residual.
  moe_route_fwd / moe_route_bwd
                     the router's choices, weights, counts per expert and losses from its logits.
  linear_cross_entropy_fwd / linear_cross_entropy_bwd
                     the loss of a linear layer over a large vocabulary, without its logits in memory.
"""
from __future__ import annotations

import ctypes
import os
import threading

import numpy as np

from . import build_ext

__all__ = [
    "MXFP8Error", "ROWWISE", "COLWISE", "SF_COMPACT", "SF_MMA", "lib", "library_path",
    "mxfp8_sf_bytes", "mxfp8_quantize", "grouped_mlp_workspace_size", "grouped_mlp_workspace_layout",
    "grouped_mlp_fwd", "grouped_mlp_fwd_noalloc", "grouped_mlp_fwd_tokens", "moe_permute",
    "moe_permute_workspace_size", "moe_combine", "moe_gather_rows", "mxfp8_check_device_error", "mxfp8_quantize_colwise_t",
    "grouped_mlp_saved_bytes", "grouped_mlp_fwd_train", "grouped_mlp_bwd_workspace_size", "grouped_mlp_bwd",
    "grouped_mlp_fwd_tokens_train", "grouped_mlp_bwd_tokens", "mxfp8_status_string", "mxfp8_abi_version",
    "mxfp8_mma_peak", "grouped_mlp_bwd_workspace_layout", "nvfp4_sf_bytes", "nvfp4_quantize", "nvfp4_grouped_mlp_workspace_size",
    "nvfp4_grouped_mlp_workspace_layout", "nvfp4_grouped_mlp_fwd", "moe_decode_workspace_size", "moe_decode_fwd",
    "nvfp4_moe_decode_fwd", "matvec_workspace_size", "mxfp8_matvec", "nvfp4_matvec",
    "residual_norm_fwd", "residual_norm_bwd", "residual_norm_bwd_workspace_size",
    "moe_route_workspace_size", "moe_route_fwd", "moe_route_bwd", "linear_cross_entropy_workspace_size",
    "linear_cross_entropy_fwd", "linear_cross_entropy_bwd_workspace_size", "linear_cross_entropy_bwd",
]

ROWWISE = 1
COLWISE = 2
SF_COMPACT = 0
SF_MMA = 1

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA, ERR_DEVICE_TIMEOUT, ERR_SPLIT_MISMATCH = range(7)

_lock = threading.Lock()
_lib = None


class MXFP8Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({mxfp8_status_string(status)})")


def library_path() -> str:
    return build_ext.LIB


def lib() -> ctypes.CDLL:
    """Load the CUDA library (raises if it has not been built: there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(build_ext.LIB):
                raise RuntimeError(f"MXFP8 CUDA library not built ({build_ext.LIB}); run "
                                   "mxfp8_block_scaled_03_gb300.build_ext.build() or __graft_entry__.build()")
            L = ctypes.CDLL(build_ext.LIB)
            P, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
            L.mxfp8_abi_version.restype = i32
            L.mxfp8_abi_version.argtypes = []
            L.mxfp8_status_string.restype = ctypes.c_char_p
            L.mxfp8_status_string.argtypes = [i32]
            L.mxfp8_sf_bytes.restype = sz
            L.mxfp8_sf_bytes.argtypes = [i64, i64, i32, i32]
            L.mxfp8_quantize.restype = i32
            L.mxfp8_quantize.argtypes = [P, i64, i64, i32, i32, P, P, P, P, P]
            L.grouped_mlp_workspace_size.restype = sz
            L.grouped_mlp_workspace_size.argtypes = [i64, i64, i64, i32]
            L.grouped_mlp_workspace_layout.restype = i32
            L.grouped_mlp_workspace_layout.argtypes = [i64, i64, i64, i32, P]
            L.grouped_mlp_fwd.restype = i32
            L.grouped_mlp_fwd.argtypes = [P, i64, i64, i64, i32, P, P, P, P, P, P, P, P, sz, P]
            L.grouped_mlp_fwd_timed.restype = i32
            L.grouped_mlp_fwd_timed.argtypes = [P, i64, i64, i64, i32, P, P, P, P, P, P, P, P, sz, P, P]
            L.grouped_mlp_saved_bytes.restype = sz
            L.grouped_mlp_saved_bytes.argtypes = [i64, i64, i64, i32]
            L.grouped_mlp_fwd_train.restype = i32
            L.grouped_mlp_fwd_train.argtypes = [P, i64, i64, i64, i32, P, P, P, P, P, P, P, P, sz, P, sz, P]
            L.grouped_mlp_bwd_workspace_size.restype = sz
            L.grouped_mlp_bwd_workspace_size.argtypes = [i64, i64, i64, i32]
            L.grouped_mlp_bwd_workspace_layout.restype = i32
            L.grouped_mlp_bwd_workspace_layout.argtypes = [i64, i64, i64, i32, P]
            L.grouped_mlp_bwd.restype = i32
            L.grouped_mlp_bwd.argtypes = [P, i64, i64, i64, i32, P, P, P, sz, P, P, P, P, P, P, P, P, P, P, sz, P]
            L.grouped_mlp_bwd_timed.restype = i32
            L.grouped_mlp_bwd_timed.argtypes = L.grouped_mlp_bwd.argtypes + [P]
            L.grouped_mlp_fwd_tokens_train.restype = i32
            L.grouped_mlp_fwd_tokens_train.argtypes = [P, i64, P, i64, i64, i64, i32, P, P, P, P, P, P, P, P, sz, P,
                                                       sz, P]
            L.grouped_mlp_bwd_tokens.restype = i32
            L.grouped_mlp_bwd_tokens.argtypes = [P, i64, P, i64, i64, i64, i32, P, P, P, sz, P, P, P, P, P, P, P, P,
                                                 P, P, sz, P]
            L.mxfp8_quantize_colwise_t.restype = i32
            L.mxfp8_quantize_colwise_t.argtypes = [P, i64, i64, i32, P, P, P]
            L.grouped_mlp_fwd_noalloc.restype = i32
            L.grouped_mlp_fwd_noalloc.argtypes = [P, i64, i64, i64, i32, P, P, P, P, P, P, P, P]
            L.grouped_mlp_fwd_tokens.restype = i32
            L.grouped_mlp_fwd_tokens.argtypes = [P, i64, P, i64, i64, i64, i32, P, P, P, P, P, P, P, P, sz, P]
            L.moe_permute_workspace_size.restype = sz
            L.moe_permute_workspace_size.argtypes = [i64, i32, i32]
            L.moe_permute.restype = i32
            L.moe_permute.argtypes = [P, P, i64, i32, i32, P, P, P, P, P, sz, P]
            L.moe_combine.restype = i32
            L.moe_combine.argtypes = [P, P, i64, i32, i64, P, P]
            L.moe_gather_rows.restype = i32
            L.moe_gather_rows.argtypes = [P, i64, i64, P, i64, P, P]
            L.mxfp8_check_device_error.restype = i32
            L.mxfp8_check_device_error.argtypes = [P, P, P]
            f32 = ctypes.c_float
            L.nvfp4_sf_bytes.restype = sz
            L.nvfp4_sf_bytes.argtypes = [i64, i64, i32]
            L.nvfp4_quantize.restype = i32
            L.nvfp4_quantize.argtypes = [P, i64, i64, i32, P, P, P, P]
            L.nvfp4_grouped_mlp_workspace_size.restype = sz
            L.nvfp4_grouped_mlp_workspace_size.argtypes = [i64, i64, i64, i32]
            L.nvfp4_grouped_mlp_workspace_layout.restype = i32
            L.nvfp4_grouped_mlp_workspace_layout.argtypes = [i64, i64, i64, i32, P]
            L.nvfp4_grouped_mlp_fwd.restype = i32
            L.nvfp4_grouped_mlp_fwd.argtypes = [P, i64, i64, i64, i32, P, P, P, P, P, P, P, P, f32, P, P, sz, P, P]
            L.mxfp8_mma_peak.restype = i32
            L.mxfp8_mma_peak.argtypes = [i64, i32, P, P, P]
            L.moe_decode_workspace_size.restype = sz
            L.moe_decode_workspace_size.argtypes = [i64, i32, i64, i64, i32]
            L.moe_decode_fwd.restype = i32
            L.moe_decode_fwd.argtypes = [P, i64, i64, i64, i32, i32, P, P, P, P, P, P, P, P, sz, P]
            L.nvfp4_moe_decode_fwd.restype = i32
            L.nvfp4_moe_decode_fwd.argtypes = [P, i64, i64, i64, i32, i32, P, P, P, P, P, P, P, P, P, P, sz, P]
            L.matvec_workspace_size.restype = sz
            L.matvec_workspace_size.argtypes = [i64, i64]
            L.mxfp8_matvec.restype = i32
            L.mxfp8_matvec.argtypes = [P, i64, i64, i64, P, P, P, P, sz, P]
            L.nvfp4_matvec.restype = i32
            L.nvfp4_matvec.argtypes = [P, i64, i64, i64, P, P, P, P, P, sz, P]
            L.residual_norm_fwd.restype = i32
            L.residual_norm_fwd.argtypes = [P, P, P, P, P, i64, i64, i32, i32, i32, f32, f32, P, P, P, P]
            L.residual_norm_bwd_workspace_size.restype = sz
            L.residual_norm_bwd_workspace_size.argtypes = [i64, i64]
            L.residual_norm_bwd.restype = i32
            L.residual_norm_bwd.argtypes = [P, P, P, P, P, P, P, P, i64, i64, i32, i32, i32, f32, P, P, P, P, P, P, sz, P]
            L.moe_route_workspace_size.restype = sz
            L.moe_route_workspace_size.argtypes = [i64, i32, i32]
            L.moe_route_fwd.restype = i32
            L.moe_route_fwd.argtypes = [P, i32, i64, i32, i32, P, i32, i32, P, P, P, P, P, P, P, sz, P]
            L.moe_route_bwd.restype = i32
            L.moe_route_bwd.argtypes = [P, i32, i64, i32, i32, P, P, P, P, P, P, P, P, i32, P, P]
            L.linear_cross_entropy_workspace_size.restype = sz
            L.linear_cross_entropy_workspace_size.argtypes = [i64, i64, i64]
            L.linear_cross_entropy_fwd.restype = i32
            L.linear_cross_entropy_fwd.argtypes = [P, P, P, i32, i64, i64, i64, P, P, P, sz, P]
            L.linear_cross_entropy_bwd_workspace_size.restype = sz
            L.linear_cross_entropy_bwd_workspace_size.argtypes = [i64, i64, i64]
            L.linear_cross_entropy_bwd.restype = i32
            L.linear_cross_entropy_bwd.argtypes = [P, P, P, P, P, i32, P, i64, i64, i64, P, P, P, sz, P]
            _lib = L
    return _lib


def _stream(stream=None) -> int:
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


def _ptr(t) -> int | None:
    return None if t is None else int(t.data_ptr())


def _check(status: int, where: str):
    if status != OK:
        raise MXFP8Error(status, where)


def mxfp8_abi_version() -> int:
    return int(lib().mxfp8_abi_version())


def mxfp8_status_string(status: int) -> str:
    return lib().mxfp8_status_string(int(status)).decode()


def mxfp8_sf_bytes(M: int, K: int, direction: int, sf_layout: int) -> int:
    return int(lib().mxfp8_sf_bytes(M, K, direction, sf_layout))


def mxfp8_quantize(x, rowwise: bool = True, colwise: bool = False, sf_layout: int = SF_COMPACT,
                   out=None, stream=None):
    """MXFP8 quantization of a contiguous bf16 CUDA tensor [M, K].

    Returns (q_row, sf_row, q_col, sf_col); entries of a direction not requested are None.  Codes
    are uint8 [M, K]; scale bytes are uint8 with mxfp8_sf_bytes(...) elements (compact layout:
    [M, K/32] row-wise, [ceil(M/32), K] column-wise).  `out` may pass preallocated outputs.
    """
    import torch
    assert x.dtype == torch.bfloat16 and x.is_cuda and x.is_contiguous() and x.dim() == 2
    M, K = x.shape
    dirs = (ROWWISE if rowwise else 0) | (COLWISE if colwise else 0)
    if out is None:
        out = [None] * 4
        if rowwise:
            out[0] = torch.empty((M, K), dtype=torch.uint8, device=x.device)
            n = mxfp8_sf_bytes(M, K, ROWWISE, sf_layout)
            out[1] = torch.empty(n, dtype=torch.uint8, device=x.device)
            if sf_layout == SF_COMPACT:
                out[1] = out[1].view(M, K // 32)
        if colwise:
            out[2] = torch.empty((M, K), dtype=torch.uint8, device=x.device)
            n = mxfp8_sf_bytes(M, K, COLWISE, sf_layout)
            out[3] = torch.empty(n, dtype=torch.uint8, device=x.device)
            if sf_layout == SF_COMPACT:
                out[3] = out[3].view((M + 31) // 32, K)
    st = lib().mxfp8_quantize(_ptr(x), M, K, dirs, sf_layout, _ptr(out[0]), _ptr(out[1]), _ptr(out[2]),
                              _ptr(out[3]), _stream(stream))
    _check(st, "mxfp8_quantize")
    return tuple(out)


def mxfp8_quantize_colwise_t(x, sf_layout: int = SF_MMA, out=None, stream=None):
    """Column-wise MXFP8 of bf16 [M, K] with the codes transposed: returns (q_t uint8 [K, M],
    sf_t) where row k of q_t holds column k of x in blocks of 32 rows (the operand form of GEMMs
    that contract over x's rows; weights quantized for the backward)."""
    import torch
    assert x.dtype == torch.bfloat16 and x.is_cuda and x.is_contiguous() and x.dim() == 2
    M, K = x.shape
    if out is None:
        q_t = torch.empty((K, M), dtype=torch.uint8, device=x.device)
        n = mxfp8_sf_bytes(K, M, ROWWISE, sf_layout)
        sf_t = torch.empty(n, dtype=torch.uint8, device=x.device)
        if sf_layout == SF_COMPACT:
            sf_t = sf_t.view(K, M // 32)
    else:
        q_t, sf_t = out
    _check(lib().mxfp8_quantize_colwise_t(_ptr(x), M, K, sf_layout, _ptr(q_t), _ptr(sf_t), _stream(stream)),
           "mxfp8_quantize_colwise_t")
    return q_t, sf_t


def grouped_mlp_workspace_size(R: int, H: int, F: int, E: int) -> int:
    return int(lib().grouped_mlp_workspace_size(R, H, F, E))


def grouped_mlp_workspace_layout(R: int, H: int, F: int, E: int) -> dict:
    arr = (ctypes.c_uint64 * 7)()
    _check(lib().grouped_mlp_workspace_layout(R, H, F, E, arr), "grouped_mlp_workspace_layout")
    keys = ["error", "schedule", "xq", "xsf", "hq", "hsf", "r_pad"]
    return {k: int(v) for k, v in zip(keys, arr)}


def grouped_mlp_fwd(x_sorted, split_sizes, gates, w1_q, w1_sf, w2_q, w2_sf, y=None, workspace=None,
                    stream=None, stage_events=None):
    """Fused MXFP8 grouped expert MLP forward.

    x_sorted bf16 [R, H]; split_sizes int32 [E] (device); gates float32 [R] or None; w1_q uint8
    [E*2F, H] with w1_sf in the tensor-core scale layout; w2_q uint8 [E*H, F] with w2_sf.
    Returns y bf16 [R, H].  `workspace` (uint8 CUDA tensor) is allocated here when not given.
    """
    import torch
    R, H = x_sorted.shape
    E = int(split_sizes.numel())
    F = int(w2_q.shape[1])
    assert x_sorted.dtype == torch.bfloat16 and split_sizes.dtype == torch.int32
    assert gates is None or gates.dtype == torch.float32
    for t in (x_sorted, split_sizes, gates, w1_q, w1_sf, w2_q, w2_sf):
        assert t is None or (t.is_cuda and t.is_contiguous())
    if y is None:
        y = torch.empty((R, H), dtype=torch.bfloat16, device=x_sorted.device)
    need = grouped_mlp_workspace_size(R, H, F, E)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=x_sorted.device)
    args = (_ptr(x_sorted), R, H, F, E, _ptr(split_sizes), _ptr(gates), _ptr(w1_q), _ptr(w1_sf), _ptr(w2_q),
            _ptr(w2_sf), _ptr(y), _ptr(workspace), workspace.numel(), _stream(stream))
    if stage_events is None:
        _check(lib().grouped_mlp_fwd(*args), "grouped_mlp_fwd")
    else:
        # 5 torch.cuda.Event(enable_timing=True), already recorded once (torch creates the CUDA
        # event lazily): re-recorded before each of the 4 kernels and after the last
        handles = [int(ev.cuda_event) for ev in stage_events]
        if len(handles) != 5 or not all(handles):
            raise ValueError("stage_events: 5 CUDA events that have been recorded at least once")
        arr = (ctypes.c_void_p * 5)(*handles)
        _check(lib().grouped_mlp_fwd_timed(*args, arr), "grouped_mlp_fwd_timed")
    return y


def grouped_mlp_saved_bytes(R: int, H: int, F: int, E: int) -> int:
    return int(lib().grouped_mlp_saved_bytes(R, H, F, E))


def grouped_mlp_bwd_workspace_size(R: int, H: int, F: int, E: int) -> int:
    return int(lib().grouped_mlp_bwd_workspace_size(R, H, F, E))


def grouped_mlp_fwd_train(x_sorted, split_sizes, gates, w1_q, w1_sf, w2_q, w2_sf, y=None, saved=None,
                          workspace=None, stream=None):
    """grouped_mlp_fwd that also keeps the bf16 pre-activations [G | U] the backward needs.
    Returns (y, saved); `saved` is a uint8 CUDA tensor of grouped_mlp_saved_bytes(...) bytes."""
    import torch
    R, H = x_sorted.shape
    E = int(split_sizes.numel())
    F = int(w2_q.shape[1])
    dev = x_sorted.device
    if y is None:
        y = torch.empty((R, H), dtype=torch.bfloat16, device=dev)
    if saved is None:
        saved = torch.empty(grouped_mlp_saved_bytes(R, H, F, E), dtype=torch.uint8, device=dev)
    if workspace is None:
        workspace = torch.empty(grouped_mlp_workspace_size(R, H, F, E), dtype=torch.uint8, device=dev)
    st = lib().grouped_mlp_fwd_train(_ptr(x_sorted), R, H, F, E, _ptr(split_sizes), _ptr(gates), _ptr(w1_q),
                                     _ptr(w1_sf), _ptr(w2_q), _ptr(w2_sf), _ptr(y), _ptr(saved), saved.numel(),
                                     _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "grouped_mlp_fwd_train")
    return y, saved


def grouped_mlp_bwd(x_sorted, split_sizes, gates, saved, w1t_q, w1t_sf, w2t_q, w2t_sf, dy, dx=None, dgates=True,
                    dw1=None, dw2=None, workspace=None, stream=None, stage_events=None):
    """Backward of the grouped MLP.  w1t_*/w2t_* are W1 [E*2F, H] and W2 [E*H, F] quantized
    along their other axis (mxfp8_quantize_colwise_t, tensor-core layout).  Returns
    (dx bf16 [R, H], dgates float32 [R] or None, dW1 float32 [E, 2F, H], dW2 float32 [E, H, F],
    workspace)."""
    import torch
    R, H = x_sorted.shape
    E = int(split_sizes.numel())
    F = int(w2t_q.shape[0])
    dev = x_sorted.device
    if dx is None:
        dx = torch.empty((R, H), dtype=torch.bfloat16, device=dev)
    if dgates is True:
        dgates = torch.empty(R, dtype=torch.float32, device=dev)
    elif dgates is False:
        dgates = None
    if dw1 is None:
        dw1 = torch.empty((E, 2 * F, H), dtype=torch.float32, device=dev)
    if dw2 is None:
        dw2 = torch.empty((E, H, F), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(grouped_mlp_bwd_workspace_size(R, H, F, E), dtype=torch.uint8, device=dev)
    args = (_ptr(x_sorted), R, H, F, E, _ptr(split_sizes), _ptr(gates), _ptr(saved), saved.numel(), _ptr(w1t_q),
            _ptr(w1t_sf), _ptr(w2t_q), _ptr(w2t_sf), _ptr(dy), _ptr(dx), _ptr(dgates), _ptr(dw1), _ptr(dw2),
            _ptr(workspace), workspace.numel(), _stream(stream))
    if stage_events is None:
        _check(lib().grouped_mlp_bwd(*args), "grouped_mlp_bwd")
    else:
        handles = [int(ev.cuda_event) for ev in stage_events]
        if len(handles) != 7 or not all(handles):
            raise ValueError("stage_events: 7 CUDA events that have been recorded at least once")
        _check(lib().grouped_mlp_bwd_timed(*args, (ctypes.c_void_p * 7)(*handles)), "grouped_mlp_bwd_timed")
    return dx, dgates, dw1, dw2, workspace


def grouped_mlp_fwd_tokens_train(x_tokens, token_of_row, split_sizes, gates_sorted, w1_q, w1_sf, w2_q, w2_sf,
                                 y=None, saved=None, workspace=None, stream=None):
    """grouped_mlp_fwd_tokens that also saves the pre-activations.  Returns (y_rows, saved)."""
    import torch
    T, H = x_tokens.shape
    R = int(token_of_row.numel())
    E = int(split_sizes.numel())
    F = int(w2_q.shape[1])
    dev = x_tokens.device
    if y is None:
        y = torch.empty((R, H), dtype=torch.bfloat16, device=dev)
    if saved is None:
        saved = torch.empty(grouped_mlp_saved_bytes(R, H, F, E), dtype=torch.uint8, device=dev)
    if workspace is None:
        workspace = torch.empty(grouped_mlp_workspace_size(R, H, F, E), dtype=torch.uint8, device=dev)
    st = lib().grouped_mlp_fwd_tokens_train(_ptr(x_tokens), T, _ptr(token_of_row), R, H, F, E, _ptr(split_sizes),
                                            _ptr(gates_sorted), _ptr(w1_q), _ptr(w1_sf), _ptr(w2_q), _ptr(w2_sf),
                                            _ptr(y), _ptr(saved), saved.numel(), _ptr(workspace), workspace.numel(),
                                            _stream(stream))
    _check(st, "grouped_mlp_fwd_tokens_train")
    return y, saved


def grouped_mlp_bwd_tokens(x_tokens, token_of_row, split_sizes, gates_sorted, saved, w1t_q, w1t_sf, w2t_q, w2t_sf,
                           d_out_tokens, workspace=None, stream=None):
    """grouped_mlp_bwd reading x and the output gradient as token rows through token_of_row.
    Returns (dx_rows bf16 [R, H], dgates_sorted float32 [R] or None, dW1, dW2, workspace)."""
    import torch
    T, H = x_tokens.shape
    R = int(token_of_row.numel())
    E = int(split_sizes.numel())
    F = int(w2t_q.shape[0])
    dev = x_tokens.device
    dx = torch.empty((R, H), dtype=torch.bfloat16, device=dev)
    dg = torch.empty(R, dtype=torch.float32, device=dev) if gates_sorted is not None else None
    dw1 = torch.empty((E, 2 * F, H), dtype=torch.float32, device=dev)
    dw2 = torch.empty((E, H, F), dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(grouped_mlp_bwd_workspace_size(R, H, F, E), dtype=torch.uint8, device=dev)
    st = lib().grouped_mlp_bwd_tokens(_ptr(x_tokens), T, _ptr(token_of_row), R, H, F, E, _ptr(split_sizes),
                                      _ptr(gates_sorted), _ptr(saved), saved.numel(), _ptr(w1t_q), _ptr(w1t_sf),
                                      _ptr(w2t_q), _ptr(w2t_sf), _ptr(d_out_tokens), _ptr(dx), _ptr(dg), _ptr(dw1),
                                      _ptr(dw2), _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "grouped_mlp_bwd_tokens")
    return dx, dg, dw1, dw2, workspace


def grouped_mlp_fwd_noalloc(x_sorted, split_sizes, gates, w1_q, w1_sf, w2_q, w2_sf, y, stream=None):
    """grouped_mlp_fwd without a workspace, for callers that cannot allocate device memory at the
    call site: scratch comes from the library's fixed 64 MiB device array (shared by all calls on
    a device; overlapping calls race).  `y` (bf16 [R, H]) must be passed in; nothing is
    allocated.  Sizes whose workspace exceeds 64 MiB raise MXFP8Error (status ERR_WORKSPACE)."""
    R, H = x_sorted.shape
    E = int(split_sizes.numel())
    F = int(w2_q.shape[1])
    st = lib().grouped_mlp_fwd_noalloc(_ptr(x_sorted), R, H, F, E, _ptr(split_sizes), _ptr(gates), _ptr(w1_q),
                                       _ptr(w1_sf), _ptr(w2_q), _ptr(w2_sf), _ptr(y), _stream(stream))
    _check(st, "grouped_mlp_fwd_noalloc")
    return y


def moe_permute_workspace_size(T: int, k: int, E: int) -> int:
    return int(lib().moe_permute_workspace_size(T, k, E))


def moe_permute(experts, gates, E: int, workspace=None, out=None, stream=None):
    """Stable device sort of the router's (token, slot) choices by expert.

    experts int32 [T, k] (CUDA), gates float32 [T, k] or None.  Returns (split_sizes [E],
    row_of_slot [T, k], token_of_row [T*k], gates_sorted [T*k] or None, workspace); `out`
    may pass the first four to be reused."""
    import torch
    T, k = experts.shape
    dev = experts.device
    if out is not None:
        split, row_of_slot, token_of_row, gates_sorted = out
    else:
        split = torch.empty(E, dtype=torch.int32, device=dev)
        row_of_slot = torch.empty((T, k), dtype=torch.int32, device=dev)
        token_of_row = torch.empty(T * k, dtype=torch.int32, device=dev)
        gates_sorted = None if gates is None else torch.empty(T * k, dtype=torch.float32, device=dev)
    if workspace is None:
        workspace = torch.empty(max(256, moe_permute_workspace_size(T, k, E)), dtype=torch.uint8, device=dev)
    st = lib().moe_permute(_ptr(experts), _ptr(gates), T, k, E, _ptr(split), _ptr(row_of_slot), _ptr(token_of_row),
                           _ptr(gates_sorted), _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "moe_permute")
    return split, row_of_slot, token_of_row, gates_sorted, workspace


def grouped_mlp_fwd_tokens(x_tokens, token_of_row, split_sizes, gates_sorted, w1_q, w1_sf, w2_q, w2_sf, y=None,
                           workspace=None, stream=None):
    """grouped_mlp_fwd that gathers its rows from x_tokens [T, H] through token_of_row [R] inside
    the activation quantize.  Returns y [R, H] bf16 in sorted-row order."""
    import torch
    T, H = x_tokens.shape
    R = int(token_of_row.numel())
    E = int(split_sizes.numel())
    F = int(w2_q.shape[1])
    if y is None:
        y = torch.empty((R, H), dtype=torch.bfloat16, device=x_tokens.device)
    if workspace is None:
        workspace = torch.empty(grouped_mlp_workspace_size(R, H, F, E), dtype=torch.uint8, device=x_tokens.device)
    st = lib().grouped_mlp_fwd_tokens(_ptr(x_tokens), T, _ptr(token_of_row), R, H, F, E, _ptr(split_sizes),
                                      _ptr(gates_sorted), _ptr(w1_q), _ptr(w1_sf), _ptr(w2_q), _ptr(w2_sf), _ptr(y),
                                      _ptr(workspace), workspace.numel(), _stream(stream))
    _check(st, "grouped_mlp_fwd_tokens")
    return y


def moe_combine(y_rows, row_of_slot, out=None, stream=None):
    """out[t] = sum_j y_rows[row_of_slot[t, j]] (bf16 out, fp32 sum)."""
    import torch
    T, k = row_of_slot.shape
    H = y_rows.shape[1]
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=y_rows.device)
    _check(lib().moe_combine(_ptr(y_rows), _ptr(row_of_slot), T, k, H, _ptr(out), _stream(stream)), "moe_combine")
    return out


def moe_gather_rows(src, index, out=None, stream=None):
    """out[i] = src[index[i]] (rows copied bit for bit; rows of an index outside [0, len(src)) are
    zeros).  src [N, ...] (rows of a multiple of 4 bytes), index int32 [n]."""
    import torch
    n = int(index.numel())
    row_shape = tuple(src.shape[1:])
    if out is None:
        out = torch.empty((n,) + row_shape, dtype=src.dtype, device=src.device)
    row_bytes = src.element_size() * (int(np.prod(row_shape)) if row_shape else 1)
    _check(lib().moe_gather_rows(_ptr(src), int(src.shape[0]), row_bytes, _ptr(index), n, _ptr(out), _stream(stream)),
           "moe_gather_rows")
    return out


def grouped_mlp_bwd_workspace_layout(R: int, H: int, F: int, E: int) -> list[int]:
    """Byte offsets in a backward workspace: [error word, dGU row-wise codes [R_pad, 2F], their
    scale bytes, dGU column-wise codes transposed [2F, R_pad], their scale bytes, h column-wise
    codes transposed [F, R_pad], their scale bytes, R_pad]; scale bytes in the tensor-core
    layout."""
    out = (ctypes.c_uint64 * 8)()
    _check(lib().grouped_mlp_bwd_workspace_layout(R, H, F, E, out), "grouped_mlp_bwd_workspace_layout")
    return list(out)


def nvfp4_sf_bytes(M: int, K: int, sf_layout: int = SF_COMPACT) -> int:
    return int(lib().nvfp4_sf_bytes(M, K, sf_layout))


def nvfp4_quantize(x, sf_layout: int = SF_COMPACT, out=None, stream=None):
    """NVFP4 of a bf16 [M, K] CUDA tensor.  Returns (codes uint8 [M, K/2], scale codes uint8,
    amax float32 [1]: max |x|, which defines the per-tensor encode scale).  `out` may pass the
    three to be reused."""
    import torch
    M, K = x.shape
    assert x.dtype == torch.bfloat16 and x.is_cuda and x.is_contiguous()
    if out is None:
        out = (torch.empty((M, K // 2), dtype=torch.uint8, device=x.device),
               torch.empty(max(1, nvfp4_sf_bytes(M, K, sf_layout)), dtype=torch.uint8, device=x.device),
               torch.empty(1, dtype=torch.float32, device=x.device))
    q, sf, amax = out
    _check(lib().nvfp4_quantize(_ptr(x), M, K, sf_layout, _ptr(q), _ptr(sf), _ptr(amax), _stream(stream)),
           "nvfp4_quantize")
    return q, sf, amax


def nvfp4_grouped_mlp_workspace_size(R: int, H: int, F: int, E: int) -> int:
    return int(lib().nvfp4_grouped_mlp_workspace_size(R, H, F, E))


def nvfp4_grouped_mlp_workspace_layout(R: int, H: int, F: int, E: int) -> list[int]:
    out = (ctypes.c_uint64 * 7)()
    _check(lib().nvfp4_grouped_mlp_workspace_layout(R, H, F, E, out), "nvfp4_grouped_mlp_workspace_layout")
    return list(out)


def nvfp4_grouped_mlp_fwd(x_sorted, split_sizes, gates, w1, w2, h_amax: float, y=None, workspace=None, stream=None,
                          stage_events=None):
    """NVFP4 grouped expert MLP forward.  w1 = (codes, scale codes in SF_MMA layout, amax) from
    nvfp4_quantize of W1 [E*2F, H]; w2 likewise of W2 [E*H, F]; h_amax: the magnitude the
    intermediate's encode scale is derived from.  Returns y bf16 [R, H]."""
    import torch
    R, H = x_sorted.shape
    E = int(split_sizes.numel())
    F = int(w2[0].shape[1]) * 2
    assert x_sorted.dtype == torch.bfloat16 and split_sizes.dtype == torch.int32
    assert gates is None or gates.dtype == torch.float32
    for t in (x_sorted, split_sizes, gates, *w1, *w2):
        assert t is None or (t.is_cuda and t.is_contiguous())
    if y is None:
        y = torch.empty((R, H), dtype=torch.bfloat16, device=x_sorted.device)
    if workspace is None:
        workspace = torch.empty(nvfp4_grouped_mlp_workspace_size(R, H, F, E), dtype=torch.uint8,
                                device=x_sorted.device)
    ev = None
    if stage_events is not None:   # 5 torch.cuda.Event(enable_timing=True), already recorded once
        handles = [int(e.cuda_event) for e in stage_events]
        if len(handles) != 5 or not all(handles):
            raise ValueError("stage_events: 5 CUDA events that have been recorded at least once")
        ev = (ctypes.c_void_p * 5)(*handles)
    _check(lib().nvfp4_grouped_mlp_fwd(_ptr(x_sorted), R, H, F, E, _ptr(split_sizes), _ptr(gates), _ptr(w1[0]),
                                       _ptr(w1[1]), _ptr(w1[2]), _ptr(w2[0]), _ptr(w2[1]), _ptr(w2[2]),
                                       float(h_amax), _ptr(y), _ptr(workspace), workspace.numel(), _stream(stream),
                                       ev), "nvfp4_grouped_mlp_fwd")
    return y


def _place(t, name: str):
    """(device, its current stream) of a call: the device of its first tensor.  The library launches on the current
    device, so it has to be that one.  A call with a stream of its own makes that stream and its device current
    first, so that what the call allocates belongs to it."""
    import torch
    dev = t.get_device()                       # -1: not on a GPU
    if dev < 0 or dev != torch._C._cuda_getDevice():
        raise ValueError(f"{name}: expected a tensor on the current CUDA device (or the stream's); got {t.device}")
    return dev, torch._C._cuda_getCurrentRawStream(dev)


def _need(t, dtype, shape, name: str, dev: int):
    """A contiguous tensor of this device, dtype and shape (an int: at least so many elements).  These calls
    are as short as the kernels behind them, so the message is put together only when it is needed."""
    if t.dtype == dtype and t.get_device() == dev and t.is_contiguous() and \
            (t.numel() >= shape if isinstance(shape, int) else t.shape == shape):
        return t.data_ptr()
    want = f"at least {shape} elements" if isinstance(shape, int) else f"shape {tuple(shape)}"
    raise ValueError(f"{name}: expected a contiguous tensor of {dtype}, {want}, on cuda:{dev}; "
                     f"got {t.dtype}, {tuple(t.shape)}, {t.device}")


def _sf_mma_bytes(nv: bool, M: int, K: int) -> int:
    """Bytes of a row-wise SF_MMA scale array (mxfp8_sf_bytes, nvfp4_sf_bytes)."""
    return (M + 127) // 128 * ((K + 255) // 256 * 4 if nv else (K // 32 + 3) // 4) * 512


def moe_decode_workspace_size(T: int, k: int, H: int, F: int, E: int) -> int:
    return int(lib().moe_decode_workspace_size(T, k, H, F, E))


def _moe_decode(name, nv, x, experts, gates, w1, w2, out, workspace, stream):
    import torch
    if stream is not None:
        with torch.cuda.stream(stream):
            return _moe_decode(name, nv, x, experts, gates, w1, w2, out, workspace, None)
    u8, f32, bf16 = torch.uint8, torch.float32, torch.bfloat16
    dev, current = _place(x, "x")
    T, H = x.shape
    T2, k = experts.shape
    per = 2 if nv else 1                       # values per code byte
    M2, F = w2[0].shape
    F *= per
    E = M2 // H if H else 0
    px, pe = _need(x, bf16, (T, H), "x", dev), _need(experts, torch.int32, (T, k), "experts", dev)
    pg = None if gates is None else _need(gates, f32, (T, k), "gates", dev)
    p1 = _need(w1[0], u8, (E * 2 * F, H // per), "W1 codes", dev)
    s1 = _need(w1[1], u8, _sf_mma_bytes(nv, E * 2 * F, H), "W1 scales", dev)
    p2 = _need(w2[0], u8, (E * H, F // per), "W2 codes", dev)
    s2 = _need(w2[1], u8, _sf_mma_bytes(nv, E * H, F), "W2 scales", dev)
    if out is None:
        out = torch.empty((T, H), dtype=bf16, device=x.device)
        po = out.data_ptr()
    else:
        po = _need(out, bf16, (T, H), "out", dev)
    if workspace is None:
        workspace = torch.empty(max(256, moe_decode_workspace_size(T, k, H, F, E)), dtype=u8, device=x.device)
    pw = _need(workspace, u8, 256, "workspace", dev)
    if nv:
        st = lib().nvfp4_moe_decode_fwd(px, T, H, F, E, k, pe, pg, p1, s1, _need(w1[2], f32, 1, "W1 amax", dev), p2, s2,
                                        _need(w2[2], f32, 1, "W2 amax", dev), po, pw, workspace.numel(), current)
    else:
        st = lib().moe_decode_fwd(px, T, H, F, E, k, pe, pg, p1, s1, p2, s2, po, pw, workspace.numel(), current)
    if st != OK:
        raise MXFP8Error(st, name)
    return out


def moe_decode_fwd(x, experts, gates, w1_q, w1_sf, w2_q, w2_sf, out=None, workspace=None, stream=None):
    """A whole MoE layer for a few tokens (T <= 64): out[t] = sum_j gates[t, j] * expert(experts[t, j])(x_t).

    x bf16 [T, H]; experts int32 [T, k] (negative: a dropped choice); gates float32 [T, k] or None;
    weights as for grouped_mlp_fwd.  The activations are not rounded to 8 bits: x is off by at most 2^-17 of its
    block's largest value, the intermediate by 2^-12.  Returns out bf16 [T, H].
    `workspace` (uint8 CUDA tensor, moe_decode_workspace_size bytes) is allocated here when not given, and its
    error word is lost with it: to learn of an id >= E, which is skipped, or of a wait that ran out, pass one and
    ask mxfp8_check_device_error."""
    return _moe_decode("moe_decode_fwd", False, x, experts, gates, (w1_q, w1_sf), (w2_q, w2_sf), out, workspace, stream)


def nvfp4_moe_decode_fwd(x, experts, gates, w1, w2, out=None, workspace=None, stream=None):
    """moe_decode_fwd from NVFP4 weights: w1 = (codes, scale codes in SF_MMA layout, amax) as for
    nvfp4_grouped_mlp_fwd, w2 likewise.  x and the intermediate are off by at most 2^-14 of their block's largest
    value plus 2^-31 of the row's."""
    return _moe_decode("nvfp4_moe_decode_fwd", True, x, experts, gates, w1, w2, out, workspace, stream)


def matvec_workspace_size(T: int = 64, K: int = 16384) -> int:
    """Bytes of a workspace for mxfp8_matvec / nvfp4_matvec calls of up to T rows of up to K values."""
    return int(lib().matvec_workspace_size(T, K))


def _matvec(name, nv, x, w, out, workspace, stream):
    import torch
    if stream is not None:
        with torch.cuda.stream(stream):
            return _matvec(name, nv, x, w, out, workspace, None)
    u8, bf16 = torch.uint8, torch.bfloat16
    dev, current = _place(x, "x")
    T, K = x.shape
    N = w[0].shape[0]
    px, pq = _need(x, bf16, (T, K), "x", dev), _need(w[0], u8, (N, K // 2 if nv else K), "codes", dev)
    ps = _need(w[1], u8, _sf_mma_bytes(nv, N, K), "scales", dev)
    if out is None:
        out = torch.empty((T, N), dtype=bf16, device=x.device)
        po = out.data_ptr()
    else:
        po = _need(out, bf16, (T, N), "out", dev)
    if workspace is None:
        workspace = torch.empty(max(256, matvec_workspace_size(T, K)), dtype=u8, device=x.device)
    pw = _need(workspace, u8, 256, "workspace", dev)
    if nv:
        st = lib().nvfp4_matvec(px, T, K, N, pq, ps, _need(w[2], torch.float32, 1, "amax", dev), po, pw,
                                workspace.numel(), current)
    else:
        st = lib().mxfp8_matvec(px, T, K, N, pq, ps, po, pw, workspace.numel(), current)
    if st != OK:
        raise MXFP8Error(st, name)
    return out


def mxfp8_matvec(x, w_q, w_sf, out=None, workspace=None, stream=None):
    """y = x W^T for a few rows of x (bf16 [T, K], T <= 64) from W quantized by mxfp8_quantize (row-wise,
    SF_MMA).  x is not rounded to 8 bits (off by at most 2^-17 of a block's largest value).  Returns bf16 [T, N].
    `workspace` (matvec_workspace_size bytes) and its error word as for moe_decode_fwd."""
    return _matvec("mxfp8_matvec", False, x, (w_q, w_sf), out, workspace, stream)


def nvfp4_matvec(x, w, out=None, workspace=None, stream=None):
    """y = x W^T for a few rows of x (bf16 [T, K], T <= 64) from 4-bit weights: w = (codes, scale codes,
    amax) as nvfp4_quantize writes them with SF_MMA.  x is off by at most 2^-14 of a block's largest value plus
    2^-31 of the row's.  Returns bf16 [T, N].  `workspace` (matvec_workspace_size bytes) as for moe_decode_fwd."""
    return _matvec("nvfp4_matvec", True, x, w, out, workspace, stream)


def _norm_args(y, res_like, w_post, gate, w_pre):
    """(device, stream, T, H, residual dtype, its code, gate kind, gate pointer, w_post pointer, w_pre pointer)."""
    import torch
    f32 = torch.float32
    dev, current = _place(y, "y")
    T, H = y.shape
    rt = res_like.dtype
    if rt is not torch.bfloat16 and rt is not f32:
        raise ValueError(f"residual: expected bfloat16 or float32, got {rt}")
    kind, pg = 0, None
    if gate is not None:
        kind = 1 if gate.dim() == 1 else 2     # [H]: per channel; [T, 1]: per token
        pg = _need(gate, f32, (H,) if kind == 1 else (T, 1), "gate", dev)
    return (dev, current, T, H, rt, 0 if rt is torch.bfloat16 else 1, kind, pg,
            None if w_post is None else _need(w_post, f32, (H,), "w_post", dev),
            None if w_pre is None else _need(w_pre, f32, (H,), "w_pre", dev))


def residual_norm_fwd(y, res, w_post=None, gate=None, w_pre=None, res_scale: float = 1.0, post_norm: bool = True,
                      eps: float = 1e-6, out=None, stream=None):
    """res_out = res_scale * res + gate * rms_norm(y) * w_post;  n = rms_norm(res_out) * w_pre.

    y bf16 [T, H]; res bf16 or float32 [T, H]; w_post, w_pre float32 [H] or None; gate float32 [H] (per
    channel), [T, 1] (per token) or None; post_norm False: no norm of y.  Returns (res_out, n bf16, stats
    float32 [2, T]); `out` may pass the three (res_out may be res)."""
    import torch
    if stream is not None:
        with torch.cuda.stream(stream):
            return residual_norm_fwd(y, res, w_post, gate, w_pre, res_scale, post_norm, eps, out)
    bf16 = torch.bfloat16
    dev, current, T, H, rt, code, kind, pg, pa, pb = _norm_args(y, res, w_post, gate, w_pre)
    py, pr = _need(y, bf16, (T, H), "y", dev), _need(res, rt, (T, H), "res", dev)
    if out is None:
        res_out, n, stats = torch.empty_like(res), torch.empty_like(y), torch.empty((2, T), dtype=torch.float32, device=y.device)
        po, pn, ps = res_out.data_ptr(), n.data_ptr(), stats.data_ptr()
    else:
        res_out, n, stats = out
        po, pn = _need(res_out, rt, (T, H), "res_out", dev), _need(n, bf16, (T, H), "n", dev)
        ps = _need(stats, torch.float32, (2, T), "stats", dev)
    st = lib().residual_norm_fwd(py, pr, pa, pg, pb, T, H, code, kind, 1 if post_norm else 0, res_scale, eps, po, pn,
                                 ps, current)
    if st != OK:
        raise MXFP8Error(st, "residual_norm_fwd")
    return res_out, n, stats


def residual_norm_bwd_workspace_size(T: int, H: int) -> int:
    return int(lib().residual_norm_bwd_workspace_size(T, H))


def residual_norm_bwd(dn, dres_out, y, res_out, stats, w_post=None, gate=None, w_pre=None, res_scale: float = 1.0,
                      post_norm: bool = True, workspace=None, stream=None):
    """Gradients of residual_norm_fwd from those of n (bf16 [T, H]) and of res_out (residual's type, or None
    for 0); y, res_out, stats as the forward read or wrote them.  Returns (dy bf16, dres, dw_post, dgate,
    dw_pre), the last three float32 shaped like the weights (None where the weight is None)."""
    import torch
    if stream is not None:
        with torch.cuda.stream(stream):
            return residual_norm_bwd(dn, dres_out, y, res_out, stats, w_post, gate, w_pre, res_scale, post_norm, workspace)
    bf16, f32 = torch.bfloat16, torch.float32
    dev, current, T, H, rt, code, kind, pg, pa, pb = _norm_args(y, res_out, w_post, gate, w_pre)
    pn, py = _need(dn, bf16, (T, H), "dn", dev), _need(y, bf16, (T, H), "y", dev)
    pr = _need(res_out, rt, (T, H), "res_out", dev)
    pd = None if dres_out is None else _need(dres_out, rt, (T, H), "dres_out", dev)
    like = torch.empty_like
    dy, dres = like(y), like(res_out)
    dw_post, dgate, dw_pre = (None if w is None else like(w) for w in (w_post, gate, w_pre))
    if workspace is None:
        workspace = torch.empty(max(16, residual_norm_bwd_workspace_size(T, H)), dtype=torch.uint8, device=y.device)
    st = lib().residual_norm_bwd(pn, pd, py, pr, _need(stats, f32, (2, T), "stats", dev), pa, pg, pb, T, H, code, kind,
                                 1 if post_norm else 0, res_scale, dy.data_ptr(), dres.data_ptr(), _ptr(dw_post),
                                 _ptr(dgate), _ptr(dw_pre), _need(workspace, torch.uint8, 0, "workspace", dev),
                                 workspace.numel(), current)
    if st != OK:
        raise MXFP8Error(st, "residual_norm_bwd")
    return dy, dres, dw_post, dgate, dw_pre


def moe_route_workspace_size(T: int, E: int, k: int) -> int:
    return int(lib().moe_route_workspace_size(T, E, k))


def _logits(logits, name: str, dev: int):
    """(T, E, code of the type, pointer) of a router's logits."""
    import torch
    if logits.dtype is not torch.bfloat16 and logits.dtype is not torch.float32 or logits.dim() != 2:
        raise ValueError(f"{name}: expected bfloat16 or float32 [T, E], got {logits.dtype}, {tuple(logits.shape)}")
    T, E = logits.shape
    return T, E, 0 if logits.dtype is torch.bfloat16 else 1, _need(logits, logits.dtype, (T, E), name, dev)


def moe_route_fwd(logits, k: int, token_mask=None, normalize: bool = True, spread: bool = False, out=None,
                  workspace=None, stream=None):
    """A router's decisions from its logits [T, E] (bf16 or float32): each token's k largest, their softmax weights
    (with `normalize` over the chosen alone), the counts, and the two losses.

    token_mask bool or uint8 [T]: tokens at 0 take no part.  A logit of -inf closes an expert.  Slots without a
    choice have gate 0 and id -1, or with `spread` (t * k + j) % E: moe_decode_fwd takes the former, moe_permute
    needs the latter.  Returns (experts int32 [T, k], gates float32 [T, k], lse float32 [T], counts int32 [E + 1]: choices
    per expert and tokens that take part, prob_sum float32 [E], losses float32 [2]: balance and mean of lse^2); `out` may
    pass the six.  `workspace`: uint8 CUDA tensor, moe_route_workspace_size bytes."""
    import torch
    if stream is not None:
        with torch.cuda.stream(stream):
            return moe_route_fwd(logits, k, token_mask, normalize, spread, out, workspace)
    f32, i32 = torch.float32, torch.int32
    dev, current = _place(logits, "logits")
    T, E, code, pl = _logits(logits, "logits", dev)
    pm = None
    if token_mask is not None:
        if token_mask.dtype is not torch.bool and token_mask.dtype is not torch.uint8:
            raise ValueError(f"token_mask: expected bool or uint8, got {token_mask.dtype}")
        pm = _need(token_mask, token_mask.dtype, (T,), "token_mask", dev)
    where = logits.device
    if out is None:
        empty = torch.empty
        out = (empty((T, k), dtype=i32, device=where), empty((T, k), dtype=f32, device=where),
               empty(T, dtype=f32, device=where), empty(E + 1, dtype=i32, device=where),
               empty(E, dtype=f32, device=where), empty(2, dtype=f32, device=where))
        experts, gates, lse, counts, prob_sum, losses = out
        pe, pg, ps = experts.data_ptr(), gates.data_ptr(), lse.data_ptr()
        pc, pp, po = counts.data_ptr(), prob_sum.data_ptr(), losses.data_ptr()
    else:
        experts, gates, lse, counts, prob_sum, losses = out
        pe, pg = _need(experts, i32, (T, k), "experts", dev), _need(gates, f32, (T, k), "gates", dev)
        ps, pc = _need(lse, f32, (T,), "lse", dev), _need(counts, i32, (E + 1,), "counts", dev)
        pp, po = _need(prob_sum, f32, (E,), "prob_sum", dev), _need(losses, f32, (2,), "losses", dev)
    if workspace is None:
        workspace = torch.empty(max(16, moe_route_workspace_size(T, E, k)), dtype=torch.uint8, device=where)
    st = lib().moe_route_fwd(pl, code, T, E, k, pm, 1 if normalize else 0, 1 if spread else 0, pe, pg, ps, pc, pp, po,
                             _need(workspace, torch.uint8, 0, "workspace", dev), workspace.numel(), current)
    if st != OK:
        raise MXFP8Error(st, "moe_route_fwd")
    return experts, gates, lse, counts, prob_sum, losses


def moe_route_bwd(logits, experts, gates, lse, counts, dgates=None, dlosses=None, row_of_slot=None, dprob_sum=None,
                  normalize: bool = True, out=None, stream=None):
    """The gradient of moe_route_fwd's logits (in their type) from those of the gates (float32 [T, k]; with row_of_slot
    from moe_permute [T * k] in sorted-row order, as grouped_mlp_bwd gives it), of the losses (float32 [2]) and of
    prob_sum (float32 [E]); None: 0.  logits, experts, gates, lse, counts, normalize as the forward had or wrote
    them; counts may be the sum over several batches."""
    import torch
    if stream is not None:
        with torch.cuda.stream(stream):
            return moe_route_bwd(logits, experts, gates, lse, counts, dgates, dlosses, row_of_slot, dprob_sum, normalize,
                                 out)
    f32, i32 = torch.float32, torch.int32
    dev, current = _place(logits, "logits")
    T, E, code, pl = _logits(logits, "logits", dev)
    _, k = experts.shape
    if row_of_slot is not None and dgates is None:
        raise ValueError("row_of_slot without dgates")
    args = (_need(experts, i32, (T, k), "experts", dev), _need(gates, f32, (T, k), "gates", dev),
            _need(lse, f32, (T,), "lse", dev), _need(counts, i32, (E + 1,), "counts", dev),
            None if dgates is None else _need(dgates, f32, (T, k) if row_of_slot is None else (T * k,), "dgates", dev),
            None if row_of_slot is None else _need(row_of_slot, i32, (T, k), "row_of_slot", dev),
            None if dprob_sum is None else _need(dprob_sum, f32, (E,), "dprob_sum", dev),
            None if dlosses is None else _need(dlosses, f32, (2,), "dlosses", dev))
    if out is None:
        out = torch.empty_like(logits)
        po = out.data_ptr()
    else:
        po = _need(out, logits.dtype, (T, E), "out", dev)
    st = lib().moe_route_bwd(pl, code, T, E, k, *args, 1 if normalize else 0, po, current)
    if st != OK:
        raise MXFP8Error(st, "moe_route_bwd")
    return out


def linear_cross_entropy_workspace_size(T: int, H: int, V: int) -> int:
    return int(lib().linear_cross_entropy_workspace_size(T, H, V))


def linear_cross_entropy_bwd_workspace_size(T: int, H: int, V: int) -> int:
    return int(lib().linear_cross_entropy_bwd_workspace_size(T, H, V))


def _lce_args(x, w, targets):
    """(device, stream, T, H, V, x pointer, w pointer, targets pointer, 1 for int64 targets)."""
    import torch
    dev, current = _place(x, "x")
    (T, H), (V, _) = x.shape, w.shape
    if targets.dtype is not torch.int32 and targets.dtype is not torch.int64:
        raise ValueError(f"targets: expected int32 or int64, got {targets.dtype}")
    return (dev, current, T, H, V, _need(x, torch.bfloat16, (T, H), "x", dev),
            _need(w, torch.bfloat16, (V, H), "w", dev), _need(targets, targets.dtype, (T,), "targets", dev),
            1 if targets.dtype is torch.int64 else 0)


def linear_cross_entropy_fwd(x, w, targets, out=None, workspace=None, stream=None):
    """Cross entropy of softmax(x W^T) against targets, without the logits in memory.

    x bf16 [T, H]; w bf16 [V, H]; targets int32 or int64 [T], negative: the row takes no part (its loss is 0).  Returns
    (loss float32 [T], lse float32 [T]); `out` may pass the two.  `workspace` (uint8 CUDA tensor,
    linear_cross_entropy_workspace_size bytes) is allocated here when not given, and its error word is lost with it: a
    target >= V then shows as a NaN loss only."""
    import torch
    if stream is not None:
        with torch.cuda.stream(stream):
            return linear_cross_entropy_fwd(x, w, targets, out, workspace)
    f32, u8 = torch.float32, torch.uint8
    dev, current, T, H, V, px, pw, pt, wide = _lce_args(x, w, targets)
    if out is None:
        loss, lse = (torch.empty(T, dtype=f32, device=x.device), torch.empty(T, dtype=f32, device=x.device))
        ptrs = loss.data_ptr(), lse.data_ptr()
    else:
        loss, lse = out
        ptrs = _need(loss, f32, (T,), "loss", dev), _need(lse, f32, (T,), "lse", dev)
    if workspace is None:
        workspace = torch.empty(max(256, linear_cross_entropy_workspace_size(T, H, V)), dtype=u8, device=x.device)
    st = lib().linear_cross_entropy_fwd(px, pw, pt, wide, T, H, V, *ptrs, _need(workspace, u8, 256, "workspace", dev),
                                        workspace.numel(), current)
    if st != OK:
        raise MXFP8Error(st, "linear_cross_entropy_fwd")
    return loss, lse


def linear_cross_entropy_bwd(dloss, x, w, targets, lse, dlse=None, out=None, workspace=None, stream=None):
    """Gradients of linear_cross_entropy_fwd from those of loss (float32 [T]) and of lse (float32 [T], or None for 0);
    x, w, targets, lse as the forward had or wrote them.  Rows without a target pass nothing on, whatever they hold.
    Returns (dx bf16 [T, H], dw bf16 [V, H]); `out` may pass the two.  `workspace`:
    linear_cross_entropy_bwd_workspace_size bytes, as for the forward."""
    import torch
    if stream is not None:
        with torch.cuda.stream(stream):
            return linear_cross_entropy_bwd(dloss, x, w, targets, lse, dlse, out, workspace)
    f32, u8 = torch.float32, torch.uint8
    dev, current, T, H, V, px, pw, pt, wide = _lce_args(x, w, targets)
    pd, ps = _need(dloss, f32, (T,), "dloss", dev), _need(lse, f32, (T,), "lse", dev)
    pe = None if dlse is None else _need(dlse, f32, (T,), "dlse", dev)
    if out is None:
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        ptrs = dx.data_ptr(), dw.data_ptr()
    else:
        dx, dw = out
        ptrs = _need(dx, torch.bfloat16, (T, H), "dx", dev), _need(dw, torch.bfloat16, (V, H), "dw", dev)
    if workspace is None:
        workspace = torch.empty(max(256, linear_cross_entropy_bwd_workspace_size(T, H, V)), dtype=u8, device=x.device)
    st = lib().linear_cross_entropy_bwd(pd, pe, px, pw, pt, wide, ps, T, H, V, *ptrs,
                                        _need(workspace, u8, 256, "workspace", dev), workspace.numel(), current)
    if st != OK:
        raise MXFP8Error(st, "linear_cross_entropy_bwd")
    return dx, dw


def mxfp8_mma_peak(iters: int, workspace, fmt: int = 0, stream=None) -> int:
    """Enqueue the block-scaled MMA rate measurement (see include/mxfp8moe.h; fmt 0 MXFP8, 1
    NVFP4); returns the number of CTA-pair clusters launched.  `workspace`: a CUDA tensor of at
    least 4 bytes."""
    n = ctypes.c_int(0)
    _check(lib().mxfp8_mma_peak(int(iters), int(fmt), _ptr(workspace), ctypes.byref(n), _stream(stream)),
           "mxfp8_mma_peak")
    return int(n.value)


def mxfp8_check_device_error(workspace, stream=None) -> tuple[int, int]:
    """(status, raw error bits) of the last grouped_mlp_fwd on this workspace (synchronizes)."""
    flags = ctypes.c_uint32(0)
    st = lib().mxfp8_check_device_error(_ptr(workspace), _stream(stream), ctypes.byref(flags))
    return int(st), int(flags.value)
