"""Thin ctypes binding of include/moe_fp8.h with the same entry-point names.

Argument marshalling only: every step runs in libmoe_fp8.so's kernels. Tensors
are torch CUDA tensors (torch provides device memory and streams); their data
pointers are passed straight through. A missing library raises at import of
the first call; there is no fallback path."""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

from .build import LIB

MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED_SHAPE = 2
MOE_ERR_UNSUPPORTED_DEVICE = 3
MOE_ERR_WORKSPACE_TOO_SMALL = 4
MOE_ERR_CAPACITY = 5
MOE_ERR_CUDA = 6
MOE_ERR_DEVICE_TIMEOUT = 7
STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED_SHAPE",
                3: "MOE_ERR_UNSUPPORTED_DEVICE", 4: "MOE_ERR_WORKSPACE_TOO_SMALL", 5: "MOE_ERR_CAPACITY",
                6: "MOE_ERR_CUDA", 7: "MOE_ERR_DEVICE_TIMEOUT"}
ROUTE_SOFTMAX_TOPK, ROUTE_HASH = 0, 1
LAYOUT_CONTIGUOUS, LAYOUT_MASKED = 0, 1
EPI_BF16, EPI_SWIGLU_FP8 = 0, 1
CONTIG_AUTO, CONTIG_SINGLE, CONTIG_PAIR = 0, 1, 2
WEIGHTS_FP8, WEIGHTS_W4 = 0, 1
TYPE_BF16, TYPE_FP32 = 0, 1
EXPORTS = ("moe_rows_capacity", "moe_workspace_size", "moe_route", "moe_permute", "moe_grouped_gemm_fp8",
           "moe_combine", "moe_forward", "moe_forward_train", "moe_get_device_status", "moe_selftest_wait_timeout", "moe_status_string",
           "moe_permute_noalloc", "moe_balance_bias", "moe_grouped_gemm_w4", "moe_set_contig_kernel",
           "moe_ep_plan", "moe_ep_plan_chunked", "moe_ep_workspace_size", "moe_ep_count", "moe_ep_dispatch",
           "moe_ep_receive", "moe_ep_receive_chunk", "moe_ep_return", "moe_backward_workspace_size", "moe_backward",
           "moe_train_logits_offset", "moe_balance_workspace_size", "moe_balance_loss", "moe_balance_loss_backward",
           "moe_router_backward_workspace_size", "moe_router_backward", "moe_orthogonalise_workspace_size",
           "moe_orthogonalise")


class MoeError(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        super().__init__(f"{call}: {STATUS_NAMES.get(status, status)} ({status_string(status)})")


class Config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("T", "H", "E", "I", "k", "routing", "cap_num", "cap_den",
                                            "layout", "masked_max_m", "weights")]

    @classmethod
    def from_moe(cls, cfg) -> "Config":
        """From an inputs.MoeConfig."""
        return cls(cfg.T, cfg.H, cfg.E, cfg.I, cfg.k,
                   ROUTE_HASH if cfg.routing == "hash" else ROUTE_SOFTMAX_TOPK,
                   cfg.cap_num, cfg.cap_den,
                   LAYOUT_MASKED if cfg.layout == "masked" else LAYOUT_CONTIGUOUS,
                   cfg.masked_max_m, WEIGHTS_W4 if getattr(cfg, "weights", "fp8") == "w4" else WEIGHTS_FP8)


_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is None:
        if not os.path.exists(LIB):
            raise RuntimeError(f"native library {LIB} is missing: run fp8_grouped_gemm_fp32_b200.build.build()")
        L = ctypes.CDLL(LIB)
        P, I, SZ, CP = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.POINTER(Config)
        L.moe_rows_capacity.argtypes = [CP]
        L.moe_workspace_size.argtypes = [CP, I]
        L.moe_route.argtypes = [CP, P, P, P, P, P, P, P, SZ, P]
        L.moe_permute.argtypes = [CP, P, P, P, P, P, P, P, P, P, P, SZ, P]
        L.moe_permute_noalloc.argtypes = [CP, P, P, P, P, P, P, P, P, P, P]
        L.moe_grouped_gemm_fp8.argtypes = [I, I, I, I, P, P, P, I, P, P, I, P, P, P]
        L.moe_grouped_gemm_w4.argtypes = [I, I, I, I, P, P, P, I, P, P, I, P, P, P]
        L.moe_combine.argtypes = [CP, P, P, P, P, P]
        L.moe_forward.argtypes = [CP, P, P, P, P, P, P, P, P, P, P, P, P, P, P, SZ, P]
        L.moe_forward_train.argtypes = [CP, P, P, P, P, P, P, P, P, P, P, P, P, P, P, SZ, P]
        L.moe_balance_bias.argtypes = [I, P, P, P, ctypes.c_float, I, P]
        L.moe_get_device_status.argtypes = [P]
        L.moe_selftest_wait_timeout.argtypes = [I, P]
        L.moe_set_contig_kernel.argtypes = [I]
        L.moe_ep_plan.argtypes = [I, I, I, ctypes.c_int64, I, I, I, P, P]
        L.moe_ep_plan_chunked.argtypes = [I, I, I, ctypes.c_int64, I, I, I, P, I, P]
        L.moe_ep_workspace_size.argtypes = [CP]
        L.moe_ep_count.argtypes = [CP, P, P, P, SZ, P]
        L.moe_ep_dispatch.argtypes = [CP, P, P, P, P, P, P, SZ, P]
        L.moe_ep_receive.argtypes = [I, P, I, P, P, P, I, P, P, P]
        L.moe_ep_receive_chunk.argtypes = [I, P, I, P, P, P, I, P, P, P]
        L.moe_ep_return.argtypes = [I, I, P, P, P, P]
        L.moe_backward_workspace_size.argtypes = [CP]
        L.moe_backward.argtypes = [CP] + [P] * 12 + [I] + [P] * 7 + [SZ, P]
        F = ctypes.c_float
        L.moe_train_logits_offset.argtypes = [CP]
        L.moe_balance_workspace_size.argtypes = [I, I, I]
        L.moe_balance_loss.argtypes = [I, I, I, P, P, P, P, I, F, F, P, P, P, P, P, P, SZ, P]
        L.moe_balance_loss_backward.argtypes = [I, I, I, P, P, P, P, P, P, I, F, F, P, P, P]
        L.moe_router_backward_workspace_size.argtypes = [I, I, I]
        L.moe_router_backward.argtypes = [I, I, I] + [P] * 10 + [SZ, P]
        L.moe_orthogonalise_workspace_size.argtypes = [I, I, I, I]
        L.moe_orthogonalise.argtypes = [I, I, I, I, P, I, I, F, F, F, F, F, P, P, SZ, P]
        sizes = ("moe_rows_capacity", "moe_workspace_size", "moe_ep_workspace_size", "moe_backward_workspace_size",
                 "moe_train_logits_offset", "moe_balance_workspace_size", "moe_router_backward_workspace_size",
                 "moe_orthogonalise_workspace_size")
        for f in sizes:
            getattr(L, f).restype = SZ
        L.moe_status_string.argtypes = [I]
        L.moe_status_string.restype = ctypes.c_char_p
        for f in EXPORTS:
            if f != "moe_status_string" and f not in sizes:
                getattr(L, f).restype = I
        _lib = L
    return _lib


def _p(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        return int(t)
    ptr = t.data_ptr()                           # 0 for a tensor without elements
    if ptr and not t.is_cuda:
        raise ValueError("moe_fp8 entry points take CUDA tensors")
    if not t.is_contiguous():
        raise ValueError("moe_fp8 entry points take contiguous tensors")
    return ptr or None


def _stream(stream):
    if stream is None:
        # the current stream's handle, without the Stream object torch.cuda.current_stream() would build
        if not torch.cuda.is_initialized():
            torch.cuda.init()
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _check(st: int, call: str):
    if st != MOE_OK:
        raise MoeError(st, call)


def status_string(st: int) -> str:
    return lib().moe_status_string(st).decode()


def moe_rows_capacity(cfg: Config) -> int:
    return int(lib().moe_rows_capacity(ctypes.byref(cfg)))


def moe_workspace_size(cfg: Config, for_forward: int = 0) -> int:
    """Scratch bytes: 0 route / permute, 1 moe_forward, 2 moe_forward_train."""
    return int(lib().moe_workspace_size(ctypes.byref(cfg), int(for_forward)))


def moe_route(cfg, x, Wg, bias, token_ids, topk_idx, topk_w, ws, stream=None):
    _check(lib().moe_route(ctypes.byref(cfg), _p(x), _p(Wg), _p(bias), _p(token_ids), _p(topk_idx), _p(topk_w),
                           _p(ws), ws.numel() * ws.element_size() if ws is not None else 0, _stream(stream)),
           "moe_route")


def moe_permute(cfg, x, topk_idx, Aq, As, counts, kept, offsets, row_src, slot_row, ws, stream=None):
    _check(lib().moe_permute(ctypes.byref(cfg), _p(x), _p(topk_idx), _p(Aq), _p(As), _p(counts), _p(kept),
                             _p(offsets), _p(row_src), _p(slot_row), _p(ws), ws.numel() * ws.element_size(),
                             _stream(stream)), "moe_permute")


def moe_permute_noalloc(cfg, x, topk_idx, Aq, As, counts, kept, offsets, row_src, slot_row, stream=None):
    """moe_permute without a workspace: for callers that may not allocate device memory.
    Uses the library's fixed device scratch; calls that overlap on the GPU race."""
    _check(lib().moe_permute_noalloc(ctypes.byref(cfg), _p(x), _p(topk_idx), _p(Aq), _p(As), _p(counts), _p(kept),
                                     _p(offsets), _p(row_src), _p(slot_row), _stream(stream)), "moe_permute_noalloc")


def moe_grouped_gemm_fp8(layout, E, N, K, A, As, group_info, M_rows, B, Bs, epilogue, D, Ds=None, stream=None):
    _check(lib().moe_grouped_gemm_fp8(layout, E, N, K, _p(A), _p(As), _p(group_info), M_rows, _p(B), _p(Bs),
                                      epilogue, _p(D), _p(Ds), _stream(stream)), "moe_grouped_gemm_fp8")


def moe_grouped_gemm_w4(layout, E, N, K, A, As, group_info, M_rows, B, Bs, epilogue, D, Ds=None, stream=None):
    """moe_grouped_gemm_fp8 with 4-bit weights: B [E, N, K/2] packed levels, Bs [E, K/128, N] row scales."""
    _check(lib().moe_grouped_gemm_w4(layout, E, N, K, _p(A), _p(As), _p(group_info), M_rows, _p(B), _p(Bs),
                                     epilogue, _p(D), _p(Ds), _stream(stream)), "moe_grouped_gemm_w4")


def moe_combine(cfg, O, slot_row, topk_w, y, stream=None):
    _check(lib().moe_combine(ctypes.byref(cfg), _p(O), _p(slot_row), _p(topk_w), _p(y), _stream(stream)),
           "moe_combine")


def moe_forward(cfg, x, Wg, bias, token_ids, W13, S13, W2, S2, y, topk_idx, topk_w, counts, slot_row, ws,
                stream=None):
    _check(lib().moe_forward(ctypes.byref(cfg), _p(x), _p(Wg), _p(bias), _p(token_ids), _p(W13), _p(S13), _p(W2),
                             _p(S2), _p(y), _p(topk_idx), _p(topk_w), _p(counts), _p(slot_row), _p(ws),
                             ws.numel() * ws.element_size(), _stream(stream)), "moe_forward")


def moe_forward_train(cfg, x, Wg, bias, token_ids, W13, S13, W2, S2, y, topk_idx, topk_w, counts, slot_row, ws,
                      stream=None):
    """moe_forward that also keeps the gate and up values in ws (moe_workspace_size(cfg, 2) bytes) for
    moe_backward(..., fwd_train=True)."""
    _check(lib().moe_forward_train(ctypes.byref(cfg), _p(x), _p(Wg), _p(bias), _p(token_ids), _p(W13), _p(S13),
                                   _p(W2), _p(S2), _p(y), _p(topk_idx), _p(topk_w), _p(counts), _p(slot_row), _p(ws),
                                   ws.numel() * ws.element_size(), _stream(stream)), "moe_forward_train")


def moe_balance_bias(E, counts, load, bias, gamma, update, stream=None):
    """Auxiliary-loss-free bias step: load (int64) += counts; if update, bias (fp32) moves by -gamma / +gamma
    for experts above / below the mean tally, and load is cleared."""
    _check(lib().moe_balance_bias(E, _p(counts), _p(load), _p(bias), float(gamma), int(bool(update)),
                                  _stream(stream)), "moe_balance_bias")


def moe_get_device_status(stream=None) -> int:
    return int(lib().moe_get_device_status(_stream(stream)))


def moe_selftest_wait_timeout(limit_us: int, stream=None):
    _check(lib().moe_selftest_wait_timeout(limit_us, _stream(stream)), "moe_selftest_wait_timeout")


def moe_set_contig_kernel(form: int):
    """Form of the contiguous-layout grouped GEMM for later calls: CONTIG_AUTO, CONTIG_SINGLE or CONTIG_PAIR."""
    _check(lib().moe_set_contig_kernel(int(form)), "moe_set_contig_kernel")


# ---------------------------------------------------------------- expert parallelism (see ep.py)
def _nbytes(t):
    return t.nbytes if t is not None else 0


def moe_ep_workspace_size(cfg: Config) -> int:
    return int(lib().moe_ep_workspace_size(ctypes.byref(cfg)))


def moe_ep_count(cfg, topk_idx, counts, ws, stream=None):
    _check(lib().moe_ep_count(ctypes.byref(cfg), _p(topk_idx), _p(counts), _p(ws), _nbytes(ws), _stream(stream)),
           "moe_ep_count")


def moe_ep_dispatch(cfg, x, topk_idx, plan_dev, send, slot_row, ws, stream=None):
    _check(lib().moe_ep_dispatch(ctypes.byref(cfg), _p(x), _p(topk_idx), _p(plan_dev), _p(send), _p(slot_row), _p(ws),
                                 _nbytes(ws), _stream(stream)), "moe_ep_dispatch")


def moe_ep_receive(H, plan_dev, rows_recv, recv, Aq, As, M_rows, offsets, group_row, stream=None):
    _check(lib().moe_ep_receive(H, _p(plan_dev), rows_recv, _p(recv) if rows_recv else None, _p(Aq), _p(As), M_rows,
                                _p(offsets), _p(group_row), _stream(stream)), "moe_ep_receive")


def moe_ep_receive_chunk(H, plan_dev, chunk, recv, Aq, As, M_rows, offsets, group_row, stream=None):
    _check(lib().moe_ep_receive_chunk(H, _p(plan_dev), chunk, _p(recv), _p(Aq), _p(As), M_rows, _p(offsets),
                                      _p(group_row), _stream(stream)), "moe_ep_receive_chunk")


def moe_ep_return(H, rows_recv, O, group_row, ret, stream=None):
    _check(lib().moe_ep_return(H, rows_recv, _p(O), _p(group_row), _p(ret), _stream(stream)), "moe_ep_return")


# ---------------------------------------------------------------- backward pass
def moe_backward_workspace_size(cfg: Config) -> int:
    return int(lib().moe_backward_workspace_size(ctypes.byref(cfg)))


def moe_backward(cfg, x, Wg, W13, S13, W13T, S13T, W2T, S2T, topk_idx, topk_w, slot_row, fwd_ws, dy, dx, dWg, db,
                 dW13, dW2, ws, stream=None, fwd_train: bool = False):
    """fwd_train: fwd_ws comes from moe_forward_train (the gate and up values are read, not recomputed)."""
    _check(lib().moe_backward(ctypes.byref(cfg), _p(x), _p(Wg), _p(W13), _p(S13), _p(W13T), _p(S13T), _p(W2T),
                              _p(S2T), _p(topk_idx), _p(topk_w), _p(slot_row), _p(fwd_ws), int(bool(fwd_train)),
                              _p(dy), _p(dx), _p(dWg), _p(db), _p(dW13), _p(dW2), _p(ws), _nbytes(ws),
                              _stream(stream)), "moe_backward")


# ---------------------------------------------------------------- balance loss, the router's gradient, updates
_F32, _I32, _BF16 = torch.float32, torch.int32, torch.bfloat16


def _args(call, *specs):
    """The pointers of (name, tensor, type, least number of elements) each (tensor None: null; type None: any), all
    checked to be of that type, large enough, contiguous and on the current device, where the library launches
    whatever device a pointer is of."""
    out, dev = [], None
    for name, t, dtype, n in specs:
        if t is None:
            out.append(None)
            continue
        if dtype is not None and t.dtype is not dtype:
            raise ValueError(f"{call}: {name} is {t.dtype}, not {dtype}")
        if t.numel() < n:
            raise ValueError(f"{call}: {name} has {t.numel()} elements, not {n}")
        if not t.is_contiguous():
            raise ValueError("moe_fp8 entry points take contiguous tensors")
        d = t.get_device()
        if d != dev:
            if dev is not None:
                raise ValueError(f"{call}: {name} is on {t.device}, the tensors before it are not")
            dev = d
        out.append(t.data_ptr())
    if dev is not None:
        if dev < 0:
            raise ValueError("moe_fp8 entry points take CUDA tensors")
        current = torch._C._cuda_getDevice()
        if dev != current:
            raise ValueError(f"{call}: tensors of cuda:{dev} in a call on the current device cuda:{current}")
    return out


def _mask(t, T):
    """The spec of a token mask: u8, or bool, whose values are 0 and 1 too."""
    return "token_mask", t, torch.bool if t is not None and t.dtype is torch.bool else torch.uint8, T


def moe_train_logits(cfg: Config, ws: torch.Tensor) -> torch.Tensor:
    """The router's logits [T, E] fp32 that moe_forward_train left in its workspace (a view of it)."""
    off = int(lib().moe_train_logits_offset(ctypes.byref(cfg)))
    if off == 0:
        raise ValueError("moe_train_logits: not a configuration of moe_forward_train")
    return ws[off:off + 4 * cfg.T * cfg.E].view(torch.float32).view(cfg.T, cfg.E)


def moe_balance_workspace_size(T: int, E: int, S: int = 1) -> int:
    return int(lib().moe_balance_workspace_size(T, E, S))


def moe_balance_loss(T, E, k, logits, topk_idx, token_mask, seq_offsets, S, alpha, beta, loss, counts, mean_prob, lse,
                     seq_valid, ws, stream=None):
    """Balance loss and z-loss of the router's logits; token_mask, seq_offsets nullable."""
    p = _args("moe_balance_loss", ("logits", logits, _F32, T * E), ("topk_idx", topk_idx, _I32, T * k), _mask(token_mask, T),
              ("seq_offsets", seq_offsets, _I32, S + 1), ("loss", loss, _F32, 2), ("counts", counts, _I32, S * E),
              ("mean_prob", mean_prob, _F32, S * E), ("lse", lse, _F32, T), ("seq_valid", seq_valid, _I32, S + 2),
              ("ws", ws, None, 0))
    _check(lib().moe_balance_loss(T, E, k, *p[:4], S, alpha, beta, *p[4:], _nbytes(ws), _stream(stream)),
           "moe_balance_loss")


def moe_balance_loss_backward(T, E, k, logits, lse, counts, seq_valid, token_mask, seq_offsets, S, alpha, beta, dloss,
                              dlogits, stream=None):
    """dlogits [T, E] of moe_balance_loss; dloss [2] nullable (ones)."""
    p = _args("moe_balance_loss_backward", ("logits", logits, _F32, T * E), ("lse", lse, _F32, T),
              ("counts", counts, _I32, S * E), ("seq_valid", seq_valid, _I32, S + 2), _mask(token_mask, T),
              ("seq_offsets", seq_offsets, _I32, S + 1), ("dloss", dloss, _F32, 2), ("dlogits", dlogits, _F32, T * E))
    _check(lib().moe_balance_loss_backward(T, E, k, *p[:6], S, alpha, beta, *p[6:], _stream(stream)),
           "moe_balance_loss_backward")


def moe_router_backward_workspace_size(T: int, H: int, E: int) -> int:
    return int(lib().moe_router_backward_workspace_size(T, H, E))


def moe_router_backward(T, H, E, x, Wg, dlogits, dx0, dWg0, db0, dx, dWg, db, ws, stream=None):
    """dx = dx0 + dlogits Wg, dWg = dWg0 + dlogits^T x, db = db0 + sum of dlogits; the bases nullable."""
    p = _args("moe_router_backward", ("x", x, _BF16, T * H), ("Wg", Wg, _F32, E * H), ("dlogits", dlogits, _F32, T * E),
              ("dx0", dx0, _BF16, T * H), ("dWg0", dWg0, _F32, E * H), ("db0", db0, _F32, E), ("dx", dx, _BF16, T * H),
              ("dWg", dWg, _F32, E * H), ("db", db, _F32, E), ("ws", ws, None, 0))
    _check(lib().moe_router_backward(T, H, E, *p, _nbytes(ws), _stream(stream)), "moe_router_backward")


def moe_orthogonalise_workspace_size(batch: int, M: int, N: int, interleaved: bool = False) -> int:
    return int(lib().moe_orthogonalise_workspace_size(batch, M, N, int(bool(interleaved))))


def moe_orthogonalise(batch, M, N, interleaved, G, steps, a, b, c, eps, scale, O, ws, stream=None):
    """O = scale * the quintic Newton-Schulz iterate of each matrix of G (bf16 or fp32) after `steps` steps."""
    f32 = G.dtype is _F32
    n = batch * M * N * (2 if interleaved else 1)
    g, o, w = _args("moe_orthogonalise", ("G", G, _F32 if f32 else _BF16, n), ("O", O, _BF16, n), ("ws", ws, None, 0))
    _check(lib().moe_orthogonalise(batch, M, N, int(bool(interleaved)), g, TYPE_FP32 if f32 else TYPE_BF16, steps, a,
                                   b, c, eps, scale, o, w, _nbytes(ws), _stream(stream)), "moe_orthogonalise")
