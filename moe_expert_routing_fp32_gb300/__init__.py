"""Python binding of libmoe, a GB300 (sm_103a) MoE feed-forward layer.

Argument marshalling only: every function below checks dtypes/devices,
allocates its outputs with torch on the input's device and calls the
same-named C entry point of ``libmoe.so`` on torch's current stream.  All
arithmetic runs in the library's CUDA kernels.  There is no fallback: if the
library is missing or no suitable GPU is present the call raises.

The layer follows "NPU HunyuanImage-3.0模型推理优化实践" (HunyuanImage-3.0 MoE
block: RMSNorm, fp32 gate, GatingTopK, init_routing, compute_expert_tokens,
grouped matmul with SwiGLU on the merged w13 weight, down projection,
finalize_routing, shared expert).  See include/moe.h for the contracts.

Two fp32 gates: ``rmsnorm_gate`` sums each logit sequentially (the oracle's
order, bit for bit); ``gate_tensor`` sums the same exact products on the
tensor cores (the weight split exactly into three bf16 parts), which the
layer uses above 512 tokens unless ``make_desc(..., gate_sequential=True)``.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
import os
import threading
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_OK = 0
STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED_SHAPE",
                3: "MOE_ERR_WORKSPACE_TOO_SMALL", 4: "MOE_ERR_CUDA", 5: "MOE_ERR_NO_DEVICE"}
DEV_BAD_EXPERT_ID, DEV_TIMEOUT, DEV_BAD_OFFSETS, DEV_UNSORTED = 1, 2, 4, 8
RENORM, RMSNORM, SHARED, OUT_F32, SHARED_F32, GATE_SEQUENTIAL, Y_F32 = 1, 2, 4, 8, 16, 32, 64
GATHER_A = 128

# every symbol include/moe.h declares
EXPORTS = ("moe_status_string", "moe_rmsnorm_gate", "moe_rmsnorm_sumsq",
           "moe_gate_tensor_workspace_size",
           "moe_gate_tensor", "moe_gate_topk",
           "moe_init_routing_workspace_size", "moe_init_routing", "moe_init_routing_noalloc",
           "moe_expert_tokens",
           "moe_grouped_mlp", "moe_finalize_routing", "moe_layer_workspace_size",
           "moe_layer_forward", "moe_layer_forward_timed", "moe_layer_forward_streams",
           "moe_layer_forward_host", "moe_local_rerouting",
           "moe_local_finalize_rerouting", "moe_selftest_wait_timeout",
           "moe_balance_loss_workspace_size", "moe_balance_loss", "moe_gate_topk_backward",
           "moe_finalize_routing_backward", "moe_fp4_scales_size", "moe_fp4_quantize",
           "moe_fp4_dequantize", "moe_fp4_grouped_matmul", "moe_fp4_grouped_swiglu",
           "moe_fp4_grouped_mlp")
NUM_STAGES = 6
STAGE_NAMES = ("router", "route_scan_scatter", "permute", "gemm_w13_swiglu", "gemm_down",
               "finalize")


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: {STATUS_NAMES.get(status, status)}")
        self.status = status


class MoeDesc(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32), ("I", ctypes.c_int32), ("I_shared", ctypes.c_int32),
                ("rms_eps", ctypes.c_float), ("flags", ctypes.c_uint32)]


class _Fp4(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("sf", ctypes.c_void_p), ("format", ctypes.c_int32),
                ("scale_exp", ctypes.c_int32)]


FP4_FORMATS = {"mx": 0, "nv": 1}

_lock = threading.Lock()
_lib = None


def build(force: bool = False) -> str:
    from . import native_build
    return native_build.build(force=force)


def lib() -> ctypes.CDLL:
    """The loaded libmoe.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"libmoe.so not found at {LIB_PATH}: build it with "
                    "`python -m moe_expert_routing_fp32_gb300.native_build` (no CPU fallback exists)")
            L = ctypes.CDLL(LIB_PATH)
            P, I32, U32, F, SZ = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32,
                                  ctypes.c_float, ctypes.c_size_t)
            PSZ = ctypes.POINTER(ctypes.c_size_t)
            sigs = {
                "moe_rmsnorm_gate": [P, P, P, P, I32, I32, I32, F, U32, P, P, P],
                "moe_rmsnorm_sumsq": [P, I32, I32, P, P],
                "moe_gate_tensor_workspace_size": [I32, I32, I32, PSZ],
                "moe_gate_tensor": [P, P, P, I32, I32, I32, P, P, SZ, P, P],
                "moe_gate_topk": [P, I32, I32, I32, U32, P, P, P],
                "moe_init_routing_workspace_size": [I32, I32, I32, PSZ],
                "moe_init_routing": [P, P, I32, I32, I32, I32, P, P, P, P, P, P, P, SZ, P, P],
                "moe_init_routing_noalloc": [P, P, I32, I32, I32, I32, P, P, P, P, P, P, P, P],
                "moe_expert_tokens": [P, I32, I32, P, P, P, P],
                "moe_grouped_mlp": [P, P, I32, P, P, I32, I32, I32, P, P, P, P],
                "moe_finalize_routing": [P, P, P, P, I32, I32, I32, U32, P, P],
                "moe_layer_workspace_size": [ctypes.POINTER(MoeDesc), PSZ],
                "moe_layer_forward": [ctypes.POINTER(MoeDesc), P, P, P, P, P, P, P, P, P, P,
                                      SZ, P, P],
                "moe_layer_forward_timed": [ctypes.POINTER(MoeDesc), P, P, P, P, P, P, P, P, P,
                                            P, SZ, P, P, P],
                "moe_layer_forward_streams": [ctypes.POINTER(MoeDesc), P, P, P, P, P, P, P, P, P,
                                              P, SZ, P, P, P, P, P, P],
                "moe_layer_forward_host": [ctypes.POINTER(MoeDesc), I32, P, P, P, P, P, P, P, P,
                                           P, P, P, P, SZ, P, P, P, P, P],
                "moe_balance_loss_workspace_size": [I32, I32, I32, PSZ],
                "moe_balance_loss": [P, P, P, P, I32, I32, I32, I32, F, P, P, P, P, P, SZ, P, P],
                "moe_gate_topk_backward": [P, P, P, P, P, I32, P, P, P, F, I32, I32, I32, U32, P,
                                           P, P],
                "moe_finalize_routing_backward": [P, P, P, P, I32, I32, I32, U32, P, P, P, P],
                "moe_fp4_scales_size": [I32, I32, I32, I32, PSZ],
                "moe_fp4_quantize": [P, I32, I32, P, I32, P, I32, P, P, P],
                "moe_fp4_dequantize": [P, I32, I32, P, I32, P, P],
                "moe_fp4_grouped_matmul": [P, P, I32, P, I32, I32, I32, U32, P, P, P],
                "moe_fp4_grouped_swiglu": [P, P, I32, P, I32, I32, I32, P, P, P, P],
                "moe_fp4_grouped_mlp": [P, P, I32, P, P, I32, I32, I32, U32, P, P, P, P],
            }
            for name, args in sigs.items():
                fn = getattr(L, name)
                fn.argtypes = args
                fn.restype = ctypes.c_int
            L.moe_local_rerouting.argtypes = [P, P, I32, I32, I32, I32, P, P, P, P, P, P]
            L.moe_local_rerouting.restype = ctypes.c_int
            L.moe_local_finalize_rerouting.argtypes = [P, P, I32, I32, P, P]
            L.moe_local_finalize_rerouting.restype = ctypes.c_int
            L.moe_selftest_wait_timeout.argtypes = [P, P]
            L.moe_selftest_wait_timeout.restype = ctypes.c_int
            L.moe_status_string.argtypes = [ctypes.c_int]
            L.moe_status_string.restype = ctypes.c_char_p
            _lib = L
    return _lib


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libmoe takes CUDA tensors only")
    if not t.is_contiguous():
        raise ValueError("libmoe takes contiguous tensors only")
    return t.data_ptr()


# the handle of a device's current stream without the Stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device) -> int:
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _call(name: str, *args):
    st = getattr(_lib or lib(), name)(*args)
    if st != MOE_OK:
        raise MoeError(name, st)


class _Here:
    """Nothing to switch: the tensors' device is the current one."""

    def __enter__(self):
        pass

    def __exit__(self, *exc):
        pass


_here = _Here()


def _on(dev):
    """The context in which a call for tensors on ``dev`` is made (entering
    torch.cuda.device costs more than the call where nothing changes)."""
    if dev.type == "cuda" and dev.index == torch.cuda.current_device():
        return _here
    return torch.cuda.device(dev)


def _check(t, dtype, name):
    if t is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")


def local_rerouting(recv_x, recv_counts, with_rows=True, status=None):
    """EP local step: -> dict(local_x, local_src, local_counts, local_offsets)."""
    _check(recv_x, torch.bfloat16, "recv_x")
    _check(recv_counts, torch.int32, "recv_counts")
    R, H = recv_x.shape
    ep, El = recv_counts.shape
    dev = recv_x.device
    lx = torch.empty_like(recv_x) if with_rows else None
    src = torch.empty(R, dtype=torch.int32, device=dev)
    lc = torch.empty(El, dtype=torch.int32, device=dev)
    lo = torch.empty(El + 1, dtype=torch.int32, device=dev)
    _call("moe_local_rerouting", _ptr(recv_x), _ptr(recv_counts), ep, El, R, H, _ptr(lx),
          _ptr(src), _ptr(lc), _ptr(lo), _ptr(status), _stream(dev))
    return dict(local_x=lx, local_src=src, local_counts=lc, local_offsets=lo)


def local_finalize_rerouting(local_y, local_src, recv_y=None):
    """EP local step: recv_y[local_src[d]] = local_y[d]."""
    _check(local_y, torch.bfloat16, "local_y")
    R, H = local_y.shape
    if recv_y is None:
        recv_y = torch.zeros_like(local_y)
    _call("moe_local_finalize_rerouting", _ptr(local_y), _ptr(local_src), R, H, _ptr(recv_y),
          _stream(local_y.device))
    return recv_y


def selftest_wait_timeout(status):
    """Enqueue the bounded-wait check (see include/moe.h); sets DEV_TIMEOUT."""
    _call("moe_selftest_wait_timeout", _ptr(status), _stream(status.device))


def new_status(device) -> torch.Tensor:
    """A zeroed device int32 for the MOE_DEV_* bits."""
    return torch.zeros(1, dtype=torch.int32, device=device)


# ----------------------------------------------------------------- operations
def rmsnorm_gate(x, wg, gamma=None, gate_bias=None, eps=1e-6, rmsnorm=True):
    """-> (xn or None, logits fp32 [T, E]); with wg None: (xn, None) from the
    RMSNorm-only pass."""
    _check(x, torch.bfloat16, "x")
    _check(wg, torch.float32, "wg")
    _check(gamma, torch.bfloat16, "gamma")
    _check(gate_bias, torch.float32, "gate_bias")
    T, H = x.shape
    if wg is None:
        xn = torch.empty_like(x)
        _call("moe_rmsnorm_gate", _ptr(x), _ptr(gamma), None, None, T, H, 1, float(eps),
              RMSNORM, _ptr(xn), None, _stream(x.device))
        return xn, None
    E = wg.shape[0]
    logits = torch.empty((T, E), dtype=torch.float32, device=x.device)
    xn = torch.empty_like(x) if rmsnorm else None
    _call("moe_rmsnorm_gate", _ptr(x), _ptr(gamma), _ptr(wg), _ptr(gate_bias), T, H, E,
          float(eps), RMSNORM if rmsnorm else 0, _ptr(xn), _ptr(logits), _stream(x.device))
    return xn, logits


def rmsnorm_sumsq(x):
    """-> float32 [T]: each row's sum of squares as the RMSNorm takes it (the
    exact sum of the bf16 squares rounded once to fp32)."""
    _check(x, torch.bfloat16, "x")
    T, H = x.shape
    ss = torch.empty(T, dtype=torch.float32, device=x.device)
    _call("moe_rmsnorm_sumsq", _ptr(x), T, H, _ptr(ss), _stream(x.device))
    return ss


def gate_tensor_workspace_size(T, H, E) -> int:
    n = ctypes.c_size_t(0)
    _call("moe_gate_tensor_workspace_size", T, H, E, ctypes.byref(n))
    return n.value


def gate_tensor(xs, wg, gate_bias=None, workspace=None, status=None):
    """The tensor-core fp32 gate on already-normalised rows -> logits fp32 [T, E]."""
    _check(xs, torch.bfloat16, "xs")
    _check(wg, torch.float32, "wg")
    _check(gate_bias, torch.float32, "gate_bias")
    T, H = xs.shape
    E = wg.shape[0]
    logits = torch.empty((T, E), dtype=torch.float32, device=xs.device)
    need = gate_tensor_workspace_size(T, H, E)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=xs.device)
    _call("moe_gate_tensor", _ptr(xs), _ptr(wg), _ptr(gate_bias), T, H, E, _ptr(logits),
          _ptr(workspace), workspace.numel(), _ptr(status), _stream(xs.device))
    return logits


def gate_topk(logits, k, renorm=True):
    """-> (topk_idx int32 [T, k], topk_w fp32 [T, k])."""
    _check(logits, torch.float32, "logits")
    T, E = logits.shape
    idx = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    w = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    _call("moe_gate_topk", _ptr(logits), T, E, k, RENORM if renorm else 0, _ptr(idx), _ptr(w),
          _stream(logits.device))
    return idx, w


def init_routing(topk_idx, x, E, with_rows=True, status=None):
    """-> dict(expanded_x, row_idx, src_token, sorted_ids, counts, offsets)."""
    _check(topk_idx, torch.int32, "topk_idx")
    _check(x, torch.bfloat16, "x")
    T, k = topk_idx.shape
    dev = topk_idx.device
    H = x.shape[1] if x is not None else 0
    N = T * k
    ex = torch.empty((N, H), dtype=torch.bfloat16, device=dev) if (with_rows and x is not None) \
        else None
    row_idx = torch.empty(N, dtype=torch.int32, device=dev)
    src = torch.empty(N, dtype=torch.int32, device=dev)
    sorted_ids = torch.empty(N, dtype=torch.int32, device=dev)
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    nbytes = ctypes.c_size_t(0)
    _call("moe_init_routing_workspace_size", T, k, E, ctypes.byref(nbytes))
    ws = torch.empty(max(nbytes.value, 256), dtype=torch.uint8, device=dev)
    _call("moe_init_routing", _ptr(topk_idx), _ptr(x if ex is not None else None), T, H, E, k,
          _ptr(ex), _ptr(row_idx), _ptr(src), _ptr(sorted_ids), _ptr(counts), _ptr(offsets),
          _ptr(ws), nbytes.value, _ptr(status), _stream(dev))
    return dict(expanded_x=ex, row_idx=row_idx, src_token=src, sorted_ids=sorted_ids,
                counts=counts, offsets=offsets)


def expert_tokens(sorted_ids, E, status=None):
    """-> (counts int32 [E], offsets int32 [E+1])."""
    _check(sorted_ids, torch.int32, "sorted_ids")
    dev = sorted_ids.device
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    _call("moe_expert_tokens", _ptr(sorted_ids), sorted_ids.numel(), E, _ptr(counts),
          _ptr(offsets), _ptr(status), _stream(dev))
    return counts, offsets


def grouped_mlp(expanded_x, offsets, w13, w2, status=None):
    """-> (act bf16 [n, I], y bf16 [n, H])."""
    _check(expanded_x, torch.bfloat16, "expanded_x")
    _check(offsets, torch.int32, "offsets")
    _check(w13, torch.bfloat16, "w13")
    _check(w2, torch.bfloat16, "w2")
    n, H = expanded_x.shape
    G, I2, _ = w13.shape
    I = I2 // 2
    act = torch.zeros((n, I), dtype=torch.bfloat16, device=expanded_x.device)
    y = torch.zeros((n, H), dtype=torch.bfloat16, device=expanded_x.device)
    _call("moe_grouped_mlp", _ptr(expanded_x), _ptr(offsets), G, _ptr(w13), _ptr(w2), n, H, I,
          _ptr(act), _ptr(y), _ptr(status), _stream(expanded_x.device))
    return act, y


def finalize_routing(y_exp, row_idx, topk_w, shared=None, out_f32=False):
    """-> out [T, H] (bf16, or fp32 with out_f32).  y_exp bf16 or fp32."""
    if y_exp.dtype != torch.float32:
        _check(y_exp, torch.bfloat16, "y_exp")
    _check(row_idx, torch.int32, "row_idx")
    _check(topk_w, torch.float32, "topk_w")
    T, k = topk_w.shape
    H = y_exp.shape[1]
    flags = (OUT_F32 if out_f32 else 0) | (Y_F32 if y_exp.dtype == torch.float32 else 0)
    if shared is not None:
        if shared.dtype == torch.float32:
            flags |= SHARED_F32
        else:
            _check(shared, torch.bfloat16, "shared")
    out = torch.empty((T, H), dtype=torch.float32 if out_f32 else torch.bfloat16,
                      device=y_exp.device)
    _call("moe_finalize_routing", _ptr(y_exp), _ptr(row_idx), _ptr(topk_w), _ptr(shared), T, H,
          k, flags, _ptr(out), _stream(y_exp.device))
    return out


# ------------------------------------------------------- training the router
def _arg(t, dtype, dev, shape, name):
    """The address of an optional tensor, checked in one place: its type, its
    device (the call's), its shape (None: any) and that it is contiguous."""
    if t is None:
        return None
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"libmoe takes contiguous tensors only ({name})")
    return t.data_ptr()


def _status_arg(status, dev):
    return _arg(status, torch.int32, dev, None, "status")


def _router_args(logits, topk_idx, token_mask, seq_offsets):
    """(T, E, k, S, device, the four addresses) of the router's operators."""
    T, E = logits.shape
    k = topk_idx.shape[-1]
    dev = logits.device
    lg = _arg(logits, torch.float32, dev, None, "logits")
    idx = _arg(topk_idx, torch.int32, dev, (T, k), "topk_idx")
    mask = seq = None
    S = 1
    if token_mask is not None:
        mask = _arg(token_mask, torch.bool if token_mask.dtype == torch.bool else torch.uint8, dev,
                    (T,), "token_mask")
    if seq_offsets is not None:
        S = seq_offsets.numel() - 1
        if S < 1:
            raise ValueError("seq_offsets: [S + 1] with S >= 1")
        seq = _arg(seq_offsets, torch.int32, dev, (S + 1,), "seq_offsets")
    return T, E, k, S, dev, (lg, idx, mask, seq)


@functools.lru_cache(maxsize=256)
def _balance_workspace(T, E, S, device_index) -> int:
    n = ctypes.c_size_t(0)
    _call("moe_balance_loss_workspace_size", T, E, S, ctypes.byref(n))
    return n.value


def balance_loss(logits, topk_idx, coef=1.0, token_mask=None, seq_offsets=None, status=None):
    """Balance loss of the router over the sequences given by ``seq_offsets``
    (int32 [S+1]; None: all tokens are one), without the tokens whose
    ``token_mask`` (bool or uint8 [T]) is zero.
    -> dict(loss fp32 [], counts int32 [S, E], prob_mean fp32 [S, E],
    n_tokens int32 [S], coef); gate_topk_backward takes the dict."""
    T, E, k, S, dev, (lg, idx, mask, seq) = _router_args(logits, topk_idx, token_mask, seq_offsets)
    st = _status_arg(status, dev)
    coef = float(coef)
    with _on(dev):
        nbytes = _balance_workspace(T, E, S, dev.index)
        loss = torch.empty((), dtype=torch.float32, device=dev)
        counts = torch.empty((S, E), dtype=torch.int32, device=dev)
        prob = torch.empty((S, E), dtype=torch.float32, device=dev)
        n_tokens = torch.empty(S, dtype=torch.int32, device=dev)
        ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        _call("moe_balance_loss", lg, idx, mask, seq, S, T, E, k, coef, loss.data_ptr(),
              counts.data_ptr(), prob.data_ptr(), n_tokens.data_ptr(), ws.data_ptr(), nbytes, st,
              _stream(dev))
    return dict(loss=loss, counts=counts, prob_mean=prob, n_tokens=n_tokens, coef=coef)


def gate_topk_backward(logits, topk_idx, d_topk_w=None, renorm=True, balance=None, d_loss=None,
                       token_mask=None, seq_offsets=None, status=None):
    """Gradient of the gate's logits (fp32 [T, E]) from ``d_topk_w`` (the
    gradient of gate_topk's weights, or None) and, with ``balance`` (what
    balance_loss returned for the same logits, mask and bounds), from the
    balance loss times ``d_loss`` (fp32 [1] or [], None: 1)."""
    T, E, k, S, dev, (lg, idx, mask, seq) = _router_args(logits, topk_idx, token_mask, seq_offsets)
    dw = _arg(d_topk_w, torch.float32, dev, (T, k), "d_topk_w")
    st = _status_arg(status, dev)
    counts = n_tokens = dl = None
    coef = 0.0
    if balance is not None:
        coef = balance["coef"]
        counts = _arg(balance["counts"], torch.int32, dev, (S, E), "counts")
        n_tokens = _arg(balance["n_tokens"], torch.int32, dev, (S,), "n_tokens")
        if d_loss is not None:
            if d_loss.numel() != 1:
                raise ValueError("d_loss must hold one value")
            dl = _arg(d_loss, torch.float32, dev, None, "d_loss")
    with _on(dev):
        d = torch.empty_like(logits)
        _call("moe_gate_topk_backward", lg, idx, dw, mask, seq, S, counts, n_tokens, dl, coef, T,
              E, k, RENORM if renorm else 0, d.data_ptr(), st, _stream(dev))
    return d


def _bf16_or_f32(t, name):
    if t.dtype != torch.float32 and t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16 or torch.float32, got {t.dtype}")
    return t.dtype


def finalize_routing_backward(d_out, y_exp, row_idx, topk_w, status=None):
    """-> (d_y_exp like y_exp, d_topk_w fp32 [T, k]) from the gradient of
    finalize_routing's output (bf16 or fp32).  The shared rows' gradient is
    d_out itself.  Rows of d_y_exp that row_idx does not name are not set."""
    T, k = topk_w.shape
    H = y_exp.shape[1]
    dev = y_exp.device
    dt, yt = _bf16_or_f32(d_out, "d_out"), _bf16_or_f32(y_exp, "y_exp")
    do = _arg(d_out, dt, dev, (T, H), "d_out")
    y = _arg(y_exp, yt, dev, (T * k, H), "y_exp")
    rows = _arg(row_idx, torch.int32, dev, None, "row_idx")
    w = _arg(topk_w, torch.float32, dev, None, "topk_w")
    st = _status_arg(status, dev)
    if row_idx.numel() != T * k:
        raise ValueError("row_idx must hold T * k rows")
    flags = (OUT_F32 if dt == torch.float32 else 0) | (Y_F32 if yt == torch.float32 else 0)
    with _on(dev):
        d_y = torch.empty_like(y_exp)
        d_w = torch.empty_like(topk_w)
        _call("moe_finalize_routing_backward", do, y, rows, w, T, H, k, flags, d_y.data_ptr(),
              d_w.data_ptr(), st, _stream(dev))
    return d_y, d_w


# ------------------------------------------------------------ 4-bit operands
@dataclasses.dataclass
class Fp4Matrix:
    """A microscaled 4-bit matrix: codes ``q`` (uint8 [rows, K/2], weights
    [G, rows, K/2]), scale tiles ``sf`` (uint8, see include/moe.h), ``fmt``
    "mx" or "nv" and, for "nv", the exponent of the whole matrix."""
    q: torch.Tensor
    sf: torch.Tensor
    fmt: str = "mx"
    scale_exp: int = 0

    @property
    def K(self) -> int:
        return self.q.shape[-1] * 2


@functools.lru_cache(maxsize=256)
def fp4_scales_size(rows, K, fmt="mx", groups=0) -> int:
    """Bytes of the scale tiles of ``rows`` rows (in ``groups`` groups; 0 for
    an ungrouped matrix such as a weight)."""
    n = ctypes.c_size_t(0)
    _call("moe_fp4_scales_size", rows, K, groups, _fp4_format(fmt), ctypes.byref(n))
    return n.value


def _fp4_format(fmt) -> int:
    if fmt not in FP4_FORMATS:
        raise ValueError(f"fmt must be one of {sorted(FP4_FORMATS)}, got {fmt!r}")
    return FP4_FORMATS[fmt]


def _fp4_empty(rows, K, fmt, scale_exp, groups, dev) -> Fp4Matrix:
    return Fp4Matrix(torch.empty((rows, K // 2), dtype=torch.uint8, device=dev),
                     torch.empty(fp4_scales_size(rows, K, fmt, groups), dtype=torch.uint8,
                                 device=dev), fmt, int(scale_exp))


def _fp4_arg(m: Fp4Matrix, name, groups, dev):
    """The C struct of a matrix, its buffers checked against the layout."""
    q, sf = m.q, m.sf
    qp = _arg(q, torch.uint8, dev, None, name)
    sp = _arg(sf, torch.uint8, dev, None, name)
    half = q.shape[-1]
    if sf.numel() < fp4_scales_size(q.numel() // half if half else 0, half * 2, m.fmt, groups):
        raise ValueError(f"{name}.sf is smaller than its scale tiles")
    return ctypes.byref(_Fp4(qp, sp, FP4_FORMATS[m.fmt], m.scale_exp))


def _groups_arg(offsets, dev):
    """(address, G) of optional group offsets."""
    if offsets is None:
        return None, 0
    return _arg(offsets, torch.int32, dev, None, "offsets"), offsets.numel() - 1


def fp4_quantize(x, fmt="mx", scale_exp=0, row_idx=None, k=1, offsets=None,
                 status=None) -> Fp4Matrix:
    """bf16 rows to 4 bits.  With ``row_idx`` (init_routing's, int32 [T*k]) and
    ``offsets``, token rows go to their k rows in expert order.  A weight
    [G, N, K] keeps its shape in ``q`` and is quantised ungrouped.  Rows that
    row_idx does not name are not set.  A block that holds an infinity or a NaN
    becomes NaN."""
    dev = x.device
    xp = _arg(x, torch.bfloat16, dev, None, "x")
    rows = _arg(row_idx, torch.int32, dev, None, "row_idx")
    off, G = _groups_arg(offsets, dev)
    st = _status_arg(status, dev)
    K = x.shape[-1]
    T = x.numel() // K if K else 0
    if row_idx is None:
        if k != 1:
            raise ValueError("k needs row_idx")
    elif row_idx.numel() != T * k:
        raise ValueError("row_idx must hold T * k rows")
    with _on(dev):
        m = _fp4_empty(T * k, K, fmt, scale_exp, G, dev)
        _call("moe_fp4_quantize", xp, T, K, rows, k, off, G, _fp4_arg(m, "out", G, dev), st,
              _stream(dev))
    if x.dim() != 2:
        m.q = m.q.view(*x.shape[:-1], K // 2)
    return m


def fp4_dequantize(m: Fp4Matrix, offsets=None):
    """-> bf16 values of a 4-bit matrix, exact (``offsets`` as it was made
    with; rows past the last group are not set)."""
    dev = m.q.device
    off, G = _groups_arg(offsets, dev)
    K = m.K
    arg = _fp4_arg(m, "m", G, dev)
    with _on(dev):
        x = torch.empty((*m.q.shape[:-1], K), dtype=torch.bfloat16, device=dev)
        _call("moe_fp4_dequantize", arg, x.numel() // K if K else 0, K, off, G, x.data_ptr(),
              _stream(dev))
    return x


def _fp4_product(a, offsets, w, name):
    """(n, K, G, rows of a group's weights, device, offsets' address)."""
    if a.q.dim() != 2 or w.q.dim() != 3 or a.q.shape[1] != w.q.shape[2]:
        raise ValueError(f"{name}: a [n, K/2] and weights [G, rows, K/2] of the same K")
    n, half = a.q.shape
    G, rows, _ = w.q.shape
    dev = a.q.device
    return n, half * 2, G, rows, dev, _arg(offsets, torch.int32, dev, (G + 1,), "offsets")


def fp4_grouped_matmul(a: Fp4Matrix, offsets, w: Fp4Matrix, out_f32=False, out=None, status=None):
    """y = a . w[group]^T -> [n, N] bf16 (fp32 with out_f32).  Rows past the
    last group are left as they were in ``out`` (not set without it)."""
    n, K, G, N, dev, off = _fp4_product(a, offsets, w, "fp4_grouped_matmul")
    aa, wa, st = _fp4_arg(a, "a", G, dev), _fp4_arg(w, "w", 0, dev), _status_arg(status, dev)
    dt = torch.float32 if out_f32 else torch.bfloat16
    with _on(dev):
        if out is None:
            out = torch.empty((n, N), dtype=dt, device=dev)
        _call("moe_fp4_grouped_matmul", aa, off, G, wa, n, K, N, Y_F32 if out_f32 else 0,
              _arg(out, dt, dev, (n, N), "out"), st, _stream(dev))
    return out


def fp4_grouped_swiglu(a: Fp4Matrix, offsets, w13: Fp4Matrix, quantize=False, scale_exp=0,
                       out=None, status=None):
    """act = SiLU(gate) * up of the merged w13 [G, 2I, K] -> bf16 [n, I], or
    with ``quantize`` the same values in 4 bits (an Fp4Matrix of a's format,
    grouped by ``offsets``; blocks with values beyond bf16's range are NaN)."""
    n, K, G, rows, dev, off = _fp4_product(a, offsets, w13, "fp4_grouped_swiglu")
    if rows % 2:
        raise ValueError("w13 must hold an even number of rows, gate then up")
    I = rows // 2
    aa, wa, st = _fp4_arg(a, "a", G, dev), _fp4_arg(w13, "w13", 0, dev), _status_arg(status, dev)
    with _on(dev):
        if quantize:
            if out is None:
                out = _fp4_empty(n, I, a.fmt, scale_exp, G, dev)
            elif out.q.shape != (n, I // 2):
                raise ValueError(f"out.q must have shape {(n, I // 2)}")
            bf, q4 = None, _fp4_arg(out, "out", G, dev)
        else:
            if out is None:
                out = torch.empty((n, I), dtype=torch.bfloat16, device=dev)
            bf, q4 = _arg(out, torch.bfloat16, dev, (n, I), "out"), None
        _call("moe_fp4_grouped_swiglu", aa, off, G, wa, n, K, I, bf, q4, st, _stream(dev))
    return out


def fp4_grouped_mlp(expanded_x: Fp4Matrix, offsets, w13: Fp4Matrix, w2: Fp4Matrix, y_f32=False,
                    act_exp=0, status=None):
    """-> (act Fp4Matrix [n, I], y bf16 [n, H], fp32 with y_f32)."""
    n, H, G, rows, dev, off = _fp4_product(expanded_x, offsets, w13, "fp4_grouped_mlp")
    I = rows // 2
    if rows % 2 or w2.q.shape != (G, H, I // 2):
        raise ValueError("w13 must be [G, 2I, H/2] and w2 [G, H, I/2]")
    xa, wa = _fp4_arg(expanded_x, "expanded_x", G, dev), _fp4_arg(w13, "w13", 0, dev)
    w2a, st = _fp4_arg(w2, "w2", 0, dev), _status_arg(status, dev)
    with _on(dev):
        act = _fp4_empty(n, I, expanded_x.fmt, act_exp, G, dev)
        y = torch.empty((n, H), dtype=torch.float32 if y_f32 else torch.bfloat16, device=dev)
        _call("moe_fp4_grouped_mlp", xa, off, G, wa, w2a, n, H, I, Y_F32 if y_f32 else 0,
              _fp4_arg(act, "act", G, dev), y.data_ptr(), st, _stream(dev))
    return act, y


def make_desc(T, H, E, k, I, I_shared=0, rmsnorm=False, eps=1e-6, renorm=True,
              out_f32=False, gate_sequential=False, y_f32=False, gather_a=False) -> MoeDesc:
    """``gate_sequential``: the sequential fp32 gate (moe_rmsnorm_gate's
    logits, bit for bit) instead of the tensor-core gate for T > 512.
    ``y_f32``: the routed expert outputs enter the weighted sum as the down
    matmul's fp32 accumulator instead of rounded to bf16 (MOE_Y_F32).
    ``gather_a``: the routed w13 matmul reads its rows by source token, with
    no permute pass, where it runs as the wide pair kernel (MOE_GATHER_A)."""
    flags = (RENORM if renorm else 0) | (RMSNORM if rmsnorm else 0) | \
        (SHARED if I_shared > 0 else 0) | (OUT_F32 if out_f32 else 0) | \
        (GATE_SEQUENTIAL if gate_sequential else 0) | (Y_F32 if y_f32 else 0) | \
        (GATHER_A if gather_a else 0)
    return MoeDesc(T, H, E, k, I, I_shared, eps, flags)


def layer_workspace_size(desc: MoeDesc) -> int:
    n = ctypes.c_size_t(0)
    _call("moe_layer_workspace_size", ctypes.byref(desc), ctypes.byref(n))
    return n.value


@dataclasses.dataclass
class LayerWeights:
    wg: torch.Tensor
    w13: torch.Tensor
    w2: torch.Tensor
    gamma: Optional[torch.Tensor] = None
    gate_bias: Optional[torch.Tensor] = None
    w13_s: Optional[torch.Tensor] = None
    w2_s: Optional[torch.Tensor] = None


def layer_forward(desc: MoeDesc, x, weights: LayerWeights, out=None, workspace=None,
                  status=None, stage_events=None, shared_stream=None, events=None):
    """The whole MoE layer.  ``workspace`` (uint8, >= layer_workspace_size)
    and ``out`` are allocated when not given.  ``stage_events``: a list of
    NUM_STAGES + 1 recorded-once torch.cuda.Event (timing enabled) to time
    the internal stages.  ``shared_stream`` (a torch.cuda.Stream) with
    ``events`` (two recorded-once torch.cuda.Event) runs the shared expert on
    that stream.  Returns ``out``."""
    _check(x, torch.bfloat16, "x")
    dev = x.device
    if out is None:
        out = torch.empty((desc.T, desc.H),
                          dtype=torch.float32 if desc.flags & OUT_F32 else torch.bfloat16,
                          device=dev)
    nbytes = layer_workspace_size(desc)
    if workspace is None:
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
    w = weights
    args = [ctypes.byref(desc), _ptr(x), _ptr(w.gamma), _ptr(w.wg), _ptr(w.gate_bias),
            _ptr(w.w13), _ptr(w.w2), _ptr(w.w13_s), _ptr(w.w2_s), _ptr(out), _ptr(workspace),
            workspace.numel(), _ptr(status), _stream(dev)]
    arr = None
    if stage_events is not None:
        assert len(stage_events) == NUM_STAGES + 1
        arr = (ctypes.c_void_p * (NUM_STAGES + 1))(*[e.cuda_event for e in stage_events])
    if shared_stream is not None:
        fork, join = events
        _call("moe_layer_forward_streams", *args, ctypes.c_void_p(shared_stream.cuda_stream),
              ctypes.c_void_p(fork.cuda_event), ctypes.c_void_p(join.cuda_event), arr)
    elif arr is None:
        _call("moe_layer_forward", *args)
    else:
        _call("moe_layer_forward_timed", *args, arr)
    return out


_host_pipes = {}


def _host_pipe(dev):
    """Per device: the two copy streams and six events of the host pipeline
    (created once; a torch event gets its CUDA handle on its first record)."""
    key = dev.index if dev.index is not None else torch.cuda.current_device()
    pipe = _host_pipes.get(key)
    if pipe is None:
        with torch.cuda.device(key):
            cin, cout = torch.cuda.Stream(), torch.cuda.Stream()
            evs = [torch.cuda.Event() for _ in range(6)]
            for e in evs:
                e.record(cin)
            cin.synchronize()
        pipe = _host_pipes[key] = (cin, cout, evs)
    return pipe


def layer_forward_host(desc: MoeDesc, x_host, weights: LayerWeights, out_host=None,
                       staging=None, workspace=None, status=None):
    """The layer on token batches in host memory (moe_layer_forward_host).
    ``x_host``: one [T, H] bf16 CPU tensor (pinned) or a list of them, one
    per batch; the outputs land in ``out_host`` (the same form; pinned CPU
    tensors are allocated when None).  Batch i+1's tokens are copied in and
    batch i-1's output copied out while batch i runs on the current stream.
    ``staging`` = (x_dev, out_dev): device tensors of 2*T*H elements
    (allocated when None).  Returns once the last output has arrived."""
    single = isinstance(x_host, torch.Tensor)
    xs = [x_host] if single else list(x_host)
    T, H = desc.T, desc.H
    odt = torch.float32 if desc.flags & OUT_F32 else torch.bfloat16
    for t in xs:
        if t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous() or \
                tuple(t.shape) != (T, H):
            raise ValueError("x_host: contiguous [T, H] bf16 CPU tensors")
    if out_host is None:
        outs = [torch.empty((T, H), dtype=odt, pin_memory=True) for _ in xs]
    else:
        outs = [out_host] if single else list(out_host)
    if len(outs) != len(xs):
        raise ValueError("one output per batch")
    for t in outs:
        if t.is_cuda or t.dtype != odt or not t.is_contiguous() or tuple(t.shape) != (T, H):
            raise ValueError(f"out_host: contiguous [T, H] {odt} CPU tensors")
    dev = weights.w13.device
    if staging is None:
        staging = (torch.empty((2, T, H), dtype=torch.bfloat16, device=dev),
                   torch.empty((2, T, H), dtype=odt, device=dev))
    x_dev, out_dev = staging
    if x_dev.numel() < 2 * T * H or out_dev.numel() < 2 * T * H or out_dev.dtype != odt:
        raise ValueError("staging: (x_dev, out_dev) with 2*T*H elements each")
    if workspace is None:
        workspace = torch.empty(max(layer_workspace_size(desc), 256), dtype=torch.uint8,
                                device=dev)
    cin, cout, evs = _host_pipe(dev)
    cur = torch.cuda.current_stream(dev)
    cin.wait_stream(cur)          # staging buffers and workspace as the caller left them
    cout.wait_stream(cur)
    n = len(xs)
    xa = (ctypes.c_void_p * n)(*[t.data_ptr() for t in xs])
    oa = (ctypes.c_void_p * n)(*[t.data_ptr() for t in outs])
    ea = (ctypes.c_void_p * 6)(*[e.cuda_event for e in evs])
    w = weights
    _call("moe_layer_forward_host", ctypes.byref(desc), n, xa, oa, _ptr(w.gamma), _ptr(w.wg),
          _ptr(w.gate_bias), _ptr(w.w13), _ptr(w.w2), _ptr(w.w13_s), _ptr(w.w2_s),
          _ptr(x_dev), _ptr(out_dev), _ptr(workspace), workspace.numel(), _ptr(status),
          _stream(dev), ctypes.c_void_p(cin.cuda_stream), ctypes.c_void_p(cout.cuda_stream), ea)
    cout.synchronize()
    return outs[0] if single else outs
