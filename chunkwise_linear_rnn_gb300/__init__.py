"""GB300-native gated linear attention (GLA): chunked prefill, its backward, and the decode step.

The computation ("Gated Linear Attention (GLA): Mathematical Foundations, ..."
(llms.blog), section "The Gated Recurrent Update"):

    S_t = diag(alpha_t) S_{t-1} + k_t^T v_t,      o_t = scale * q_t S_t

runs entirely in the hand-written sm_103a kernels of ``libgla.so``; this module
only checks and marshals PyTorch tensors into the C ABI of ``include/gla.h``
(device pointers, sizes and the current CUDA stream).

Layouts (contiguous, head-first): q, k ``[B,H,T,dk]`` bf16; v ``[B,H,T,dv]``
bf16; log_alpha ``[B,H,T,dk]`` fp32; o ``[B,H,T,dv]`` bf16; h0 / hT
``[B,H,dk,dv]`` fp32.
"""

from __future__ import annotations

import ctypes
import functools

import torch

from . import _lib
from ._lib import GlaChunkOptions, GlaError, status_string  # noqa: F401

__all__ = ["gla_chunk_fwd", "gla_chunk_fwd_varlen", "gla_chunk_fwd_varlen_plan",
           "gla_chunk_fwd_plan", "gla_chunk_bwd", "gla_chunk_bwd_plan", "gla_chunk_bwd_varlen",
           "gla_chunk", "gla_chunk_varlen", "gla_gdn_fwd",
           "gla_scan_fwd", "gla_scan_bwd", "gla_scan", "gla_scan_step", "gla_scan_fwd_varlen",
           "gla_scan_bwd_varlen", "gla_scan_varlen", "gla_scan_checkpoints",
           "gla_qk_norm_rope_fwd", "gla_qk_norm_rope_bwd", "gla_qk_norm_rope",
           "gla_rope_frequencies",
           "gla_recurrent_step", "gla_last_device_status", "GlaError", "status_string",
           "library_path"]

library_path = _lib.LIB_PATH


def _stream(device: torch.device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


@functools.lru_cache(maxsize=None)
def _entry(name: str):
    return getattr(_lib.lib(), name)


def _call(name: str, device: torch.device, *args) -> None:
    """A C entry point on the current stream of `device`; raises GlaError on a bad status."""
    index = device.index
    if torch.cuda.current_device() == index:
        st = _entry(name)(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(device):
            st = _entry(name)(*args, torch._C._cuda_getCurrentRawStream(index))
    if st:
        _lib.check(st, name)


def _once(backward):
    """`backward` of an autograd.Function whose gradients have no derivative of their own.

    A plain backward pass runs it as it is; one that builds a graph of the gradients gets
    torch's wrapper, which refuses the second derivative when it is asked for.
    """
    refusing = torch.autograd.function.once_differentiable(backward)

    def run(ctx, *grads):
        return (refusing if torch.is_grad_enabled() else backward)(ctx, *grads)

    return run


def _like(grad, dtype):
    """A gradient as the kernels take it: contiguous, of this type, at a multiple of 16 bytes;
    None stays None."""
    if grad is None:
        return None
    if grad.dtype is not dtype or not grad.is_contiguous():
        grad = grad.to(dtype).contiguous()
    return grad.clone() if grad.data_ptr() % 16 else grad


def _meta(t):
    """What the checks of a tensor argument look at."""
    return None if t is None else (t.shape, t.stride(), t.dtype, t.device)


def _fits(meta, name: str, dtype: torch.dtype, shape: tuple, device) -> None:
    """`_need` for a tensor's `_meta`; None fits."""
    if meta is None:
        return
    has, strides, kind, dev = meta
    if dev != device:
        raise ValueError(f"{name} must be on the CUDA device {device}")
    if kind != dtype:
        raise TypeError(f"{name} must be {dtype}, got {kind}")
    if tuple(has) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(has)}")
    step = 1
    for size, stride in zip(reversed(has), reversed(strides)):
        if size != 1 and stride != step and 0 not in has:
            raise ValueError(f"{name} must be contiguous")
        step *= size


def _all_tensors(**tensors) -> None:
    """Refuses an argument that is no tensor."""
    for name, t in tensors.items():
        if t is not None and not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")


def _apart(out, name: str, *others, also: str = "an input") -> None:
    """Refuses an output that shares memory with an input, or with what `also` names."""
    first, last = out.data_ptr(), out.data_ptr() + out.numel() * out.element_size()
    for t in others:
        if t is not None and first < t.data_ptr() + t.numel() * t.element_size() and \
                t.data_ptr() < last:
            raise ValueError(f"{name} must not share memory with {also}")


def _ints(*sizes) -> None:
    """Refuses sizes that the C calls' ints do not hold."""
    if max(sizes) > 0x7fffffff:
        raise ValueError("sizes must be below 2^31")


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, shape: tuple, device) -> None:
    """Checks a tensor argument; `device` is a CUDA device, or the CPU for host entry points."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and
            t.device == device and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if device is not None and device.type == "cpu":
        if t.device.type != "cpu":
            raise ValueError(f"{name} must be a CPU tensor")
    elif t.device.type != "cuda" or (device is not None and t.device != device):
        raise ValueError(f"{name} must be on the CUDA device {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def gla_chunk_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_alpha: torch.Tensor,
                  scale: float | None = None, h0: torch.Tensor | None = None,
                  output_final_state: bool = True, *, out: torch.Tensor | None = None,
                  final_state: torch.Tensor | None = None, segments: int = 0, dv_tile: int = 0,
                  force_exact: bool = False, cta_pair: int = 0):
    """Chunkwise-parallel GLA forward over whole sequences.

    ``log_alpha`` is ``[B, H, T, dk]`` (one gate per key channel) or
    ``[B, H, T]`` (one gate per token and head, used for every channel).
    Returns ``(o, hT)``; ``hT`` is None when ``output_final_state`` is False.
    ``final_state`` may be ``h0`` itself (in-place state update).
    ``segments``, ``dv_tile``, ``force_exact`` and ``cta_pair`` are the C ABI's
    options (0 / False = automatic; ``cta_pair=-1`` keeps the value tiles of a
    head in independent CTAs).
    """
    if q.dim() != 4:
        raise ValueError("q must be [B, H, T, dk]")
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("q must be on a CUDA device (gla_chunk_fwd_host takes CPU tensors)")
    _need(q, "q", torch.bfloat16, (B, H, T, dk), dev)
    _need(k, "k", torch.bfloat16, (B, H, T, dk), dev)
    _need(v, "v", torch.bfloat16, (B, H, T, dv), dev)
    # a [B, H, T] gate is one decay per token and head, the same for every channel
    per_head = log_alpha.dim() == 3
    _need(log_alpha, "log_alpha", torch.float32, (B, H, T) if per_head else (B, H, T, dk), dev)
    if h0 is not None:
        _need(h0, "h0", torch.float32, (B, H, dk, dv), dev)
    if out is None:
        out = torch.empty(B, H, T, dv, dtype=torch.bfloat16, device=dev)
    _need(out, "out", torch.bfloat16, (B, H, T, dv), dev)
    hT = None
    if output_final_state:
        hT = final_state if final_state is not None else torch.empty(
            B, H, dk, dv, dtype=torch.float32, device=dev)
        _need(hT, "final_state", torch.float32, (B, H, dk, dv), dev)
    if scale is None:
        scale = dk ** -0.5
    opts = GlaChunkOptions(segments=int(segments), dv_tile=int(dv_tile),
                           force_exact=1 if force_exact else 0, cta_pair=int(cta_pair),
                           gate_per_head=1 if per_head else 0)
    with torch.cuda.device(dev):
        st = _lib.lib().gla_chunk_fwd_ex(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), log_alpha.data_ptr(), float(scale),
            None if h0 is None else h0.data_ptr(), out.data_ptr(),
            None if hT is None else hT.data_ptr(), B, H, T, dk, dv, ctypes.byref(opts),
            _stream(dev))
    _lib.check(st, "gla_chunk_fwd")
    return out, hT


def gla_chunk_fwd_varlen(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                         log_alpha: torch.Tensor, cu_seqlens, scale: float | None = None,
                         h0: torch.Tensor | None = None, output_final_state: bool = True, *,
                         out: torch.Tensor | None = None, final_state: torch.Tensor | None = None,
                         segments: int = 0, dv_tile: int = 0, force_exact: bool = False,
                         cta_pair: int = 0):
    """Chunkwise-parallel GLA forward over a packed batch of variable-length sequences.

    ``q``, ``k``, ``log_alpha`` are ``[H, T_total, dk]`` and ``v`` is
    ``[H, T_total, dv]`` (a leading batch dimension of 1 is accepted too);
    sequence ``n`` holds rows ``cu_seqlens[n] : cu_seqlens[n+1]`` of every head.
    ``cu_seqlens`` is a host sequence of ``N + 1`` ints (list, tuple or CPU
    tensor).  ``h0`` and the returned ``hT`` are ``[N, H, dk, dv]``.
    Returns ``(o, hT)`` with ``o`` shaped like ``v``.
    """
    squeeze = q.dim() == 4
    if squeeze:
        if q.shape[0] != 1:
            raise ValueError("a packed batch has a leading dimension of 1")
        q, k, v, log_alpha = q[0], k[0], v[0], log_alpha[0]
        if out is not None:
            out = out[0]
    if q.dim() != 3:
        raise ValueError("q must be [H, T_total, dk]")
    H, T_total, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("q must be on a CUDA device")
    cu = [int(x) for x in (cu_seqlens.tolist() if torch.is_tensor(cu_seqlens) else cu_seqlens)]
    N = len(cu) - 1
    if N < 1:
        raise ValueError("cu_seqlens needs at least two entries")
    _need(q, "q", torch.bfloat16, (H, T_total, dk), dev)
    _need(k, "k", torch.bfloat16, (H, T_total, dk), dev)
    _need(v, "v", torch.bfloat16, (H, T_total, dv), dev)
    _need(log_alpha, "log_alpha", torch.float32, (H, T_total, dk), dev)
    if h0 is not None:
        _need(h0, "h0", torch.float32, (N, H, dk, dv), dev)
    if out is None:
        out = torch.empty(H, T_total, dv, dtype=torch.bfloat16, device=dev)
    _need(out, "out", torch.bfloat16, (H, T_total, dv), dev)
    hT = None
    if output_final_state:
        hT = final_state if final_state is not None else torch.empty(
            N, H, dk, dv, dtype=torch.float32, device=dev)
        _need(hT, "final_state", torch.float32, (N, H, dk, dv), dev)
    if scale is None:
        scale = dk ** -0.5
    opts = GlaChunkOptions(segments=int(segments), dv_tile=int(dv_tile),
                           force_exact=1 if force_exact else 0, cta_pair=int(cta_pair))
    cu_arr = (ctypes.c_int * len(cu))(*cu)
    with torch.cuda.device(dev):
        st = _lib.lib().gla_chunk_fwd_varlen_ex(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), log_alpha.data_ptr(), float(scale),
            None if h0 is None else h0.data_ptr(), out.data_ptr(),
            None if hT is None else hT.data_ptr(), cu_arr, N, H, T_total, dk, dv,
            ctypes.byref(opts), _stream(dev))
    _lib.check(st, "gla_chunk_fwd_varlen")
    return (out.unsqueeze(0) if squeeze else out), hT


def gla_chunk_fwd_varlen_plan(cu_seqlens, H: int, dk: int, dv: int, *, segments: int = 0,
                              dv_tile: int = 0, force_exact: bool = False,
                              cta_pair: int = 0) -> dict:
    """The launch plan gla_chunk_fwd_varlen would use for this packed batch (no GPU work)."""
    cu = [int(x) for x in (cu_seqlens.tolist() if torch.is_tensor(cu_seqlens) else cu_seqlens)]
    opts = GlaChunkOptions(segments=int(segments), dv_tile=int(dv_tile),
                           force_exact=1 if force_exact else 0, cta_pair=int(cta_pair))
    nseg, tile, launches = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    sb = ctypes.c_ulong()
    st = _lib.lib().gla_chunk_fwd_varlen_plan((ctypes.c_int * len(cu))(*cu), len(cu) - 1, H,
                                               cu[-1], dk, dv, ctypes.byref(opts),
                                               ctypes.byref(nseg), ctypes.byref(tile),
                                               ctypes.byref(launches), ctypes.byref(sb))
    _lib.check(st, "gla_chunk_fwd_varlen_plan")
    return {"segments": nseg.value, "dv_tile": tile.value, "launches": launches.value,
            "scratch_bytes": sb.value}


def gla_chunk_fwd_host(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_alpha: torch.Tensor,
                       scale: float | None = None, h0: torch.Tensor | None = None,
                       output_final_state: bool = True, *, out: torch.Tensor | None = None,
                       final_state: torch.Tensor | None = None, device: int | None = None):
    """gla_chunk_fwd on CPU tensors, end to end (copies in, forward, copies out).

    The inputs are CPU tensors; pin them (``tensor.pin_memory()``) for the
    copies to overlap the computation.  The outputs are CPU tensors too;
    when not given, they are allocated pinned.  The work is enqueued on the
    current stream of ``device`` (default: the current CUDA device).  The
    results are valid once that stream has completed; call
    ``torch.cuda.synchronize`` or wait on an event before reading them.
    Returns ``(o, hT)``.
    """
    if q.dim() != 4:
        raise ValueError("q must be [B, H, T, dk]")
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    cpu = torch.device("cpu")
    _need(q, "q", torch.bfloat16, (B, H, T, dk), cpu)
    _need(k, "k", torch.bfloat16, (B, H, T, dk), cpu)
    _need(v, "v", torch.bfloat16, (B, H, T, dv), cpu)
    _need(log_alpha, "log_alpha", torch.float32, (B, H, T, dk), cpu)
    if h0 is not None:
        _need(h0, "h0", torch.float32, (B, H, dk, dv), cpu)
    if out is None:
        out = torch.empty(B, H, T, dv, dtype=torch.bfloat16, pin_memory=True)
    _need(out, "out", torch.bfloat16, (B, H, T, dv), cpu)
    hT = None
    if output_final_state:
        hT = final_state if final_state is not None else torch.empty(
            B, H, dk, dv, dtype=torch.float32, pin_memory=True)
        _need(hT, "final_state", torch.float32, (B, H, dk, dv), cpu)
    if scale is None:
        scale = dk ** -0.5
    dev = torch.device("cuda", torch.cuda.current_device() if device is None else device)
    with torch.cuda.device(dev):
        st = _lib.lib().gla_chunk_fwd_host(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), log_alpha.data_ptr(), float(scale),
            None if h0 is None else h0.data_ptr(), out.data_ptr(),
            None if hT is None else hT.data_ptr(), B, H, T, dk, dv, _stream(dev))
    _lib.check(st, "gla_chunk_fwd_host")
    return out, hT


def gla_chunk_fwd_plan(B: int, H: int, T: int, dk: int, dv: int, *, segments: int = 0,
                       dv_tile: int = 0, force_exact: bool = False, cta_pair: int = 0) -> dict:
    """The launch plan gla_chunk_fwd would use on the current device (no GPU work)."""
    opts = GlaChunkOptions(segments=int(segments), dv_tile=int(dv_tile),
                           force_exact=1 if force_exact else 0, cta_pair=int(cta_pair))
    nseg, tile, launches = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    scratch = ctypes.c_ulong()
    st = _lib.lib().gla_chunk_fwd_plan(B, H, T, dk, dv, ctypes.byref(opts), ctypes.byref(nseg),
                                       ctypes.byref(tile), ctypes.byref(launches),
                                       ctypes.byref(scratch))
    _lib.check(st, "gla_chunk_fwd_plan")
    return {"segments": nseg.value, "dv_tile": tile.value, "launches": launches.value,
            "scratch_bytes": scratch.value}


def gla_chunk_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_alpha: torch.Tensor,
                  d_o: torch.Tensor, scale: float | None = None, h0: torch.Tensor | None = None,
                  dhT: torch.Tensor | None = None, *, need_dh0: bool = True,
                  force_exact: bool = False):
    """Gradients of L = sum <d_o, o> + <dhT, hT> through the chunked forward.

    Inputs as for ``gla_chunk_fwd`` (gates ``[B,H,T,dk]``, or ``[B,H,T]`` for one
    gate per token and head; ``dlog_alpha`` then has the same shape), with
    ``d_o`` ``[B,H,T,dv]`` bf16 and ``dhT`` ``[B,H,dk,dv]`` fp32 or None (zero).
    Returns ``(dq, dk, dv, dlog_alpha, dh0)``: bf16, bf16, bf16, fp32, and fp32
    or None when ``need_dh0`` is False.  The states are recomputed on the GPU.
    """
    if q.dim() != 4:
        raise ValueError("q must be [B, H, T, dk]")
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("q must be on a CUDA device")
    _need(q, "q", torch.bfloat16, (B, H, T, dk), dev)
    _need(k, "k", torch.bfloat16, (B, H, T, dk), dev)
    _need(v, "v", torch.bfloat16, (B, H, T, dv), dev)
    per_head = log_alpha.dim() == 3
    _need(log_alpha, "log_alpha", torch.float32, (B, H, T) if per_head else (B, H, T, dk), dev)
    _need(d_o, "d_o", torch.bfloat16, (B, H, T, dv), dev)
    if h0 is not None:
        _need(h0, "h0", torch.float32, (B, H, dk, dv), dev)
    if dhT is not None:
        _need(dhT, "dhT", torch.float32, (B, H, dk, dv), dev)
    if scale is None:
        scale = dk ** -0.5
    dq = torch.empty_like(q)
    dkk = torch.empty_like(k)
    dvv = torch.empty_like(v)
    da = torch.empty_like(log_alpha)
    dh0 = torch.empty(B, H, dk, dv, dtype=torch.float32, device=dev) if need_dh0 else None
    opts = GlaChunkOptions(force_exact=1 if force_exact else 0, gate_per_head=1 if per_head else 0)
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    with torch.cuda.device(dev):
        st = _lib.lib().gla_chunk_bwd_ex(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), log_alpha.data_ptr(), float(scale),
            ptr(h0), d_o.data_ptr(), ptr(dhT), dq.data_ptr(), dkk.data_ptr(), dvv.data_ptr(),
            da.data_ptr(), ptr(dh0), B, H, T, dk, dv, ctypes.byref(opts), _stream(dev))
    _lib.check(st, "gla_chunk_bwd")
    return dq, dkk, dvv, da, dh0


def gla_chunk_bwd_varlen(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                         log_alpha: torch.Tensor, d_o: torch.Tensor, cu_seqlens,
                         scale: float | None = None, h0: torch.Tensor | None = None,
                         dhT: torch.Tensor | None = None, *, need_dh0: bool = True,
                         force_exact: bool = False):
    """Gradients of gla_chunk_fwd_varlen over a packed batch of sequences.

    ``q``, ``k``, ``log_alpha`` ``[H, T_total, dk]``; ``v``, ``d_o``
    ``[H, T_total, dv]``; ``h0``, ``dhT`` ``[N, H, dk, dv]`` or None (zero);
    ``cu_seqlens`` a host sequence of ``N + 1`` ints.  Returns
    ``(dq, dk, dv, dlog_alpha, dh0)`` shaped like their inputs (``dh0`` None
    when ``need_dh0`` is False).
    """
    if q.dim() != 3:
        raise ValueError("q must be [H, T_total, dk]")
    H, T_total, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("q must be on a CUDA device")
    cu = [int(x) for x in (cu_seqlens.tolist() if torch.is_tensor(cu_seqlens) else cu_seqlens)]
    N = len(cu) - 1
    if N < 1:
        raise ValueError("cu_seqlens needs at least two entries")
    _need(q, "q", torch.bfloat16, (H, T_total, dk), dev)
    _need(k, "k", torch.bfloat16, (H, T_total, dk), dev)
    _need(v, "v", torch.bfloat16, (H, T_total, dv), dev)
    _need(log_alpha, "log_alpha", torch.float32, (H, T_total, dk), dev)
    _need(d_o, "d_o", torch.bfloat16, (H, T_total, dv), dev)
    if h0 is not None:
        _need(h0, "h0", torch.float32, (N, H, dk, dv), dev)
    if dhT is not None:
        _need(dhT, "dhT", torch.float32, (N, H, dk, dv), dev)
    if scale is None:
        scale = dk ** -0.5
    dq, dkk, dvv, da = (torch.empty_like(t) for t in (q, k, v, log_alpha))
    dh0 = torch.empty(N, H, dk, dv, dtype=torch.float32, device=dev) if need_dh0 else None
    opts = GlaChunkOptions(force_exact=1 if force_exact else 0)
    cu_arr = (ctypes.c_int * len(cu))(*cu)
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    with torch.cuda.device(dev):
        st = _lib.lib().gla_chunk_bwd_varlen_ex(
            q.data_ptr(), k.data_ptr(), v.data_ptr(), log_alpha.data_ptr(), float(scale),
            ptr(h0), d_o.data_ptr(), ptr(dhT), dq.data_ptr(), dkk.data_ptr(), dvv.data_ptr(),
            da.data_ptr(), ptr(dh0), cu_arr, N, H, T_total, dk, dv, ctypes.byref(opts),
            _stream(dev))
    _lib.check(st, "gla_chunk_bwd_varlen")
    return dq, dkk, dvv, da, dh0


def gla_chunk_bwd_plan(B: int, H: int, T: int, dk: int, dv: int) -> dict:
    """Chunk length, launches and scratch bytes of gla_chunk_bwd for a shape (no GPU work)."""
    chunk, launches, scratch = ctypes.c_int(), ctypes.c_int(), ctypes.c_ulong()
    st = _lib.lib().gla_chunk_bwd_plan(B, H, T, dk, dv, ctypes.byref(chunk),
                                       ctypes.byref(launches), ctypes.byref(scratch))
    _lib.check(st, "gla_chunk_bwd_plan")
    return {"chunk": chunk.value, "launches": launches.value, "scratch_bytes": scratch.value}


class _GlaChunk(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, log_alpha, h0, scale):
        o, hT = gla_chunk_fwd(q, k, v, log_alpha, scale, h0)
        ctx.save_for_backward(q, k, v, log_alpha, h0)
        ctx.scale = scale
        return o, hT

    @staticmethod
    def backward(ctx, d_o, dhT):
        q, k, v, log_alpha, h0 = ctx.saved_tensors
        if d_o is None:
            d_o = torch.zeros(*q.shape[:-1], v.shape[-1], dtype=torch.bfloat16, device=q.device)
        d_o = d_o.to(torch.bfloat16).contiguous()
        dhT = None if dhT is None else dhT.float().contiguous()
        dq, dk, dv, da, dh0 = gla_chunk_bwd(q, k, v, log_alpha, d_o, ctx.scale, h0, dhT,
                                            need_dh0=h0 is not None and ctx.needs_input_grad[4])
        return dq, dk, dv, da, dh0, None


def gla_chunk(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_alpha: torch.Tensor,
              scale: float | None = None, h0: torch.Tensor | None = None):
    """Differentiable chunked GLA: ``(o, hT)`` with gradients through ``gla_chunk_bwd``.

    Gates ``[B,H,T,dk]`` or ``[B,H,T]``.  The backward recomputes the states
    from the saved inputs; ``d_o`` is taken in bf16, ``dhT`` in fp32.
    """
    if scale is None:
        scale = q.shape[-1] ** -0.5
    return _GlaChunk.apply(q, k, v, log_alpha, h0, float(scale))


class _GlaChunkVarlen(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, log_alpha, h0, cu, scale):
        o, hT = gla_chunk_fwd_varlen(q, k, v, log_alpha, cu, scale, h0)
        ctx.save_for_backward(q, k, v, log_alpha, h0)
        ctx.cu, ctx.scale = cu, scale
        return o, hT

    @staticmethod
    def backward(ctx, d_o, dhT):
        q, k, v, log_alpha, h0 = ctx.saved_tensors
        if d_o is None:
            d_o = torch.zeros(*q.shape[:-1], v.shape[-1], dtype=torch.bfloat16, device=q.device)
        d_o = d_o.to(torch.bfloat16).contiguous()
        dhT = None if dhT is None else dhT.float().contiguous()
        dq, dk, dv, da, dh0 = gla_chunk_bwd_varlen(
            q, k, v, log_alpha, d_o, ctx.cu, ctx.scale, h0, dhT,
            need_dh0=h0 is not None and ctx.needs_input_grad[4])
        return dq, dk, dv, da, dh0, None, None


def gla_chunk_varlen(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_alpha: torch.Tensor,
                     cu_seqlens, scale: float | None = None, h0: torch.Tensor | None = None):
    """Differentiable packed-batch GLA: ``(o, hT)`` of ``gla_chunk_fwd_varlen`` with gradients
    through ``gla_chunk_bwd_varlen``.  ``q`` etc. are ``[H, T_total, .]``; ``h0`` is
    ``[N, H, dk, dv]`` or None."""
    if scale is None:
        scale = q.shape[-1] ** -0.5
    cu = [int(x) for x in (cu_seqlens.tolist() if torch.is_tensor(cu_seqlens) else cu_seqlens)]
    return _GlaChunkVarlen.apply(q, k, v, log_alpha, h0, cu, float(scale))


def gla_gdn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                beta: torch.Tensor, scale: float | None = None, h0: torch.Tensor | None = None,
                output_final_state: bool = True, chunked: bool = False, *,
                qk_l2norm: bool = False, norm_eps: float = 1e-6):
    """Gated delta rule (Gated DeltaNet) forward: ``(o, hT)``.

    q, k ``[B,H,T,dk]`` bf16 (as given, or with ``qk_l2norm=True`` each row
    divided by its length first, ``gla_qk_norm_rope_fwd`` with ``norm="l2"`` and
    ``norm_eps``); v ``[B,H,T,dv]`` bf16; g (log alpha) and beta ``[B,H,T]`` fp32;
    h0 ``[B,H,dk,dv]`` fp32 or None.
    ``chunked=True`` calls gla_gdn_chunk_fwd (the chunk algorithm on the tensor
    cores, dk = 128), else gla_gdn_fwd (token-recurrent).
    """
    if q.dim() != 4:
        raise ValueError("q must be [B, H, T, dk]")
    B, H, T, dk = q.shape
    dv = v.shape[-1]
    dev = q.device
    if dev.type != "cuda":
        raise ValueError("q must be on a CUDA device")
    _need(q, "q", torch.bfloat16, (B, H, T, dk), dev)
    _need(k, "k", torch.bfloat16, (B, H, T, dk), dev)
    _need(v, "v", torch.bfloat16, (B, H, T, dv), dev)
    _need(g, "g", torch.float32, (B, H, T), dev)
    _need(beta, "beta", torch.float32, (B, H, T), dev)
    if h0 is not None:
        _need(h0, "h0", torch.float32, (B, H, dk, dv), dev)
    if qk_l2norm:
        q, k = gla_qk_norm_rope_fwd(q.transpose(1, 2), k.transpose(1, 2), norm="l2", eps=norm_eps)
    if scale is None:
        scale = dk ** -0.5
    o = torch.empty(B, H, T, dv, dtype=torch.bfloat16, device=dev)
    hT = torch.empty(B, H, dk, dv, dtype=torch.float32, device=dev) if output_final_state else None
    with torch.cuda.device(dev):
        fn = _lib.lib().gla_gdn_chunk_fwd if chunked else _lib.lib().gla_gdn_fwd
        st = fn(q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(),
                float(scale), None if h0 is None else h0.data_ptr(), o.data_ptr(),
                None if hT is None else hT.data_ptr(), B, H, T, dk, dv, _stream(dev))
    _lib.check(st, "gla_gdn_chunk_fwd" if chunked else "gla_gdn_fwd")
    return o, hT


def gla_recurrent_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_alpha: torch.Tensor,
                       h: torch.Tensor, scale: float | None = None, *,
                       out: torch.Tensor | None = None) -> torch.Tensor:
    """One decode token for every (batch, head): ``h`` is updated in place, returns o.

    q, k, log_alpha: ``[B,H,dk]``; v: ``[B,H,dv]``; h: ``[B,H,dk,dv]`` fp32.
    """
    if h.dim() != 4:
        raise ValueError("h must be [B, H, dk, dv]")
    B, H, dk, dv = h.shape
    dev = h.device
    if dev.type != "cuda":
        raise ValueError("h must be on a CUDA device")
    _need(h, "h", torch.float32, (B, H, dk, dv), dev)
    _need(q, "q", torch.bfloat16, (B, H, dk), dev)
    _need(k, "k", torch.bfloat16, (B, H, dk), dev)
    _need(v, "v", torch.bfloat16, (B, H, dv), dev)
    _need(log_alpha, "log_alpha", torch.float32, (B, H, dk), dev)
    if out is None:
        out = torch.empty(B, H, dv, dtype=torch.bfloat16, device=dev)
    _need(out, "out", torch.bfloat16, (B, H, dv), dev)
    if scale is None:
        scale = dk ** -0.5
    with torch.cuda.device(dev):
        st = _lib.lib().gla_recurrent_step(q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                           log_alpha.data_ptr(), float(scale), h.data_ptr(),
                                           out.data_ptr(), B, H, dk, dv, _stream(dev))
    _lib.check(st, "gla_recurrent_step")
    return out


def _ptr(t):
    return None if t is None else t.data_ptr()


_DTYPES = {torch.bfloat16: _lib.GLA_BF16, torch.float32: _lib.GLA_F32}


def _dtype(t: torch.Tensor, name: str) -> int:
    dtype = _DTYPES.get(t.dtype) if isinstance(t, torch.Tensor) else None
    if dtype is None:
        raise TypeError(f"{name} must be a torch.bfloat16 or torch.float32 tensor")
    return dtype


def _bounds(cu_seqlens) -> list:
    """The bounds of a packed batch as ints."""
    return [int(c) for c in (cu_seqlens.tolist() if torch.is_tensor(cu_seqlens) else cu_seqlens)]


@functools.lru_cache(maxsize=256)
def _scan_fixed(x, log_alpha, h0):
    """`_scan_sizes` for a batch of one length, with the inputs' checks: functions of their
    `_meta`s alone."""
    shape, _, kind, dev = x
    if dev.type != "cuda":
        raise ValueError("x must be on a CUDA device")
    if kind not in _DTYPES:
        raise TypeError("x must be a torch.bfloat16 or torch.float32 tensor")
    if len(shape) not in (3, 4):
        raise ValueError("x must be [B, T, D] or [B, H, T, D]")
    lead, T, D = tuple(shape[:-2]), shape[-2], shape[-1]
    H = lead[0] if len(lead) == 1 else lead[0] * lead[1]
    _ints(H, T, D)
    state = (*lead, D)
    if log_alpha is not None:
        _fits(x, "x", kind, shape, dev)
        _fits(log_alpha, "log_alpha", torch.float32, shape, dev)
        _fits(h0, "h0", torch.float32, state, dev)
    return state, (*lead, -(-T // _lib.SCAN_BLOCK), D), (H, T, D, _DTYPES[kind])


def _scan_sizes(x: torch.Tensor, cu):
    """(shape of a state, shape of the checkpoints, the C call's sizes) of a scan over `x`."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if cu is None:
        return _scan_fixed(_meta(x), None, None)
    if not x.is_cuda:
        raise ValueError("x must be on a CUDA device")
    shape, dtype = x.shape, _dtype(x, "x")
    if len(shape) not in (2, 3):
        raise ValueError("x must be [T_total, D] or [H, T_total, D]")
    T, D, N = shape[-2], shape[-1], len(cu) - 1
    if N < 1:
        raise ValueError("cu_seqlens needs at least two entries")
    if cu[0] != 0 or cu[-1] != T or any(b < a for a, b in zip(cu, cu[1:])):
        raise ValueError("cu_seqlens must run from 0 to T_total without decreasing")
    lead = shape[:-2]
    _ints(T, D, *lead)
    blocks = sum(-(-(b - a) // _lib.SCAN_BLOCK) for a, b in zip(cu, cu[1:]))
    sizes = ((ctypes.c_int * len(cu))(*cu), N, lead[0] if lead else 1, T, D, dtype)
    return (N, *lead, D), (*lead, blocks, D), sizes


def _scan_inputs(x, log_alpha, cu, h0):
    """`_scan_sizes`, and the checks of these inputs."""
    if x is None or log_alpha is None:
        raise TypeError("x and log_alpha must be torch.Tensors")
    if cu is None:
        try:
            return _scan_fixed(_meta(x), _meta(log_alpha), _meta(h0))
        except AttributeError:
            _all_tensors(x=x, log_alpha=log_alpha, h0=h0)
            raise
    sizes = _scan_sizes(x, cu)
    dev = x.device
    _need(x, "x", x.dtype, x.shape, dev)
    _need(log_alpha, "log_alpha", torch.float32, x.shape, dev)
    if h0 is not None:
        _need(h0, "h0", torch.float32, sizes[0], dev)
    return sizes


def _scan_fwd(x, log_alpha, cu, h0, output_final_state, out, final_state, checkpoints,
              write_h=True, with_checkpoints=False):
    state, ckpt, sizes = _scan_inputs(x, log_alpha, cu, h0)
    dev = x.device
    if out is not None:
        _need(out, "out", x.dtype, x.shape, dev)
        _apart(out, "out", x, log_alpha, h0)
    elif write_h:
        out = torch.empty_like(x)
    hT = final_state if output_final_state else None
    if hT is not None:
        _need(hT, "final_state", torch.float32, state, dev)
        _apart(hT, "final_state", x, log_alpha, None if h0 is None or
               h0.data_ptr() == hT.data_ptr() else h0)
        _apart(hT, "final_state", out, also="another output")
    elif output_final_state:
        hT = torch.empty(state, dtype=torch.float32, device=dev)
    if with_checkpoints:
        checkpoints = torch.empty(ckpt, dtype=torch.float32, device=dev)
    elif checkpoints is not None:
        _need(checkpoints, "checkpoints", torch.float32, ckpt, dev)
        _apart(checkpoints, "checkpoints", x, log_alpha, h0)
        _apart(checkpoints, "checkpoints", out, hT, also="another output")
    _call("gla_scan_fwd" if cu is None else "gla_scan_fwd_varlen", dev, x.data_ptr(),
          log_alpha.data_ptr(), _ptr(h0), _ptr(out), _ptr(hT), _ptr(checkpoints), *sizes)
    return (out, hT, checkpoints) if with_checkpoints else (out, hT)


def _scan_bwd(x, log_alpha, d_h, cu, h0, dhT, checkpoints, need_dx, need_dlog_alpha, need_dh0):
    state, ckpt, sizes = _scan_inputs(x, log_alpha, cu, None)
    dev = x.device
    if d_h is not None:
        _need(d_h, "d_h", x.dtype, x.shape, dev)
    if dhT is not None:
        _need(dhT, "dhT", torch.float32, state, dev)
    if checkpoints is None:
        checkpoints = _scan_fwd(x, log_alpha, cu, h0, False, None, None, None, False, True)[2]
    else:
        _need(checkpoints, "checkpoints", torch.float32, ckpt, dev)
    dx = torch.empty_like(x) if need_dx else None
    da = torch.empty_like(log_alpha) if need_dlog_alpha else None
    dh0 = torch.empty(state, dtype=torch.float32, device=dev) if need_dh0 else None
    if need_dx or need_dlog_alpha or need_dh0:
        _call("gla_scan_bwd" if cu is None else "gla_scan_bwd_varlen", dev, x.data_ptr(),
              log_alpha.data_ptr(), checkpoints.data_ptr(), _ptr(d_h), _ptr(dhT), _ptr(dx),
              _ptr(da), _ptr(dh0), *sizes)
    return dx, da, dh0


def gla_scan_checkpoints(x: torch.Tensor, cu_seqlens=None) -> torch.Tensor:
    """An empty buffer for the states that enter each block of 64 tokens (fp32).

    ``gla_scan_fwd`` fills it and ``gla_scan_bwd`` reads it: ``[B, ceil(T/64), D]``
    for ``x`` ``[B, T, D]`` (``[B, H, ceil(T/64), D]`` for four dimensions); for a
    packed batch ``[sum of ceil(length/64), D]`` (``[H, ..., D]``).
    """
    shape = _scan_sizes(x, None if cu_seqlens is None else _bounds(cu_seqlens))[1]
    return torch.empty(shape, dtype=torch.float32, device=x.device)


def gla_scan_fwd(x: torch.Tensor, log_alpha: torch.Tensor, h0: torch.Tensor | None = None,
                 output_final_state: bool = True, *, out: torch.Tensor | None = None,
                 final_state: torch.Tensor | None = None,
                 checkpoints: torch.Tensor | None = None):
    """The gated linear recurrence ``h_t = exp(log_alpha_t) h_{t-1} + x_t``, elementwise.

    ``x`` ``[B, T, D]`` or ``[B, H, T, D]``, bf16 or fp32, contiguous as all tensors
    here; ``log_alpha`` the same shape in fp32, <= 0 (-inf is a gate of zero); ``h0``
    ``[B, D]`` / ``[B, H, D]`` fp32 or None (zero).  Returns ``(h, hT)``: every state
    in ``x``'s type, kept in fp32 on the way, and the last one in fp32 (None when
    ``output_final_state`` is False).  ``final_state`` may be ``h0`` itself; no other
    output may share memory with an input, and no output with another.
    ``checkpoints`` (from ``gla_scan_checkpoints``) is filled for ``gla_scan_bwd``.
    """
    return _scan_fwd(x, log_alpha, None, h0, output_final_state, out, final_state, checkpoints)


def gla_scan_fwd_varlen(x: torch.Tensor, log_alpha: torch.Tensor, cu_seqlens,
                        h0: torch.Tensor | None = None, output_final_state: bool = True, *,
                        out: torch.Tensor | None = None, final_state: torch.Tensor | None = None,
                        checkpoints: torch.Tensor | None = None):
    """``gla_scan_fwd`` over a packed batch: ``x`` ``[T_total, D]`` or ``[H, T_total, D]``.

    Sequence ``n`` holds rows ``cu_seqlens[n] : cu_seqlens[n+1]``; ``cu_seqlens`` is a
    host sequence of ``N + 1`` ints (list, tuple or CPU tensor).  ``h0`` and ``hT``
    are ``[N, D]`` / ``[N, H, D]``; an empty sequence keeps its state.
    """
    return _scan_fwd(x, log_alpha, _bounds(cu_seqlens), h0, output_final_state, out, final_state,
                     checkpoints)


def gla_scan_bwd(x: torch.Tensor, log_alpha: torch.Tensor, d_h: torch.Tensor | None,
                 h0: torch.Tensor | None = None, dhT: torch.Tensor | None = None, *,
                 checkpoints: torch.Tensor | None = None, need_dx: bool = True,
                 need_dlog_alpha: bool = True, need_dh0: bool = True):
    """Gradients of ``sum <d_h, h> + <dhT, hT>`` through ``gla_scan_fwd``.

    ``d_h`` is like ``x`` and ``dhT`` like ``h0`` (each None: zero).  Returns
    ``(dx, dlog_alpha, dh0)``, in ``x``'s type, fp32 and fp32; each None when not
    needed.  ``checkpoints`` are those that ``gla_scan_fwd`` filled for the same
    ``x``, ``log_alpha`` and ``h0``; without them a pass over ``x`` recomputes them.
    """
    return _scan_bwd(x, log_alpha, d_h, None, h0, dhT, checkpoints, need_dx, need_dlog_alpha,
                     need_dh0)


def gla_scan_bwd_varlen(x: torch.Tensor, log_alpha: torch.Tensor, d_h: torch.Tensor | None,
                        cu_seqlens, h0: torch.Tensor | None = None,
                        dhT: torch.Tensor | None = None, *,
                        checkpoints: torch.Tensor | None = None, need_dx: bool = True,
                        need_dlog_alpha: bool = True, need_dh0: bool = True):
    """``gla_scan_bwd`` over a packed batch (shapes of ``gla_scan_fwd_varlen``)."""
    return _scan_bwd(x, log_alpha, d_h, _bounds(cu_seqlens), h0, dhT, checkpoints, need_dx,
                     need_dlog_alpha, need_dh0)


class _GlaScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, log_alpha, h0, cu):
        ctx.set_materialize_grads(False)
        h, hT, ckpt = _scan_fwd(x, log_alpha, cu, h0, True, None, None, None,
                                with_checkpoints=True)
        ctx.save_for_backward(x, log_alpha, ckpt)
        ctx.cu = cu
        return h, hT

    @staticmethod
    @_once
    def backward(ctx, d_h, dhT):
        x, log_alpha, ckpt = ctx.saved_tensors
        if d_h is None and dhT is None:
            return None, None, None, None
        # checked again: what was saved may come back elsewhere (hooks on saved tensors)
        return (*_scan_bwd(x, log_alpha, _like(d_h, x.dtype), ctx.cu, None,
                           _like(dhT, torch.float32), ckpt, *ctx.needs_input_grad[:3]), None)


def gla_scan(x: torch.Tensor, log_alpha: torch.Tensor, h0: torch.Tensor | None = None):
    """Differentiable ``gla_scan_fwd``: ``(h, hT)`` with gradients through ``gla_scan_bwd``."""
    return _GlaScan.apply(x, log_alpha, h0, None)


def gla_scan_varlen(x: torch.Tensor, log_alpha: torch.Tensor, cu_seqlens,
                    h0: torch.Tensor | None = None):
    """Differentiable ``gla_scan_fwd_varlen``."""
    return _GlaScan.apply(x, log_alpha, h0, _bounds(cu_seqlens))


@functools.lru_cache(maxsize=256)
def _step_checked(x, log_alpha, h):
    """The checks of a step's arguments and the C call's sizes, of the tensors' `_meta`s alone."""
    shape, _, kind, dev = x
    if len(shape) not in (2, 3):
        raise ValueError("x must be [B, D] or [B, H, D]")
    if dev.type != "cuda":
        raise ValueError("x must be on a CUDA device")
    if kind not in _DTYPES:
        raise TypeError("x must be a torch.bfloat16 or torch.float32 tensor")
    _fits(x, "x", kind, shape, dev)
    _fits(log_alpha, "log_alpha", torch.float32, shape, dev)
    _fits(h, "h", torch.float32, shape, dev)
    B, D = shape[:-1].numel(), shape[-1]
    _ints(B, D)
    return B, D, _DTYPES[kind]


def gla_scan_step(x: torch.Tensor, log_alpha: torch.Tensor, h: torch.Tensor, *,
                  out: torch.Tensor | None = None) -> torch.Tensor:
    """One decode token of ``gla_scan_fwd``: ``h`` is updated in place, returns it in ``x``'s type.

    x ``[B, D]`` or ``[B, H, D]`` bf16 or fp32; log_alpha and h the same shape in fp32.
    ``out`` (or ``h``) may be another argument of the same element size itself, such as
    ``out=x``; tensors that share memory in any other way are refused.
    """
    if x is None or log_alpha is None or h is None:
        raise TypeError("x, log_alpha and h must be torch.Tensors")
    try:
        sizes = _step_checked(_meta(x), _meta(log_alpha), _meta(h))
    except AttributeError:
        _all_tensors(x=x, log_alpha=log_alpha, h=h)
        raise
    if out is None:
        out = torch.empty_like(x)
    else:
        _need(out, "out", x.dtype, x.shape, x.device)
    _call("gla_scan_step", x.device, x.data_ptr(), log_alpha.data_ptr(), h.data_ptr(),
          out.data_ptr(), *sizes)
    return out


_NORMS = {"rms": _lib.GLA_NORM_RMS, "l2": _lib.GLA_NORM_L2}


@functools.lru_cache(maxsize=256)
def _qk_checked(q, k, q_weight, k_weight, positions, inv_freq, norm, eps, interleaved):
    """The checks of a gla_qk_norm_rope call's arguments and the C call's sizes, layout and
    options: functions of the tensors' `_meta`s and of the options alone."""
    if q is None or k is None:
        raise TypeError("q and k must be torch.Tensors")
    (qn, qs, kind, dev), (kn, ks, k_kind, k_dev) = q, k
    if kind not in _DTYPES:
        raise TypeError("q must be a torch.bfloat16 or torch.float32 tensor")
    if dev.type != "cuda" or k_dev != dev:
        raise ValueError("q and k must be on the same CUDA device")
    if len(qn) != 4 or len(kn) != 4:
        raise ValueError("q and k must be [B, T, H, d]")
    if qs[3] != 1 or ks[3] != 1:
        raise ValueError("the last dimension of q and k must be contiguous")
    B, T, Hq, d = qn
    Hk = kn[2]
    if k_kind is not kind:
        raise TypeError(f"k must be {kind}, got {k_kind}")
    if kn[0] != B or kn[1] != T or kn[3] != d:
        raise ValueError(f"k must have shape {(B, T, Hk, d)}, got {tuple(kn)}")
    if norm not in _NORMS:
        raise ValueError("norm must be 'rms' or 'l2'")
    _fits(q_weight, "q_weight", torch.float32, (d,), dev)
    _fits(k_weight, "k_weight", torch.float32, (d,), dev)
    rot = 0
    if inv_freq is not None:
        rot = 2 * inv_freq[0].numel()
        _fits(inv_freq, "inv_freq", torch.float64, (rot // 2,), dev)
    pos_sb = 0
    if positions is not None:
        one = len(positions[0]) == 1
        _fits(positions, "positions", torch.int64, (T,) if one else (B, T), dev)
        pos_sb = 0 if one else T
    _ints(B, T, Hq, Hk, d, rot)
    # a dimension of one entry is never stepped over, whatever its stride says
    layout = _lib.GlaQkLayout(qs[0] if B != 1 else 0, qs[1] if T != 1 else 0,
                              qs[2] if Hq != 1 else 0, ks[0] if B != 1 else 0,
                              ks[1] if T != 1 else 0, ks[2] if Hk != 1 else 0, pos_sb)
    options = _lib.GlaQkOptions(dtype=_DTYPES[kind], norm=_NORMS[norm],
                                interleaved=int(interleaved), eps=eps)
    return B, T, Hq, Hk, d, rot, ctypes.byref(layout), ctypes.byref(options)


def _qk_sizes(q, k, q_weight, k_weight, positions, inv_freq, norm, eps, interleaved):
    """Checks the arguments of a gla_qk_norm_rope call: (the inputs' pointers, the C call's
    sizes)."""
    try:
        sizes = _qk_checked(_meta(q), _meta(k), _meta(q_weight), _meta(k_weight),
                            _meta(positions), _meta(inv_freq), norm, float(eps),
                            bool(interleaved))
    except AttributeError:
        _all_tensors(q=q, k=k, q_weight=q_weight, k_weight=k_weight, positions=positions,
                     inv_freq=inv_freq)
        raise
    return (q.data_ptr(), k.data_ptr(), _ptr(q_weight), _ptr(k_weight), _ptr(positions),
            _ptr(inv_freq)), sizes


def _qk_fwd(q, pointers, sizes):
    B, T, Hq, Hk, d = sizes[:5]
    q_out = torch.empty((B, Hq, T, d), dtype=q.dtype, device=q.device)
    k_out = torch.empty((B, Hk, T, d), dtype=q.dtype, device=q.device)
    _call("gla_qk_norm_rope_fwd", q.device, *pointers, q_out.data_ptr(), k_out.data_ptr(), *sizes)
    return q_out, k_out


def gla_rope_frequencies(rot: int, base: float = 10000.0, device=None) -> torch.Tensor:
    """``base^(-2i/rot)`` for ``i < rot/2``, fp64: the angles per position of each rotated pair."""
    if rot <= 0 or rot % 8:
        raise ValueError("rot must be a positive multiple of 8")
    return float(base) ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)


def gla_qk_norm_rope_fwd(q: torch.Tensor, k: torch.Tensor, q_weight: torch.Tensor | None = None,
                         k_weight: torch.Tensor | None = None,
                         positions: torch.Tensor | None = None,
                         inv_freq: torch.Tensor | None = None, *, norm: str = "rms",
                         eps: float = 1e-6, interleaved: bool = False):
    """Norms of the query and key rows and their rotation by position, in one pass.

    q ``[B, T, Hq, d]`` and k ``[B, T, Hk, d]``, bf16 or fp32, as a projection
    leaves them: strided views with a contiguous last dimension are read in place
    (strides in multiples of 8 elements, 16-byte aligned).  Returns
    ``(q', k')``, ``[B, Hq, T, d]`` and ``[B, Hk, T, d]`` contiguous, as
    ``gla_chunk`` and ``gla_gdn_fwd`` take them.

    Each row is divided by its norm (``norm="rms"``: the root of its mean square,
    ``"l2"``: its length; ``eps`` under the root), multiplied by its weight (``[d]``
    fp32 or None) and, with ``inv_freq`` (fp64 ``[rot/2]``, see
    ``gla_rope_frequencies``), the pairs of its first ``rot`` values are turned by
    ``position * inv_freq``: pairs ``(i, i + rot/2)``, or ``(2i, 2i + 1)`` when
    ``interleaved``.  ``positions`` is int64 ``[B, T]`` or ``[T]``, contiguous (None: 0 .. T-1).
    d and rot are multiples of 8, up to 256.
    """
    return _qk_fwd(q, *_qk_sizes(q, k, q_weight, k_weight, positions, inv_freq, norm, eps,
                                 interleaved))


def gla_qk_norm_rope_bwd(q: torch.Tensor, k: torch.Tensor, d_q: torch.Tensor, d_k: torch.Tensor,
                         q_weight: torch.Tensor | None = None,
                         k_weight: torch.Tensor | None = None,
                         positions: torch.Tensor | None = None,
                         inv_freq: torch.Tensor | None = None, *, norm: str = "rms",
                         eps: float = 1e-6, interleaved: bool = False,
                         need_dweights: bool = True):
    """Gradients of ``<d_q, q'> + <d_k, k'>`` through ``gla_qk_norm_rope_fwd``.

    d_q, d_k are contiguous like q', k'.  Returns ``(dq, dk, dq_weight, dk_weight)``:
    contiguous ``[B, T, H, d]`` in q's type, and fp32 ``[d]`` sums over every row
    (None without a weight, or when not needed).
    """
    pointers, sizes = _qk_sizes(q, k, q_weight, k_weight, positions, inv_freq, norm, eps,
                                interleaved)
    B, T, Hq, Hk, d = sizes[:5]
    _need(d_q, "d_q", q.dtype, (B, Hq, T, d), q.device)
    _need(d_k, "d_k", q.dtype, (B, Hk, T, d), q.device)
    return _qk_grads(q, d_q, d_k, q_weight, k_weight, pointers, sizes, need_dweights)


def _qk_grads(q, d_q, d_k, q_weight, k_weight, pointers, sizes, need_dweights):
    B, T, Hq, Hk, d = sizes[:5]
    dev = q.device
    dq = torch.empty((B, T, Hq, d), dtype=q.dtype, device=dev)
    dk = torch.empty((B, T, Hk, d), dtype=q.dtype, device=dev)
    dwq = torch.empty_like(q_weight) if q_weight is not None and need_dweights else None
    dwk = torch.empty_like(k_weight) if k_weight is not None and need_dweights else None
    scratch, size = None, 0
    if dwq is not None or dwk is not None:
        size = _entry("gla_qk_norm_rope_bwd_scratch")(d)
        scratch = torch.empty(size, dtype=torch.uint8, device=dev)
    _call("gla_qk_norm_rope_bwd", dev, *pointers, d_q.data_ptr(), d_k.data_ptr(), dq.data_ptr(),
          dk.data_ptr(), _ptr(dwq), _ptr(dwk), *sizes, _ptr(scratch), size)
    return dq, dk, dwq, dwk


class _GlaQkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, positions, inv_freq, norm, eps, interleaved):
        pointers, sizes = _qk_sizes(q, k, q_weight, k_weight, positions, inv_freq, norm, eps,
                                    interleaved)
        ctx.save_for_backward(q, k, q_weight, k_weight, positions, inv_freq)
        ctx.options = norm, eps, interleaved
        return _qk_fwd(q, pointers, sizes)

    @staticmethod
    @_once
    def backward(ctx, d_q, d_k):
        saved = ctx.saved_tensors
        q, wq, wk = saved[0], saved[2], saved[3]
        # checked again: what was saved may come back with other strides (hooks on saved tensors)
        pointers, sizes = _qk_sizes(*saved, *ctx.options)
        need = ctx.needs_input_grad
        grads = _qk_grads(q, _like(d_q, q.dtype), _like(d_k, q.dtype), wq, wk, pointers, sizes,
                          need[2] or need[3])
        return (*grads, None, None, None, None, None)


def gla_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, q_weight: torch.Tensor | None = None,
                     k_weight: torch.Tensor | None = None, positions: torch.Tensor | None = None,
                     inv_freq: torch.Tensor | None = None, *, norm: str = "rms",
                     eps: float = 1e-6, interleaved: bool = False):
    """Differentiable ``gla_qk_norm_rope_fwd``: gradients of q, k and the weights."""
    return _GlaQkNormRope.apply(q, k, q_weight, k_weight, positions, inv_freq, norm, eps,
                                interleaved)


def gla_last_device_status(device: torch.device | int | None = None) -> int:
    """Synchronise the current stream and read/clear the library's device status word."""
    dev = torch.device("cuda", torch.cuda.current_device() if device is None else
                       (device if isinstance(device, int) else device.index))
    with torch.cuda.device(dev):
        return int(_lib.lib().gla_last_device_status(_stream(dev)))
