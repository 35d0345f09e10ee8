"""Linear attention with one decay per head (include/kda_linear.h):

    S_t = a_t S_{t-1} + k_t v_t^T,   o_t = S_t^T q_t,   a_t = exp(log_decay_t)

with a 128 x 128 fp32 state per head, a_t one scalar per token and head or one
constant per head.  Query and key heads may be shared: q and k have Hq heads,
v and the states H, a multiple of Hq; head h reads query and key head
h // (H // Hq).

    o, final_state = linear_chunk_fwd(q, k, v, log_decay, initial_state, cu_seqlens)
    dq, dk, dv, d_log_decay, d_initial_state = linear_chunk_bwd(q, k, v, log_decay, d_o, ...)
    o, final_state = chunk_linear(q, k, v, log_decay, initial_state)   # torch.autograd
    o = linear_decode_step(state, q, k, v, log_decay)                  # state updated in place
"""
from __future__ import annotations

import contextlib
from typing import Optional, Tuple

import torch

from . import D, KDA_OK, KDAError, _check, _DTYPES, _load


# The calls for single tokens take a few microseconds on the GPU, so what the
# host does for each counts: addresses and the stream go to ctypes as plain
# integers, the latter without a torch.cuda.Stream around it.
_HERE = contextlib.nullcontext()
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _on(dev: torch.device):
    """The kernels run on the tensors' device, whichever is current."""
    return _HERE if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)


def _stream(dev: torch.device) -> int:
    if _raw_stream is not None:
        return _raw_stream(dev.index)
    return torch.cuda.current_stream(dev).cuda_stream


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _sizes(q, k, v, log_decay, cu_seqlens, lead):
    """Checks the tensors of one call; (N, rows, H, Hq, decay_per_head)."""
    for name, t in (("q", q), ("k", k), ("v", v), ("log_decay", log_decay)):
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s must be a torch.Tensor" % name)
    if q.dim() != 3 or q.shape[2] != D:
        raise ValueError("q must be [%s, Hq, 128]" % lead)
    if v.dim() != 3 or v.shape[2] != D:
        raise ValueError("v must be [%s, H, 128]" % lead)
    rows, hq = q.shape[0], q.shape[1]
    h = v.shape[1]
    if hq < 1 or h < 1 or h % hq != 0:
        raise ValueError("the heads of v (%d) must be a multiple of the heads of q and k (%d)" % (h, hq))
    dev, dt = q.device, q.dtype
    if dt not in _DTYPES:
        raise TypeError("q/k/v must be float32 or bfloat16")
    if dev.type != "cuda":
        raise ValueError("tensors must be on a HIP device")
    _check(q, "q", (rows, hq, D), dt, dev)
    _check(k, "k", (rows, hq, D), dt, dev)
    _check(v, "v", (rows, h, D), dt, dev)
    per_head = log_decay.dim() == 1
    _check(log_decay, "log_decay", (h,) if per_head else (rows, h), torch.float32, dev)
    n = 1
    if cu_seqlens is not None:
        if not isinstance(cu_seqlens, torch.Tensor):
            raise TypeError("cu_seqlens must be a torch.Tensor")
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must be [N+1]")
        n = cu_seqlens.numel() - 1
        _check(cu_seqlens, "cu_seqlens", (n + 1,), torch.int32, dev)
    return n, rows, h, hq, int(per_head)


def _workspace(workspace, need, dev):
    if workspace is not None:
        if workspace.device != dev:
            raise ValueError("workspace is on %s, expected %s" % (workspace.device, dev))
        if not workspace.is_contiguous():  # (an expanded tensor has less memory than elements)
            raise ValueError("workspace must be contiguous")
    if need > 0 and (workspace is None or workspace.numel() * workspace.element_size() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    return workspace, 0 if workspace is None else workspace.numel() * workspace.element_size()


def linear_chunk_fwd_workspace_bytes(num_seqs: int, total_tokens: int, num_heads: int,
                                     dtype: torch.dtype = torch.bfloat16, *, num_qk_heads: Optional[int] = None,
                                     segment_tokens: int = 0) -> int:
    """Workspace bytes of linear_chunk_fwd on the current device."""
    return int(_load().kda_linear_chunk_fwd_workspace_bytes(num_seqs, total_tokens, num_heads,
                                                            num_qk_heads or num_heads, D, D, _DTYPES[dtype],
                                                            segment_tokens))


def linear_chunk_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                     initial_state: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None, *,
                     out: Optional[torch.Tensor] = None, final_state: Optional[torch.Tensor] = None,
                     output_final_state: bool = True, workspace: Optional[torch.Tensor] = None,
                     segment_tokens: int = 0) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """Prefill over a packed batch (kda_linear_chunk_fwd).

    q, k: [T, Hq, 128] and v: [T, H, 128], float32 or bfloat16; log_decay
    float32 <= 0 (-inf included), [T, H] or one constant per head, [H];
    initial_state [N, H, 128, 128] float32 or None; cu_seqlens int32 [N+1] on
    the device or None.  segment_tokens: 0 lets the library choose whether
    segments of a sequence run side by side, a positive multiple of 64 forces
    segments of that length, a negative value keeps one walk per sequence.
    Returns (o [T, H, 128], final_state float32 or None); final_state may be
    the same tensor as initial_state (in-place continuation)."""
    lib = _load()
    n, t, h, hq, per_head = _sizes(q, k, v, log_decay, cu_seqlens, "T")
    dev, dt = q.device, q.dtype
    if initial_state is not None:
        _check(initial_state, "initial_state", (n, h, D, D), torch.float32, dev)
    if out is None:
        out = torch.empty((t, h, D), dtype=dt, device=dev)
    else:
        _check(out, "out", (t, h, D), dt, dev)
    if final_state is None and output_final_state:
        final_state = torch.empty((n, h, D, D), dtype=torch.float32, device=dev)
    elif final_state is not None:
        _check(final_state, "final_state", (n, h, D, D), torch.float32, dev)
    with _on(dev):
        need = int(lib.kda_linear_chunk_fwd_workspace_bytes(n, t, h, hq, D, D, _DTYPES[dt], segment_tokens))
        workspace, ws_bytes = _workspace(workspace, need, dev)
        rc = lib.kda_linear_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(initial_state),
                                      _ptr(cu_seqlens), n, t, h, hq, per_head, D, D, _DTYPES[dt], segment_tokens,
                                      _ptr(out), _ptr(final_state), _ptr(workspace), ws_bytes, _stream(dev))
    if rc != KDA_OK:
        raise KDAError(rc, "kda_linear_chunk_fwd")
    return out, final_state


def linear_chunk_bwd_workspace_bytes(num_seqs: int, total_tokens: int, num_heads: int,
                                     dtype: torch.dtype = torch.bfloat16, *, num_qk_heads: Optional[int] = None,
                                     decay_per_head: bool = False, need_d_log_decay: bool = True,
                                     with_d_final_state: bool = True, segment_tokens: int = 0) -> int:
    """Workspace bytes of linear_chunk_bwd on the current device."""
    return int(_load().kda_linear_chunk_bwd_workspace_bytes(num_seqs, total_tokens, num_heads,
                                                            num_qk_heads or num_heads, int(decay_per_head),
                                                            int(need_d_log_decay), int(with_d_final_state), D, D,
                                                            _DTYPES[dtype], segment_tokens))


def linear_chunk_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor, d_o: torch.Tensor,
                     initial_state: Optional[torch.Tensor] = None, cu_seqlens: Optional[torch.Tensor] = None,
                     d_final_state: Optional[torch.Tensor] = None, *, need_d_log_decay: bool = True,
                     need_d_initial_state: bool = True, workspace: Optional[torch.Tensor] = None,
                     segment_tokens: int = 0):
    """Gradients of sum <d_o, o> + <d_final_state, S_T> through
    linear_chunk_fwd (kda_linear_chunk_bwd).

    Inputs as linear_chunk_fwd; d_o [T, H, 128] in the I/O dtype;
    d_final_state [N, H, 128, 128] float32 or None (zero).  Returns (dq, dk,
    dv, d_log_decay, d_initial_state) with the shapes and dtypes of q, k, v,
    log_decay and the initial state: dq and dk summed over the heads that
    share a query and key head, d_log_decay of a constant decay over all
    tokens.  The last two are None when not needed; without d_log_decay the
    call does less work (and bf16 dq and dk may differ in their last bit)."""
    lib = _load()
    n, t, h, hq, per_head = _sizes(q, k, v, log_decay, cu_seqlens, "T")
    dev, dt = q.device, q.dtype
    _check(d_o, "d_o", (t, h, D), dt, dev)
    for name, x in (("initial_state", initial_state), ("d_final_state", d_final_state)):
        if x is not None:
            _check(x, name, (n, h, D, D), torch.float32, dev)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    dg = torch.empty_like(log_decay) if need_d_log_decay else None
    ds = torch.empty((n, h, D, D), dtype=torch.float32, device=dev) if need_d_initial_state else None
    with _on(dev):
        need = int(lib.kda_linear_chunk_bwd_workspace_bytes(n, t, h, hq, per_head, int(need_d_log_decay),
                                                            int(d_final_state is not None), D, D, _DTYPES[dt],
                                                            segment_tokens))
        workspace, ws_bytes = _workspace(workspace, need, dev)
        rc = lib.kda_linear_chunk_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), _ptr(initial_state),
                                      _ptr(cu_seqlens), _ptr(d_o), _ptr(d_final_state), n, t, h, hq, per_head, D, D,
                                      _DTYPES[dt], segment_tokens, _ptr(dq), _ptr(dk), _ptr(dv), _ptr(dg), _ptr(ds),
                                      _ptr(workspace), ws_bytes, _stream(dev))
    if rc != KDA_OK:
        raise KDAError(rc, "kda_linear_chunk_bwd")
    return dq, dk, dv, dg, ds


_STREAM = "chunk_linear.stream"


def _mark_accumulators(out: torch.Tensor) -> None:
    """Notes on the leaves' gradient accumulators the stream they were made on.
    One lives as long as some graph of its leaf, and a captured backward whose
    accumulator belongs to a stream outside the capture ends the process."""
    if out.grad_fn is not None:
        stream = torch.cuda.current_stream(out.device).cuda_stream
        for node, _ in out.grad_fn.next_functions:
            if hasattr(node, "variable"):
                node.metadata.setdefault(_STREAM, stream)


class _ChunkLinear(torch.autograd.Function):
    """linear_chunk_fwd forward, linear_chunk_bwd backward (which needs only
    the forward's inputs)."""

    @staticmethod
    def forward(ctx, q, k, v, log_decay, initial_state, cu_seqlens):
        o, final_state = linear_chunk_fwd(q, k, v, log_decay, initial_state, cu_seqlens)
        ctx.save_for_backward(q, k, v, log_decay, initial_state, cu_seqlens)
        ctx.set_materialize_grads(False)
        return o, final_state

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, d_o, d_final_state):
        if torch.cuda.is_current_stream_capturing():
            stream = torch.cuda.current_stream().cuda_stream
            for node, _ in ctx.next_functions:
                if hasattr(node, "variable") and node.metadata.get(_STREAM, stream) != stream:
                    raise RuntimeError("chunk_linear: a gradient is accumulated by a node that was made outside the "
                                       "graph capture; free the outputs of earlier eager calls with the same leaves, "
                                       "and capture the forward with the backward")
        q, k, v, log_decay, initial_state, cu_seqlens = ctx.saved_tensors
        d_o = torch.zeros_like(v) if d_o is None else d_o.to(v.dtype).contiguous()
        if d_final_state is not None:
            d_final_state = d_final_state.to(torch.float32).contiguous()
        need_ds = initial_state is not None and ctx.needs_input_grad[4]
        dq, dk, dv, dg, ds = linear_chunk_bwd(q, k, v, log_decay, d_o, initial_state, cu_seqlens, d_final_state,
                                              need_d_log_decay=ctx.needs_input_grad[3],
                                              need_d_initial_state=need_ds)
        return dq, dk, dv, dg, ds, None


def chunk_linear(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                 initial_state: Optional[torch.Tensor] = None,
                 cu_seqlens: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Differentiable prefill (torch.autograd): (o, final_state) as
    linear_chunk_fwd, with gradients for q, k, v, log_decay (when it requires
    one) and the initial state from linear_chunk_bwd, once (no gradients of
    gradients).  A graph capture has to hold the forward and the backward, with
    no output of an eager call with the same leaves alive: a backward that
    would accumulate through such a call's nodes is refused.  That is seen for
    leaves that are arguments here and for calls of this function; leaves in
    front of them, and graphs that other operations made of the same leaves, are
    the caller's to free, as with any operation of torch."""
    o, final_state = _ChunkLinear.apply(q, k, v, log_decay, initial_state, cu_seqlens)
    _mark_accumulators(o)
    return o, final_state


def linear_decode_step(state: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                       log_decay: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token for every (sequence, head); ``state`` [N, H, 128, 128] float32
    is advanced in place (kda_linear_decode_step).  q, k [N, Hq, 128] and
    v [N, H, 128], float32 or bfloat16; log_decay float32 [N, H] or [H].
    Returns o [N, H, 128]."""
    lib = _load()
    _, n, h, hq, per_head = _sizes(q, k, v, log_decay, None, "N")
    dev, dt = q.device, q.dtype
    _check(state, "state", (n, h, D, D), torch.float32, dev)
    if out is None:
        out = torch.empty_like(v)
    else:
        _check(out, "out", (n, h, D), dt, dev)
    with _on(dev):
        rc = lib.kda_linear_decode_step(_ptr(state), _ptr(q), _ptr(k), _ptr(v), _ptr(log_decay), n, h, hq, per_head,
                                        D, D, _DTYPES[dt], _ptr(out), _stream(dev))
    if rc != KDA_OK:
        raise KDAError(rc, "kda_linear_decode_step")
    return out
