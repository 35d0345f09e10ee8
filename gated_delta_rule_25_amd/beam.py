"""Beam search over recurrent states (include/kda_beam.h).

A group is one prompt with K hypotheses; beam k of group b is row b * K + k of
every tensor that holds something per sequence.  One step of the search:

    o = linear_decode_step(state, q, k, v, log_decay)         # or decode_step
    ...                                                       # logits [B, K, V]
    scores, tokens, parents, finished = beam_select(logits, scores, finished, end_token=2)
    beam_reorder([state, conv_q_state, conv_k_state], parents)  # in place
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Sequence, Tuple, Union

import torch

from . import KDA_OK, KDAError, _check, _DTYPES, _load
from .linear import _on, _ptr, _stream, _workspace

BEAM_MAX = 16
BEAM_REORDER_MAX = 8


@functools.lru_cache(maxsize=64)
def _select_bytes(groups: int, beams: int, vocab: int, dtype: int) -> int:
    return int(_load().kda_beam_select_workspace_bytes(groups, beams, vocab, dtype))


def beam_select_workspace_bytes(groups: int, beams: int, vocab: int, dtype: torch.dtype = torch.bfloat16) -> int:
    """Workspace bytes of beam_select."""
    return _select_bytes(groups, beams, vocab, _DTYPES[dtype])


def beam_select(logits: torch.Tensor, scores: torch.Tensor, finished: Optional[torch.Tensor] = None, *,
                end_token: Optional[int] = None, out: Optional[Tuple] = None,
                workspace: Optional[torch.Tensor] = None):
    """The K best continuations of each group's K beams (kda_beam_select).

    logits [B, K, V] float32 or bfloat16, K <= 16 (-inf and NaN: masked
    tokens); scores [B, K] float32, the beams' scores so far (-inf: no such
    beam, as all but one at the first step); finished [B, K] bool or None: a
    finished beam has only end_token, at its own score.  A candidate's score
    is scores[b, k] + log_softmax(logits[b, k])[t]; the best K are taken in
    descending order, ties to the lowest k * V + t.

    Returns (scores [B, K] float32, tokens [B, K] int32, parents [B, K] int32,
    finished [B, K] bool, or None without finished).  out: the four tensors to
    write them to; its scores and finished may be the arguments themselves."""
    lib = _load()
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a torch.Tensor")
    if logits.dim() != 3:
        raise ValueError("logits must be [B, K, V]")
    b, k, v = logits.shape
    dev, dt = logits.device, logits.dtype
    if dt not in _DTYPES:
        raise TypeError("logits must be float32 or bfloat16")
    if dev.type != "cuda":
        raise ValueError("tensors must be on a HIP device")
    _check(logits, "logits", (b, k, v), dt, dev)
    _check(scores, "scores", (b, k), torch.float32, dev)
    if finished is not None:
        _check(finished, "finished", (b, k), torch.bool, dev)
        if end_token is None or not 0 <= int(end_token) < v:
            raise ValueError("finished needs an end_token in [0, V)")
    if out is None:
        out = (torch.empty_like(scores), torch.empty((b, k), dtype=torch.int32, device=dev),
               torch.empty((b, k), dtype=torch.int32, device=dev),
               None if finished is None else torch.empty_like(finished))
    new_scores, tokens, parents, new_finished = out
    _check(new_scores, "out scores", (b, k), torch.float32, dev)
    _check(tokens, "out tokens", (b, k), torch.int32, dev)
    _check(parents, "out parents", (b, k), torch.int32, dev)
    if finished is None:
        if new_finished is not None:
            raise ValueError("out finished without finished")
    else:
        _check(new_finished, "out finished", (b, k), torch.bool, dev)
    with _on(dev):
        workspace, ws_bytes = _workspace(workspace, _select_bytes(b, k, v, _DTYPES[dt]), dev)
        rc = lib.kda_beam_select(_ptr(logits), _ptr(scores), _ptr(finished), b, k, v,
                                 0 if finished is None else int(end_token), _DTYPES[dt], _ptr(new_scores),
                                 _ptr(tokens), _ptr(parents), _ptr(new_finished), _ptr(workspace), ws_bytes,
                                 _stream(dev))
    if rc != KDA_OK:
        raise KDAError(rc, "kda_beam_select")
    return new_scores, tokens, parents, new_finished


def _refuse_reorder(ranges, parents) -> None:
    """Refuses, before any of them is moved, the tensors that kda_beam_reorder
    would refuse in a later one of several calls.  ranges: (address, bytes,
    bytes of a row) of each state; parents: its (address, bytes)."""
    used = sorted((a, a + n) for a, n, _ in [*ranges, (*parents, 0)] if n > 0)
    for (_, end), (begin, _) in zip(used, used[1:]):
        if begin < end:
            raise ValueError("the states and parents must not overlap")
    for i in range(0, len(ranges), BEAM_REORDER_MAX):
        blocks = 0
        for a, _, row in ranges[i:i + BEAM_REORDER_MAX]:
            unit = 16 if (a | row) % 16 == 0 else 4 if (a | row) % 4 == 0 else 1
            blocks += (row // unit + 255) // 256
        if blocks * 256 > 2 ** 32 - 1:
            raise ValueError("the states' rows are too long")


def beam_reorder(states: Union[torch.Tensor, Sequence[torch.Tensor]], parents: torch.Tensor):
    """Rows of the states follow the selected parents, in place
    (kda_beam_reorder): row b * K + k becomes what row b * K + parents[b, k]
    was, for all k of a group at once.

    states: a contiguous tensor, or several, of any dtype, [B * K, ...] or
    [B, K, ...]; parents [B, K] int32, K <= 16 (a parent outside [0, K) leaves
    its row as it is).  Returns states."""
    lib = _load()
    many = [states] if isinstance(states, torch.Tensor) else list(states)
    if not isinstance(parents, torch.Tensor):
        raise TypeError("parents must be a torch.Tensor")
    if parents.dim() != 2:
        raise ValueError("parents must be [B, K]")
    b, k = parents.shape
    dev = parents.device
    if dev.type != "cuda":
        raise ValueError("tensors must be on a HIP device")
    _check(parents, "parents", (b, k), torch.int32, dev)
    if not many:
        raise ValueError("no states")
    held = []  # (address, bytes, bytes of a row)
    for t in many:
        if not isinstance(t, torch.Tensor):
            raise TypeError("states must be torch.Tensors")
        if t.shape[:1] != (b * k,) and t.shape[:2] != (b, k):
            raise ValueError("a state has shape %s, expected [%d, ...] or [%d, %d, ...]" % (tuple(t.shape), b * k, b, k))
        if t.device != dev:
            raise ValueError("a state is on %s, expected %s" % (t.device, dev))
        if not t.is_contiguous():
            raise ValueError("states must be contiguous")
        n = t.nbytes
        held.append((t.data_ptr(), n, n // (b * k) if b * k else 0))
    if len(many) > 1:
        at = [a for a, n, _ in held if n]
        if len(set(at)) != len(at):
            raise ValueError("the same state is given twice")
    if len(many) > BEAM_REORDER_MAX:
        _refuse_reorder(held, (parents.data_ptr(), parents.nbytes))
    with _on(dev):
        for i in range(0, len(many), BEAM_REORDER_MAX):
            part = held[i:i + BEAM_REORDER_MAX]
            ptrs = (ctypes.c_void_p * len(part))(*[a for a, _, _ in part])
            rows = (ctypes.c_int64 * len(part))(*[r for _, _, r in part])
            rc = lib.kda_beam_reorder(ptrs, rows, len(part), _ptr(parents), b, k, _stream(dev))
            if rc != KDA_OK:
                raise KDAError(rc, "kda_beam_reorder")
    return states
