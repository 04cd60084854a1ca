"""Binding of the sequence operators: short causal convolution (conv_*), selective
state space scan (ssm_*) and sparse attention over selected blocks (block_*).

Argument marshalling only, as in sdm.py: shapes, types, devices and aliasing are
checked before anything is launched, and every product runs in the library's
kernels.  The marshalling itself is compiled (binding/sequence.cpp, the module
_sequence): a single-token pass is shorter than a Python function that checks its
arguments.  Tensors are [B, H, T, d] views with a dense last axis and any other
strides, so slices of a token-major projection [B, T, C] go in as they are
(`xbc[..., :H * d].view(B, T, H, d).transpose(1, 2)`); results come in the layout
of the tensor they belong to.  Work is enqueued on `stream` (default: the current
stream of the tensors' device) and workspaces and results are allocated for it.
"""
from __future__ import annotations

import os
from typing import Dict, Optional

import torch

from .sdm import _IN_DTYPES

_HERE = os.path.dirname(os.path.abspath(__file__))
_module = None


def _host():
    """The compiled host side, loaded on the first call (raises if it was not built)."""
    global _module
    if _module is None:
        if not os.path.exists(os.path.join(_HERE, "_sequence.so")):
            raise RuntimeError("_sequence.so not found in %s; build it with "
                               "`python -m sparse_memory_linear_scoring_b200.build`" % _HERE)
        from . import _sequence
        _module = _sequence
    return _module


def _on(stream, t, call, *args):
    """call(*args) on `stream` of t's device."""
    if not t.is_cuda:
        raise ValueError("all tensors must be CUDA tensors (there is no CPU path)")
    if stream.device != t.device:
        raise ValueError("stream belongs to another device than the tensors")
    with torch.cuda.stream(stream):
        return call(*args)


# ---------------------------------------------------------------- convolution
def conv_forward(x, w, bias=None, state=None, *, silu: bool = True,
                 lengths: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """Short causal convolution along T (sdm_conv_forward).  x [B,H,T,d]; w [H,d,K]
    with 2 <= K <= 8; bias [H,d] or None; state [B,H,K-1,d] (contiguous), the K - 1
    inputs before the call, updated in place to the last ones -- one token at a time
    is T = 1.  All of x's dtype.  lengths [B] int32: steps at or past it are not read
    and give 0.  Returns y [B,H,T,d] = silu(p), or p with silu=False."""
    if stream is not None:
        return _on(stream, x, _host().conv_forward, x, w, bias, state, bool(silu), lengths, y)
    return _host().conv_forward(x, w, bias, state, bool(silu), lengths, y)


def conv_backward(x, w, dy, bias=None, state0=None, dstate=None, *, silu: bool = True,
                  workspace: Optional[torch.Tensor] = None, stream=None) -> Dict[str, torch.Tensor]:
    """Gradients of conv_forward at full length (sdm_conv_backward).  state0: the state
    the forward started from (a copy; None for zeros); dstate [B,H,K-1,d] float32: the
    gradient of the state it left.  For a padded batch: dy = 0 behind each row's length, and
    the gradient of the state left, which are the K - 1 inputs before that, is added to
    their rows of the result instead of given as dstate.  Returns x (x's dtype), w [H,d,K] and, where bias /
    state0 or dstate are given, bias [H,d] and state [B,H,K-1,d], float32."""
    if stream is not None:
        return _on(stream, x, _host().conv_backward, x, w, dy, bias, state0, dstate, bool(silu), workspace)
    return _host().conv_backward(x, w, dy, bias, state0, dstate, bool(silu), workspace)


# ---------------------------------------------------------------- selective scan
def ssm_workspace_bytes(B, H, G, T, d_k, d_v, in_dtype) -> int:
    """Bytes ssm_forward's workspace needs (0 for sizes it does not take)."""
    dt = _IN_DTYPES[in_dtype] if isinstance(in_dtype, torch.dtype) else int(in_dtype)
    return _host().ssm_workspace_bytes(B, H, G, T, d_k, d_v, dt)


def ssm_forward(x, dt, A, Bm, Cm, S, D=None, *, lengths: Optional[torch.Tensor] = None,
                y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """Selective state space scan (sdm_ssm_forward): per head
    S_t = exp(dt_t A) S_{t-1} + dt_t x_t Bm_t^T, y_t = S_t Cm_t + D x_t.
    x [B,H,T,d_v] and Bm, Cm [B,G,T,d_k] share one dtype (float32 or bfloat16), G
    divides H; dt [B,H,T], A [H], D [H] or None, float32; S [B,H,d_v,d_k] float32,
    updated in place.  lengths [B] int32: later steps leave S alone and give 0.
    Returns y [B,H,T,d_v] of x's dtype."""
    if stream is not None:
        return _on(stream, x, _host().ssm_forward, False, x, dt, A, Bm, Cm, S, D, lengths, y, workspace)
    return _host().ssm_forward(False, x, dt, A, Bm, Cm, S, D, lengths, y, workspace)


def ssm_step(x, dt, A, Bm, Cm, S, D=None, *, y: Optional[torch.Tensor] = None,
             stream=None) -> torch.Tensor:
    """ssm_forward for one token or a few at a time (sdm_ssm_step): one kernel that
    reads and writes S once, no workspace.  A row without a token takes dt = 0."""
    if stream is not None:
        return _on(stream, x, _host().ssm_forward, True, x, dt, A, Bm, Cm, S, D, None, y, None)
    return _host().ssm_forward(True, x, dt, A, Bm, Cm, S, D, None, y, None)


def ssm_backward(x, dt, A, Bm, Cm, S0, dy, dS_T=None, *, D=None,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> Dict[str, torch.Tensor]:
    """Gradients of ssm_forward at full length (sdm_ssm_backward); for a padded batch, dt = 0
    and dy = 0 behind each row's length.  S0: the state it
    started from (a copy; None for zeros); dS_T: the gradient of the state it left
    (None: 0).  Returns x, Bm, Cm (x's dtype), dt [B,H,T], A [H], S0 [B,H,d_v,d_k] and,
    where D is given, D [H], float32."""
    if stream is not None:
        return _on(stream, x, _host().ssm_backward, x, dt, A, Bm, Cm, S0, dy, dS_T, D, workspace)
    return _host().ssm_backward(x, dt, A, Bm, Cm, S0, dy, dS_T, D, workspace)


# ---------------------------------------------------------------- block attention
def block_pool(k, kc: Optional[torch.Tensor] = None, *, block: int = 64, first: int = 0,
               stream=None) -> torch.Tensor:
    """Means of the complete blocks of k [B,G,Tk,d] (sdm_block_pool), in k's dtype:
    blocks first .. Tk // block - 1 of kc [B,G,n,d], n >= Tk // block (default: a new one
    with n = Tk // block).  With a cache that grows, first = the blocks already there."""
    if stream is not None:
        return _on(stream, k, _host().block_pool, k, kc, block, first)
    return _host().block_pool(k, kc, block, first)


def block_select(q, kc, *, n_sel: int, block: int = 64, Tk: Optional[int] = None,
                 lengths: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Lists of blocks per query and key head (sdm_block_select): the query's own block,
    then the best n_sel - 1 before it by the group's summed q . kc, best first, lower
    index at ties, then -1.  q [B,H,Tq,d] are the last Tq of Tk keys (default Tk = Tq),
    or of lengths[b] <= Tk in row b (caches; a batch of prompts padded behind needs no
    lengths, here or in block_forward: its live queries see nothing behind them); kc [B,G,n,d] from block_pool.  Returns idx
    [B,G,Tq,n_sel] int32."""
    if stream is not None:
        return _on(stream, q, _host().block_select, q, kc, n_sel, block, Tk, lengths)
    return _host().block_select(q, kc, n_sel, block, Tk, lengths)


def block_forward(q, k, v, idx, *, block: int = 64, scale: Optional[float] = None,
                  lengths: Optional[torch.Tensor] = None, o: Optional[torch.Tensor] = None,
                  return_lse: bool = False, workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of q [B,H,Tq,d], the last Tq of each row's keys, to the keys at or before
    its position in the listed blocks of k, v [B,G,Tk,d] (sdm_block_forward).  idx
    [B,G,Tq,n_sel] int32: any lists; an entry that is no block or lies behind the query
    adds nothing, a repeated one counts as often as listed.  scale defaults to d**-0.5.
    Returns o [B,H,Tq,d] (0 for a query without keys), or (o, lse [B,H,Tq] float32)."""
    if stream is not None:
        return _on(stream, q, _host().block_forward, q, k, v, idx, block, scale, lengths, o, return_lse, workspace)
    return _host().block_forward(q, k, v, idx, block, scale, lengths, o, return_lse, workspace)


def block_backward(q, k, v, idx, o, lse, d_o, *, block: int = 64, scale: Optional[float] = None,
                   lengths: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> Dict[str, torch.Tensor]:
    """Gradients of block_forward at its lists (sdm_block_backward): q, k, v in their
    dtype, given its o and lse and d_o = dL/do [B,H,Tq,d]."""
    if stream is not None:
        return _on(stream, q, _host().block_backward, q, k, v, idx, o, lse, d_o, block, scale, lengths, workspace)
    return _host().block_backward(q, k, v, idx, o, lse, d_o, block, scale, lengths, workspace)
