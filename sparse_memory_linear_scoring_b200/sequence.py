"""Binding of the sequence operators: short causal convolution (conv_*), selective
state space scan (ssm_*) and sparse attention over selected blocks (block_*).

Argument marshalling only, as in sdm.py: shapes, types, devices and aliasing are
checked before anything is launched, and every product runs in the library's
kernels.  Tensors are [B, H, T, d] views with a dense last axis and any other
strides, so slices of a token-major projection [B, T, C] go in as they are
(`xbc[..., :H * d].view(B, T, H, d).transpose(1, 2)`); results come in the layout
of the tensor they belong to.  Work is enqueued on `stream` (default: the current
stream of the tensors' device) and workspaces and results are allocated for it.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import Dict, Optional

import torch

from .sdm import _IN_DTYPES, SDMError, _check, _expect, _nbytes, _ptr, load_library

_F32 = (torch.float32,)


class Strides(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in ("b", "h", "t")]


class ConvDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "H", "T", "d", "K", "silu", "in_dtype")]


class SsmDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "H", "G", "T", "d_k", "d_v", "in_dtype")]


class SsmViews(ctypes.Structure):
    _fields_ = [(n, Strides) for n in ("x", "dt", "B", "C", "y")]


class BlockDims(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("B", "H", "G", "Tq", "Tk", "d", "block", "n_sel", "in_dtype")] + \
               [("scale", ctypes.c_float)]


class BlockViews(ctypes.Structure):
    _fields_ = [(n, Strides) for n in ("q", "k", "v", "o", "kc")]


_bound = None


def _lib():
    """The library with these entry points' argument types set (once)."""
    global _bound
    if _bound is None:
        lib = load_library()
        P, S, I = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int32
        SP, CD, SD, SV = (ctypes.POINTER(t) for t in (Strides, ConvDims, SsmDims, SsmViews))
        BD, BV = ctypes.POINTER(BlockDims), ctypes.POINTER(BlockViews)
        for name, args in (
                ("conv_forward", [P] * 6 + [CD, SP, SP, P]),
                ("conv_backward", [P] * 10 + [CD, SP, SP, SP, P, S, P]),
                ("ssm_forward", [P] * 9 + [SD, SV, P, S, P]),
                ("ssm_step", [P] * 8 + [SD, SV, P]),
                ("ssm_backward", [P] * 16 + [SD, SV, SV, P, S, P]),
                ("block_pool", [P, P, I, BD, BV, P]),
                ("block_select", [P, P, I, P, P, BD, BV, P]),
                ("block_forward", [P] * 7 + [BD, BV, P, S, P]),
                ("block_backward", [P] * 11 + [BD, BV, BV, P, S, P])):
            fn = getattr(lib, "sdm_" + name)
            fn.argtypes, fn.restype = args, ctypes.c_int
        for name, d in (("conv_backward", CD), ("ssm", SD), ("ssm_backward", SD), ("block", BD),
                        ("block_backward", BD)):
            fn = getattr(lib, "sdm_%s_workspace_bytes" % name)
            fn.argtypes, fn.restype = [d], S
        _bound = lib
    return _bound


def _dims_ok(t: torch.Tensor, name: str, layout: str) -> None:
    if t.dim() != 4:
        raise ValueError("%s must be %s, got shape %s" % (name, layout, tuple(t.shape)))
    if t.dtype not in _IN_DTYPES:
        raise TypeError("%s has dtype %s, expected torch.float32 or torch.bfloat16" % (name, t.dtype))


def _same_device(named, dense=()) -> torch.device:
    dev = named[0][1].device
    for name, t in named:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("all tensors must be CUDA tensors (there is no CPU path)")
        if t.device != dev:
            raise ValueError("all tensors must be on one device")
        if name in dense:
            if not t.is_contiguous():
                raise ValueError("%s must be contiguous" % name)
        elif t.dim() == 4 and t.shape[3] > 1 and t.stride(3) != 1:
            raise ValueError("the last axis of %s must be dense" % name)
    return dev


def _strides(t: torch.Tensor) -> Strides:
    # the stride of an axis of one element says nothing and would hide alignment
    s, n = t.stride(), t.shape
    return Strides(s[0] if n[0] > 1 else 0, s[1] if n[1] > 1 else 0, s[2] if n[2] > 1 else 0)


def _span(t: torch.Tensor):
    n = 1 + sum((s - 1) * st for s, st in zip(t.shape, t.stride())) if t.numel() else 0
    return t.data_ptr(), t.data_ptr() + n * t.element_size()


def _apart(outs, ins) -> None:
    """Given outputs must not overlap each other, themselves or an input."""
    for i, (no, o) in enumerate(outs):
        if o is None or o.numel() == 0:
            continue
        need = 0
        for st, s in sorted((st, s) for s, st in zip(o.shape, o.stride()) if s > 1):
            if st <= need:
                raise ValueError("rows of %s overlap" % no)
            need += (s - 1) * st
        a0, a1 = _span(o)
        for nt, t in outs[i + 1:] + ins:
            if t is None or t.numel() == 0:
                continue
            b0, b1 = _span(t)
            if a0 < b1 and b0 < a1:
                raise ValueError("%s overlaps %s; outputs must not alias other tensors" % (no, nt))


class _On:
    """Device and stream of a call: `with _On(dev, stream) as s` makes the device
    current (only if another one is) and allocations belong to `stream`."""

    def __init__(self, dev, stream):
        self.dev, self.stream, self.stack = dev, stream, None

    def __enter__(self):
        if self.stream is None and torch.cuda.current_device() == self.dev.index:
            return ctypes.c_void_p(torch.cuda.current_stream(self.dev).cuda_stream)
        self.stack = contextlib.ExitStack()
        self.stack.enter_context(torch.cuda.device(self.dev))
        if self.stream is not None:
            if self.stream.device != self.dev:
                self.stack.close()
                raise ValueError("stream belongs to another device than the tensors")
            self.stack.enter_context(torch.cuda.stream(self.stream))
        return ctypes.c_void_p(torch.cuda.current_stream(self.dev).cuda_stream)

    def __exit__(self, *exc):
        if self.stack is not None:
            self.stack.close()
        return False


def _like(t: torch.Tensor, shape=None, dtype=None) -> torch.Tensor:
    """Empty [B, H, T(, d)], token-major where t is."""
    shape = tuple(t.shape) if shape is None else tuple(shape)
    dtype = t.dtype if dtype is None else dtype
    if t.shape[1] > 1 and t.shape[2] > 1 and t.stride(2) > t.stride(1):
        swapped = (shape[0], shape[2], shape[1]) + shape[3:]
        return torch.empty(swapped, dtype=dtype, device=t.device).transpose(1, 2)
    return torch.empty(shape, dtype=dtype, device=t.device)


def _workspace_for(need: int, given: Optional[torch.Tensor], dev) -> torch.Tensor:
    if given is None:
        return torch.empty(need, dtype=torch.uint8, device=dev)
    if given.device != dev or _nbytes(given) < need or not given.is_contiguous():
        raise SDMError(4, "workspace too small, not contiguous or on another device")
    return given


def _lengths_ok(lengths: Optional[torch.Tensor], B: int) -> None:
    if lengths is not None:
        _expect(lengths, "lengths", (B,), (torch.int32,))


# ---------------------------------------------------------------- convolution
def _conv_args(x, w, bias, silu):
    _dims_ok(x, "x", "[B, H, T, d]")
    B, H, T, d = x.shape
    if w.dim() != 3:
        raise ValueError("w must be [H, d, K], got shape %s" % (tuple(w.shape),))
    K = w.shape[2]
    _expect(w, "w", (H, d, K), (x.dtype,))
    if bias is not None:
        _expect(bias, "bias", (H, d), (x.dtype,))
    return ConvDims(B, H, T, d, K, int(bool(silu)), _IN_DTYPES[x.dtype])


def conv_forward(x, w, bias=None, state=None, *, silu: bool = True,
                 lengths: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """Short causal convolution along T (sdm_conv_forward).  x [B,H,T,d]; w [H,d,K]
    with 2 <= K <= 8; bias [H,d] or None; state [B,H,K-1,d] (contiguous), the K - 1
    inputs before the call, updated in place to the last ones -- one token at a time
    is T = 1.  All of x's dtype.  lengths [B] int32: steps at or past it are not read
    and give 0.  Returns y [B,H,T,d] = silu(p), or p with silu=False."""
    dims = _conv_args(x, w, bias, silu)
    if state is not None:
        _expect(state, "state", (dims.B, dims.H, max(dims.K - 1, 0), dims.d), (x.dtype,))
    _lengths_ok(lengths, dims.B)
    if y is not None:
        _expect(y, "y", x.shape, (x.dtype,))
    dev = _same_device([("x", x), ("w", w), ("bias", bias), ("state", state), ("lengths", lengths),
                        ("y", y)], ("w", "bias", "state", "lengths"))
    _apart([("state", state), ("y", y)], [("x", x), ("w", w), ("bias", bias), ("lengths", lengths)])
    with _On(dev, stream) as s:
        if y is None:
            y = _like(x)
        _check(_lib().sdm_conv_forward(_ptr(x), _ptr(w), _ptr(bias), _ptr(state), _ptr(lengths),
                                       _ptr(y), ctypes.byref(dims), ctypes.byref(_strides(x)),
                                       ctypes.byref(_strides(y)), s))
    return y


def conv_backward(x, w, dy, bias=None, state0=None, dstate=None, *, silu: bool = True,
                  workspace: Optional[torch.Tensor] = None, stream=None) -> Dict[str, torch.Tensor]:
    """Gradients of conv_forward at full length (sdm_conv_backward).  state0: the state
    the forward started from (a copy; None for zeros); dstate [B,H,K-1,d] float32: the
    gradient of the state it left.  Returns x (x's dtype), w [H,d,K] and, where bias /
    state0 or dstate are given, bias [H,d] and state [B,H,K-1,d], float32."""
    dims = _conv_args(x, w, bias, silu)
    B, H, T, d, K = dims.B, dims.H, dims.T, dims.d, dims.K
    _expect(dy, "dy", x.shape, (x.dtype,))
    if state0 is not None:
        _expect(state0, "state0", (B, H, max(K - 1, 0), d), (x.dtype,))
    if dstate is not None:
        _expect(dstate, "dstate", (B, H, max(K - 1, 0), d), _F32)
    dev = _same_device([("x", x), ("w", w), ("dy", dy), ("bias", bias), ("state0", state0),
                        ("dstate", dstate)], ("w", "bias", "state0", "dstate"))
    lib = _lib()
    need = int(lib.sdm_conv_backward_workspace_bytes(ctypes.byref(dims)))
    if need == 0 or T == 0:
        _check(lib.sdm_conv_backward(*([None] * 10), ctypes.byref(dims), None, None, None, None, 0,
                                     None))
    with _On(dev, stream) as s:
        f32 = dict(dtype=torch.float32, device=dev)
        g = {"x": _like(x), "w": torch.empty(H, d, K, **f32)}
        if bias is not None:
            g["bias"] = torch.empty(H, d, **f32)
        if state0 is not None or dstate is not None:
            g["state"] = torch.empty(B, H, K - 1, d, **f32)
        ws = _workspace_for(need, workspace, dev)
        _check(lib.sdm_conv_backward(
            _ptr(x), _ptr(w), _ptr(bias), _ptr(state0), _ptr(dy), _ptr(dstate), _ptr(g["x"]),
            _ptr(g["w"]), _ptr(g.get("bias")), _ptr(g.get("state")), ctypes.byref(dims),
            ctypes.byref(_strides(x)), ctypes.byref(_strides(dy)), ctypes.byref(_strides(g["x"])),
            _ptr(ws), _nbytes(ws), s))
    return g


# ---------------------------------------------------------------- selective scan
def _ssm_args(x, dt, A, Bm, Cm, D):
    _dims_ok(x, "x", "[B, H, T, d_v]")
    B, H, T, P = x.shape
    if Bm.dim() != 4:
        raise ValueError("Bm must be [B, G, T, d_k], got shape %s" % (tuple(Bm.shape),))
    G, N = Bm.shape[1], Bm.shape[3]
    _expect(Bm, "Bm", (B, G, T, N), (x.dtype,))
    _expect(Cm, "Cm", (B, G, T, N), (x.dtype,))
    _expect(dt, "dt", (B, H, T), _F32)
    _expect(A, "A", (H,), _F32)
    if D is not None:
        _expect(D, "D", (H,), _F32)
    return SsmDims(B, H, G, T, N, P, _IN_DTYPES[x.dtype])


def ssm_workspace_bytes(B, H, G, T, d_k, d_v, in_dtype) -> int:
    """Bytes ssm_forward's workspace needs (0 for sizes it does not take)."""
    dt = _IN_DTYPES[in_dtype] if isinstance(in_dtype, torch.dtype) else int(in_dtype)
    return int(_lib().sdm_ssm_workspace_bytes(ctypes.byref(SsmDims(B, H, G, T, d_k, d_v, dt))))


def _ssm_views(x, dt, Bm, Cm, y) -> SsmViews:
    return SsmViews(_strides(x), _strides(dt), _strides(Bm), _strides(Cm), _strides(y))


def _ssm_forward(step, x, dt, A, Bm, Cm, S, D, lengths, y, workspace, stream):
    dims = _ssm_args(x, dt, A, Bm, Cm, D)
    _expect(S, "S", (dims.B, dims.H, dims.d_v, dims.d_k), _F32)
    _lengths_ok(lengths, dims.B)
    if y is not None:
        _expect(y, "y", x.shape, (x.dtype,))
    dev = _same_device([("x", x), ("dt", dt), ("A", A), ("Bm", Bm), ("Cm", Cm), ("S", S), ("D", D),
                        ("lengths", lengths), ("y", y)], ("A", "S", "D", "lengths"))
    _apart([("S", S), ("y", y)], [("x", x), ("dt", dt), ("A", A), ("Bm", Bm), ("Cm", Cm), ("D", D),
                                  ("lengths", lengths)])
    lib = _lib()
    with _On(dev, stream) as s:
        if y is None:
            y = _like(x)
        v = _ssm_views(x, dt, Bm, Cm, y)
        if step:
            _check(lib.sdm_ssm_step(_ptr(x), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(D), _ptr(S),
                                    _ptr(y), ctypes.byref(dims), ctypes.byref(v), s))
            return y
        ws = _workspace_for(int(lib.sdm_ssm_workspace_bytes(ctypes.byref(dims))), workspace, dev)
        _check(lib.sdm_ssm_forward(_ptr(x), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(D), _ptr(S),
                                   _ptr(lengths), _ptr(y), ctypes.byref(dims), ctypes.byref(v),
                                   _ptr(ws), _nbytes(ws), s))
    return y


def ssm_forward(x, dt, A, Bm, Cm, S, D=None, *, lengths: Optional[torch.Tensor] = None,
                y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """Selective state space scan (sdm_ssm_forward): per head
    S_t = exp(dt_t A) S_{t-1} + dt_t x_t Bm_t^T, y_t = S_t Cm_t + D x_t.
    x [B,H,T,d_v] and Bm, Cm [B,G,T,d_k] share one dtype (float32 or bfloat16), G
    divides H; dt [B,H,T], A [H], D [H] or None, float32; S [B,H,d_v,d_k] float32,
    updated in place.  lengths [B] int32: later steps leave S alone and give 0.
    Returns y [B,H,T,d_v] of x's dtype."""
    return _ssm_forward(False, x, dt, A, Bm, Cm, S, D, lengths, y, workspace, stream)


def ssm_step(x, dt, A, Bm, Cm, S, D=None, *, y: Optional[torch.Tensor] = None,
             stream=None) -> torch.Tensor:
    """ssm_forward for one token or a few at a time (sdm_ssm_step): one kernel that
    reads and writes S once, no workspace."""
    return _ssm_forward(True, x, dt, A, Bm, Cm, S, D, None, y, None, stream)


def ssm_backward(x, dt, A, Bm, Cm, S0, dy, dS_T=None, *, D=None,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> Dict[str, torch.Tensor]:
    """Gradients of ssm_forward at full length (sdm_ssm_backward).  S0: the state it
    started from (a copy; None for zeros); dS_T: the gradient of the state it left
    (None: 0).  Returns x, Bm, Cm (x's dtype), dt [B,H,T], A [H], S0 [B,H,d_v,d_k] and,
    where D is given, D [H], float32."""
    dims = _ssm_args(x, dt, A, Bm, Cm, D)
    B, H, P, N = dims.B, dims.H, dims.d_v, dims.d_k
    _expect(dy, "dy", x.shape, (x.dtype,))
    for name, t in (("S0", S0), ("dS_T", dS_T)):
        if t is not None:
            _expect(t, name, (B, H, P, N), _F32)
    dev = _same_device([("x", x), ("dt", dt), ("A", A), ("Bm", Bm), ("Cm", Cm), ("S0", S0), ("dy", dy),
                        ("dS_T", dS_T), ("D", D)], ("A", "S0", "dS_T", "D"))
    lib = _lib()
    need = int(lib.sdm_ssm_backward_workspace_bytes(ctypes.byref(dims)))
    if need == 0 or dims.T == 0:
        _check(lib.sdm_ssm_backward(*([None] * 16), ctypes.byref(dims), None, None, None, 0, None))
    with _On(dev, stream) as s:
        f32 = dict(dtype=torch.float32, device=dev)
        g = {"x": _like(x), "dt": _like(dt), "A": torch.empty(H, **f32), "Bm": _like(Bm),
             "Cm": _like(Cm), "S0": torch.empty(B, H, P, N, **f32)}
        if D is not None:
            g["D"] = torch.empty(H, **f32)
        ws = _workspace_for(need, workspace, dev)
        v, gv = _ssm_views(x, dt, Bm, Cm, dy), _ssm_views(g["x"], g["dt"], g["Bm"], g["Cm"], g["x"])
        _check(lib.sdm_ssm_backward(
            _ptr(x), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(D), _ptr(S0), _ptr(dy), _ptr(dS_T),
            _ptr(g["x"]), _ptr(g["dt"]), _ptr(g["A"]), _ptr(g["Bm"]), _ptr(g["Cm"]), _ptr(g.get("D")),
            _ptr(g["S0"]), ctypes.byref(dims), ctypes.byref(v), ctypes.byref(gv), _ptr(ws),
            _nbytes(ws), s))
    return g


# ---------------------------------------------------------------- block attention
_NONE = Strides(0, 0, 0)


def block_pool(k, kc: Optional[torch.Tensor] = None, *, block: int = 64, first: int = 0,
               stream=None) -> torch.Tensor:
    """Means of the complete blocks of k [B,G,Tk,d] (sdm_block_pool), in k's dtype:
    blocks first .. Tk // block - 1 of kc [B,G,n,d], n >= Tk // block (default: a new one
    with n = Tk // block).  With a cache that grows, first = the blocks already there."""
    _dims_ok(k, "k", "[B, G, Tk, d]")
    B, G, Tk, d = k.shape
    n = Tk // int(block) if block > 0 else 0
    if kc is not None:
        if kc.dim() != 4 or kc.shape[2] < n:
            raise ValueError("kc must be [B, G, n >= %d, d], got shape %s" % (n, tuple(kc.shape)))
        _expect(kc, "kc", (B, G, kc.shape[2], d), (k.dtype,))
    elif first:
        raise ValueError("first needs the kc that holds the blocks before it")
    dev = _same_device([("k", k), ("kc", kc)])
    _apart([("kc", kc)], [("k", k)])
    dims = BlockDims(B, G, G, 0, Tk, d, int(block), 1, _IN_DTYPES[k.dtype], 1.0)
    with _On(dev, stream) as s:
        if kc is None:
            kc = torch.empty(B, G, n, d, dtype=k.dtype, device=dev)
        v = BlockViews(_NONE, _strides(k), _NONE, _NONE, _strides(kc))
        _check(_lib().sdm_block_pool(_ptr(k), _ptr(kc), int(first), ctypes.byref(dims),
                                     ctypes.byref(v), s))
    return kc


def block_select(q, kc, *, n_sel: int, block: int = 64, Tk: Optional[int] = None,
                 lengths: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Lists of blocks per query and key head (sdm_block_select): the query's own block,
    then the best n_sel - 1 before it by the group's summed q . kc, best first, lower
    index at ties, then -1.  q [B,H,Tq,d] are the last Tq of Tk keys (default Tk = Tq),
    or of lengths[b] <= Tk in row b; kc [B,G,n,d] from block_pool.  Returns idx
    [B,G,Tq,n_sel] int32."""
    _dims_ok(q, "q", "[B, H, Tq, d]")
    B, H, Tq, d = q.shape
    if kc.dim() != 4:
        raise ValueError("kc must be [B, G, n, d], got shape %s" % (tuple(kc.shape),))
    G, n = kc.shape[1], kc.shape[2]
    _expect(kc, "kc", (B, G, n, d), (q.dtype,))
    _lengths_ok(lengths, B)
    dev = _same_device([("q", q), ("kc", kc), ("lengths", lengths)], ("lengths",))
    dims = BlockDims(B, H, G, Tq, Tq if Tk is None else int(Tk), d, int(block), int(n_sel),
                     _IN_DTYPES[q.dtype], 1.0)
    with _On(dev, stream) as s:
        idx = torch.empty(B, G, Tq, max(int(n_sel), 0), dtype=torch.int32, device=dev)
        v = BlockViews(_strides(q), _NONE, _NONE, _NONE, _strides(kc))
        _check(_lib().sdm_block_select(_ptr(q), _ptr(kc), n, _ptr(lengths), _ptr(idx),
                                       ctypes.byref(dims), ctypes.byref(v), s))
    return idx


def _block_args(q, k, v, idx, block, scale, lengths):
    _dims_ok(q, "q", "[B, H, Tq, d]")
    B, H, Tq, d = q.shape
    if k.dim() != 4:
        raise ValueError("k must be [B, G, Tk, d], got shape %s" % (tuple(k.shape),))
    G, Tk = k.shape[1], k.shape[2]
    _expect(k, "k", (B, G, Tk, d), (q.dtype,))
    _expect(v, "v", (B, G, Tk, d), (q.dtype,))
    if idx.dim() != 4:
        raise ValueError("idx must be [B, G, Tq, n_sel], got shape %s" % (tuple(idx.shape),))
    _expect(idx, "idx", (B, G, Tq, idx.shape[3]), (torch.int32,))
    _lengths_ok(lengths, B)
    return BlockDims(B, H, G, Tq, Tk, d, int(block), idx.shape[3], _IN_DTYPES[q.dtype],
                     d ** -0.5 if scale is None else float(scale))


def block_forward(q, k, v, idx, *, block: int = 64, scale: Optional[float] = None,
                  lengths: Optional[torch.Tensor] = None, o: Optional[torch.Tensor] = None,
                  return_lse: bool = False, workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of q [B,H,Tq,d], the last Tq of each row's keys, to the keys at or before
    its position in the listed blocks of k, v [B,G,Tk,d] (sdm_block_forward).  idx
    [B,G,Tq,n_sel] int32: any lists; an entry that is no block or lies behind the query
    adds nothing, a repeated one counts as often as listed.  scale defaults to d**-0.5.
    Returns o [B,H,Tq,d] (0 for a query without keys), or (o, lse [B,H,Tq] float32)."""
    dims = _block_args(q, k, v, idx, block, scale, lengths)
    if o is not None:
        _expect(o, "o", q.shape, (q.dtype,))
    dev = _same_device([("q", q), ("k", k), ("v", v), ("idx", idx), ("lengths", lengths), ("o", o)],
                       ("idx", "lengths"))
    _apart([("o", o)], [("q", q), ("k", k), ("v", v), ("idx", idx), ("lengths", lengths)])
    lib = _lib()
    with _On(dev, stream) as s:
        if o is None:
            o = _like(q)
        lse = torch.empty(q.shape[:3], dtype=torch.float32, device=dev) if return_lse else None
        views = BlockViews(_strides(q), _strides(k), _strides(v), _strides(o), _NONE)
        ws = _workspace_for(int(lib.sdm_block_workspace_bytes(ctypes.byref(dims))), workspace, dev)
        _check(lib.sdm_block_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(idx), _ptr(lengths), _ptr(o),
                                     _ptr(lse), ctypes.byref(dims), ctypes.byref(views), _ptr(ws),
                                     _nbytes(ws), s))
    return (o, lse) if return_lse else o


def block_backward(q, k, v, idx, o, lse, d_o, *, block: int = 64, scale: Optional[float] = None,
                   lengths: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None) -> Dict[str, torch.Tensor]:
    """Gradients of block_forward at its lists (sdm_block_backward): q, k, v in their
    dtype, given its o and lse and d_o = dL/do [B,H,Tq,d]."""
    dims = _block_args(q, k, v, idx, block, scale, lengths)
    _expect(o, "o", q.shape, (q.dtype,))
    _expect(d_o, "d_o", q.shape, (q.dtype,))
    _expect(lse, "lse", q.shape[:3], _F32)
    dev = _same_device([("q", q), ("k", k), ("v", v), ("idx", idx), ("o", o), ("lse", lse),
                        ("d_o", d_o), ("lengths", lengths)], ("idx", "lse", "lengths"))
    lib = _lib()
    need = int(lib.sdm_block_backward_workspace_bytes(ctypes.byref(dims)))
    with _On(dev, stream) as s:
        g = {"q": _like(q), "k": _like(k), "v": _like(v)}
        ws = _workspace_for(need, workspace, dev)
        views = BlockViews(_strides(q), _strides(k), _strides(v), _strides(o), _NONE)
        gv = BlockViews(_strides(g["q"]), _strides(g["k"]), _strides(g["v"]), _strides(d_o), _NONE)
        _check(lib.sdm_block_backward(
            _ptr(q), _ptr(k), _ptr(v), _ptr(idx), _ptr(lengths), _ptr(o), _ptr(lse), _ptr(d_o),
            _ptr(g["q"]), _ptr(g["k"]), _ptr(g["v"]), ctypes.byref(dims), ctypes.byref(views),
            ctypes.byref(gv), _ptr(ws), _nbytes(ws), s))
    return g
