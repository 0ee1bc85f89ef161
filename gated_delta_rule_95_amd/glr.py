"""Torch front of the gated linear recurrence entry points (C ABI: include/glr.h).

    glr_fwd_scan(x, g, h0=None, cu_seqlens=None, ...) -> (h, h_T) or (h, h_T, kept)
    glr_fwd_scan_gated(x, r, i, rate, ...) -> the same             (gates fused)
    glr_bwd_scan(x, g, dh, ...) -> (dx, dg, dh0)
    glr_bwd_scan_gated(x, r, i, rate, dh, ...) -> (dx, dr, di, drate, dh0)
    glr_decode_step(x, g, S, slots=None, ...) -> h                 (pool S updated in place)
    glr_decode_step_gated(x, r, i, rate, S, slots=None, ...) -> h

Marshalling only: outputs and workspaces are allocated through torch, the
work runs in the library's kernels on the inputs' device and its current
stream.
"""
from __future__ import annotations

from typing import Optional, Tuple

import torch

from . import _lib
from .gdr import _need, _ptr, _stream

__all__ = ["glr_fwd_scan", "glr_fwd_scan_gated", "glr_bwd_scan", "glr_bwd_scan_gated",
           "glr_decode_step", "glr_decode_step_gated", "glr_fwd_workspace_bytes",
           "glr_bwd_workspace_bytes"]

_DT = {torch.bfloat16: _lib.KDA_BF16, torch.float32: _lib.KDA_F32}
_F32 = torch.float32


def _run(dev: torch.device, fn, *args) -> None:
    """Calls the library with `dev` current, on its current stream."""
    if torch.cuda.current_device() == dev.index:
        st = fn(*args, _stream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, _stream(dev))
    if st:
        _lib.check(st)


def _check(dev: torch.device, *what) -> None:
    """what: (tensor or None, name, dtype, shape), each as _need checks it."""
    for t, name, dtype, shape in what:
        if t is not None and not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
                                  and t.is_contiguous() and t.device == dev):
            _need(t, name, dtype, shape, dev)


def _given(*what) -> None:
    """what: (tensor, name) that must not be None."""
    for t, name in what:
        if t is None:
            raise TypeError(f"{name} must be a torch.Tensor")


def _int32(*what) -> None:
    """what: (size, name) that the library takes in 32 bits."""
    for n, name in what:
        if n >> 31:
            raise ValueError(f"{name} must be below 2^31 (got {n})")


class _Batch:
    """Sizes of a batch of x [B, T, D] or packed [N, D]; checks everything
    whose shape follows from them."""

    def __init__(self, x, gates, cu_seqlens):
        if not isinstance(x, torch.Tensor):
            raise TypeError("x must be a torch.Tensor")
        self.dev = dev = x.device
        if dev.type != "cuda":
            raise ValueError(f"x is on {dev}: the kernels run on a GPU, there is no CPU fallback")
        self.shape = shape = x.shape
        dims, dt = len(shape), x.dtype
        if dims not in (2, 3):
            raise ValueError("x must be [B, T, D] or [N, D]")
        if dt not in _DT:
            raise TypeError(f"unsupported dtype {dt}; the gated linear recurrence takes bfloat16 or float32")
        self.dt, self.D = _DT[dt], shape[-1]
        if self.D < 1:
            raise ValueError("x must have a channel")
        self.N = shape[0] if dims == 2 else shape[0] * shape[1]
        if cu_seqlens is not None:
            if dims == 3 and shape[0] != 1:
                raise ValueError("cu_seqlens needs packed input ([N, D] or [1, N, D])")
            if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
                raise ValueError("cu_seqlens must be a 1-D tensor of n_seqs + 1 entries")
            _need(cu_seqlens, "cu_seqlens", torch.int32, cu_seqlens.shape, dev)
            self.n_seqs = cu_seqlens.numel() - 1
        else:
            self.n_seqs = shape[0] if dims == 3 else 1
        if (self.D | self.n_seqs) >> 31:
            _int32((self.D, "D"), (self.n_seqs, "n_seqs"))
        if len(gates) == 1:
            g, = gates
            _given((g, "g"))
            _check(dev, (x, "x", dt, shape), (g, "g", _F32, shape))
            self.ins = (x.data_ptr(), g.data_ptr())
        else:
            r, i, rate = gates
            _given((r, "r"), (i, "i"), (rate, "rate"))
            _check(dev, (x, "x", dt, shape), (r, "r", dt, shape), (i, "i", dt, shape), (rate, "rate", _F32, (self.D,)))
            self.ins = (x.data_ptr(), r.data_ptr(), i.data_ptr(), rate.data_ptr())
        self.state = (self.n_seqs, self.D)

    def kept(self):
        """The shape of the kept states, from the bytes the library asks for."""
        return _lib.load().glr_kept_bytes(self.N, self.D) // (4 * self.D), self.D

    def workspace(self, need, given):
        if given is not None:
            _need(given, "workspace", torch.uint8, getattr(given, "shape", None), self.dev)
            return given
        return torch.empty(need, dtype=torch.uint8, device=self.dev) if need else None


def glr_fwd_workspace_bytes(n_tokens: int, D: int) -> int:
    """Bytes of workspace glr_fwd_scan and glr_fwd_scan_gated need for these sizes (0: none, or sizes that they refuse)."""
    return 0 if D >> 31 or n_tokens >> 63 else int(_lib.load().glr_fwd_workspace_bytes(n_tokens, D))


def glr_bwd_workspace_bytes(n_tokens: int, D: int) -> int:
    """Bytes of workspace glr_bwd_scan and glr_bwd_scan_gated need for these sizes (0: none, or sizes that they refuse)."""
    return 0 if D >> 31 or n_tokens >> 63 else int(_lib.load().glr_bwd_workspace_bytes(n_tokens, D))


def _fwd(fn, x, gates, h0, cu_seqlens, output_final_state, keep, h, h_T, workspace):
    b = _Batch(x, gates, cu_seqlens)
    _check(b.dev, (h0, "h0", _F32, b.state), (h, "h", x.dtype, b.shape), (h_T, "h_T", _F32, b.state))
    if h is None:
        h = torch.empty_like(x)
    if h_T is None and output_final_state:
        h_T = torch.empty(b.state, dtype=_F32, device=b.dev)
    kept = torch.empty(b.kept(), dtype=_F32, device=b.dev) if keep else None
    ws = b.workspace(_lib.load().glr_fwd_workspace_bytes(b.N, b.D), workspace)
    _run(b.dev, fn, *b.ins, _ptr(h0), _ptr(cu_seqlens), b.n_seqs, b.N, b.D, b.dt, h.data_ptr(), _ptr(h_T), _ptr(kept),
         _ptr(ws), 0 if ws is None else ws.numel())
    return (h, h_T, kept) if keep else (h, h_T)


def glr_fwd_scan(x: torch.Tensor, g: torch.Tensor, h0: Optional[torch.Tensor] = None,
                 cu_seqlens: Optional[torch.Tensor] = None, output_final_state: bool = True,
                 keep: bool = False, h: Optional[torch.Tensor] = None,
                 h_T: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None
                 ) -> Tuple[Optional[torch.Tensor], ...]:
    """h_t = exp(g_t) h_{t-1} + x_t for each channel, over a batch of sequences.

    x  : [B, T, D] or packed [N, D] (bf16 or fp32)
    g  : like x, fp32 log-decay <= 0 (-inf allowed)
    h0 : [n_seqs, D] fp32 or None
    cu_seqlens : int32 [n_seqs + 1] on the device (packed input only); rows of tokens behind
        its last entry are left as they are in a given h, unset in one allocated here
    keep : also return what the backward wants, the state before every 32nd token of the batch
    Returns (h in x's dtype, h_T fp32 or None), with keep (h, h_T, kept).
    """
    return _fwd(_lib.load().glr_fwd_scan, x, (g,), h0, cu_seqlens, output_final_state, keep, h, h_T, workspace)


def glr_fwd_scan_gated(x: torch.Tensor, r: torch.Tensor, i: torch.Tensor, rate: torch.Tensor,
                       h0: Optional[torch.Tensor] = None,
                       cu_seqlens: Optional[torch.Tensor] = None, output_final_state: bool = True,
                       keep: bool = False, h: Optional[torch.Tensor] = None,
                       h_T: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None
                       ) -> Tuple[Optional[torch.Tensor], ...]:
    """h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sigmoid(i_t) x_t with a_t = exp(-rate
    sigmoid(r_t)), the gates formed inside.  r, i : like x; rate : [D] fp32 >= 0;
    the rest as in glr_fwd_scan."""
    return _fwd(_lib.load().glr_fwd_scan_gated, x, (r, i, rate), h0, cu_seqlens, output_final_state, keep, h, h_T,
                workspace)


def _bwd(fn, x, gates, dh, h0, dh_T, cu_seqlens, kept, workspace):
    b = _Batch(x, gates, cu_seqlens)
    _given((dh, "dh"))
    _check(b.dev, (dh, "dh", x.dtype, b.shape), (h0, "h0", _F32, b.state), (dh_T, "dh_T", _F32, b.state))
    if kept is not None:
        _check(b.dev, (kept, "kept", _F32, b.kept()))
    ws = b.workspace(_lib.load().glr_bwd_workspace_bytes(b.N, b.D), workspace)
    # the gradients of x and of the gates are shaped like them
    out = [torch.empty_like(x)] + [torch.empty_like(t) for t in gates]
    out.append(torch.empty(b.state, dtype=_F32, device=b.dev))
    _run(b.dev, fn, *b.ins, _ptr(h0), _ptr(cu_seqlens), b.n_seqs, b.N, b.D, b.dt, _ptr(kept), dh.data_ptr(), _ptr(dh_T),
         *[t.data_ptr() for t in out], _ptr(ws), 0 if ws is None else ws.numel())
    return tuple(out)


def glr_bwd_scan(x: torch.Tensor, g: torch.Tensor, dh: torch.Tensor,
                 h0: Optional[torch.Tensor] = None, dh_T: Optional[torch.Tensor] = None,
                 cu_seqlens: Optional[torch.Tensor] = None, kept: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, ...]:
    """Gradients of glr_fwd_scan: dx in x's dtype, dg and dh0 in fp32.  dh has
    h's shape and dtype, dh_T is the final states' cotangent or None, kept is
    what the forward of these inputs returned (formed again where None).  Rows
    of tokens behind cu_seqlens' last entry are unset.  The workspace (uint8)
    is allocated through torch unless given."""
    return _bwd(_lib.load().glr_bwd_scan, x, (g,), dh, h0, dh_T, cu_seqlens, kept, workspace)


def glr_bwd_scan_gated(x: torch.Tensor, r: torch.Tensor, i: torch.Tensor, rate: torch.Tensor,
                       dh: torch.Tensor, h0: Optional[torch.Tensor] = None,
                       dh_T: Optional[torch.Tensor] = None,
                       cu_seqlens: Optional[torch.Tensor] = None,
                       kept: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, ...]:
    """Gradients of glr_fwd_scan_gated: dx, dr, di in x's dtype, drate [D]
    (summed over the tokens) and dh0 in fp32; the rest as in glr_bwd_scan."""
    return _bwd(_lib.load().glr_bwd_scan_gated, x, (r, i, rate), dh, h0, dh_T, cu_seqlens, kept, workspace)


def _decode(fn, x, gates, S, slots, h):
    b = _Batch(x, gates, None)
    shape = b.shape
    if len(shape) != 2:
        raise ValueError("x must be [N, D]")
    if not isinstance(S, torch.Tensor) or S.dim() != 2:
        raise ValueError("S must be [n_slots, D]")
    n_slots = S.shape[0]
    if (b.N | n_slots) >> 31:
        _int32((b.N, "N"), (n_slots, "n_slots"))
    _check(b.dev, (S, "S", _F32, (n_slots, b.D)), (slots, "slots", torch.int32, shape[:1]), (h, "h", x.dtype, shape))
    if h is None:
        h = torch.empty_like(x)
    _run(b.dev, fn, *b.ins, S.data_ptr(), None if slots is None else slots.data_ptr(), n_slots, b.N, b.D, b.dt,
         h.data_ptr())
    return h


def glr_decode_step(x: torch.Tensor, g: torch.Tensor, S: torch.Tensor,
                    slots: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None
                    ) -> torch.Tensor:
    """One token for each request.  x [N, D]; g [N, D] fp32; S : a pool
    [n_slots, D] fp32, updated in place; slots : int32 [N] on the device, each
    request's state (all different; one outside the pool marks a padded row,
    whose h is zeros), or None for states 0 .. N - 1.  Returns h in x's dtype."""
    return _decode(_lib.load().glr_decode_step, x, (g,), S, slots, h)


def glr_decode_step_gated(x: torch.Tensor, r: torch.Tensor, i: torch.Tensor, rate: torch.Tensor,
                          S: torch.Tensor, slots: Optional[torch.Tensor] = None,
                          h: Optional[torch.Tensor] = None) -> torch.Tensor:
    """glr_decode_step with the gates of glr_fwd_scan_gated formed inside: r, i
    like x, rate [D] fp32."""
    return _decode(_lib.load().glr_decode_step_gated, x, (r, i, rate), S, slots, h)
