"""Torch front of the gated delta rule entry points (C ABI: include/gdr.h).

    gdr_fwd_chunked(q, k, v, g, beta, S0=None, cu_seqlens=None, ...) -> (o, S_T)
    gdr_decode_step(q, k, v, g, beta, S, slots=None, ...) -> o      (pool S updated in place)
    gdr_bwd_chunked(q, k, v, g, beta, dO, ...) -> (dq, dk, dv, dg, dbeta, dS0)
    gdr_save8(q, k, v) -> Saved8;  gdr_load8(saved) -> (q, k, v)
    gdr_bwd_chunked_saved8(saved, g, beta, dO, ...) -> (dq, dk, dv, dg, dbeta, dS0)

Marshalling only: outputs and workspaces are allocated through torch, the
work runs in the library's kernels on the inputs' device and its current
stream.
"""
from __future__ import annotations

from typing import NamedTuple, Optional, Tuple

import torch

from . import _lib

__all__ = ["gdr_fwd_chunked", "gdr_decode_step", "gdr_bwd_chunked", "gdr_bwd_workspace_bytes",
           "gdr_save8", "gdr_load8", "gdr_bwd_chunked_saved8", "Saved8"]


class Saved8(NamedTuple):
    """q, k, v in 8 bits: e4m3 bytes shaped like the inputs, and one exponent
    byte for each block of min(32, d) channels ([..., H, d / min(32, d)])."""
    q8: torch.Tensor
    qe: torch.Tensor
    k8: torch.Tensor
    ke: torch.Tensor
    v8: torch.Tensor
    ve: torch.Tensor


_DT = {torch.bfloat16: _lib.KDA_BF16, torch.float32: _lib.KDA_F32}


def _dt(t: torch.dtype) -> int:
    if t not in _DT:
        raise TypeError(f"unsupported dtype {t}; the gated delta rule takes bfloat16 or float32")
    return _DT[t]


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, name: str, dtype, shape, device) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.device == device:
        return
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype} (got {t.dtype})")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    raise ValueError(f"{name} must be contiguous")


# the current stream's handle (the private form costs a tenth of the public one's 3 us)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device: torch.device) -> int:
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


class _Dims:
    """Sizes of a batch of q, k [B, T, H_k, d_k] or packed [N, H_k, d_k] and
    v [..., H_v, d_v]; checks everything whose shape follows from them."""

    def __init__(self, q, k, v, g, beta, cu_seqlens, dtype=None, gates=True):
        if not isinstance(q, torch.Tensor) or not isinstance(v, torch.Tensor):
            raise TypeError("q and v must be torch.Tensors")
        self.dev = dev = q.device
        if dev.type != "cuda":
            raise ValueError(f"q is on {dev}: the kernels run on a GPU, there is no CPU fallback")
        if q.dim() not in (3, 4):
            raise ValueError("q must be [B, T, H_k, d_k] or [N, H_k, d_k]")
        if v.dim() != q.dim():
            raise ValueError("v must have as many dimensions as q")
        self.lead = lead = q.shape[:-2]
        self.Hk, self.dk = q.shape[-2:]
        self.Hv, self.dv = v.shape[-2:]
        self.N = lead[0] if len(lead) == 1 else lead[0] * lead[1]
        if cu_seqlens is not None:
            if q.dim() == 4 and q.shape[0] != 1:
                raise ValueError("cu_seqlens needs packed input ([N, H, d] or [1, N, H, d])")
            if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
                raise ValueError("cu_seqlens must be a 1-D tensor of n_seqs + 1 entries")
            _need(cu_seqlens, "cu_seqlens", torch.int32, cu_seqlens.shape, dev)
            self.n_seqs = cu_seqlens.numel() - 1
        else:
            self.n_seqs = lead[0] if q.dim() == 4 else 1
        dt = q.dtype if dtype is None else dtype
        _need(q, "q", dt, q.shape, dev)
        _need(k, "k", dt, q.shape, dev)
        _need(v, "v", dt, lead + (self.Hv, self.dv), dev)
        if self.dk < 1 or self.dv < 1:
            raise ValueError("d_k and d_v must be positive")
        if gates:
            _need(g, "g", torch.float32, lead + (self.Hv,), dev)
            _need(beta, "beta", torch.float32, lead + (self.Hv,), dev)
        self.state = torch.Size((self.n_seqs, self.Hv, self.dk, self.dv))

    def scale(self, scale):
        return self.dk ** -0.5 if scale is None else float(scale)

    def run(self, fn, *args):
        """Calls the library with the inputs' device current, on its current stream."""
        if torch.cuda.current_device() == self.dev.index:
            st = fn(*args, _stream(self.dev))
        else:
            with torch.cuda.device(self.dev):
                st = fn(*args, _stream(self.dev))
        if st:
            _lib.check(st)


def gdr_fwd_chunked(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                    beta: torch.Tensor, S0: Optional[torch.Tensor] = None,
                    cu_seqlens: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                    output_final_state: bool = True, o: Optional[torch.Tensor] = None,
                    S_T: Optional[torch.Tensor] = None
                    ) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """The gated delta rule over a batch of sequences.

    q, k : [B, T, H_k, d_k] or packed [N, H_k, d_k] (bf16 or fp32)
    v    : [..., H_v, d_v], H_v a multiple of H_k (value head h reads key head h // (H_v // H_k))
    g    : [..., H_v] fp32 log-decay <= 0 (-inf allowed);  beta : [..., H_v] fp32
    S0   : [n_seqs, H_v, d_k, d_v] fp32 or None
    cu_seqlens : int32 [n_seqs + 1] on the device (packed input only); rows of tokens behind
        its last entry are left as they are in a given o, unset in one allocated here
    scale : multiplies o; d_k ** -0.5 by default
    Returns (o in q's dtype, S_T fp32 or None).
    """
    d = _Dims(q, k, v, g, beta, cu_seqlens)
    if S0 is not None:
        _need(S0, "S0", torch.float32, d.state, d.dev)
    if o is None:
        o = torch.empty_like(v)                         # in q's dtype, which v has
    else:
        _need(o, "o", q.dtype, v.shape, d.dev)
    if S_T is not None:
        _need(S_T, "S_T", torch.float32, d.state, d.dev)
    elif output_final_state:
        S_T = torch.empty(d.state, dtype=torch.float32, device=d.dev)
    d.run(_lib.load().gdr_fwd_chunked, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S0),
          _ptr(cu_seqlens), d.n_seqs, d.N, d.Hk, d.Hv, d.dk, d.dv, d.scale(scale), _dt(q.dtype),
          _ptr(o), _ptr(S_T))
    return o, S_T


def gdr_decode_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                    beta: torch.Tensor, S: torch.Tensor, slots: Optional[torch.Tensor] = None,
                    scale: Optional[float] = None, o: Optional[torch.Tensor] = None
                    ) -> torch.Tensor:
    """One token for each request.  q, k : [N, H_k, d_k]; v : [N, H_v, d_v];
    g, beta : [N, H_v] fp32; S : a pool [n_slots, H_v, d_k, d_v] fp32, updated
    in place; slots : int32 [N] on the device, each request's state (all
    different; one outside the pool marks a padded row, whose o is zeros), or
    None for states 0 .. N - 1.  Returns o in q's dtype."""
    if isinstance(q, torch.Tensor) and q.dim() != 3:
        raise ValueError("q must be [N, H_k, d_k]")
    d = _Dims(q, k, v, g, beta, None)
    if not isinstance(S, torch.Tensor) or S.dim() != 4:
        raise ValueError("S must be [n_slots, H_v, d_k, d_v]")
    _need(S, "S", torch.float32, S.shape[:1] + d.state[1:], d.dev)
    if slots is not None:
        _need(slots, "slots", torch.int32, q.shape[:1], d.dev)
    if o is None:
        o = torch.empty_like(v)                         # in q's dtype, which v has
    else:
        _need(o, "o", q.dtype, v.shape, d.dev)
    d.run(_lib.load().gdr_decode_step, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(S),
          _ptr(slots), S.shape[0], d.N, d.Hk, d.Hv, d.dk, d.dv, d.scale(scale), _dt(q.dtype),
          _ptr(o))
    return o


def gdr_bwd_workspace_bytes(n_seqs: int, n_tokens: int, H_k: int, H_v: int, d_k: int, d_v: int,
                            dtype: torch.dtype = torch.bfloat16) -> int:
    """Bytes of workspace gdr_bwd_chunked (and, with bf16, gdr_bwd_chunked_saved8)
    needs for these sizes."""
    return int(_lib.load().gdr_bwd_workspace_bytes(n_seqs, n_tokens, H_k, H_v, d_k, d_v, _dt(dtype)))


def _bwd(d, dt, fn, args, g, beta, dO, S0, dS_T, cu_seqlens, scale, workspace):
    _need(dO, "dO", dt, d.lead + (d.Hv, d.dv), d.dev)
    if S0 is not None:
        _need(S0, "S0", torch.float32, d.state, d.dev)
    if dS_T is not None:
        _need(dS_T, "dS_T", torch.float32, d.state, d.dev)
    if workspace is None:
        need = gdr_bwd_workspace_bytes(d.n_seqs, d.N, d.Hk, d.Hv, d.dk, d.dv, dt)
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=d.dev)
    else:
        _need(workspace, "workspace", torch.uint8, workspace.shape, d.dev)
    new = lambda shape, t: torch.empty(shape, dtype=t, device=d.dev)   # noqa: E731
    dq, dk = new(d.lead + (d.Hk, d.dk), dt), new(d.lead + (d.Hk, d.dk), dt)
    dv, dS0 = torch.empty_like(dO), new(d.state, torch.float32)
    dg, db = torch.empty_like(g), torch.empty_like(g)
    d.run(fn, *args[0], _ptr(g), _ptr(beta), _ptr(S0), _ptr(cu_seqlens), d.n_seqs, d.N, d.Hk, d.Hv,
          d.dk, d.dv, d.scale(scale), *args[1], _ptr(dO), _ptr(dS_T), _ptr(dq), _ptr(dk), _ptr(dv),
          _ptr(dg), _ptr(db), _ptr(dS0), _ptr(workspace), workspace.numel())
    return dq, dk, dv, dg, db, dS0


def gdr_bwd_chunked(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                    beta: torch.Tensor, dO: torch.Tensor, S0: Optional[torch.Tensor] = None,
                    dS_T: Optional[torch.Tensor] = None,
                    cu_seqlens: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                    workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, ...]:
    """Gradients of gdr_fwd_chunked: dq, dk (summed over the value heads of a
    key head) and dv in q's dtype, dg, dbeta, dS0 in fp32.  dO has o's shape
    and q's dtype, dS_T is the final states' cotangent or None.  Rows of tokens
    behind cu_seqlens' last entry are unset.  The workspace (uint8) is
    allocated through torch unless given."""
    d = _Dims(q, k, v, g, beta, cu_seqlens)
    return _bwd(d, q.dtype, _lib.load().gdr_bwd_chunked, ((_ptr(q), _ptr(k), _ptr(v)), (_dt(q.dtype),)),
                g, beta, dO, S0, dS_T, cu_seqlens, scale, workspace)


def _exp_shape(shape):
    return shape[:-1] + (shape[-1] // min(32, shape[-1]),)


def gdr_save8(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor) -> Saved8:
    """Keeps bf16 q, k, v for the backward in 8 bits (half their bytes):
    e4m3 elements and a power-of-two scale for each 32 channels.  The inputs
    move by 2.7% of their norms, the gradients formed from them by 4 to 6%."""
    d = _Dims(q, k, v, None, None, None, torch.bfloat16, gates=False)
    b = lambda shape: torch.empty(shape, dtype=torch.uint8, device=d.dev)   # noqa: E731
    s = Saved8(b(q.shape), b(_exp_shape(q.shape)), b(k.shape), b(_exp_shape(k.shape)), b(v.shape),
               b(_exp_shape(v.shape)))
    d.run(_lib.load().gdr_save8, _ptr(q), _ptr(k), _ptr(v), d.N, d.Hk, d.Hv, d.dk, d.dv,
          *(_ptr(x) for x in s))
    return s


def _saved(s: Saved8, g, beta, cu_seqlens, gates=True) -> _Dims:
    if not isinstance(s, Saved8):
        raise TypeError("saved must be what gdr_save8 returned")
    d = _Dims(s.q8, s.k8, s.v8, g, beta, cu_seqlens, torch.uint8, gates)
    for name, x, e in (("qe", s.q8, s.qe), ("ke", s.k8, s.ke), ("ve", s.v8, s.ve)):
        _need(e, name, torch.uint8, _exp_shape(x.shape), d.dev)
    return d


def gdr_load8(saved: Saved8) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """The bf16 q, k, v that `saved` stands for."""
    d = _saved(saved, None, None, None, gates=False)
    out = tuple(torch.empty(x.shape, dtype=torch.bfloat16, device=d.dev)
                for x in (saved.q8, saved.k8, saved.v8))
    d.run(_lib.load().gdr_load8, *(_ptr(x) for x in saved), d.N, d.Hk, d.Hv, d.dk, d.dv,
          *(_ptr(x) for x in out))
    return out


def gdr_bwd_chunked_saved8(saved: Saved8, g: torch.Tensor, beta: torch.Tensor, dO: torch.Tensor,
                           S0: Optional[torch.Tensor] = None,
                           dS_T: Optional[torch.Tensor] = None,
                           cu_seqlens: Optional[torch.Tensor] = None,
                           scale: Optional[float] = None,
                           workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, ...]:
    """gdr_bwd_chunked at the inputs that gdr_save8 kept: the gradients are
    those at gdr_load8(saved), bit for bit."""
    d = _saved(saved, g, beta, cu_seqlens)
    return _bwd(d, torch.bfloat16, _lib.load().gdr_bwd_chunked_saved8,
                (tuple(_ptr(x) for x in saved), ()), g, beta, dO, S0, dS_T, cu_seqlens, scale,
                workspace)
