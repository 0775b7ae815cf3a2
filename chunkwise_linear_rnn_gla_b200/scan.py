"""Elementwise gated recurrence (vector state): thin binding over ``gla_scan_fwd`` / ``gla_scan_bwd`` /
``gla_scan_step`` (include/gla.h). Argument checks, output allocation and the current stream only; every
step runs in libgla's kernels.

Per sequence, head and channel, with a_t = exp(log_a_t):
    h_t = a_t h_{t-1} + w_t x_t,    w_t = 1 (write="input") or 1 - a_t (write="leak"),
with h_{-1} = h0 and hT the last state. It is the layer's gated memory without a key dimension, for
recurrent layers that stand beside GLA layers in a stack.

Shapes: x, h [B,H,L,D] (a [B,L,D] tensor is the H=1 case: x.unsqueeze(1)); log_a [B,H,L,D] fp32;
states h0, hT [B,H,D] fp32. Packed sequences: x, log_a [1,H,T,D] and cu_seqlens (int32 [N+1], device);
sequence n holds the rows cu_seqlens[n] .. cu_seqlens[n+1]-1, may be empty, and has row n of the states
[N,H,D]. Rows outside every sequence are left as they were in a buffer that the caller passes, and are 0 in
one that is allocated here.
gate="preact": log_a holds the gate's argument z, log a = logsigmoid(z) / tau.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import _dt, _enqueue, _finish_checks, _guarded, _lib, _same, _workspace, make_desc
from ._lib import load

__all__ = ["scan_fwd", "scan_bwd", "scan_step", "scan_workspace_size", "scan_workspace"]


def _write(write: str) -> int:
    w = _lib.SCAN_WRITE.get(write)
    if w is None:
        raise ValueError("write must be one of %s, got %r" % (sorted(_lib.SCAN_WRITE), write))
    return w


def _addr(t):
    return None if t is None else t.data_ptr()


def _index(t, name, n, dev):
    _same(t, name, (n,), torch.int32, dev)


def _sizes(x, cu_seqlens):
    """(sequences, H, rows, D) of x, which is [B,H,L,D], or [1,H,T,D] with cu_seqlens."""
    if not isinstance(x, torch.Tensor) or x.dim() != 4:
        raise ValueError("x must be a [B, H, L, D] tensor")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    B, H, L, D = x.shape
    if cu_seqlens is None:
        return B, H, L, D
    if B != 1:
        raise ValueError("packed sequences need x of shape [1, H, T, D], got %s" % (tuple(x.shape),))
    if not isinstance(cu_seqlens, torch.Tensor) or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens must be an int32 [N + 1] tensor, N >= 1")
    _index(cu_seqlens, "cu_seqlens", cu_seqlens.numel(), x.device)
    return cu_seqlens.numel() - 1, H, L, D


@functools.lru_cache(maxsize=256)
def _desc_ref(B, H, L, D, dtype, gate, tau, flags):
    """A descriptor (which the library only reads) as an argument; made once per set of sizes and options."""
    return ctypes.byref(make_desc(B, H, L, D, 1, dtype, flags=flags, gate=gate, tau=tau))


def _desc(x, B, H, L, D, gate, tau, flags):
    return _desc_ref(B, H, L, D, _dt(x), gate, tau, flags)


def _flags(checks, ws_from_fwd=False):
    return (_lib.FLAG_WS_FROM_FWD if ws_from_fwd else 0) | (_lib.FLAG_CHECKS if checks else 0)


def _finish(dev, guards, what):
    with torch.cuda.device(dev):
        _finish_checks(guards, what)


def scan_workspace_size(desc, packed: bool = False) -> int:
    """Workspace bytes of scan_fwd / scan_bwd for a descriptor (Dk = channels, Dv ignored)."""
    return int(load().gla_scan_workspace_size(ctypes.byref(desc), 1 if packed else 0))


def scan_workspace(x, cu_seqlens=None, checks=False) -> torch.Tensor:
    """A workspace for scan_fwd and the scan_bwd that follows it."""
    B, H, L, D = _sizes(x, cu_seqlens)
    n = load().gla_scan_workspace_size(_desc(x, B, H, L, D, "channel", 0.0, _flags(checks)), cu_seqlens is not None)
    return torch.empty(n, dtype=torch.uint8, device=x.device)


def _buffer(t, like, name, packed, guards):
    """An output: the caller's, or a new one, in checking mode (guards) between canaries."""
    if t is None:
        if guards is None:
            return torch.zeros_like(like) if packed else torch.empty_like(like)
        t = _guarded(like.shape, like.dtype, like.device, guards)
        return t.zero_() if packed else t
    _same(t, name, like.shape, like.dtype, like.device)
    return t


def scan_fwd(x, log_a, h0=None, *, cu_seqlens=None, write="input", gate="channel", tau=0.0, h=None, hT=None,
             want_hT=True, workspace: Optional[torch.Tensor] = None, checks=False):
    """Forward. Returns (h, hT); hT is None when want_hT is False and no hT buffer is given. A `workspace`
    (scan_workspace) keeps what scan_bwd(ws_from_fwd=True) reuses. checks=True: the library's checking mode
    (gate domain, finite outputs; of packed rows those that belong to a sequence) with canaries around the outputs
    allocated here, synchronous, raises GlaError on a failure."""
    lib = load()
    B, H, L, D = _sizes(x, cu_seqlens)
    dev = x.device
    _same(log_a, "log_a", x.shape, torch.float32, dev)
    if h0 is not None:
        _same(h0, "h0", (B, H, D), torch.float32, dev)
    desc = _desc(x, B, H, L, D, gate, tau, _flags(checks))
    guards = [] if checks else None
    h = _buffer(h, x, "h", cu_seqlens is not None, guards)
    if hT is not None:
        _same(hT, "hT", (B, H, D), torch.float32, dev)
    elif want_hT:
        hT = (torch.empty(B, H, D, dtype=torch.float32, device=dev) if guards is None else
              _guarded((B, H, D), torch.float32, dev, guards))
    ws, nbytes = None, 0
    if workspace is not None:
        ws, nbytes = _workspace(lib.gla_scan_workspace_size(desc, cu_seqlens is not None), dev, workspace)
    _enqueue(dev, "gla_scan_fwd", lib.gla_scan_fwd, desc, _write(write), x.data_ptr(), log_a.data_ptr(),
             _addr(cu_seqlens), _addr(h0), h.data_ptr(), _addr(hT), _addr(ws), nbytes)
    if checks:
        _finish(dev, guards, "gla_scan_fwd")
    return h, hT


def scan_bwd(x, log_a, dh, h0=None, dhT=None, *, cu_seqlens=None, write="input", gate="channel", tau=0.0,
             want_dh0=True, workspace: Optional[torch.Tensor] = None, ws_from_fwd=False, out=None, checks=False):
    """Backward of <dh, h> + <dhT, hT>. Returns a dict with dx, dlog_a (dL/dz for gate="preact") and dh0
    (None when want_dh0 is False and `out` has no buffer for it). `out` may hold buffers under these names.
    With ws_from_fwd=True the workspace must be the one the matching scan_fwd was given (same inputs, same
    options)."""
    lib = load()
    B, H, L, D = _sizes(x, cu_seqlens)
    dev = x.device
    packed = cu_seqlens is not None
    _same(log_a, "log_a", x.shape, torch.float32, dev)
    _same(dh, "dh", x.shape, x.dtype, dev)
    for t, n in ((h0, "h0"), (dhT, "dhT")):
        if t is not None:
            _same(t, n, (B, H, D), torch.float32, dev)
    if ws_from_fwd and workspace is None:
        raise ValueError("ws_from_fwd needs the forward's workspace")
    desc = _desc(x, B, H, L, D, gate, tau, _flags(checks, ws_from_fwd))
    out, guards = dict(out or {}), [] if checks else None
    dx = _buffer(out.get("dx"), x, "dx", packed, guards)
    dla = _buffer(out.get("dlog_a"), log_a, "dlog_a", packed, guards)
    dh0 = out.get("dh0")
    if dh0 is not None:
        _same(dh0, "dh0", (B, H, D), torch.float32, dev)
    elif want_dh0:
        dh0 = (torch.empty(B, H, D, dtype=torch.float32, device=dev) if guards is None else
               _guarded((B, H, D), torch.float32, dev, guards))
    ws, nbytes = _workspace(lib.gla_scan_workspace_size(desc, packed), dev, workspace)
    _enqueue(dev, "gla_scan_bwd", lib.gla_scan_bwd, desc, _write(write), x.data_ptr(), log_a.data_ptr(),
             _addr(cu_seqlens), _addr(h0), dh.data_ptr(), _addr(dhT), dx.data_ptr(), dla.data_ptr(), _addr(dh0),
             _addr(ws), nbytes)
    if checks:
        _finish(dev, guards, "gla_scan_bwd")
    return {"dx": dx, "dlog_a": dla, "dh0": dh0}


def scan_step(x, log_a, state, slots=None, *, write="input", gate="channel", tau=0.0, h=None, checks=False):
    """One token per row: x, log_a [B,H,D]; state [pool,H,D] fp32, updated in place. slots (int32 [B], device)
    names each row's entry of the pool (None: row b has entry b); a negative slot is a padding row, whose h is
    0. Returns h [B,H,D]. A slot outside the pool, or named twice in one call, is treated as padding and
    reported by gla_check_device_error."""
    lib = load()
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a [B, H, D] tensor")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    dev, shape = x.device, x.shape
    B, H, D = shape
    _same(log_a, "log_a", shape, torch.float32, dev)
    if not isinstance(state, torch.Tensor) or state.dim() != 3:
        raise ValueError("state must be a [pool, H, D] tensor")
    _same(state, "state", (state.shape[0], H, D), torch.float32, dev)
    if slots is not None:
        _index(slots, "slots", B, dev)
    elif state.shape[0] < B:
        raise ValueError("state has %d entries for %d rows" % (state.shape[0], B))
    guards = [] if checks else None
    if h is None:
        h = torch.empty_like(x) if guards is None else _guarded(shape, x.dtype, dev, guards)
    else:
        _same(h, "h", shape, x.dtype, dev)
    desc = _desc(x, B, H, 1, D, gate, tau, _flags(checks))
    _enqueue(dev, "gla_scan_step", lib.gla_scan_step, desc, _write(write), x.data_ptr(), log_a.data_ptr(),
             _addr(slots), state.shape[0], state.data_ptr(), h.data_ptr())
    if checks:
        _finish(dev, guards, "gla_scan_step")
    return h
