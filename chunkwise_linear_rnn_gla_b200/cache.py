"""Recurrent-state cache: thin binding over ``gla_cache_store`` / ``gla_cache_load`` / ``gla_cache_step``
(include/gla.h). The matrix states of many sequences live in a pool of slots, in 8 bits with one scale per
state row and 128 columns, and the last few tokens of each beside them; a decode step reads both and rounds
the state back only when its window of tokens is full.

    cache = StateCache.empty(slots, H, Dk, Dv)          # one per layer
    o, hT = gla_fwd(q, k, v, log_a)                     # prefill
    cache_store(cache, hT, slots)                       # quantised into its slots; lengths = 0
    o_t = cache_step(cache, q1, k1, v1, log_a1, slots, lengths); lengths += 1
    S = cache_load(cache, slots, lengths)               # fp32, e.g. the h0 of the next gla_fwd

`lengths` (int32, device) counts each row's tokens since its state was stored; the caller advances it. A
negative slot is a padding row (its output row is 0). A slot outside the pool, a negative length, or a slot
named twice in one store or step is treated as padding and reported by gla_check_device_error.
"""
from __future__ import annotations

import ctypes

import torch

from . import _dt, _enqueue, _finish_checks, _guarded, _lib, _need, _same, gate_shape, make_desc
from ._lib import load

__all__ = ["StateCache", "cache_store", "cache_load", "cache_step"]

_FORMATS = {torch.int8: "int8", torch.float8_e4m3fn: "e4m3"}
_CODES = {v: k for k, v in _FORMATS.items()}


class StateCache:
    """The tensors of a pool: codes [slots,H,Dk,Dv] (torch.int8 or torch.float8_e4m3fn), scale
    [slots,H,Dk,ceil(Dv/128)] fp32, and the windows k [slots,H,W,Dk], v [slots,H,W,Dv] (fp32 or bf16, the
    type of the layer's q, k, v) and log_a [slots,H,W,Dk] fp32."""

    def __init__(self, codes, scale, k, v, log_a):
        if not isinstance(codes, torch.Tensor) or codes.dim() != 4:
            raise ValueError("codes must be a [slots, H, Dk, Dv] tensor")
        if codes.dtype not in _FORMATS:
            raise TypeError("codes must be int8 or float8_e4m3fn, got %s" % codes.dtype)
        self.slots, self.H, self.Dk, self.Dv = codes.shape
        if not isinstance(k, torch.Tensor) or k.dim() != 4:
            raise ValueError("k must be a [slots, H, window, Dk] tensor")
        self.window = k.shape[2]
        _dt(k)
        self._tensors = (codes, scale, k, v, log_a)
        self._ptrs = tuple(t.data_ptr for t in self._tensors)
        self.format, self.dtype, self.device = _FORMATS[codes.dtype], k.dtype, codes.device
        self._descs = {}
        self._at = self._ref = None
        self._pool()

    def _pool(self):
        """The pool as an argument of the library. Its tensors' storage may have been exchanged since the last call
        (`t.data = ...`): the addresses are those of now, and new ones are looked over like the first."""
        codes, scale, k, v, log_a = self._ptrs
        at = (codes(), scale(), k(), v(), log_a())
        if at != self._at:
            codes, scale, k, v, log_a = self._tensors
            P, H, K, V, W, dev = self.slots, self.H, self.Dk, self.Dv, self.window, self.device
            _need(codes, "codes", (P, H, K, V), _CODES[self.format], dev)
            _need(scale, "scale", (P, H, K, -(-V // _lib.CACHE_GROUP)), torch.float32, dev)
            _need(k, "k", (P, H, W, K), self.dtype, dev)
            _need(v, "v", (P, H, W, V), self.dtype, dev)
            _need(log_a, "log_a", (P, H, W, K), torch.float32, dev)
            self._ref = ctypes.byref(_lib.GlaCache(*at, P, W, _lib.CACHE_FORMAT[self.format]))
            self._at = at
        return self._ref

    @property
    def codes(self):
        return self._tensors[0]

    @property
    def scale(self):
        return self._tensors[1]

    @property
    def k(self):
        return self._tensors[2]

    @property
    def v(self):
        return self._tensors[3]

    @property
    def log_a(self):
        return self._tensors[4]

    @classmethod
    def empty(cls, slots, H, Dk, Dv, *, window=16, format="int8", dtype=torch.bfloat16, device="cuda"):
        """A pool of zero states."""
        if format not in _CODES:
            raise ValueError("format must be one of %s, got %r" % (sorted(_CODES), format))
        f32 = dict(dtype=torch.float32, device=device)
        return cls(torch.zeros(slots, H, Dk, Dv, dtype=torch.uint8, device=device).view(_CODES[format]),
                   torch.zeros(slots, H, Dk, -(-Dv // _lib.CACHE_GROUP), **f32),
                   torch.zeros(slots, H, window, Dk, dtype=dtype, device=device),
                   torch.zeros(slots, H, window, Dv, dtype=dtype, device=device),
                   torch.zeros(slots, H, window, Dk, **f32))

    def _desc(self, B, gate="channel", tau=0.0, checks=False):
        """A descriptor (which the library only reads) as an argument; made once per batch size and options."""
        key = (B, gate, tau, checks)
        d = self._descs.get(key)
        if d is None:
            if len(self._descs) >= 256:  # a server that has met many batch sizes starts afresh
                self._descs.clear()
            d = self._descs[key] = ctypes.byref(make_desc(
                B, self.H, 1, self.Dk, self.Dv, "bf16" if self.dtype == torch.bfloat16 else "f32",
                flags=_lib.FLAG_CHECKS if checks else 0, gate=gate, tau=tau))
        return d


def _rows(cache, slots, lengths=None):
    """(rows, the pool as an argument) of a call."""
    if not isinstance(cache, StateCache):
        raise TypeError("cache must be a StateCache")
    if not isinstance(slots, torch.Tensor) or slots.dim() != 1:
        raise ValueError("slots must be an int32 [B] tensor")
    pool = cache._pool()
    _same(slots, "slots", slots.shape, torch.int32, cache.device)
    if lengths is not None:
        _same(lengths, "lengths", slots.shape, torch.int32, cache.device)
    return slots.shape[0], pool


def _finish(dev, guards, what):
    with torch.cuda.device(dev):
        _finish_checks(guards, what)


def cache_store(cache, S, slots, *, checks=False):
    """Quantise the states S [B,H,Dk,Dv] (fp32) into their slots (int32 [B], device). Their lengths are 0 then."""
    lib = load()
    B, pool = _rows(cache, slots)
    dev = cache.device
    _same(S, "S", (B, cache.H, cache.Dk, cache.Dv), torch.float32, dev)
    desc = cache._desc(B, checks=checks)
    _enqueue(dev, "gla_cache_store", lib.gla_cache_store, desc, pool, S.data_ptr(), slots.data_ptr())
    if checks:
        _finish(dev, [], "gla_cache_store")


def cache_load(cache, slots, lengths=None, S=None, *, checks=False):
    """The states of the slots, S [B,H,Dk,Dv] fp32, with the tokens in their windows applied (lengths None: as
    stored)."""
    lib = load()
    B, pool = _rows(cache, slots, lengths)
    dev = cache.device
    guards = [] if checks else None
    if S is None:
        S = (torch.empty(B, cache.H, cache.Dk, cache.Dv, dtype=torch.float32, device=dev) if guards is None else
             _guarded((B, cache.H, cache.Dk, cache.Dv), torch.float32, dev, guards))
    else:
        _same(S, "S", (B, cache.H, cache.Dk, cache.Dv), torch.float32, dev)
    desc = cache._desc(B, checks=checks)
    _enqueue(dev, "gla_cache_load", lib.gla_cache_load, desc, pool, slots.data_ptr(),
             None if lengths is None else lengths.data_ptr(), S.data_ptr())
    if checks:
        _finish(dev, guards, "gla_cache_load")
    return S


def cache_step(cache, q, k, v, log_a, slots, lengths, o=None, *, gate="channel", tau=0.0, checks=False):
    """One decode step through the cache: q, k [B,H,Dk], v [B,H,Dv] (the cache's dtype), log_a as for gla_step
    (fp32; every gate kind). Returns o [B,H,Dv]. The caller adds 1 to `lengths` afterwards."""
    lib = load()
    B, pool = _rows(cache, slots, lengths)
    if lengths is None:
        raise TypeError("cache_step needs lengths")
    dev, dt, H, Dk, Dv = cache.device, cache.dtype, cache.H, cache.Dk, cache.Dv
    _same(q, "q", (B, H, Dk), dt, dev)
    _same(k, "k", (B, H, Dk), dt, dev)
    _same(v, "v", (B, H, Dv), dt, dev)
    desc = cache._desc(B, gate, tau, checks)
    _same(log_a, "log_a", gate_shape(gate, B, H, None, Dk), torch.float32, dev)
    guards = [] if checks else None
    if o is None:
        o = torch.empty(B, H, Dv, dtype=dt, device=dev) if guards is None else _guarded((B, H, Dv), dt, dev, guards)
    else:
        _same(o, "o", (B, H, Dv), dt, dev)
    _enqueue(dev, "gla_cache_step", lib.gla_cache_step, desc, pool, q.data_ptr(), k.data_ptr(), v.data_ptr(),
             log_a.data_ptr(), slots.data_ptr(), lengths.data_ptr(), o.data_ptr())
    if checks:
        _finish(dev, guards, "gla_cache_step")
    return o
