"""Binding of the operators that decoding with drafted tokens needs beside retrieval: rotary
positions, attention over a paged K/V cache, and the cache's page operations.

Like the rest of the package it checks arguments, allocates outputs and scratch with
PyTorch and passes device pointers; the calls run on the current stream of their tensors'
device.  Unlike the calls that take a grown workspace, these allocate their scratch per
call, so that calls on several streams and captured graphs share none; the error word is
that of `ws`, by default `cache_workspace(device)`.
"""
from __future__ import annotations

import ctypes

import torch

from . import (CHUNK, LIB, MAX_DRAFT, Cache, Heads, Workspace, _check, _dtype, _need)

_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "parts": 3}
_SCRATCH = {}     # argument sizes -> scratch bytes
_WS = {}          # device index -> Workspace with the error word of these calls
_ERR_BYTES = 256


def cache_workspace(device) -> Workspace:
    """The workspace whose error word the calls of this module use by default (it never
    grows; `cache_workspace(device).check()` raises what a kernel flagged)."""
    d = torch.device(device)
    key = d.index if d.index is not None else torch.cuda.current_device()
    ws = _WS.get(key)
    if ws is None:
        ws = _WS[key] = Workspace(torch.device("cuda", key))
    return ws


class _On:
    """The device of a call's tensors made current, and its current stream."""
    __slots__ = ("dev", "old")

    def __init__(self, *tensors):
        dev = None
        for t in tensors:
            if t is not None:
                if not t.is_cuda:
                    raise ValueError("tensors must live on a CUDA device")
                i = t.get_device()
                if dev is None:
                    dev = i
                elif i != dev:
                    raise ValueError("tensors must live on one device")
        self.dev = dev
        self.old = torch.cuda.current_device()

    def __enter__(self):
        if self.old != self.dev:
            torch.cuda.set_device(self.dev)
        return torch.cuda.current_stream(self.dev).cuda_stream

    def __exit__(self, *exc):
        if self.old != self.dev:
            torch.cuda.set_device(self.old)


def _heads(t: torch.Tensor) -> Heads:
    # The stride of an axis of one is no address: torch may have left any number there.
    b, n, h, _ = t.shape
    s = t.stride()
    return Heads(t.data_ptr(), s[0] if b > 1 else 0, s[1] if n > 1 else 0, s[2] if h > 1 else 0)


def _scratch(key, size, device) -> torch.Tensor:
    n = _SCRATCH.get(key)
    if n is None:
        n = _SCRATCH[key] = size()
    return torch.empty(n, dtype=torch.uint8, device=device)


def _int32(t, shape, what):
    _need(t.dtype == torch.int32 and tuple(t.shape) == shape and t.is_contiguous(),
          f"{what} must be a contiguous int32 {list(shape)} tensor")


def _ws_ptr(ws, device):
    buf = (ws or cache_workspace(device)).buf
    return buf.data_ptr(), buf.numel()


# --------------------------------------------------------------------------- rotary positions
def rotary_frequencies(rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                       context: float = 0.0, low: float = 1.0, high: float = 32.0, device=None) -> torch.Tensor:
    """Turning speeds of the rot/2 pairs (gca_rotary_frequencies) as an int64 device tensor
    for rotary(): base^(-2i/rot) per position, with scaling "none", "linear", "ntk" or
    "parts" (which keeps the pairs that turn more than `high` times in `context` tokens and
    stretches those below `low` turns by `factor`)."""
    _need(scaling in _SCALINGS, f"scaling must be one of {sorted(_SCALINGS)}")
    buf = (ctypes.c_uint64 * max(1, rot // 2))()
    _check(LIB.gca_rotary_frequencies(rot, base, _SCALINGS[scaling], factor, context, low, high, buf))
    return torch.frombuffer(bytearray(bytes(buf)), dtype=torch.int64).to(device or "cuda")


def _rotary(q, k, freq, positions, interleaved, gain, q_out, k_out, backward):
    B, L, H, dh = q.shape
    Hkv = 0
    code = _dtype(q)
    if q.stride(3) != 1:
        raise ValueError("q must have unit stride in its last dim")
    if k is not None:
        Hkv = k.shape[2]
        if k.shape[0] != B or k.shape[1] != L or k.shape[3] != dh or k.dtype != q.dtype or k.stride(3) != 1:
            raise ValueError("k must be [B, L, Hkv, dh] like q, with unit stride in its last dim")
    if freq.dtype != torch.int64 or freq.dim() != 1 or not freq.is_contiguous():
        raise ValueError("freq must be what rotary_frequencies returned")
    pos_bs = 0
    if positions is not None:
        if positions.dtype != torch.int32 or positions.shape not in ((B, L), (1, L), (L,)) or positions.stride(-1) != 1 and L > 1:
            raise ValueError("positions must be int32 [B, L] or [L], with unit stride in the last dim")
        pos_bs = positions.stride(0) if positions.dim() == 2 and positions.shape[0] == B and B > 1 else 0
    with _On(q, k, freq, positions, q_out, k_out) as stream:
        if q_out is None:
            q_out = torch.empty((B, L, H, dh), dtype=q.dtype, device=q.device)
        if k is not None and k_out is None:
            k_out = torch.empty((B, L, Hkv, dh), dtype=k.dtype, device=k.device)
        for o, i in ((q_out, q), (k_out, k)):
            if i is None:
                _need(o is None, "k_out needs k")
            else:
                _need(o.shape == i.shape and o.dtype == i.dtype and o.stride(3) == 1, "an output must be like its input")
        hq, hqo = _heads(q), _heads(q_out)
        hk, hko = (ctypes.byref(_heads(k)), ctypes.byref(_heads(k_out))) if k is not None else (None, None)
        _check(LIB.gca_rotary(ctypes.byref(hq), hk, ctypes.byref(hqo), hko, code, B, L, H, Hkv, dh, 2 * freq.shape[0],
                              1 if interleaved else 0, backward, freq.data_ptr(),
                              positions.data_ptr() if positions is not None else None, pos_bs, gain, stream))
    return q_out, k_out


def rotary(q: torch.Tensor, k, freq: torch.Tensor, positions: torch.Tensor = None, interleaved: bool = False,
           gain: float = 1.0, q_out: torch.Tensor = None, k_out: torch.Tensor = None):
    """Rotary positions (gca_rotary).  q [B, L, H, dh], k [B, L, Hkv, dh] or None, with any
    strides but the last (views of a fused projection work); freq from
    rotary_frequencies(rot, ...): the first rot elements of a head turn, the others are
    copied.  positions int32 [B, L] or [L] (default: 0 .. L-1).  Pass q_out=q, k_out=k to
    work in place.  Returns (q_out, k_out)."""
    return _rotary(q, k, freq, positions, interleaved, gain, q_out, k_out, 0)


def rotary_backward(dq: torch.Tensor, dk, freq: torch.Tensor, positions: torch.Tensor = None,
                    interleaved: bool = False, gain: float = 1.0, q_out: torch.Tensor = None,
                    k_out: torch.Tensor = None):
    """Gradients of rotary() (gca_rotary with backward): dq, dk are the gradients of its
    outputs; returns those of its inputs."""
    return _rotary(dq, dk, freq, positions, interleaved, gain, q_out, k_out, 1)


# --------------------------------------------------------------------------- drafted tokens
def tree_plan(parents: torch.Tensor, lengths: torch.Tensor, ws: Workspace = None):
    """Mask and positions of a draft (gca_tree_plan), once for all layers of a step.
    parents int32 [B, T]: the earlier draft token that each follows, -1 for the cache's last
    token, -2 for padding; lengths int32 [B].  Returns mask int64 [B, T, ceil(T/64)] (bit u
    of row t: t sees u) and positions int32 [B, T] (-1 for padding)."""
    B, T = parents.shape
    _int32(parents, (B, T), "parents")
    _int32(lengths, (B,), "lengths")
    with _On(parents, lengths) as stream:
        mask = torch.empty((B, T, (T + 63) // 64), dtype=torch.int64, device=parents.device)
        positions = torch.empty((B, T), dtype=torch.int32, device=parents.device)
        wp, wn = _ws_ptr(ws, parents.device)
        _check(LIB.gca_tree_plan(parents.data_ptr(), lengths.data_ptr(), B, T, mask.data_ptr(), positions.data_ptr(),
                                 wp, wn, stream))
    return mask, positions


def _pool_struct(k_pages, v_pages, table, lengths, refs=None) -> Cache:
    if (k_pages.dim() != 4 or k_pages.shape[1] != CHUNK or v_pages.shape != k_pages.shape
            or v_pages.dtype != k_pages.dtype or not k_pages.is_contiguous() or not v_pages.is_contiguous()):
        raise ValueError("k_pages, v_pages must be contiguous [pages, 64, heads, dh] tensors of one type")
    if table.dtype != torch.int32 or table.dim() != 2 or not table.is_contiguous():
        raise ValueError("table must be a contiguous int32 [slots, width] tensor")
    slots, width = table.shape
    if lengths.dtype != torch.int32 or lengths.shape != (slots,) or not lengths.is_contiguous():
        raise ValueError("lengths must be a contiguous int32 [slots] tensor")
    pages, _, heads, dh = k_pages.shape
    if refs is not None:
        _int32(refs, (pages,), "refs")
    return Cache(k_pages.data_ptr(), v_pages.data_ptr(), _dtype(k_pages), heads, dh, pages, table.data_ptr(), slots,
                 width, lengths.data_ptr(), refs.data_ptr() if refs is not None else None)


def _attend(c: Cache, q, k_new, v_new, mask, positions, window, scale, out, lse, ws, stream):
    B, T, H, dh = q.shape
    if dh != c.dh or _dtype(q) != c.dtype or q.stride(3) != 1:
        raise ValueError("q must be [B, T, H, dh] of the pages' type and head dim, with unit stride in its last dim")
    for t in (k_new, v_new):
        if t.shape != (B, T, c.heads, dh) or t.dtype != q.dtype or t.stride(3) != 1:
            raise ValueError("k_new, v_new must be [B, T, heads, dh] of the pages' type, with unit stride in the last dim")
    if mask is not None and (mask.dtype != torch.int64 or mask.shape != (B, T, (T + 63) // 64) or not mask.is_contiguous()):
        raise ValueError("mask must be a contiguous int64 [B, T, ceil(T/64)] tensor")
    if positions is not None:
        _int32(positions, (B, T), "positions")
    if out is None:
        out = torch.empty((B, T, H, dh), dtype=q.dtype, device=q.device)
    else:
        _need(out.shape == q.shape and out.dtype == q.dtype and out.is_contiguous(), "out must be contiguous, like q")
    if lse is None:
        lse = torch.empty((B, T, H), dtype=torch.float32, device=q.device)
    else:
        _need(lse.shape == (B, T, H) and lse.dtype == torch.float32 and lse.is_contiguous(),
              "lse must be a contiguous float32 [B, T, H] tensor")
    _need(1 <= T <= MAX_DRAFT, f"T must be in 1..{MAX_DRAFT}")
    scratch = _scratch((B, T, H, c.heads, dh, c.dtype),
                       lambda: LIB.gca_tree_attention_scratch_size(B, T, H, c.heads, dh, c.dtype), q.device)
    wp, wn = _ws_ptr(ws, q.device)
    hq, hk, hv = _heads(q), _heads(k_new), _heads(v_new)
    _check(LIB.gca_tree_attention(ctypes.byref(hq), ctypes.byref(hk), ctypes.byref(hv), ctypes.byref(c), B, T, H,
                                  mask.data_ptr() if mask is not None else None,
                                  positions.data_ptr() if positions is not None else None, window,
                                  dh ** -0.5 if scale is None else scale, out.data_ptr(), lse.data_ptr(), wp, wn,
                                  scratch.data_ptr(), scratch.numel(), stream))
    return out, lse


def tree_attention(q: torch.Tensor, k_new: torch.Tensor, v_new: torch.Tensor, k_pages: torch.Tensor,
                   v_pages: torch.Tensor, table: torch.Tensor, lengths: torch.Tensor, mask: torch.Tensor = None,
                   positions: torch.Tensor = None, window: int = 0, scale: float = None, out: torch.Tensor = None,
                   lse: torch.Tensor = None, ws: Workspace = None):
    """Attention of T new tokens per sequence over a paged cache and one another
    (gca_tree_attention): single tokens, runs, or trees of drafted tokens.

    q [B, T, H, dh], k_new, v_new [B, T, heads, dh]; k_pages, v_pages [pages, 64, heads, dh];
    table int32 [slots >= B, width], lengths int32 [slots]; mask and positions from
    tree_plan (default: token t sees tokens 0 .. t of the draft and is at lengths + t).
    window > 0 keeps the last `window` positions of each token.  Returns O [B, T, H, dh] and
    LSE float32 [B, T, H]; the new tokens' keys and values go into the cache with
    PagedCache.append."""
    with _On(q, k_new, v_new, k_pages, v_pages, table, lengths, mask, positions, out, lse) as stream:
        return _attend(_pool_struct(k_pages, v_pages, table, lengths), q, k_new, v_new, mask, positions, window, scale,
                       out, lse, ws, stream)


# --------------------------------------------------------------------------- pages
class PagedCache:
    """A K/V cache in pages of 64 tokens, over the caller's tensors: k_pages, v_pages
    [pages, 64, heads, dh]; table int32 [slots, width] (-1: no page); lengths int32 [slots];
    refs int32 [pages], the slots that hold each page (0: free).

    The pool is also a K/V store for gca_forward: gca_forward(q, *cache.store(),
    cache.lookup(idx), scores, shift=0, kv_shared=True) attends to retrieved chunks where
    they lie.  Calls change the state in place, in stream order; no call waits for the
    device.  What a call could not do is flagged in the error word (see check())."""

    def __init__(self, k_pages, v_pages, table, lengths, refs, ws: Workspace = None):
        self.c = _pool_struct(k_pages, v_pages, table, lengths, refs)
        _On(k_pages, v_pages, table, lengths, refs)
        self.k_pages, self.v_pages, self.table, self.lengths, self.refs = k_pages, v_pages, table, lengths, refs
        self.ws = ws

    @classmethod
    def empty(cls, pages: int, slots: int, width: int, heads: int, dh: int, dtype=torch.bfloat16, device="cuda",
              ws: Workspace = None) -> "PagedCache":
        """A cache with every page free and every slot empty (the pages' contents are undefined)."""
        return cls(torch.empty((pages, CHUNK, heads, dh), dtype=dtype, device=device),
                   torch.empty((pages, CHUNK, heads, dh), dtype=dtype, device=device),
                   torch.full((slots, width), -1, dtype=torch.int32, device=device),
                   torch.zeros(slots, dtype=torch.int32, device=device),
                   torch.zeros(pages, dtype=torch.int32, device=device), ws)

    def _call(self, *tensors):
        return _On(self.table, *tensors)

    def _entries(self, slots, n):
        if slots is not None:
            _int32(slots, (n,), "slots")
            return slots.data_ptr()
        _need(n == self.c.slots, "without `slots` the call has one entry for each slot")
        return None

    def append(self, k_new: torch.Tensor, v_new: torch.Tensor, counts: torch.Tensor, path: torch.Tensor = None,
               slots: torch.Tensor = None):
        """Adds counts[i] tokens (int32 [n], 0 .. T) behind the last of slots[i] (default:
        entry i is slot i): rows 0 .. of k_new, v_new [n, T, heads, dh], or the rows that
        path int32 [n, T] names (an accepted path of a draft).  See gca_cache_append."""
        if k_new.dim() != 4:
            raise ValueError("k_new, v_new must be [n, T, heads, dh]")
        n, T, heads, dh = k_new.shape
        c = self.c
        for t in (k_new, v_new):
            if t.shape != (n, T, c.heads, c.dh) or _dtype(t) != c.dtype or t.stride(3) != 1:
                raise ValueError("k_new, v_new must be [n, T, heads, dh] of the pages' type, with unit stride in the last dim")
        _int32(counts, (n,), "counts")
        if path is not None:
            _int32(path, (n, T), "path")
        with self._call(k_new, v_new, counts, path, slots) as stream:
            ids = self._entries(slots, n)
            scratch = _scratch((n, T), lambda: LIB.gca_cache_append_scratch_size(n, T), counts.device)
            hk, hv = _heads(k_new), _heads(v_new)
            wp, wn = _ws_ptr(self.ws, counts.device)
            _check(LIB.gca_cache_append(ctypes.byref(c), ctypes.byref(hk), ctypes.byref(hv), n, T, ids, counts.data_ptr(),
                                        path.data_ptr() if path is not None else None, wp, wn, scratch.data_ptr(),
                                        scratch.numel(), stream))

    def fork(self, src: torch.Tensor, dst: torch.Tensor):
        """Slots dst[i] (int32 [n], empty) become copies of slots src[i] that share their
        pages; a shared last page is copied when one of them appends (gca_cache_fork)."""
        n = src.shape[0]
        _int32(src, (n,), "src")
        _int32(dst, (n,), "dst")
        with self._call(src, dst) as stream:
            wp, wn = _ws_ptr(self.ws, src.device)
            _check(LIB.gca_cache_fork(ctypes.byref(self.c), n, src.data_ptr(), dst.data_ptr(), wp, wn, stream))

    def _trim(self, begin, end, slots, release):
        given = begin if begin is not None else end if end is not None else slots
        n = given.shape[0] if given is not None else self.c.slots
        for t, what in ((begin, "begin"), (end, "end")):
            if t is not None:
                _int32(t, (n,), what)
        with self._call(begin, end, slots) as stream:
            ids = self._entries(slots, n)
            wp, wn = _ws_ptr(self.ws, self.table.device)
            _check(LIB.gca_cache_trim(ctypes.byref(self.c), n, ids, begin.data_ptr() if begin is not None else None,
                                      end.data_ptr() if end is not None else None, release, wp, wn, stream))

    def trim(self, begin: torch.Tensor = None, end: torch.Tensor = None, slots: torch.Tensor = None):
        """Keeps tokens begin[i] .. end[i]-1 (int32 [n]) of the slots and gives back the pages
        outside: `end` takes back the last tokens, `begin` lets go of pages that a window has
        passed (gca_cache_trim)."""
        self._trim(begin, end, slots, 0)

    def free(self, slots: torch.Tensor = None):
        """Empties the slots (int32 [n]; default: all) and gives back their pages."""
        self._trim(None, None, slots, 1)

    def compact(self) -> torch.Tensor:
        """Moves the pages in use to the lowest numbers (gca_cache_compact); returns their
        count, an int32 [1] device tensor: the pages from there on are free."""
        dev = self.table.device
        with self._call() as stream:
            live = torch.empty(1, dtype=torch.int32, device=dev)
            scratch = _scratch(self.c.pages, lambda: LIB.gca_cache_compact_scratch_size(self.c.pages), dev)
            wp, wn = _ws_ptr(self.ws, dev)
            _check(LIB.gca_cache_compact(ctypes.byref(self.c), live.data_ptr(), wp, wn, scratch.data_ptr(),
                                         scratch.numel(), stream))
        return live

    def lookup(self, idx: torch.Tensor, slots: torch.Tensor = None) -> torch.Tensor:
        """Page numbers of retrieved chunks (gca_cache_lookup): idx int32 [n, ...], chunk j of
        entry i's slot or -1; returns int32 like idx."""
        _need(idx.dtype == torch.int32 and idx.dim() >= 2 and idx.is_contiguous(), "idx must be a contiguous int32 [n, ...] tensor")
        n, per = idx.shape[0], idx[0].numel()
        with self._call(idx, slots) as stream:
            ids = self._entries(slots, n) if slots is not None else None
            out = torch.empty_like(idx)
            wp, wn = _ws_ptr(self.ws, idx.device)
            _check(LIB.gca_cache_lookup(ctypes.byref(self.c), n, per, ids, idx.data_ptr(), out.data_ptr(), wp, wn, stream))
        return out

    def store(self):
        """The pools as a K/V store shared by all sequences, for gca_forward and gather_chunks:
        k, v [pages*64, heads, dh]."""
        return self.k_pages.flatten(0, 1), self.v_pages.flatten(0, 1)

    def attention(self, q, k_new, v_new, mask=None, positions=None, window: int = 0, scale: float = None, out=None,
                  lse=None):
        """tree_attention over this cache: sequence b is slot b."""
        with self._call(q, k_new, v_new, mask, positions, out, lse) as stream:
            return _attend(self.c, q, k_new, v_new, mask, positions, window, scale, out, lse, self.ws, stream)

    def check(self):
        """Synchronise the current stream and raise GCAError if a call flagged an entry since
        the last check (the flag is cleared)."""
        with self._call():
            (self.ws or cache_workspace(self.table.device)).check()
