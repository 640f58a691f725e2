"""The operators that decoding with drafted tokens needs beside retrieval: rotary positions,
attention over a paged K/V cache, and the cache's page operations.

The binding proper is native (csrc/binding.cpp): it checks the arguments, allocates outputs
and scratch with PyTorch and calls the C ABI on the current stream of the tensors' device
(which need not be the current one).  Scratch is allocated per call, so that calls on several
streams and captured graphs share none; the error word is that of `ws`, by default
`cache_workspace(device)`.
"""
from __future__ import annotations

import ctypes

import torch

from . import CHUNK, EXT, LIB, Workspace, _check, _need

_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "parts": 3}


class _ErrorWord(Workspace):
    """The default error word of a device: a workspace that never grows."""

    def __init__(self, index: int):
        self.device = torch.device("cuda", index)
        self.buf = EXT.error_word(index)

    def check(self):
        with torch.cuda.device(self.device):
            super().check()


def cache_workspace(device) -> Workspace:
    """The workspace whose error word the calls of this module use by default;
    `cache_workspace(device).check()` raises what a kernel flagged."""
    d = torch.device(device)
    return _ErrorWord(d.index if d.index is not None else torch.cuda.current_device())


def _word(ws):
    return None if ws is None else ws.buf


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


def rotary(q: torch.Tensor, k, freq: torch.Tensor, positions: torch.Tensor = None, interleaved: bool = False,
           gain: float = 1.0, q_out: torch.Tensor = None, k_out: torch.Tensor = None):
    """Rotary positions (gca_rotary).  q [B, L, H, dh], k [B, L, Hkv, dh] or None, with any
    strides but the last (views of a fused projection work); freq from
    rotary_frequencies(rot, ...): the first rot elements of a head turn, the others are
    copied.  positions int32 [B, L] or [L] (default: 0 .. L-1).  Pass q_out=q, k_out=k to
    work in place.  Returns (q_out, k_out)."""
    return EXT.rotary(q, k, freq, positions, interleaved, gain, q_out, k_out, 0)


def rotary_backward(dq: torch.Tensor, dk, freq: torch.Tensor, positions: torch.Tensor = None,
                    interleaved: bool = False, gain: float = 1.0, q_out: torch.Tensor = None,
                    k_out: torch.Tensor = None):
    """Gradients of rotary() (gca_rotary with backward): dq, dk are the gradients of its
    outputs; returns those of its inputs."""
    return EXT.rotary(dq, dk, freq, positions, interleaved, gain, q_out, k_out, 1)


# --------------------------------------------------------------------------- drafted tokens
def tree_plan(parents: torch.Tensor, lengths: torch.Tensor, ws: Workspace = None):
    """Mask and positions of a draft (gca_tree_plan), once for all layers of a step.
    parents int32 [B, T]: the earlier draft token that each follows, -1 for the cache's last
    token, -2 for padding; lengths int32 [slots >= B].  Returns mask int64 [B, T, ceil(T/64)] (bit u
    of row t: t sees u) and positions int32 [B, T] (-1 for padding)."""
    return EXT.tree_plan(parents, lengths, _word(ws))


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
    return EXT.tree_attention(q, k_new, v_new, k_pages, v_pages, table, lengths, None, mask, positions, window, scale, out,
                              lse, _word(ws))


# --------------------------------------------------------------------------- pages
class PagedCache:
    """A K/V cache in pages of 64 tokens, over the caller's tensors: k_pages, v_pages
    [pages, 64, heads, dh]; table int32 [slots, width] (-1: no page); lengths int32 [slots];
    refs int32 [pages], the slots that hold each page (0: free).

    The pool is also a K/V store for gca_forward: gca_forward(q, *cache.store(),
    cache.lookup(idx), scores, shift=0, kv_shared=True) attends to retrieved chunks where
    they lie.  Calls change the state in place, in stream order; no call waits for the
    device.  What a call could not do is flagged in the error word (see check()).  A page
    operation takes up to MAX_CACHE_ENTRIES entries; where no slots are named, entry i is slot i
    and a call may have fewer entries than there are slots.

    The five tensors are all there is: each call takes them as they are then, so that one of
    them may be replaced (a larger pool, a wider table) and a copy is a cache of its own."""

    __slots__ = ("k_pages", "v_pages", "table", "lengths", "refs", "ws")

    def __init__(self, k_pages, v_pages, table, lengths, refs, ws: Workspace = None):
        EXT.check_pool(k_pages, v_pages, table, lengths, refs)
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

    def append(self, k_new: torch.Tensor, v_new: torch.Tensor, counts: torch.Tensor, path: torch.Tensor = None,
               slots: torch.Tensor = None):
        """Adds counts[i] tokens (int32 [n], 0 .. T) behind the last of slots[i] (default:
        entry i is slot i): rows 0 .. of k_new, v_new [n, T, heads, dh], or the rows that
        path int32 [n, T] names (an accepted path of a draft).  See gca_cache_append."""
        EXT.append(self.k_pages, self.v_pages, self.table, self.lengths, self.refs, k_new, v_new, counts, path, slots,
                   _word(self.ws))

    def fork(self, src: torch.Tensor, dst: torch.Tensor):
        """Slots dst[i] (int32 [n], empty) become copies of slots src[i] that share their
        pages; a shared last page is copied when one of them appends (gca_cache_fork)."""
        EXT.fork(self.k_pages, self.v_pages, self.table, self.lengths, self.refs, src, dst, _word(self.ws))

    def trim(self, begin: torch.Tensor = None, end: torch.Tensor = None, slots: torch.Tensor = None):
        """Keeps tokens begin[i] .. end[i]-1 (int32 [n]) of the slots and gives back the pages
        outside: `end` takes back the last tokens, `begin` lets go of pages that a window has
        passed (gca_cache_trim)."""
        EXT.trim(self.k_pages, self.v_pages, self.table, self.lengths, self.refs, begin, end, slots, 0, _word(self.ws))

    def free(self, slots: torch.Tensor = None):
        """Empties the slots (int32 [n]; default: all) and gives back their pages."""
        EXT.trim(self.k_pages, self.v_pages, self.table, self.lengths, self.refs, None, None, slots, 1, _word(self.ws))

    def compact(self) -> torch.Tensor:
        """Moves the pages in use to the lowest numbers (gca_cache_compact); returns their
        count, an int32 [1] device tensor: the pages from there on are free."""
        return EXT.compact(self.k_pages, self.v_pages, self.table, self.lengths, self.refs, _word(self.ws))

    def lookup(self, idx: torch.Tensor, slots: torch.Tensor = None) -> torch.Tensor:
        """Page numbers of retrieved chunks (gca_cache_lookup): idx int32 [n, ...], chunk j of
        slot slots[i] (default: entry i is slot i) or -1; returns int32 like idx."""
        return EXT.lookup(self.k_pages, self.v_pages, self.table, self.lengths, self.refs, idx, slots, _word(self.ws))

    def store(self):
        """The pools as a K/V store shared by all sequences, for gca_forward and gather_chunks:
        k, v [pages*64, heads, dh]."""
        return self.k_pages.flatten(0, 1), self.v_pages.flatten(0, 1)

    def attention(self, q, k_new, v_new, mask=None, positions=None, window: int = 0, scale: float = None, out=None,
                  lse=None):
        """tree_attention over this cache: sequence b is slot b."""
        return EXT.tree_attention(q, k_new, v_new, self.k_pages, self.v_pages, self.table, self.lengths, self.refs, mask,
                                  positions, window, scale, out, lse, _word(self.ws))

    def check(self):
        """Synchronise the current stream and raise GCAError if a call flagged an entry since
        the last check (one kind a call: see Workspace.check)."""
        with torch.cuda.device(self.table.device):
            (self.ws or cache_workspace(self.table.device)).check()
