"""The operators of a prompt's way through the attention block: norms of queries and keys with their
rotary positions, causal attention over packed sequences with its gradients, and a cache that holds
what it computed in 8 bits.

As for the decoding operators, the binding proper is native (csrc/binding.cpp): calls run on the
current stream of the tensors' device, scratch is allocated per call, and the error word is that of
`ws`, by default `cache_workspace(device)`.
"""
from __future__ import annotations

import torch

from . import CHUNK, EXT, GCA_E4M3, LIB, Workspace, _need
from .decoding import PagedCache, _word


# --------------------------------------------------------------------------- norms with rotary positions
def norm_rotary(q: torch.Tensor, k, q_weight: torch.Tensor, k_weight, freq: torch.Tensor, positions: torch.Tensor = None,
                interleaved: bool = False, gain: float = 1.0, eps: float = 1e-6, q_out: torch.Tensor = None,
                k_out: torch.Tensor = None):
    """RMS norm of every head of q and k, and their rotary positions, in one pass (gca_norm_rotary):
    gain R(p) (x w / sqrt(mean(x^2) + eps)); elements that do not turn are normed alone.

    q [B, L, H, dh], k [B, L, Hkv, dh] or None, with any strides but the last; q_weight, k_weight
    float32 [dh]; freq, positions, interleaved and gain as in rotary().  Pass q_out=q, k_out=k to
    work in place (not where the gradients are needed: they take q and k as they were); outputs
    share no memory with inputs or each other otherwise.  Returns (q_out, k_out)."""
    return EXT.norm_rotary(q, k, q_weight, k_weight, freq, positions, interleaved, gain, eps, q_out, k_out)


def norm_rotary_backward(q: torch.Tensor, k, dq_out: torch.Tensor, dk_out, q_weight: torch.Tensor, k_weight,
                         freq: torch.Tensor, positions: torch.Tensor = None, interleaved: bool = False, gain: float = 1.0,
                         eps: float = 1e-6, dq: torch.Tensor = None, dk: torch.Tensor = None):
    """Gradients of norm_rotary() (gca_norm_rotary_backward): q, k are its inputs, dq_out, dk_out the
    gradients of its outputs.  Returns dq, dk (like q and k; pass dq=dq_out, dk=dk_out to work in
    place) and the weights' gradients, float32 [dh] (None without k)."""
    return EXT.norm_rotary_backward(q, k, dq_out, dk_out, q_weight, k_weight, freq, positions, interleaved, gain, eps, dq, dk)


# --------------------------------------------------------------------------- packed sequences
def prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, offsets: torch.Tensor, window: int = 0,
                     scale: float = None, out: torch.Tensor = None, lse: torch.Tensor = None, ws: Workspace = None):
    """Causal attention over packed sequences (gca_prompt_attention): sequence b is rows offsets[b] ..
    offsets[b+1]-1, and its row t sees its rows t - window + 1 .. t (window 0: 0 .. t).

    q [N, H, dh], k, v [N, Hkv, dh] (H a multiple of Hkv; views of a fused projection work), offsets
    int32 [B + 1], read on the device.  Returns O like q (contiguous) and LSE float32 [N, H]; rows that
    no sequence has are not written.  out= and lse= may share no memory with an input or each other."""
    return EXT.prompt_attention(q, k, v, offsets, window, scale, out, lse, _word(ws))


def prompt_attention_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, dout: torch.Tensor,
                              lse: torch.Tensor, offsets: torch.Tensor, window: int = 0, scale: float = None,
                              dq: torch.Tensor = None, dk: torch.Tensor = None, dv: torch.Tensor = None,
                              ws: Workspace = None):
    """Gradients of prompt_attention() (gca_prompt_attention_backward): o, lse as it returned them, dout
    [N, H, dh] the gradient of o.  Returns (dq, dk, dv); dq=, dk=, dv= may be views of one tensor, but
    share no memory with each other or an input.  Rows that no sequence has are not written."""
    return EXT.prompt_attention_backward(q, k, v, o, dout, lse, offsets, window, scale, dq, dk, dv, _word(ws))


# --------------------------------------------------------------------------- a cache in 8 bits
class QuantisedCache(PagedCache):
    """A PagedCache whose pages hold e4m3 numbers with one power of two a token and head: half the
    bytes of bf16.  k_pages, v_pages uint8 [pages, 64, row], where a row is heads x dh numbers, then an
    exponent a head (row_bytes(heads, dh) bytes; see gca_cache_append_quantised for the numbers); table,
    lengths and refs as in PagedCache, and fork, trim, free, compact and lookup too.

    append and append_packed quantise as they write; read widens the chunks that retrieval names, for
    gca_forward.  The pages are no K/V store for it themselves, and tree_attention does not read them."""

    __slots__ = ("heads", "dh")

    def __init__(self, k_pages, v_pages, table, lengths, refs, heads: int, dh: int, ws: Workspace = None):
        EXT.check_quantised(k_pages, v_pages, table, lengths, refs, heads, dh)
        self.k_pages, self.v_pages, self.table, self.lengths, self.refs = k_pages, v_pages, table, lengths, refs
        self.heads, self.dh, self.ws = heads, dh, ws

    @staticmethod
    def row_bytes(heads: int, dh: int) -> int:
        """Bytes of a token's row in a page."""
        return int(LIB.gca_cache_row_bytes(GCA_E4M3, heads, dh))

    @classmethod
    def empty(cls, pages: int, slots: int, width: int, heads: int, dh: int, device="cuda",
              ws: Workspace = None) -> "QuantisedCache":
        """A cache with every page free and every slot empty (the pages' contents are undefined)."""
        row = cls.row_bytes(heads, dh)
        return cls(torch.empty((pages, CHUNK, row), dtype=torch.uint8, device=device),
                   torch.empty((pages, CHUNK, row), dtype=torch.uint8, device=device),
                   torch.full((slots, width), -1, dtype=torch.int32, device=device),
                   torch.zeros(slots, dtype=torch.int32, device=device),
                   torch.zeros(pages, dtype=torch.int32, device=device), heads, dh, ws)

    def append(self, k_new: torch.Tensor, v_new: torch.Tensor, counts: torch.Tensor, path: torch.Tensor = None,
               slots: torch.Tensor = None):
        """PagedCache.append of rows in bfloat16 or float32, quantised as they are written
        (gca_cache_append_quantised)."""
        EXT.append_quantised(self.k_pages, self.v_pages, self.table, self.lengths, self.refs, self.heads, self.dh, k_new,
                             v_new, counts, path, None, slots, _word(self.ws))

    def append_packed(self, k: torch.Tensor, v: torch.Tensor, offsets: torch.Tensor, slots: torch.Tensor = None):
        """Rows offsets[i] .. offsets[i+1]-1 (int32 [n + 1]) of k, v [N, heads, dh] go behind the last token
        of slots[i] (default: entry i is slot i): the packed prompts of prompt_attention."""
        EXT.append_quantised(self.k_pages, self.v_pages, self.table, self.lengths, self.refs, self.heads, self.dh, k, v,
                             None, None, offsets, slots, _word(self.ws))

    def read(self, idx: torch.Tensor, slots: torch.Tensor = None, dtype=torch.bfloat16):
        """Chunks idx int32 [n, ...] of slots[i] (default: entry i is slot i), -1: none, widened to
        bfloat16 or float32 (gca_cache_read; exactly).  Returns k, v [n, per * 64, heads, dh] and idx_local
        like idx, so that gca_forward(q, k, v, idx_local, scores, shift=0) attends to them."""
        _need(dtype in (torch.bfloat16, torch.float32), "dtype must be bfloat16 or float32")
        return EXT.read_quantised(self.k_pages, self.v_pages, self.table, self.lengths, self.refs, self.heads, self.dh, idx,
                                  slots, dtype == torch.float32, _word(self.ws))

    def numbers(self):
        """Views of the pages: k, v float8_e4m3fn [pages, 64, heads, dh], and their exponents uint8 [pages, 64,
        heads].  A value is its number times two to the power exponent - 127."""
        n = self.heads * self.dh
        split = lambda p: (p.view(torch.float8_e4m3fn)[..., :n].unflatten(-1, (self.heads, self.dh)),  # noqa: E731
                           p[..., n:n + self.heads])
        (k, ke), (v, ve) = split(self.k_pages), split(self.v_pages)
        return k, v, ke, ve

    def store(self):
        raise TypeError("a quantised cache is no K/V store: read() its chunks")

    def attention(self, *args, **kw):
        raise TypeError("tree_attention does not read a quantised cache")
