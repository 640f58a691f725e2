"""Float64 CPU oracle of the decoding operators: rotary positions, attention of drafted
tokens over a paged cache, and the cache's page operations.

Written from the operators' definitions with numpy, one value or one row at a time; it
shares no code with the GPU path.
"""
from __future__ import annotations

import math

import numpy as np

PAGE = 64


# ------------------------------------------------------------------ rotary positions
def speeds(rot, base=10000.0, scaling="none", factor=1.0, context=0.0, low=1.0, high=32.0):
    """Radians per position of the rot / 2 pairs."""
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    out = []
    for i in range(rot // 2):
        w = base ** (-2.0 * i / rot)
        if scaling == "linear":
            w /= factor
        elif scaling == "parts":
            c = min(1.0, max(0.0, (context * w / (2 * math.pi) - low) / (high - low)))
            w = c * w + (1 - c) * w / factor
        out.append(w)
    return np.array(out)


def rotary(x, positions, w, interleaved=False, gain=1.0, backward=False):
    """x [B, L, H, dh], positions [B, L]; the first 2 len(w) elements of each head turn."""
    x = np.asarray(x, dtype=np.float64)
    half = len(w)
    angle = positions[:, :, None, None].astype(np.float64) * w
    c, s = gain * np.cos(angle), gain * np.sin(angle) * (-1.0 if backward else 1.0)
    y = x.copy()
    i1 = np.arange(half) * 2 if interleaved else np.arange(half)
    i2 = i1 + 1 if interleaved else i1 + half
    y[..., i1] = x[..., i1] * c - x[..., i2] * s
    y[..., i2] = x[..., i1] * s + x[..., i2] * c
    return y


# ------------------------------------------------------------------ trees
def tree(parents, length):
    """Mask [T, T] (row t sees itself and its ancestors) and positions [T] of one draft."""
    T = len(parents)
    see, pos = np.zeros((T, T), dtype=bool), np.full(T, -1)
    for t, p in enumerate(parents):
        if p == -1:
            pos[t] = length
        elif 0 <= p < t and pos[p] >= 0:
            pos[t] = pos[p] + 1
            see[t] = see[p]
        else:
            continue
        see[t, t] = True
    return see, pos


def pack_mask(see):
    """Mask [B, T, T] as int64 words [B, T, ceil(T / 64)]."""
    B, T, _ = see.shape
    words = np.zeros((B, T, (T + 63) // 64), dtype=np.uint64)
    for u in range(T):
        words[:, :, u // 64] |= see[:, :, u].astype(np.uint64) << np.uint64(u % 64)
    return words.view(np.int64)


def tree_attention(q, k_new, v_new, k_pages, v_pages, table, lengths, see, pos, window=0, scale=None):
    """One row at a time.  see [B, T, T], pos [B, T] (-1: padding).  Returns O, LSE, and per
    output the weighted mean of |v| and per row the largest sum of |q k| scale and the number
    of keys (what the error bounds are made of)."""
    B, T, H, dh = q.shape
    Hkv = k_pages.shape[2]
    scale = dh ** -0.5 if scale is None else scale
    o, lse = np.zeros((B, T, H, dh)), np.full((B, T, H), -np.inf)
    mean_abs, dot_abs, keys = np.zeros((B, T, H, dh)), np.zeros((B, T, H)), np.zeros((B, T, H))
    for b in range(B):
        n = int(lengths[b])
        for m in range(Hkv):
            ks, vs, at = [], [], []
            for j in range(n):
                page = table[b, j // PAGE]
                if 0 <= page < k_pages.shape[0]:
                    ks.append(k_pages[page, j % PAGE, m])
                    vs.append(v_pages[page, j % PAGE, m])
                    at.append(j)
            ks, vs = np.array(ks).reshape(-1, dh), np.array(vs).reshape(-1, dh)
            at = np.array(at, dtype=np.int64)
            for t in range(T):
                if pos[b, t] < 0:
                    continue
                p = max(int(pos[b, t]), n)
                low = p - window if window else -1
                past = at > low
                new = [u for u in range(T) if see[b, t, u] and pos[b, u] >= 0 and (not window or max(pos[b, u], n) > low)]
                kk = np.concatenate([ks[past], k_new[b, new, m].reshape(-1, dh)])
                vv = np.concatenate([vs[past], v_new[b, new, m].reshape(-1, dh)])
                if not len(kk):
                    continue
                for h in range(m * (H // Hkv), (m + 1) * (H // Hkv)):
                    s = kk @ q[b, t, h] * scale
                    top = s.max()
                    e = np.exp(s - top)
                    w = e / e.sum()
                    o[b, t, h], lse[b, t, h] = w @ vv, top + np.log(e.sum())
                    mean_abs[b, t, h] = w @ np.abs(vv)
                    dot_abs[b, t, h] = (np.abs(kk) @ np.abs(q[b, t, h])).max() * scale
                    keys[b, t, h] = len(kk)
    return o, lse, mean_abs, dot_abs, keys


# ------------------------------------------------------------------ pages
class Pages:
    """The cache's state as plain lists, its operations one entry at a time.  `flagged` and
    `full` tell whether a call left an entry out."""

    def __init__(self, k_pages, v_pages, table, lengths, refs):
        self.k, self.v = k_pages.copy(), v_pages.copy()
        self.table, self.lengths, self.refs = table.copy(), lengths.copy(), refs.copy()
        self.flagged = self.full = False

    def _slots(self, slots, n):
        out, seen = [], set()
        for i in range(n):
            s = int(slots[i]) if slots is not None else i
            if not 0 <= s < len(self.lengths) or s in seen:
                self.flagged = True
                out.append(-1)
            else:
                out.append(s)
            seen.add(s)
        return out

    def append(self, k_new, v_new, counts, path=None, slots=None):
        n, T = k_new.shape[:2]
        width = self.table.shape[1]
        free = [p for p in range(len(self.refs)) if self.refs[p] == 0]
        shared_before = self.refs.copy()
        drop, stopped = [], False
        k_old, v_old = self.k.copy(), self.v.copy()
        for i, s in enumerate(self._slots(slots, n)):
            if s < 0:
                continue
            c, old = int(counts[i]), int(self.lengths[s])
            if not 0 <= c <= T:
                self.flagged = True
                continue
            if old + c > width * PAGE:
                self.full = True
                continue
            if c == 0:
                continue
            last = int(self.table[s, old // PAGE]) if old % PAGE else -1
            if old % PAGE and not 0 <= last < len(self.refs):
                self.flagged = True
                continue
            copy = last >= 0 and shared_before[last] > 1
            first = old // PAGE if copy else -(-old // PAGE)
            need = -(-(old + c) // PAGE) - first
            if stopped or need > len(free):
                stopped = self.full = True
                continue
            for p in range(first, first + need):
                page = free.pop(0)
                self.table[s, p] = page
                self.refs[page] = 1
            if copy:
                drop.append(last)
                r = old % PAGE
                self.k[self.table[s, old // PAGE], :r] = k_old[last, :r]
                self.v[self.table[s, old // PAGE], :r] = v_old[last, :r]
            for t in range(c):
                row = t if path is None else int(path[i, t])
                if not 0 <= row < T:
                    self.flagged = True
                    continue
                page, at = self.table[s, (old + t) // PAGE], (old + t) % PAGE
                self.k[page, at], self.v[page, at] = k_new[i, row], v_new[i, row]
            self.lengths[s] = old + c
        for page in drop:
            self.refs[page] -= 1

    def fork(self, src, dst):
        slots = len(self.lengths)
        targets = [int(d) for d in dst]
        empty = [n == 0 for n in self.lengths]
        for i, (s, d) in enumerate(zip((int(x) for x in src), targets)):
            if not (0 <= s < slots and 0 <= d < slots) or s in targets or d in targets[:i] or not empty[d]:
                self.flagged = True
                continue
            self.table[d] = self.table[s]
            self.lengths[d] = self.lengths[s]
            for p in self.table[s]:
                if p >= 0:
                    self.refs[p] += 1

    def trim(self, begin=None, end=None, slots=None, n=None, release=False):
        for given in (begin, end, slots):
            n = len(given) if n is None and given is not None else n
        n = len(self.lengths) if n is None else n
        for i, s in enumerate(self._slots(slots, n)):
            if s < 0:
                continue
            length = int(self.lengths[s])
            hi = 0 if release else length if end is None else min(max(int(end[i]), 0), length)
            lo = 0 if begin is None or release else min(max(int(begin[i]), 0), hi)
            for p in range(self.table.shape[1]):
                page = int(self.table[s, p])
                if page >= 0 and ((p + 1) * PAGE <= lo or p * PAGE >= hi):
                    self.table[s, p] = -1
                    self.refs[page] -= 1
            self.lengths[s] = hi

    def compact(self):
        live = int((self.refs > 0).sum())
        moved = [p for p in range(live, len(self.refs)) if self.refs[p] > 0]
        holes = [p for p in range(live) if self.refs[p] == 0]
        held = self.refs > 0
        to = {a: b for a, b in zip(moved, holes)}
        for a, b in to.items():
            self.k[b], self.v[b] = self.k[a], self.v[a]
            self.refs[b], self.refs[a] = self.refs[a], 0
        for e, page in np.ndenumerate(self.table):
            if page == -1:
                continue
            if not 0 <= page < len(held) or not held[page]:  # no page, or a free one
                self.flagged = True
                self.table[e] = -1
            else:
                self.table[e] = to.get(int(page), page)
        return live

    def tokens(self, s):
        """The K rows of slot s, in order."""
        return np.array([self.k[self.table[s, j // PAGE], j % PAGE] for j in range(int(self.lengths[s]))])
