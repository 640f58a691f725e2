"""Float64 CPU oracle of a prompt's operators, written from their definitions: norms of queries and
keys with rotary positions, causal attention over packed sequences with its gradients, and the numbers
of a quantised cache.  Test infrastructure only."""
from __future__ import annotations

import numpy as np

from .decode_oracle import rotary


def norm_rotary(x, weight, positions, w, eps, interleaved=False, gain=1.0):
    """gain R(p) (x weight / sqrt(mean(x^2) + eps)) of x [B, L, heads, dh]; w the pairs' speeds."""
    x = np.asarray(x, np.float64)
    y = x * weight / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return rotary(y, positions, w, interleaved=interleaved, gain=gain)


def norm_rotary_backward(x, dy, weight, positions, w, eps, interleaved=False, gain=1.0):
    """Gradients of norm_rotary: of x and of weight."""
    x = np.asarray(x, np.float64)
    u = rotary(np.asarray(dy, np.float64), positions, w, interleaved=interleaved, gain=gain, backward=True)
    rms = np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    dweight = (u * x / rms).sum((0, 1, 2))
    g = u * weight
    return g / rms - x * (g * x).mean(-1, keepdims=True) / rms ** 3, dweight


def _sees(n, window):
    t, j = np.arange(n)[:, None], np.arange(n)[None, :]
    return (j <= t) & (j > t - window) if window else j <= t


def prompt_attention(q, k, v, offsets, window=0, scale=None, dout=None):
    """Causal attention over packed sequences, q [N, H, dh], k, v [N, Hkv, dh]: o, lse, and with dout the
    gradients dq, dk, dv, too.  Rows of no sequence are NaN.  Also returns bounds of the terms that were
    summed: sum p |v| per output, and so on (see the tests' tolerances)."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    N, H, dh = q.shape
    g = H // k.shape[1]
    scale = dh ** -0.5 if scale is None else scale
    full = lambda x: np.full(x.shape, np.nan)  # noqa: E731
    r = dict(o=full(q), lse=np.full((N, H), np.nan), o_abs=full(q), s_abs=np.full((N, H), np.nan))
    if dout is not None:
        dout = np.asarray(dout, np.float64)
        for name, like in (("dq", q), ("dk", k), ("dv", v)):
            r[name], r[name + "_abs"] = full(like), full(like)
    for a, z in zip(offsets, offsets[1:]):
        n = z - a
        if n <= 0:
            continue
        see = _sees(n, window)
        if dout is not None:
            for name in ("dk", "dv", "dk_abs", "dv_abs"):
                r[name][a:z] = 0.0
        for h in range(H):
            m = h // g
            s = scale * q[a:z, h] @ k[a:z, m].T
            top = np.where(see, s, -np.inf).max(1)
            e = np.where(see, np.exp(s - top[:, None]), 0.0)
            p = e / e.sum(1, keepdims=True)
            o = p @ v[a:z, m]
            r["o"][a:z, h], r["lse"][a:z, h] = o, top + np.log(e.sum(1))
            r["o_abs"][a:z, h] = p @ np.abs(v[a:z, m])
            r["s_abs"][a:z, h] = (scale * np.where(see, np.abs(q[a:z, h]) @ np.abs(k[a:z, m]).T, 0.0)).max(1)
            if dout is None:
                continue
            do = dout[a:z, h]
            dp = do @ v[a:z, m].T
            ds = p * (dp - (do * o).sum(1, keepdims=True)) * scale
            # What a rounding of dS counts against: its own terms, not their difference.
            mag = p * (np.abs(do) @ np.abs(v[a:z, m]).T + (np.abs(do) @ np.abs(r["o_abs"][a:z, h]).T).diagonal()[:, None]) * scale
            r["dq"][a:z, h], r["dq_abs"][a:z, h] = ds @ k[a:z, m], mag @ np.abs(k[a:z, m])
            r["dk"][a:z, m] += ds.T @ q[a:z, h]
            r["dk_abs"][a:z, m] += mag.T @ np.abs(q[a:z, h])
            r["dv"][a:z, m] += p.T @ do
            r["dv_abs"][a:z, m] += p.T @ np.abs(do)
    return r


def quantise(x):
    """e4m3 numbers and exponents of x [..., dh]: the least e >= -120 by which the largest finite magnitude is
    448 2^e at most, and x 2^-e to the nearest e4m3 number (ties to even).  Infinities become NaN."""
    x = np.asarray(x, np.float64)
    finite = np.isfinite(x)
    m = np.where(finite, np.abs(x), 0.0).max(-1)
    e = np.full(m.shape, -120)
    while (m > 448.0 * 2.0 ** e).any():
        e = e + (m > 448.0 * 2.0 ** e)
    y = np.where(finite, x, 0.0) / 2.0 ** e[..., None]
    _, at = np.frexp(y)
    step = 2.0 ** (np.maximum(at - 1, -6) - 3)
    return np.where(finite, np.round(y / step) * step, np.nan), e
