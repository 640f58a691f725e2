"""GPU parity of the decoding operators (rotary positions, attention of drafted tokens over a
paged cache, the cache's page operations) against the float64 oracle, and their use together.

Tolerances count roundings.  u = 2^-24 is float32's half step, h the output type's
(bf16 2^-8, float32 2^-24).
"""
import ctypes

import numpy as np
import pytest
import torch

import oracle.decode_oracle as orc
from retrieval_sparse_attention_causal_gb300 import synth
from tests.gpu_helpers import dev, host

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
TORCH = {"bf16": torch.bfloat16, "f32": torch.float32}


def _g():
    import retrieval_sparse_attention_causal_gb300 as g
    return g


@pytest.fixture(autouse=True)
def _clean_error_word(request):
    yield
    if not getattr(request.function, "flags", False):
        _g().cache_workspace("cuda").check()


def flags(test):
    """A test that sets the error word and reads it itself."""
    test.flags = True
    return test


def ints(x):
    return torch.as_tensor(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def within(got, ref, lim, what):
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf]), f"{what}: infinities differ"
    assert not np.isnan(got).any(), f"{what}: NaN"
    over = np.abs(got[~inf] - ref[~inf]) - np.broadcast_to(lim, ref.shape)[~inf]
    assert over.size == 0 or over.max() <= 0, f"{what}: {int((over > 0).sum())} of {over.size} beyond the bound by {over.max():.3g}"


# ------------------------------------------------------------------ rotary positions
def rotary_bound(x, y, w, positions, gain, half, dtype, interleaved):
    """Angle: the float that sincospif takes is within 2^-25 of its value (half a step at 1),
    pi 2^-25 radians, and base^(-2i/rot) / 2 pi within 2^-51 of itself, |p| w 2^-51 radians.
    Sine and cosine within one step (2 u); the gain, two products and their sum round once
    each (fma or not): 4 u.  All relative to the pair's length."""
    i1 = np.arange(half) * 2 if interleaved else np.arange(half)
    i2 = i1 + 1 if interleaved else i1 + half
    r = gain * np.hypot(x[..., i1], x[..., i2])
    ang = np.abs(positions)[:, :, None, None] * w * 2.0 ** -51
    lim = HALF[dtype] * np.abs(y)
    for i in (i1, i2):
        lim[..., i] += (1 + HALF[dtype]) * r * np.sqrt(2) * (np.pi * U / 2 + 6 * U + ang)
    return lim + 1e-40


ROTARY = [  # B, L, H, Hkv, dh, rot, dtype, interleaved, scaling
    (1, 1, 1, 1, 2, 2, "f32", False, "none"),
    (2, 5, 3, 1, 64, 64, "bf16", False, "none"),
    (1, 33, 12, 12, 64, 32, "bf16", True, "parts"),
    (3, 17, 5, 1, 72, 40, "f32", False, "linear"),
    (2, 9, 4, 2, 40, 6, "bf16", True, "ntk"),
    (1, 7, 2, 2, 50, 34, "bf16", False, "none"),
    (2, 3, 6, 3, 256, 256, "f32", True, "parts"),
    (1, 700, 16, 4, 128, 96, "bf16", False, "ntk"),
    (4, 1, 12, 12, 64, 64, "bf16", True, "linear"),
]


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("B,L,H,Hkv,dh,rot,dtype,interleaved,scaling", ROTARY)
def test_rotary_against_oracle(B, L, H, Hkv, dh, rot, dtype, interleaved, scaling, backward):
    g = _g()
    kw = dict(base=10000.0, scaling=scaling, factor=4.0, context=2048.0)
    q, k = synth.normal(1, 0, (B, L, H, dh), 1.0, dtype), synth.normal(1, 1, (B, L, Hkv, dh), 1.0, dtype)
    pos = np.random.default_rng(3).integers(0, 1 << 24, (B, L))
    pos[0, 0] = (1 << 31) - 1
    w = orc.speeds(rot, **kw)
    turn = g.rotary_backward if backward else g.rotary
    qo, ko = turn(dev(q, dtype), dev(k, dtype), g.rotary_frequencies(rot, **kw), positions=ints(pos),
                  interleaved=interleaved, gain=1.25)
    for got, x, what in ((qo, q, "q"), (ko, k, "k")):
        ref = orc.rotary(x, pos, w, interleaved, 1.25, backward)
        lim = rotary_bound(x, ref, w, pos, 1.25, rot // 2, dtype, interleaved)
        lim[..., rot:] = 0  # copied
        within(host(got), ref, lim, what)


@pytest.mark.parametrize("dtype,offset", [("bf16", 0), ("bf16", 1), ("f32", 0), ("f32", 1)])
def test_rotary_views_and_in_place(dtype, offset):
    """Views of a fused projection (also at odd addresses), heads-first storage, a broadcast
    key head, default and shared positions, and the in-place form give what contiguous
    tensors give; what lies around the views stays as it was."""
    g = _g()
    B, L, H, Hkv, dh, rot = 2, 11, 4, 2, 64, 48
    n = (H + 2 * Hkv) * dh
    raw = torch.randn(B * L * n + 8, device="cuda").to(TORCH[dtype])
    qkv = raw[offset:offset + B * L * n].view(B, L, H + 2 * Hkv, dh)
    q, k = qkv[:, :, :H], qkv[:, :, H:H + Hkv]
    freq = g.rotary_frequencies(rot)
    want = g.rotary(q.contiguous(), k.contiguous(), freq, positions=torch.arange(L, dtype=torch.int32, device="cuda"))
    got = g.rotary(q, k, freq)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    qt = q.transpose(1, 2).contiguous().transpose(1, 2)
    assert torch.equal(g.rotary(qt, None, freq)[0], want[0])
    one = k[:, :, :1].expand(B, L, 3, dh)
    assert torch.equal(g.rotary(q, one, freq)[1], want[1][:, :, :1].expand(B, L, 3, dh))
    before = raw.clone()
    g.rotary(q, k, freq, q_out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    rest = qkv[:, :, H + Hkv:]
    assert torch.equal(rest, before[offset:offset + B * L * n].view(B, L, -1, dh)[:, :, H + Hkv:])
    assert torch.equal(raw[:offset], before[:offset]) and torch.equal(raw[offset + B * L * n:], before[offset + B * L * n:])


def test_rotary_gradient_against_differences():
    """<dy, rotary(x + e d) - rotary(x - e d)> / 2e = <rotary_backward(dy), d>.  rotary is
    linear in x, so the difference has no truncation error; both sides are sums of n float32
    products of values of order 1, each within 16 u of its terms' sizes (see rotary_bound),
    and the difference of two values of size ~3 is within 3 * 2 u / (2 e) of itself, e = 1/2."""
    g = _g()
    B, L, H, dh, rot = 2, 13, 3, 32, 24
    x, d, dy = (torch.from_numpy(synth.normal(5, s, (B, L, H, dh))).float().cuda() for s in (0, 1, 2))
    freq = g.rotary_frequencies(rot, scaling="linear", factor=3.0)
    pos = ints(np.random.default_rng(0).integers(0, 5000, (B, L)))
    f = lambda t: g.rotary(t, None, freq, positions=pos, gain=0.7)[0].double()  # noqa: E731
    left = (dy.double() * (f(x + 0.5 * d) - f(x - 0.5 * d))).sum()
    back = g.rotary_backward(dy, None, freq, positions=pos, gain=0.7)[0].double()
    right = (back * d.double()).sum()
    size = (dy.abs().double() * (x.abs() + d.abs()).double().amax()).sum()
    assert abs(left - right) <= 40 * U * size


# ------------------------------------------------------------------ trees
@pytest.mark.parametrize("T", [1, 2, 13, 64, 65, 200, 256])
def test_tree_plan_against_oracle(T):
    rng = np.random.default_rng(T)
    B = 6
    parents = np.full((B, T), -2)
    for b in range(B):
        for t in range(T):
            parents[b, t] = rng.integers(-1, t) if t else -1
        if b == 1:  # a chain: the deepest tree
            parents[b] = np.arange(T) - 1
        if b == 2:  # padding in the middle: what follows it is padding too
            parents[b, T // 3] = -2
        if b == 3:
            parents[b, T // 2:] = -2
        if b == 4:
            parents[b] = -2
    lengths = np.array([0, 5, 1000, 63, 64, 2 ** 30])
    mask, pos = _g().tree_plan(ints(parents), ints(lengths))
    want = [orc.tree(parents[b], lengths[b]) for b in range(B)]
    assert np.array_equal(pos.cpu().numpy(), np.stack([w[1] for w in want]))
    assert np.array_equal(mask.cpu().numpy(), orc.pack_mask(np.stack([w[0] for w in want])))


@flags
def test_tree_plan_flags_bad_parents():
    g = _g()
    mask, pos = g.tree_plan(ints([[-1, 0, 2, 1, -5, 3]]), ints([7]))  # tokens 2 and 4 are not trees
    assert pos.cpu().tolist() == [[7, 8, -1, 9, -1, 10]]
    assert mask.cpu().flatten().tolist() == [1, 3, 0, 11, 0, 43]
    with pytest.raises(g.GCAError) as e:
        g.cache_workspace("cuda").check()
    assert e.value.status == g.GCA_ERR_DEVICE_INDEX


# ------------------------------------------------------------------ attention
def random_cache(rng, lengths, Hkv, dh, dtype, spare=2, width_spare=1, seed=0):
    """Pages in random order; rows behind the lengths, and free pages, hold NaN."""
    held = [-(-n // 64) for n in lengths]
    pages = sum(held) + spare
    order = rng.permutation(pages)
    table = np.full((len(lengths), max(held + [0]) + width_spare), -1)
    k = synth.normal(seed, 20, (pages, 64, Hkv, dh), 1.0, dtype)
    v = synth.normal(seed, 21, (pages, 64, Hkv, dh), 1.0, dtype)
    used, at = np.zeros((pages, 64), dtype=bool), 0
    for b, n in enumerate(lengths):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
        for j in range(n):
            used[table[b, j // 64], j % 64] = True
    k[~used], v[~used] = np.nan, np.nan
    refs = np.zeros(pages, dtype=np.int32)
    refs[table[table >= 0]] = 1
    return k, v, table, refs


def random_draft(rng, B, T, lengths, kind):
    """(see, pos): 'chain' (None, None), 'padded chain' (None, pos), 'tree' with padding, 'wild': any
    mask, rows that see nothing."""
    if kind == "chain":
        return None, None
    if kind == "padded chain":
        return None, np.array([[lengths[b] + t if t < max(1, T - 2 * b) else -1 for t in range(T)] for b in range(B)])
    see, pos = np.zeros((B, T, T), dtype=bool), np.full((B, T), -1)
    for b in range(B):
        if kind == "tree":
            parents = [int(rng.integers(-1, t)) if t else -1 for t in range(T)]
            if b % 3 == 1:
                parents[max(1, T // 2):] = [-2] * (T - max(1, T // 2))
            see[b], pos[b] = orc.tree(parents, int(lengths[b]))
        else:
            see[b] = rng.random((T, T)) < 0.3
            see[b, T // 2] = False
            pos[b] = lengths[b] + rng.integers(-3, 9, T)
            pos[b, pos[b] < 0] = 0
            pos[b, T // 3::5] = -1
    return see, pos


def attend_and_check(rng, lengths, T, H, Hkv, dh, dtype, kind, window=0, scale=None, holes=False, views=False, seed=0, width_spare=1,
                     rise=0.0):
    g = _g()
    B = len(lengths)
    k, v, table, _ = random_cache(rng, lengths, Hkv, dh, dtype, seed=seed, width_spare=width_spare)
    if rise:  # keys that grow along the context, rounded to the type once more
        for b, n in enumerate(lengths):
            for j in range(n):
                k[table[b, j // 64], j % 64] *= 1 + rise * j / n
        k = host(dev(k, dtype))
    if holes:  # pages that are not held
        for b in range(B):
            table[b, rng.random(table.shape[1]) < 0.3] = -1
    q = synth.normal(seed, 22, (B, T, H, dh), 1.0, dtype)
    kn, vn = synth.normal(seed, 23, (B, T, Hkv, dh), 1.0, dtype), synth.normal(seed, 24, (B, T, Hkv, dh), 1.0, dtype)
    see, pos = random_draft(rng, B, T, lengths, kind)
    rsee = np.tril(np.ones((B, T, T), dtype=bool)) if see is None else see
    rpos = np.array(lengths)[:, None] + np.arange(T) if pos is None else pos
    if kind in ("tree", "padded chain"):  # padding holds anything
        kn[rpos < 0], vn[rpos < 0], q[rpos < 0] = np.nan, np.inf, np.nan
    if views:
        fused = torch.full((B, T, H + 2 * Hkv + 1, dh), float("nan"), dtype=TORCH[dtype], device="cuda")
        qd, kd, vd = fused[:, :, :H], fused[:, :, H:H + Hkv], fused[:, :, H + Hkv:H + 2 * Hkv]
        qd.copy_(dev(q, dtype)), kd.copy_(dev(kn, dtype)), vd.copy_(dev(vn, dtype))
    else:
        qd, kd, vd = dev(q, dtype), dev(kn, dtype), dev(vn, dtype)
    o, lse = g.tree_attention(qd, kd, vd, dev(k, dtype), dev(v, dtype), ints(table), ints(lengths),
                              mask=None if see is None else torch.from_numpy(orc.pack_mask(see)).cuda(),
                              positions=None if pos is None else ints(pos), window=window, scale=scale)
    ro, rl, mean_abs, dot_abs, keys = orc.tree_attention(q, kn, vn, k, v, table, lengths, rsee, rpos, window, scale)
    # Logits: dh products and sums of float32 (a tensor core may cut where it could round: 2 u
    # each), the scale and log2 e: ds.  A weight: ds, exp2's two steps (4 u) and the rounding of
    # its argument (|s| log2 e u, |s| <= dot_abs), bf16's half step where it is rounded; sums over n keys and the rescaling
    # of each block of 32: n u + n / 32 * 6 u.
    ds = (2 * dh + 4) * U * dot_abs
    dw = 2 * ds + 4 * U * dot_abs + 8 * U + 1.2 * keys * U
    within(host(lse), rl, ds + dw + np.where(np.isfinite(rl), 4 * U * (1 + np.abs(rl)), 0), "lse")
    weight = HALF["bf16"] if dtype == "bf16" else 0.0
    lim = ((np.expm1(2 * dw) if rise else 2 * dw) + weight)[..., None] * mean_abs * (1 + 2 * HALF[dtype]) + 2 * HALF[dtype] * np.abs(ro) + 1e-38
    within(host(o), ro, lim, "o")
    return o, lse


ATTENTION = [  # lengths, T, H, Hkv, dh, dtype, kind, window
    ([0], 1, 1, 1, 64, "bf16", "chain", 0),
    ([1], 1, 4, 4, 32, "bf16", "chain", 0),
    ([64, 0, 63, 65], 1, 12, 12, 64, "bf16", "chain", 0),
    ([700, 3, 129], 1, 16, 4, 128, "bf16", "chain", 0),
    ([1000, 17, 0], 1, 8, 1, 64, "bf16", "chain", 100),
    ([130, 64], 2, 6, 2, 64, "bf16", "chain", 1),
    ([200, 0, 64], 5, 4, 4, 64, "bf16", "tree", 0),
    ([333, 64, 1, 0], 16, 12, 12, 64, "bf16", "tree", 64),
    ([333, 90], 13, 6, 2, 32, "bf16", "tree", 7),
    ([500, 20], 64, 4, 1, 64, "bf16", "tree", 0),
    ([260, 64, 0], 48, 3, 3, 64, "bf16", "tree", 128),
    ([150, 70], 65, 4, 2, 128, "bf16", "tree", 0),
    ([129, 0], 200, 2, 1, 64, "bf16", "tree", 90),
    ([90], 256, 2, 2, 64, "bf16", "chain", 0),
    ([200, 65], 100, 6, 2, 32, "bf16", "wild", 0),
    ([200, 65], 33, 8, 1, 64, "bf16", "wild", 5),
    ([100, 65], 9, 8, 2, 128, "bf16", "wild", 40),
    ([90, 0], 100, 32, 1, 64, "bf16", "tree", 0),
    ([70, 3], 130, 24, 1, 128, "bf16", "tree", 50),
    ([300, 65, 7], 12, 4, 4, 64, "bf16", "padded chain", 0),
    ([300, 65, 7], 70, 6, 3, 64, "bf16", "padded chain", 20),
    ([80, 65, 7], 9, 4, 2, 32, "f32", "padded chain", 3),
    ([64, 30], 40, 40, 2, 32, "f32", "tree", 0),
    ([0, 1, 200], 1, 4, 4, 32, "f32", "chain", 0),
    ([200, 31], 13, 6, 2, 32, "f32", "tree", 0),
    ([130, 64], 70, 4, 1, 64, "f32", "tree", 33),
    ([70, 10], 11, 2, 1, 128, "f32", "wild", 0),
]


@pytest.mark.parametrize("lengths,T,H,Hkv,dh,dtype,kind,window", ATTENTION)
def test_tree_attention_against_oracle(lengths, T, H, Hkv, dh, dtype, kind, window):
    attend_and_check(np.random.default_rng(T * 7 + dh), lengths, T, H, Hkv, dh, dtype, kind, window)


@pytest.mark.parametrize("dtype,T,H,dh", [("bf16", 1, 8, 64), ("bf16", 20, 12, 64), ("bf16", 64, 8, 128), ("f32", 3, 4, 32)])
def test_tree_attention_strides_holes_and_scale(dtype, T, H, dh):
    """Views of a fused projection, pages that are not held, a scale of one's own."""
    attend_and_check(np.random.default_rng(9), [400, 70], T, H, 4, dh, dtype, "tree", scale=0.3, holes=True, views=True)


@pytest.mark.parametrize("T,H,Hkv,dh,dtype", [(1, 4, 4, 64, "bf16"), (1, 8, 1, 128, "bf16"), (32, 2, 2, 64, "bf16"),
                                              (64, 4, 1, 64, "bf16"), (40, 2, 1, 32, "bf16"), (2, 2, 2, 64, "f32")])
def test_tree_attention_long_ragged(T, H, Hkv, dh, dtype):
    """Work split over many CTAs, a long sequence between short ones."""
    attend_and_check(np.random.default_rng(4), [0, 20000, 5, 64, 1], T, H, Hkv, dh, dtype, "tree", seed=3)


TENSOR = [  # lengths, T, H, Hkv, dh, kind, window, rise: of the tensor-core kernel
    ([0], 1, 1, 1, 64, "chain", 0, 0),
    ([64, 0, 63, 65], 1, 12, 12, 64, "chain", 0, 0),
    ([700, 3, 129], 1, 16, 4, 128, "chain", 0, 0),
    ([333, 64, 1, 0], 16, 12, 12, 64, "tree", 0, 0),
    ([500, 20], 64, 4, 1, 64, "tree", 0, 0),
    ([150, 70], 65, 4, 2, 128, "tree", 0, 0),
    ([129, 0], 200, 2, 1, 64, "tree", 0, 0),
    ([200, 65], 33, 8, 1, 64, "wild", 0, 0),
    ([100, 65], 9, 8, 2, 128, "wild", 0, 0),
    ([300, 65, 7], 70, 6, 3, 64, "padded chain", 0, 0),
    ([260, 64, 0, 1, 130, 99] * 2, 48, 12, 12, 64, "tree", 100, 0),
    ([200, 65, 130, 64, 1, 0] * 2, 33, 24, 6, 64, "wild", 40, 0),
    ([100, 65, 300] * 2, 20, 16, 4, 128, "padded chain", 70, 0),
    ([2000, 700], 3, 4, 1, 64, "chain", 0, 12.0),
    ([1500, 64], 64, 4, 2, 64, "tree", 0, 8.0),
    ([900], 40, 4, 1, 128, "wild", 0, 10.0),
]


@pytest.mark.parametrize("lengths,T,H,Hkv,dh,kind,window,rise", TENSOR)
def test_tree_attention_on_the_tensor_cores(lengths, T, H, Hkv, dh, kind, window, rise):
    """Odd sizes, masks and windows where a wide table (or many heads) makes it the kernel that is taken;
    logits that outgrow the reference of a row's weights again and again."""
    g = _g()
    g.profile_begin()
    attend_and_check(np.random.default_rng(T * 5 + dh), lengths, T, H, Hkv, dh, "bf16", kind, window, width_spare=1 if window else 1000,
                     rise=rise)
    assert "tree_tc" in g.profile_end()


ROWS = [  # lengths, T, H, Hkv, dh, kind, window, pages of the table behind the longest: of the kernel of 16 rows
    ([64, 0, 63, 65], 1, 12, 12, 64, "chain", 0, 24),
    ([700, 3, 129], 1, 16, 4, 128, "chain", 0, 15),
    ([130, 64], 2, 6, 2, 64, "chain", 0, 24),
    ([200, 0, 64], 5, 4, 4, 64, "tree", 0, 24),
    ([333, 64, 1, 0], 16, 12, 12, 64, "tree", 0, 24),
    ([500, 20], 64, 4, 1, 64, "tree", 0, 14),
    ([150, 70], 65, 4, 2, 128, "tree", 0, 7),
    ([200, 65], 33, 8, 1, 64, "wild", 0, 18),
    ([100, 65], 9, 8, 2, 128, "wild", 0, 24),
    ([300, 65, 7], 12, 4, 4, 64, "padded chain", 0, 24),
    ([260, 64, 0, 1, 130, 99] * 6, 5, 12, 12, 64, "tree", 70, 1),
    ([260, 64, 0, 1, 130, 99] * 7, 3, 48, 12, 128, "wild", 40, 1),
    ([260, 64, 0, 1, 130, 99] * 7, 16, 16, 16, 64, "padded chain", 9, 1),
]


@pytest.mark.parametrize("lengths,T,H,Hkv,dh,kind,window,spare", ROWS)
def test_tree_attention_of_sixteen_rows(lengths, T, H, Hkv, dh, kind, window, spare):
    """The same where there is little to read, but too much for whole tiles of the other kernel."""
    g = _g()
    g.profile_begin()
    attend_and_check(np.random.default_rng(T * 3 + dh), lengths, T, H, Hkv, dh, "bf16", kind, window, width_spare=spare)
    assert "tree_rows" in g.profile_end()


WHOLE = [  # lengths, T, H, Hkv, dh, dtype, kind, window: a tile a CTA, nothing to join
    ([0], 1, 1, 1, 64, "bf16", "chain", 0),
    ([64, 0, 63, 65], 1, 12, 12, 64, "bf16", "chain", 0),
    ([500, 20, 800], 64, 16, 4, 64, "bf16", "tree", 0),
    ([700, 3, 129] * 5, 48, 12, 12, 64, "bf16", "tree", 512),
    ([700, 3, 129] * 2, 150, 8, 4, 128, "bf16", "wild", 300),
    ([100, 0, 65] * 84, 2, 4, 4, 32, "bf16", "tree", 0),
    ([100, 0, 300] * 32, 1, 12, 12, 64, "bf16", "chain", 0),
]


@pytest.mark.parametrize("lengths,T,H,Hkv,dh,dtype,kind,window", WHOLE)
def test_tree_attention_of_whole_tiles(lengths, T, H, Hkv, dh, dtype, kind, window):
    g = _g()
    g.profile_begin()
    attend_and_check(np.random.default_rng(T * 2 + dh), lengths, T, H, Hkv, dh, dtype, kind, window)
    names = g.profile_end()
    assert "tree_join" not in names and ("tree_rows" in names or "tree_tc" in names)


def test_tree_attention_many_sequences():
    attend_and_check(np.random.default_rng(8), [int(x) for x in np.random.default_rng(1).integers(0, 90, 300)], 1, 2, 1, 32,
                     "bf16", "chain")


def test_tree_attention_large_logits():
    """Logits up to about 500: the running maximum carries the softmax."""
    g = _g()
    rng = np.random.default_rng(0)
    for T, H in ((1, 2), (64, 2)):
        k, v, table, _ = random_cache(rng, [300], 1, 64, "bf16")
        k *= 16
        q = synth.normal(0, 22, (1, T, H, 64), 4.0, "bf16")
        kn, vn = synth.normal(0, 23, (1, T, 1, 64), 16.0, "bf16"), synth.normal(0, 24, (1, T, 1, 64), 1.0, "bf16")
        o, lse = g.tree_attention(*(dev(x, "bf16") for x in (q, kn, vn, k, v)), ints(table), ints([300]))
        ro, rl, mean_abs, dot_abs, keys = orc.tree_attention(q, kn, vn, k, v, table, [300], np.tril(np.ones((1, T, T), bool)),
                                                             300 + np.arange(T)[None])
        ds = (2 * 64 + 4) * U * dot_abs
        dw = 2 * ds + 4 * U * dot_abs + 8 * U + 1.2 * keys * U
        within(host(lse), rl, ds + dw + 4 * U * np.abs(rl), "lse")
        # exp(dw) - 1 where dw is not small
        within(host(o), ro, (np.expm1(2 * dw) + HALF["bf16"])[..., None] * mean_abs * 1.01 + 2 * HALF["bf16"] * np.abs(ro), "o")


@flags
def test_tree_attention_flags_bad_pages_and_lengths():
    """A page number outside the pool is left out like a page that is not held, and flagged;
    so is a length that the table has no room for, which is read as the table's width."""
    g = _g()
    rng = np.random.default_rng(2)
    k, v, table, _ = random_cache(rng, [200, 100], 2, 64, "bf16")
    q, kn, vn = (dev(synth.normal(0, s, (2, 1, n, 64), 1.0, "bf16"), "bf16") for s, n in ((22, 4), (23, 2), (24, 2)))
    kd, vd = dev(k, "bf16"), dev(v, "bf16")
    bad, gone = table.copy(), table.copy()
    bad[0, 1], gone[0, 1] = k.shape[0], -1
    a = g.tree_attention(q, kn, vn, kd, vd, ints(bad), ints([200, 100]))
    with pytest.raises(g.GCAError) as e:
        g.cache_workspace("cuda").check()
    assert e.value.status == g.GCA_ERR_DEVICE_INDEX
    b = g.tree_attention(q, kn, vn, kd, vd, ints(gone), ints([200, 100]))
    g.cache_workspace("cuda").check()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    g.tree_attention(q, kn, vn, kd, vd, ints(gone), ints([1 << 20, -4]))
    with pytest.raises(g.GCAError):
        g.cache_workspace("cuda").check()


def test_tree_attention_is_deterministic_and_keeps_to_its_stream():
    """Equal calls give equal bits, on other streams than the current one too, two at a time."""
    g = _g()
    rng = np.random.default_rng(5)
    k, v, table, _ = random_cache(rng, [3000, 40, 777], 4, 64, "bf16")
    args = [dev(x, "bf16") for x in (synth.normal(0, 22, (3, 20, 8, 64), 1.0, "bf16"), synth.normal(0, 23, (3, 20, 4, 64), 1.0, "bf16"),
                                     synth.normal(0, 24, (3, 20, 4, 64), 1.0, "bf16"), k, v)] + [ints(table), ints([3000, 40, 777])]
    first = g.tree_attention(*args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(g.tree_attention(*args))
    torch.cuda.synchronize()
    for o, lse in outs:
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("T,H,Hkv,dh,top", [(1, 16, 4, 128, 32768), (8, 16, 4, 128, 20000), (40, 8, 4, 128, 9000), (24, 12, 12, 64, 9000),
                                            (64, 16, 4, 64, 9000), (1, 12, 12, 64, 40000)])
def test_tree_attention_repeats_bit_for_bit(T, H, Hkv, dh, top):
    """Many ends of sequences among long ones, thirty times: the handing over of blanked, masked
    and streamed pages must not depend on timing."""
    g = _g()
    rng = np.random.default_rng(dh + T)
    lengths = [int(x) for x in rng.integers(1, top, 16)]
    held = [-(-n // 64) for n in lengths]
    table = np.full((16, max(held) + 1), -1)
    order = rng.permutation(sum(held))
    for b, n in enumerate(held):
        table[b, :n] = order[sum(held[:b]):sum(held[:b + 1])]
    kp, vp = (synth.device_normal(0, s, (sum(held), 64, Hkv, dh), 1.0, torch.bfloat16) for s in (20, 21))
    q, kn, vn = (synth.device_normal(0, s, (16, T, n, dh), 1.0, torch.bfloat16) for s, n in ((22, H), (23, Hkv), (24, Hkv)))
    outs = [g.tree_attention(q, kn, vn, kp, vp, ints(table), ints(lengths)) for _ in range(30)]
    for o, lse in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])


def test_captured_steps_follow_the_cache():
    """Two captured steps (plan, attention, append) on two caches, replayed in turn and at once
    on two streams: each follows its own lengths and tables, and equals eager calls."""
    g = _g()
    rng = np.random.default_rng(6)
    T, B, H, Hkv, dh = 6, 2, 4, 2, 64
    graphs = []
    for i in range(2):
        k, v, table, refs = random_cache(rng, [100 + 50 * i, 0], Hkv, dh, "bf16", spare=20, width_spare=8, seed=i)
        mk = lambda: g.PagedCache(dev(k, "bf16"), dev(v, "bf16"), ints(table), ints([100 + 50 * i, 0]), ints(refs))  # noqa: E731,B023
        cache, twin = mk(), mk()
        q, kn, vn = (dev(synth.normal(i, s, (B, T, n, dh), 1.0, "bf16"), "bf16") for s, n in ((22, H), (23, Hkv), (24, Hkv)))
        parents, counts, path = ints([[-1, 0, 0, 1, 2, 3]] * B), ints([3, 2]), ints([[0, 1, 3, 0, 0, 0]] * B)

        def step(c, q=q, kn=kn, vn=vn, parents=parents, counts=counts, path=path):
            mask, pos = g.tree_plan(parents, c.lengths)
            out = c.attention(q, kn, vn, mask, pos, window=300)
            c.append(kn, vn, counts, path=path)
            return out

        graph = torch.cuda.CUDAGraph()
        side = torch.cuda.Stream()
        state = [t.clone() for t in (cache.table, cache.lengths, cache.refs, cache.k_pages, cache.v_pages)]
        with torch.cuda.stream(side):
            step(cache)  # sets the kernels' attributes
        torch.cuda.synchronize()
        for t, s in zip((cache.table, cache.lengths, cache.refs, cache.k_pages, cache.v_pages), state):
            t.copy_(s)
        with torch.cuda.graph(graph):
            out = step(cache)
        graphs.append((graph, out, cache, twin, step, torch.cuda.Stream()))
    for _ in range(6):
        torch.cuda.synchronize()
        for graph, _, _, _, _, s in graphs:
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        for _, out, cache, twin, step, _ in graphs:
            want = step(twin)
            torch.cuda.synchronize()
            assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
            assert torch.equal(cache.lengths, twin.lengths) and torch.equal(cache.table, twin.table)
            live = cache.refs > 0
            assert torch.equal(cache.refs, twin.refs)
            assert torch.equal(cache.k_pages[live].nan_to_num(7.0), twin.k_pages[live].nan_to_num(7.0))


def test_offsets_beyond_32_bits():
    """Pages that lie behind element 2^31 of the pool are read, appended to and compacted."""
    g = _g()
    Hkv, dh = 12, 128
    pages = 2 ** 31 // (64 * Hkv * dh) + 40
    kp = torch.empty((pages, 64, Hkv, dh), dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    table = np.full((1, 4), -1)
    table[0, :3] = pages - 1 - np.arange(3) * 7
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[:4] = 1
    k, v = synth.normal(0, 20, (3, 64, Hkv, dh), 1.0, "bf16"), synth.normal(0, 21, (3, 64, Hkv, dh), 1.0, "bf16")
    at = torch.from_numpy(table[0, :3]).cuda()
    kp[at], vp[at], refs[at] = dev(k, "bf16"), dev(v, "bf16"), 1
    refs[4:pages - 40] = 1  # so that the next free page lies far behind too
    cache = g.PagedCache(kp, vp, ints(table), ints([190]), refs)
    q, kn, vn = (synth.normal(0, s, (1, 4, n, dh), 1.0, "bf16") for s, n in ((22, 24), (23, Hkv), (24, Hkv)))
    small = orc.Pages(k, v, np.array([[0, 1, 2, -1]]), np.array([190]), np.ones(3))
    ro, _, mean_abs, _, _ = orc.tree_attention(q, kn, vn, small.k, small.v, small.table, [190], np.tril(np.ones((1, 4, 4), bool)),
                                               190 + np.arange(4)[None])
    o, _ = cache.attention(*(dev(x, "bf16") for x in (q, kn, vn)))
    within(host(o), ro, 2 ** -7 * (mean_abs + np.abs(ro)), "o")
    cache.append(dev(kn, "bf16"), dev(vn, "bf16"), ints([4]))
    row = cache.table[0].tolist()
    assert row[3] == pages - 40 and cache.lengths.tolist() == [194]
    assert np.array_equal(host(kp[row[3], :2]), kn[0, 2:]) and np.array_equal(host(kp[row[2], 62:]), kn[0, :2])
    refs[4:pages - 40] = 0
    assert int(cache.compact()) == 8
    assert cache.table.tolist() == [[7, 6, 5, 4]]
    assert np.array_equal(host(vp[7]), v[0]) and np.array_equal(host(kp[6]), k[1])


# ------------------------------------------------------------------ pages
def cache_pair(rng, lengths, width, pages, Hkv=2, dh=32, dtype="bf16", share=()):
    """A cache on the GPU and its model: slot s of `share` (s, t) shares the pages of slot t."""
    table, refs = np.full((len(lengths), width), -1), np.zeros(pages, dtype=np.int64)
    order = list(rng.permutation(pages))
    for s, n in enumerate(lengths):
        if s in dict(share):
            table[s] = table[dict(share)[s]]
            table[s, -(-n // 64):] = -1
        else:
            for p in range(-(-n // 64)):
                table[s, p] = order.pop()
        for p in table[s][table[s] >= 0]:
            refs[p] += 1
    k, v = (synth.normal(0, s, (pages, 64, Hkv, dh), 1.0, dtype) for s in (20, 21))
    g = _g()
    return (g.PagedCache(dev(k, dtype), dev(v, dtype), ints(table), ints(lengths), ints(refs)),
            orc.Pages(k, v, table, np.array(lengths), refs))


def same_state(cache, model):
    torch.cuda.synchronize()
    assert np.array_equal(cache.lengths.cpu().numpy(), model.lengths), "lengths"
    assert np.array_equal(cache.table.cpu().numpy(), model.table), "table"
    assert np.array_equal(cache.refs.cpu().numpy(), model.refs), "refs"
    assert np.array_equal(host(cache.k_pages), model.k), "k"
    assert np.array_equal(host(cache.v_pages), model.v), "v"


def new_rows(seed, n, T, Hkv=2, dh=32, dtype="bf16"):
    return tuple(synth.normal(seed, s, (n, T, Hkv, dh), 1.0, dtype) for s in (23, 24))


@pytest.mark.parametrize("T,counts", [(1, [1, 1, 1, 1]), (7, [0, 7, 3, 1]), (64, [64, 1, 63, 64]), (300, [300, 0, 129, 64])])
@pytest.mark.parametrize("path", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append(T, counts, path, dtype):
    rng = np.random.default_rng(T)
    cache, model = cache_pair(rng, [0, 64, 63, 130], 8, 40, dtype=dtype)
    kn, vn = new_rows(1, 4, T, dtype=dtype)
    p = np.array([np.sort(rng.permutation(T)) if T < 9 else rng.integers(0, T, T) for _ in range(4)]) if path else None
    cache.append(dev(kn, dtype), dev(vn, dtype), ints(counts), path=None if p is None else ints(p))
    model.append(kn, vn, counts, p)
    same_state(cache, model)


def test_append_slots_and_views():
    """Named slots out of order, rows out of a fused projection."""
    cache, model = cache_pair(np.random.default_rng(0), [10, 0, 70, 5, 64], 4, 20)
    kn, vn = new_rows(2, 3, 9)
    fused = torch.zeros((3, 9, 6, 32), dtype=torch.bfloat16, device="cuda")
    fused[:, :, 1:3], fused[:, :, 4:] = dev(kn, "bf16"), dev(vn, "bf16")
    cache.append(fused[:, :, 1:3], fused[:, :, 4:], ints([9, 2, 5]), slots=ints([4, 0, 2]))
    model.append(kn, vn, [9, 2, 5], slots=[4, 0, 2])
    same_state(cache, model)


def test_append_copies_a_shared_last_page():
    """Holders of one last page, some cut back to fewer of its rows, append in one call: each
    gets a page of its own with its rows; the one that does not append keeps the page."""
    for all_append in (False, True):
        cache, model = cache_pair(np.random.default_rng(1), [100, 100, 80, 100, 64], 4, 30, share=[(1, 0), (2, 0), (3, 0)])
        kn, vn = new_rows(3, 5, 40)
        counts = [3, 40, 1, 2 if all_append else 0, 1]
        cache.append(dev(kn, "bf16"), dev(vn, "bf16"), ints(counts))
        model.append(kn, vn, counts)
        same_state(cache, model)


@flags
@pytest.mark.parametrize("pages", [10, 11, 12, 13, 14, 20])
def test_append_without_room(pages):
    """Entries are served in order until the free pages run out; one that the table has no room
    for is left out.  The last of them needs no page, and is not served either."""
    g = _g()
    cache, model = cache_pair(np.random.default_rng(2), [64, 10, 200, 130, 1], 4, pages)
    kn, vn = new_rows(4, 5, 70)
    counts = [65, 60, 70, 70, 63]
    cache.append(dev(kn, "bf16"), dev(vn, "bf16"), ints(counts))
    model.append(kn, vn, counts)
    same_state(cache, model)
    assert model.full  # 200 + 70 tokens do not fit in four pages
    with pytest.raises(g.GCAError) as e:
        cache.check()
    assert e.value.status == g.GCA_ERR_CACHE_FULL


@flags
def test_append_flags_bad_entries():
    g = _g()
    cache, model = cache_pair(np.random.default_rng(3), [10, 20, 30, 64], 4, 20)
    cache.table[2, 0], model.table[2, 0] = -1, -1  # a last page that is not held
    kn, vn = new_rows(5, 6, 4)
    slots, counts = [0, 1, 2, 0, 9, 3], [2, 5, 3, 1, 1, 4]  # too many; no page; named twice; no slot
    path = [[0, 1, 2, 3], [0] * 4, [0] * 4, [0] * 4, [0] * 4, [3, 4, -1, 0]]
    cache.append(dev(kn, "bf16"), dev(vn, "bf16"), ints(counts), path=ints(path), slots=ints(slots))
    model.append(kn, vn, counts, np.array(path), slots)
    assert model.flagged
    same_state(cache, model)
    with pytest.raises(g.GCAError) as e:
        cache.check()
    assert e.value.status == g.GCA_ERR_DEVICE_INDEX


def test_fork_trim_free():
    cache, model = cache_pair(np.random.default_rng(4), [100, 0, 0, 300, 0, 64], 6, 30)
    cache.fork(ints([0, 3, 0]), ints([1, 4, 2]))
    model.fork([0, 3, 0], [1, 4, 2])
    same_state(cache, model)
    for kw in (dict(end=[90, 64, 0, 299, 500, -3]), dict(begin=[64, 63, 5, 200, 1000, 0]),
               dict(begin=[0, 65], end=[70, 256], slots=[0, 4]), dict(end=[10], slots=[3])):
        cache.trim(**{n: ints(x) for n, x in kw.items()})
        model.trim(**kw)
        same_state(cache, model)
    cache.free(ints([4, 1]))
    model.trim(slots=[4, 1], release=True)
    same_state(cache, model)
    cache.free()
    model.trim(release=True)
    same_state(cache, model)
    assert not model.refs.any()


@flags
def test_fork_and_trim_flag_bad_entries():
    g = _g()
    cache, model = cache_pair(np.random.default_rng(5), [100, 0, 0, 70, 0], 4, 30)
    src, dst = [0, 3, 1, 0, 7, 0, 3], [1, 1, 2, 3, 4, 4, 9]
    cache.fork(ints(src), ints(dst))
    model.fork(src, dst)
    assert model.flagged
    same_state(cache, model)
    with pytest.raises(g.GCAError):
        cache.check()
    cache.trim(end=ints([5, 6, 7, 8]), slots=ints([0, 0, -1, 3]))
    model.trim(end=[5, 6, 7, 8], slots=[0, 0, -1, 3])
    same_state(cache, model)
    with pytest.raises(g.GCAError):
        cache.check()


@pytest.mark.parametrize("pages,seed", [(1, 0), (9, 1), (200, 2), (1000, 3), (8191, 4), (8192, 5), (8193, 6), (11000, 7)])
def test_compact(pages, seed):
    rng = np.random.default_rng(seed)
    lengths = []
    while sum(-(-n // 64) for n in lengths) < pages * 2 // 3:
        lengths.append(int(min(rng.integers(1, 400), 64 * (pages - sum(-(-n // 64) for n in lengths)))))
    cache, model = cache_pair(rng, lengths + [0], 7, pages, Hkv=1, dh=32)
    if lengths:
        cache.fork(ints([0]), ints([len(lengths)]))
        model.fork([0], [len(lengths)])
    gone = [s for s in range(1, len(lengths)) if rng.random() < 0.4][:1024]
    if gone:
        cache.free(ints(gone))
        model.trim(slots=gone, release=True)
    live = cache.compact()
    assert int(live) == model.compact()
    same_state(cache, model)


@pytest.mark.parametrize("pages", [64, 8192, 8256])
def test_compact_of_a_full_and_of_an_empty_pool(pages):
    cache, model = cache_pair(np.random.default_rng(0), [4096] * (pages // 64), 64, pages, Hkv=1, dh=32)
    assert int(cache.compact()) == model.compact() == pages
    same_state(cache, model)
    cache.free()
    model.trim(slots=list(range(pages // 64)), release=True)
    assert int(cache.compact()) == model.compact() == 0
    same_state(cache, model)


def test_random_operations():
    """A long run of mixed operations keeps equal to the model, and the tokens to what was appended."""
    rng = np.random.default_rng(11)
    cache, model = cache_pair(rng, [0] * 6, 5, 40)
    for step in range(60):
        kind = rng.choice(["append", "append", "append", "fork", "trim", "free", "compact"])
        if kind == "append":
            T = int(rng.integers(1, 100))
            kn, vn = new_rows(100 + step, 6, T)
            counts = [int(min(rng.integers(0, T + 1), 320 - model.lengths[s])) for s in range(6)]
            need = sum(counts) // 64 + 12
            if (model.refs == 0).sum() < need:
                kind = "free"
            else:
                cache.append(dev(kn, "bf16"), dev(vn, "bf16"), ints(counts))
                model.append(kn, vn, counts)
        if kind == "fork":
            empty = [s for s in range(6) if model.lengths[s] == 0]
            full = [s for s in range(6) if model.lengths[s] > 0]
            if empty and full:
                cache.fork(ints([full[0]]), ints([empty[0]]))
                model.fork([full[0]], [empty[0]])
        if kind == "trim":
            end = [int(rng.integers(0, n + 1)) if rng.random() < 0.5 else int(n) for n in model.lengths]
            cache.trim(end=ints(end))
            model.trim(end=end)
        if kind == "free":
            s = int(np.argmax(model.lengths))
            cache.free(ints([s]))
            model.trim(slots=[s], release=True)
        if kind == "compact":
            cache.compact()
            model.compact()
        same_state(cache, model)


# ------------------------------------------------------------------ together
def test_lookup_feeds_gca():
    """Retrieved chunks are read where they lie: gca_forward on the pool equals gca_forward on
    the contiguous store."""
    g = _g()
    rng = np.random.default_rng(0)
    B, nC, H, dh, topk = 2, 9, 4, 64, 4
    k, v = (synth.normal(0, s, (B, nC * 64, H, dh), 1.0, "bf16") for s in (20, 21))
    cache = g.PagedCache.empty(32, B, nC + 1, H, dh)
    cache.append(dev(k, "bf16"), dev(v, "bf16"), ints([nC * 64] * B))
    idx = np.stack([rng.permutation(nC)[:topk] for _ in range(B)])[:, None].astype(np.int32)
    idx[1, 0, 2] = -1
    sc = torch.randn((B, 1, topk), device="cuda")
    q = torch.randn((B, 64, H, dh), device="cuda").bfloat16()
    want, _ = g.gca_forward(q, dev(k, "bf16"), dev(v, "bf16"), ints(idx), sc, shift=0)
    got, _ = g.gca_forward(q, *cache.store(), cache.lookup(ints(idx)), sc, shift=0, kv_shared=True)
    assert torch.equal(got, want)


def test_decode_paged_equals_decode():
    g = _g()
    from retrieval_sparse_attention_causal_gb300 import pipeline
    B, nC, H, dh, D = 3, 12, 4, 64, 256
    k, v = (synth.normal(1, s, (B, nC * 64, H, dh), 1.0, "bf16") for s in (20, 21))
    lm = synth.landmark_inputs(1, B, 1, nC, D, "bf16")
    q = torch.randn((B, 64, H, dh), device="cuda").bfloat16()
    cache = g.PagedCache.empty(B * nC + 5, B, nC, H, dh)
    cache.append(dev(k, "bf16"), dev(v, "bf16"), ints([nC * 64] * B))
    want = pipeline.decode(q, dev(k, "bf16"), dev(v, "bf16"), dev(lm["q_lmk"], "bf16"), dev(lm["k_lmk"], "bf16"), topk=4)
    got = pipeline.decode_paged(q, cache, dev(lm["q_lmk"], "bf16"), dev(lm["k_lmk"], "bf16"), topk=4)
    for n in ("idx", "scores", "o", "lse"):
        assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("dtype,H,dh,L,W", [("f32", 2, 32, 192, 64), ("bf16", 3, 64, 320, 128)])
def test_window_step_against_oracle(dtype, H, dh, L, W):
    """Rotary, window attention, its gradients and rotary's, as one training step.  Tolerances of
    the window tests (tests/gpu_helpers.py), with the rounding of the turned queries and keys:
    one more half step of values up to 5 in a sum of dh terms of size 1/sqrt(dh), so twice them."""
    import oracle.gca_oracle as gorc
    from retrieval_sparse_attention_causal_gb300 import pipeline
    from tests.gpu_helpers import TOL, assert_close
    B, rot = 2, dh // 2
    q, k, v, do = (synth.normal(2, s, (B, L, H, dh), 1.0, dtype) for s in (synth.S_Q, synth.S_K, synth.S_V, synth.S_DO))
    pos = np.arange(L)[None].repeat(B, 0) + np.array([[0], [70000]])
    w = orc.speeds(rot)
    r = pipeline.window_step(*(dev(x, dtype) for x in (q, k, v, do)), _g().rotary_frequencies(rot), window=W, positions=ints(pos))
    qr, kr = orc.rotary(q, pos, w), orc.rotary(k, pos, w)
    o, lse = gorc.swa_forward(qr, kr, v, W)
    dq, dk, dv = gorc.swa_backward(qr, kr, v, do, W)
    dq, dk = orc.rotary(dq, pos, w, backward=True), orc.rotary(dk, pos, w, backward=True)
    for got, ref, n in ((r["o"], o, "o"), (r["dq"], dq, "dq"), (r["dk"], dk, "dk"), (r["dv"], dv, "dv")):
        assert_close(host(got), ref, 2 * TOL[dtype], n)


@pytest.mark.parametrize("dtype,T,H,Hkv,dh,window", [("bf16", 6, 4, 2, 64, 0), ("bf16", 40, 4, 4, 64, 96), ("f32", 5, 2, 1, 32, 70),
                                                     ("bf16", 1, 8, 2, 64, 128)])
def test_drafts_accepted_step_by_step(dtype, T, H, Hkv, dh, window):
    """A run of decoding steps: every step drafts a tree, attends, and accepts a random path of it;
    pages behind the window are given back.  The output of each accepted token equals dense causal
    attention (float64) over the tokens accepted before it, at their positions."""
    g = _g()
    from retrieval_sparse_attention_causal_gb300 import pipeline
    rng = np.random.default_rng(T + dh)
    B, rot = 3, dh
    w, freq = orc.speeds(rot), g.rotary_frequencies(rot)
    cache = g.PagedCache.empty(60, B, 24, Hkv, dh, dtype=TORCH[dtype])
    prompt = [0, 70, 130]
    kp, vp = (synth.normal(0, s, (B, 130, Hkv, dh), 1.0, dtype) for s in (20, 21))
    kept = [[(kp[b, j], vp[b, j]) for j in range(prompt[b])] for b in range(B)]  # before rotary
    kr, _ = g.rotary(dev(kp, dtype), None, freq)
    cache.append(kr, dev(vp, dtype), ints(prompt))
    graph = 0
    for step in range(8):
        q, k, v = (synth.normal(10 + step, s, (B, T, n, dh), 1.0, dtype) for s, n in ((22, H), (23, Hkv), (24, Hkv)))
        parents = np.array([[int(rng.integers(-1, t)) if t else -1 for t in range(T)] for _ in range(B)])
        out = pipeline.draft_step(dev(q, dtype), dev(k, dtype), dev(v, dtype), ints(parents), cache, freq, window=window)
        paths = []
        for b in range(B):
            node, path = int(rng.integers(0, T)), []
            while node >= 0:
                path.insert(0, node)
                node = parents[b, node]
            paths.append(path if rng.random() < 0.9 else [])
        got = host(out["o"])
        for b, path in enumerate(paths):
            seq = kept[b] + [(k[b, t], v[b, t]) for t in path]
            for i, t in enumerate(path):
                n = len(kept[b]) + i + 1
                lo = max(0, n - window) if window else 0
                at = np.arange(lo, n)[None]
                ks = orc.rotary(np.stack([x[0] for x in seq[lo:n]])[None], at, w)[0]
                vs = np.stack([x[1] for x in seq[lo:n]])
                qr = orc.rotary(q[b:b + 1, t:t + 1], np.array([[n - 1]]), w)[0, 0]
                for h in range(H):
                    m = h // (H // Hkv)
                    s = ks[:, m] @ qr[h] / np.sqrt(dh)
                    e = np.exp(s - s.max())
                    ref = e @ vs[:, m] / e.sum()
                    # The turned q and k are rounded: ds <= 2 half steps of sum |q k| / sqrt(dh); the
                    # weights' own rounding and the output's: two more.
                    ds = 2.2 * HALF[dtype] * (np.abs(ks[:, m]) @ np.abs(qr[h])).max() / np.sqrt(dh) + 1e-5
                    lim = (np.expm1(2 * ds) + 2 * HALF[dtype] + 1e-5) * (e @ np.abs(vs[:, m]) / e.sum()) + HALF[dtype] * np.abs(ref)
                    assert np.all(np.abs(got[b, t, h] - ref) <= lim), (step, b, t, h)
                    graph += 1
        counts = [len(p) for p in paths]
        begin = [max(0, len(kept[b]) + counts[b] - window + 1) if window else 0 for b in range(B)]
        pipeline.accept_draft(out, cache, ints(counts), ints([p + [0] * (T - len(p)) for p in paths]), begin=ints(begin))
        for b, path in enumerate(paths):
            kept[b] += [(k[b, t], v[b, t]) for t in path]
    assert cache.lengths.tolist() == [len(x) for x in kept] and graph > 40
    held = (cache.table >= 0).sum().item()
    assert held == (cache.refs > 0).sum().item()
    if window:
        assert held <= B * (window // 64 + 2)
    cache.free()
    assert not cache.refs.any()


@flags
def test_lookup_flags():
    g = _g()
    cache, _ = cache_pair(np.random.default_rng(0), [100, 70], 4, 8)
    got = cache.lookup(ints([[[0, 1, -1, 4]], [[-2, 1, 0, 3]], [[0, 1, 2, 3]]]), slots=ints([1, 0, 2])).cpu().numpy()
    t = cache.table.cpu().numpy()
    assert got.tolist() == [[[t[1, 0], t[1, 1], -1, -1]], [[-1, t[0, 1], t[0, 0], -1]], [[-1] * 4]]
    with pytest.raises(g.GCAError):
        cache.check()


def test_copies_and_replaced_tensors_of_a_cache():
    """A deep copy (and an unpickled cache) is a cache of its own; a larger pool, a wider table and
    more slots take effect at the next call; tensors that do not fit together are refused."""
    import copy
    import pickle
    g = _g()
    cache, model = cache_pair(np.random.default_rng(7), [100, 0, 64], 3, 12)
    kn, vn = new_rows(8, 3, 40)
    before = copy.deepcopy(model)
    for twin in (copy.deepcopy(cache), pickle.loads(pickle.dumps(cache))):
        other = copy.deepcopy(before)
        twin.append(dev(kn, "bf16"), dev(vn, "bf16"), ints([3, 40, 1]))
        other.append(kn, vn, [3, 40, 1])
        same_state(twin, other)
        same_state(cache, model)
        del twin
    cache.append(dev(kn, "bf16"), dev(vn, "bf16"), ints([1, 2, 3]))
    model.append(kn, vn, [1, 2, 3])
    same_state(cache, model)
    more = synth.normal(3, 20, (5, 64, 2, 32), 1.0, "bf16")
    cache.k_pages, cache.v_pages = (torch.cat([p, dev(more, "bf16")]) for p in (cache.k_pages, cache.v_pages))
    with pytest.raises(ValueError):
        cache.compact()  # the counts are those of the smaller pool
    cache.refs = torch.cat([cache.refs, ints([0] * 5)])
    cache.table = torch.cat([cache.table, ints([[-1] * 2] * 3)], 1)
    model.k, model.v = (np.concatenate([p, more]) for p in (model.k, model.v))
    model.refs = np.concatenate([model.refs, np.zeros(5, dtype=np.int64)])
    model.table = np.concatenate([model.table, np.full((3, 2), -1)], 1)
    kn, vn = new_rows(9, 3, 200)
    cache.append(dev(kn, "bf16"), dev(vn, "bf16"), ints([200, 150, 140]))
    model.append(kn, vn, [200, 150, 140])
    assert not model.full
    same_state(cache, model)
    cache.check()
    q, k1, v1 = (dev(synth.normal(4, s, (3, 1, n, 32), 1.0, "bf16"), "bf16") for s, n in ((22, 4), (23, 2), (24, 2)))
    o, _ = cache.attention(q, k1, v1)
    want, _ = g.tree_attention(q, k1, v1, cache.k_pages, cache.v_pages, cache.table, cache.lengths)
    assert torch.equal(o, want)


@flags
@pytest.mark.parametrize("pages", [40, 8192, 8193, 9000])
def test_compact_clears_entries_that_name_free_pages(pages):
    """Entries with a page that nothing counts, below and above the pages that stay, and numbers
    outside the pool: each becomes -1 and is flagged, and no slot ends with a page of another."""
    g = _g()
    rng = np.random.default_rng(pages)
    lengths = [64 * (pages // 5)] * 3 + [130, 64]
    cache, model = cache_pair(rng, lengths, pages // 5 + 4, pages, Hkv=1, dh=32)
    live = int((model.refs > 0).sum())
    free = [p for p in range(pages) if model.refs[p] == 0]
    low, high = [p for p in free if p < live], [p for p in free if p >= live]
    bad = [(0, -1, low[0]), (1, -1, low[0]), (2, -2, low[-1]), (3, -1, high[0]), (4, 3, high[-1]), (4, 2, pages), (3, -2, -7),
           (0, -2, model.table[1, 0])]  # the last is held: it moves like any other
    for s, p, page in bad:
        cache.table[s, p] = int(page)
        model.table[s, p] = page
    assert int(cache.compact()) == model.compact() == live
    assert model.flagged and (model.table >= 0).sum() == live + 1
    same_state(cache, model)
    with pytest.raises(g.GCAError) as e:
        cache.check()
    assert e.value.status == g.GCA_ERR_DEVICE_INDEX
    assert int(cache.compact()) == live  # nothing left to move or to clear
    same_state(cache, model)
    cache.check()


@flags
def test_checks_report_one_kind_after_the_other():
    """An append that names a bad slot and runs out of pages, behind a wait that ran out, in one error
    word: each check reports one kind and leaves the others."""
    g = _g()
    for waited in (False, True):
        cache, model = cache_pair(np.random.default_rng(6), [64, 0, 64], 4, 4)
        cache.ws = g.Workspace()
        if waited:
            g.selftest_timeout(cache.ws, spins=64)
        kn, vn = new_rows(6, 3, 128)
        cache.append(dev(kn, "bf16"), dev(vn, "bf16"), ints([128, 1, 128]), slots=ints([0, 7, 2]))
        model.append(kn, vn, [128, 1, 128], slots=[0, 7, 2])
        assert model.flagged and model.full
        same_state(cache, model)
        for status in [g.GCA_ERR_TIMEOUT] * waited + [g.GCA_ERR_DEVICE_INDEX, g.GCA_ERR_CACHE_FULL]:
            with pytest.raises(g.GCAError) as e:
                cache.check()
            assert e.value.status == status
            assert ("index 7" in str(e.value)) == (status == g.GCA_ERR_DEVICE_INDEX)
        cache.check()


def test_rotary_turns_by_whole_numbers_exactly():
    """From the table on, positions cost no precision: the angle is p f mod 2^64 (whole numbers here, so that
    the speeds' own rounding has no part in it), off by the cut to 32 bits, 2 pi 2^-32, and the float that
    sincospif takes, pi 2^-25.  The rest as in rotary_bound."""
    g = _g()
    rot, H = 64, 2
    pos = np.array([[0, 1, -1, -12345, 1 << 24, (1 << 31) - 1, -(1 << 31), (1 << 31) - 64]])
    x = synth.normal(6, 0, (1, pos.shape[1], H, rot), 1.0, "f32")
    freq = g.rotary_frequencies(rot)
    turns = [[(p * f) % 2 ** 64 / 2.0 ** 64 for f in freq.tolist()] for p in pos[0].tolist()]
    angle = 2 * np.pi * np.array(turns)[None, :, None, :]
    got = host(g.rotary(dev(x, "f32"), None, freq, positions=ints(pos))[0])
    a, b = x[..., :rot // 2], x[..., rot // 2:]
    ref = np.concatenate([a * np.cos(angle) - b * np.sin(angle), a * np.sin(angle) + b * np.cos(angle)], -1)
    lim = np.hypot(a, b) * np.sqrt(2) * (np.pi * (2.0 ** -25 + 2.0 ** -31) + 6 * U) + 1e-40
    within(got, ref, np.concatenate([lim, lim], -1) + U * np.abs(ref), "rotary")


SHARES = [  # lengths, T, H, Hkv, dh, kind: blocks and leads of a set of heads, and the limit
    ([25000], 16, 4, 1, 64, "tree"),             # 396 of 400: shares of four blocks or more
    ([25344], 16, 4, 1, 64, "wild"),             # 401 of 400: shares of eight or more
    ([30000], 16, 4, 1, 64, "tree"),             # 474 of 400
    ([30000], 40, 8, 2, 64, "tree"),             # two row groups of two key heads: too few shares for a limit
    ([33333], 130, 1, 1, 64, "padded chain"),    # two row groups: 528 of 400
    ([1, 78000, 100], 8, 8, 1, 128, "wild"),     # 1237 of 1200: one long among three
    ([27000, 26000], 20, 4, 2, 64, "padded chain"),  # 839 of 800
]


@pytest.mark.parametrize("lengths,T,H,Hkv,dh,kind", SHARES)
def test_tree_attention_over_many_blocks_of_few_heads(lengths, T, H, Hkv, dh, kind):
    """Long contexts of one or two key heads, where a share's least length grows: the kernel and the
    join must divide the work alike on both sides of the limit."""
    g = _g()
    g.profile_begin()
    attend_and_check(np.random.default_rng(T + dh), lengths, T, H, Hkv, dh, "bf16", kind, seed=5)
    names = g.profile_end()
    assert "tree_tc" in names and "tree_join" in names


def test_steps_over_the_first_slots_of_a_cache():
    """A batch may be smaller than the cache: entry i is slot i where no slots are named, and the slots
    behind keep their state."""
    g = _g()
    from retrieval_sparse_attention_causal_gb300 import pipeline
    rng = np.random.default_rng(12)
    cache, model = cache_pair(rng, [70, 0, 64, 130, 5], 6, 30)
    freq = g.rotary_frequencies(32)
    for B, T in ((2, 3), (1, 1), (3, 70)):
        q, k, v = (dev(synth.normal(B, s, (B, T, n, 32), 1.0, "bf16"), "bf16") for s, n in ((22, 4), (23, 2), (24, 2)))
        parents = ints([[t - 1 for t in range(T)]] * B)
        step = pipeline.draft_step(q, k, v, parents, cache, freq, window=0)
        mask, pos = g.tree_plan(parents, cache.lengths[:B].clone())
        assert torch.equal(step["plan"][0], mask) and torch.equal(step["plan"][1], pos)
        counts = [T, 1, T // 2][:B]
        path = [list(range(T))] * B
        begin = [64, 0, 0][:B]
        pipeline.accept_draft(step, cache, ints(counts), ints(path), begin=ints(begin))
        model.append(host(step["k"]), host(v), counts, np.array(path))
        model.trim(begin=begin)
        same_state(cache, model)
    with pytest.raises(ValueError):
        cache.trim(end=ints([1] * 6))  # more entries than slots
    with pytest.raises(ValueError):
        g.tree_plan(ints([[-1]] * 6), cache.lengths)
    same_state(cache, model)


UNSEEN = [  # lengths, T, H, Hkv, dh, dtype, kind, window, pages of the table behind the longest, kernel
    ([300, 64, 1000, 90], 1, 8, 4, 64, "bf16", "late", 50, 1, None),
    ([300, 64, 1000, 90] * 40, 1, 12, 12, 64, "bf16", "late", 130, 1, "tree_rows"),
    ([300, 64, 1000, 90], 5, 4, 4, 32, "bf16", "late", 70, 1, "tree_rows"),
    ([300, 64, 700, 90], 70, 4, 2, 64, "bf16", "late", 100, 1, "tree_tc"),
    ([300, 64, 700, 90], 20, 24, 6, 128, "bf16", "late", 200, 1, "tree_tc"),
    ([300, 64, 700], 150, 4, 2, 64, "bf16", "late", 33, 1, "tree_tc"),
    ([300, 64, 700], 9, 4, 2, 32, "f32", "late", 70, 1, "tree_simt"),
    ([300, 64, 700], 70, 4, 2, 64, "f32", "late", 100, 1, "tree_simt"),
    ([100, 65, 0], 12, 4, 4, 32, "bf16", "far apart", 7, 1, "tree_rows"),
    ([100, 65, 0], 40, 8, 2, 64, "bf16", "far apart", 9, 1, "tree_tc"),
    ([100, 65, 0] * 30, 10, 16, 16, 64, "bf16", "far apart", 9, 1, "tree_rows"),
    ([100, 65, 0], 100, 2, 1, 128, "bf16", "far apart", 60, 1, "tree_tc"),
    ([100, 65, 0], 70, 2, 1, 32, "f32", "far apart", 30, 1, "tree_simt"),
    ([100, 65, 3000], 40, 4, 2, 64, "bf16", "far apart", 0, 1000, "tree_tc"),
]


@pytest.mark.parametrize("lengths,T,H,Hkv,dh,dtype,kind,window,spare,kernel", UNSEEN)
def test_tree_attention_does_not_use_what_no_row_sees(lengths, T, H, Hkv, dh, dtype, kind, window, spare, kernel):
    """NaN and infinities in every token of the cache and of the draft that no row sees: behind lengths, in
    padding, outside all masks, and passed by the window of every row, which is not only what the
    length tells where positions lie behind it ('late') or a mask names tokens that the window has passed
    ('far apart')."""
    g = _g()
    rng = np.random.default_rng(T + dh + len(lengths))
    B = len(lengths)
    k, v, table, _ = random_cache(rng, lengths, Hkv, dh, dtype, width_spare=spare)
    q = synth.normal(1, 22, (B, T, H, dh), 1.0, dtype)
    kn, vn = synth.normal(1, 23, (B, T, Hkv, dh), 1.0, dtype), synth.normal(1, 24, (B, T, Hkv, dh), 1.0, dtype)
    n = np.array(lengths)[:, None]
    if kind == "late":
        pos = n + rng.integers(0, 60, (B, 1)) + np.arange(T)
        see = rng.random((B, T, T)) < 0.5
    else:
        pos = n + rng.integers(0, 4 * max(window, 5), (B, T))
        see = rng.random((B, T, T)) < 0.2
    pos[:, 1::7] = -1
    low = pos - window if window else np.full((B, T), -1)
    for b in range(B):
        rows = [t for t in range(T) if pos[b, t] >= 0]
        first = min(low[b, t] for t in rows) + 1
        for j in range(max(0, min(first, lengths[b]))):
            k[table[b, j // 64], j % 64], v[table[b, j // 64], j % 64] = np.nan, (np.inf if j % 2 else np.nan)
        for u in range(T):
            if pos[b, u] < 0 or not any(see[b, t, u] and pos[b, u] > low[b, t] for t in rows):
                kn[b, u], vn[b, u] = np.nan, (-np.inf if u % 2 else np.nan)
    assert np.isnan(kn).any()
    g.profile_begin()
    o, lse = g.tree_attention(*(dev(x, dtype) for x in (q, kn, vn, k, v)), ints(table), ints(lengths),
                              mask=torch.from_numpy(orc.pack_mask(see)).cuda(), positions=ints(pos), window=window)
    names = g.profile_end()
    assert kernel is None or kernel in names, names
    ro, rl, mean_abs, dot_abs, keys = orc.tree_attention(q, kn, vn, k, v, table, lengths, see, pos, window)
    ds = (2 * dh + 4) * U * dot_abs  # the bounds of attend_and_check
    dw = 2 * ds + 4 * U * dot_abs + 8 * U + 1.2 * keys * U
    within(host(lse), rl, ds + dw + np.where(np.isfinite(rl), 4 * U * (1 + np.abs(rl)), 0), "lse")
    weight = HALF["bf16"] if dtype == "bf16" else 0.0
    within(host(o), ro, (2 * dw + weight)[..., None] * mean_abs * (1 + 2 * HALF[dtype]) + 2 * HALF[dtype] * np.abs(ro) + 1e-38, "o")


@pytest.mark.parametrize("lengths,T,H,Hkv,dh,dtype,window", [
    ([100, 0, 700], 1, 4, 2, 32, "f32", 0), ([700, 64], 1, 8, 1, 64, "f32", 0), ([300, 5000], 3, 2, 2, 128, "f32", 100),
    ([100, 0, 700], 1, 4, 2, 32, "bf16", 0), ([100, 64, 5000], 1, 12, 12, 64, "bf16", 0), ([100, 700], 2, 4, 4, 128, "bf16", 50),
    ([100, 0, 9000], 70, 4, 2, 64, "bf16", 0), ([100, 700], 200, 4, 2, 64, "bf16", 90)])
def test_tree_attention_of_padding_alone(lengths, T, H, Hkv, dh, dtype, window):
    """A sequence whose draft is padding sees nothing, whatever its cache holds: zeros and -inf, beside
    sequences that are not changed by it."""
    g = _g()
    rng = np.random.default_rng(dh)
    B = len(lengths)
    k, v, table, _ = random_cache(rng, lengths, Hkv, dh, dtype)
    q = synth.normal(1, 22, (B, T, H, dh), 1.0, dtype)
    kn, vn = synth.normal(1, 23, (B, T, Hkv, dh), 1.0, dtype), synth.normal(1, 24, (B, T, Hkv, dh), 1.0, dtype)
    pos = np.array(lengths)[:, None] + np.arange(T)
    args = lambda: ([dev(x, dtype) for x in (q, kn, vn, k, v)] + [ints(table), ints(lengths)])  # noqa: E731
    want, wlse = g.tree_attention(*args(), positions=ints(pos), window=window)
    pos[-1] = -1
    for p in table[-1][table[-1] >= 0]:
        k[p], v[p] = np.nan, np.inf
    q[-1], kn[-1], vn[-1] = np.inf, np.nan, np.nan
    o, lse = g.tree_attention(*args(), positions=ints(pos), window=window)
    assert torch.equal(o[:-1], want[:-1]) and torch.equal(lse[:-1], wlse[:-1])
    assert not o[-1].any() and bool((lse[-1] == -float("inf")).all())
