"""CPU tests of a prompt's operators: refusals before anything is launched, and the oracle's own rules."""
import ctypes

import numpy as np
import pytest
import torch

import oracle.decode_oracle as dorc
import oracle.prompt_oracle as orc

FAKE = 0x100000  # 256-byte aligned, never dereferenced: every call below fails validation


@pytest.fixture(scope="module")
def gca():
    import __graft_entry__
    __graft_entry__.build()
    import retrieval_sparse_attention_causal_gb300 as m
    return m


def heads(g, data=FAKE, bs=64 * 12 * 64, ts=12 * 64, hs=64):
    return ctypes.byref(g.Heads(data, bs, ts, hs))


def test_prompt_attention_refusals(gca):
    L = gca.LIB

    def call(q=None, k=None, v=None, dt=gca.GCA_BF16, N=100, B=3, H=12, Hkv=12, dh=64, off=FAKE, window=0, scale=0.125, o=FAKE,
             lse=FAKE, ws=FAKE, wsb=256):
        h = lambda x: heads(gca) if x is None else x  # noqa: E731
        return L.gca_prompt_attention(h(q), h(k), h(v), dt, N, B, H, Hkv, dh, off, window, scale, o, lse, ws, wsb, None)
    for bad in (dict(dt=2), dict(N=-1), dict(N=(1 << 30) + 1), dict(B=0), dict(B=1025), dict(H=0), dict(Hkv=0), dict(H=10, Hkv=4),
                dict(H=70000, Hkv=70000), dict(window=-1), dict(scale=0.0), dict(scale=float("nan")), dict(scale=float("inf")),
                dict(off=0), dict(off=FAKE + 2), dict(o=0), dict(lse=0), dict(o=FAKE + 8), dict(q=heads(gca, 0)),
                dict(k=heads(gca, FAKE + 8)), dict(v=heads(gca, ts=12 * 64 + 4)), dict(q=heads(gca, ts=0)), dict(k=heads(gca, hs=-64)),
                dict(v=heads(gca, ts=1 << 37))):
        assert call(**bad) == gca.GCA_ERR_INVALID_ARG, bad
    assert call(dh=96) == gca.GCA_ERR_UNSUPPORTED
    assert call(N=1 << 30, H=4096, Hkv=4096) == gca.GCA_ERR_UNSUPPORTED
    assert call(ws=0) == gca.GCA_ERR_WORKSPACE and call(wsb=100) == gca.GCA_ERR_WORKSPACE
    assert call(N=0, q=heads(gca, 0), o=0, lse=0) == gca.GCA_OK  # no row: nothing to do


def test_prompt_attention_backward_refusals(gca):
    L = gca.LIB
    need = L.gca_prompt_attention_backward_scratch_size(100, 3, 12, 12, 64, gca.GCA_BF16)
    assert need >= 2 * 100 * 12 * 4
    assert L.gca_prompt_attention_backward_scratch_size(100, 3, 12, 12, 64, gca.GCA_F32) > need  # parts of few tiles

    def call(dt=gca.GCA_BF16, N=100, B=3, H=12, Hkv=12, dh=64, o=FAKE, dout=None, lse=FAKE, dq=None, dk=None, dv=None, scratch=FAKE,
             size=need):
        h = lambda x: heads(gca) if x is None else x  # noqa: E731
        return L.gca_prompt_attention_backward(heads(gca), heads(gca), heads(gca), o, h(dout), lse, dt, N, B, H, Hkv, dh, FAKE, 0, 0.125,
                                               h(dq), h(dk), h(dv), FAKE, 256, scratch, size, None)
    for bad in (dict(o=0), dict(lse=0), dict(dout=heads(gca, 0)), dict(dq=heads(gca, FAKE + 4)), dict(dk=heads(gca, ts=0)),
                dict(dv=heads(gca, ts=64, hs=64)), dict(dq=heads(gca, hs=32)), dict(dk=heads(gca, ts=12 * 64, hs=0))):
        assert call(**bad) == gca.GCA_ERR_INVALID_ARG, bad
    assert b"overlap" in L.gca_last_error_detail()
    assert call(scratch=0) == gca.GCA_ERR_WORKSPACE and call(size=need - 1) == gca.GCA_ERR_WORKSPACE
    assert call(scratch=FAKE + 128) == gca.GCA_ERR_WORKSPACE
    assert call(dh=48) == gca.GCA_ERR_UNSUPPORTED


def test_norm_rotary_refusals(gca):
    L = gca.LIB

    def call(q=None, k=None, qo=None, ko=None, dt=gca.GCA_BF16, B=2, n=64, H=12, Hkv=12, dh=64, rot=64, eps=1e-6, qw=FAKE, kw=FAKE,
             freq=FAKE, pbs=0):
        h = lambda x: heads(gca) if x is None else x  # noqa: E731
        return L.gca_norm_rotary(h(q), h(k), h(qo), h(ko), dt, B, n, H, Hkv, dh, rot, 0, eps, qw, kw, freq, None, pbs, 1.0, None)
    for bad in (dict(dt=2), dict(q=heads(gca, 0)), dict(ko=heads(gca, 0)), dict(B=0), dict(Hkv=0), dict(rot=63), dict(rot=66),
                dict(eps=-1.0), dict(eps=float("inf")), dict(qw=0), dict(kw=0), dict(qw=FAKE + 2), dict(freq=0), dict(pbs=-1),
                dict(qo=heads(gca, hs=32)), dict(q=heads(gca, FAKE + 1))):
        assert call(**bad) == gca.GCA_ERR_INVALID_ARG, bad
    assert call(dh=300) == gca.GCA_ERR_UNSUPPORTED
    need = L.gca_norm_rotary_backward_scratch_size(64)

    def back(dqo=None, dq=None, dqw=FAKE, dkw=FAKE, scratch=FAKE, size=need):
        h = lambda x: heads(gca) if x is None else x  # noqa: E731
        return L.gca_norm_rotary_backward(heads(gca), heads(gca), h(dqo), heads(gca), h(dq), heads(gca), gca.GCA_BF16, 2, 64, 12, 12, 64,
                                          64, 0, 1e-6, FAKE, FAKE, FAKE, None, 0, 1.0, dqw, dkw, scratch, size, None)
    for bad in (dict(dqo=heads(gca, 0)), dict(dq=heads(gca, 0)), dict(dqw=0), dict(dkw=0), dict(dkw=FAKE + 2), dict(dq=heads(gca, hs=0))):
        assert back(**bad) == gca.GCA_ERR_INVALID_ARG, bad
    assert back(scratch=0) == gca.GCA_ERR_WORKSPACE and back(size=need - 1) == gca.GCA_ERR_WORKSPACE


def test_quantised_cache_refusals(gca):
    L = gca.LIB
    assert L.gca_cache_row_bytes(gca.GCA_E4M3, 12, 64) == 784 and L.gca_cache_row_bytes(gca.GCA_BF16, 12, 64) == 1536
    assert L.gca_cache_row_bytes(gca.GCA_E4M3, 16, 32) == 528 and L.gca_cache_row_bytes(gca.GCA_E4M3, 17, 32) == 576

    def pool(**kw):
        a = dict(k_pages=FAKE, v_pages=FAKE, dtype=gca.GCA_E4M3, heads=4, dh=64, pages=100, table=FAKE, slots=8, width=10, lengths=FAKE,
                 refs=FAKE)
        a.update(kw)
        return ctypes.byref(gca.Cache(**a))
    need = L.gca_cache_append_quantised_scratch_size(4, 100, 0)
    new = lambda **kw: heads(gca, **{**dict(bs=100 * 256, ts=256, hs=64), **kw})  # noqa: E731

    def append(c=None, k=None, dt=gca.GCA_BF16, n=4, T=100, counts=FAKE, path=None, off=None, scratch=FAKE, size=need):
        return L.gca_cache_append_quantised(c or pool(), k or new(), new(), dt, n, T, None, counts, path, off, FAKE, 256, scratch, size, None)
    for bad in (dict(c=pool(dtype=gca.GCA_BF16)), dict(c=pool(dtype=3)), dict(c=pool(refs=0)), dict(dt=gca.GCA_E4M3), dict(n=0), dict(n=9),
                dict(T=0), dict(counts=None), dict(counts=FAKE, off=FAKE), dict(counts=None, off=FAKE, path=FAKE), dict(k=new(data=0)),
                dict(k=new(ts=260)), dict(k=new(hs=128))):
        assert append(**bad) == gca.GCA_ERR_INVALID_ARG, bad
    assert append(c=pool(dh=80)) == gca.GCA_ERR_UNSUPPORTED
    assert append(size=need - 1) == gca.GCA_ERR_WORKSPACE

    def read(c=None, n=4, per=8, idx=FAKE, dt=gca.GCA_BF16, k=FAKE, v=FAKE):
        return L.gca_cache_read(c or pool(), n, per, None, idx, dt, k, v, None, FAKE, 256, None)
    for bad in (dict(c=pool(dtype=gca.GCA_F32)), dict(n=9), dict(per=0), dict(idx=0), dict(k=0), dict(v=FAKE + 8), dict(dt=gca.GCA_E4M3)):
        assert read(**bad) == gca.GCA_ERR_INVALID_ARG, bad
    # What reads numbers does not take quantised pages.
    h = heads(gca)
    assert L.gca_cache_append(pool(), h, h, 4, 100, None, FAKE, None, FAKE, 256, FAKE, 1 << 20, None) == gca.GCA_ERR_INVALID_ARG
    assert L.gca_tree_attention(h, h, h, pool(), 2, 1, 12, None, None, 0, 0.125, FAKE, FAKE, FAKE, 256, FAKE, 1 << 30, None) == gca.GCA_ERR_INVALID_ARG
    # (A pool of another type is still refused as one.)
    assert L.gca_cache_fork(pool(dtype=3), 1, FAKE, FAKE, FAKE, 256, None) == gca.GCA_ERR_INVALID_ARG


def test_quantised_rows_of_any_width_have_page_operations(gca):
    """A row as one head of what is left beside its exponents, as the Python cache gives it: not refused for its width."""
    row = gca.LIB.gca_cache_row_bytes(gca.GCA_E4M3, 520, 128)
    pool = ctypes.byref(gca.Cache(k_pages=FAKE, v_pages=FAKE, dtype=gca.GCA_E4M3, heads=1, dh=row - 16, pages=100, table=FAKE, slots=8, width=10,
                                  lengths=FAKE, refs=FAKE))
    assert row == 520 * 128 + 528 and gca.LIB.gca_cache_row_bytes(gca.GCA_E4M3, 1, row - 16) == row
    assert gca.LIB.gca_cache_fork(pool, 0, FAKE, FAKE, FAKE, 256, None) == gca.GCA_ERR_INVALID_ARG
    assert b"n must be in" in gca.LIB.gca_last_error_detail()  # what is refused is the call without an entry


def test_python_refusals(gca):
    """Tensors that a call cannot take are refused before a device is looked for."""
    x = torch.zeros(10, 4, 64, dtype=torch.bfloat16)
    off = torch.tensor([0, 10], dtype=torch.int32)
    for args in ((x[0], x, x, off), (x, x[:9], x, off), (x, x, x.float(), off), (x.half(), x.half(), x.half(), off), (x, x, x, off.long()),
                 (x, x, x, off[:1]), (x.transpose(1, 2), x, x, off)):
        with pytest.raises((ValueError, TypeError)):
            gca.prompt_attention(*args)
    with pytest.raises(ValueError, match="CUDA"):
        gca.prompt_attention(x, x, x, off)
    q, w, freq = torch.zeros(1, 10, 4, 64), torch.ones(64), gca.rotary_frequencies(64, device="cpu")
    for args in ((q, q, w[:32], w, freq), (q, q, w, w.double(), freq), (q, q, w, None, freq), (q, q[:, :5], w, w, freq), (q, None, w, w, freq.int())):
        with pytest.raises((ValueError, TypeError)):
            gca.norm_rotary(*args)
    state = (torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(5, dtype=torch.int32))
    with pytest.raises(ValueError):
        gca.QuantisedCache(torch.zeros(5, 64, 100, dtype=torch.uint8), torch.zeros(5, 64, 100, dtype=torch.uint8), *state, 1, 64)
    with pytest.raises(ValueError):
        gca.PagedCache(torch.zeros(5, 64, 80, dtype=torch.uint8), torch.zeros(5, 64, 80), *state)


def test_outputs_that_are_inputs_and_bytes_as_a_plain_cache_are_refused(gca):
    L, h = gca.LIB, heads(gca)
    other = lambda n: heads(gca, FAKE + n * 0x1000000)  # noqa: E731
    assert L.gca_prompt_attention(h, h, h, gca.GCA_BF16, 100, 3, 12, 12, 64, FAKE, 0, 0.125, FAKE, FAKE, FAKE, 256, None) == gca.GCA_ERR_INVALID_ARG
    assert b"input" in L.gca_last_error_detail()
    for dq, dk, dv, what in ((h, other(1), other(2), b"input"), (other(1), other(2), h, b"input"), (other(1), other(2), other(2), b"one tensor"),
                             (other(1), other(2), other(1), b"one tensor")):
        st = L.gca_prompt_attention_backward(h, h, h, FAKE, h, FAKE, gca.GCA_BF16, 100, 3, 12, 12, 64, FAKE, 0, 0.125, dq, dk, dv, FAKE, 256,
                                             FAKE, 1 << 30, None)
        assert st == gca.GCA_ERR_INVALID_ARG and what in L.gca_last_error_detail()
    pages = torch.zeros(5, 64, 80, dtype=torch.uint8)
    with pytest.raises((ValueError, TypeError), match="k_pages"):
        gca.PagedCache(pages, pages, torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), torch.zeros(5, dtype=torch.int32))


def test_outputs_that_overlap_are_refused(gca):
    """At whatever addresses: shifted, inside, one in rows of the other, interleaved with too little room."""
    L = gca.LIB
    n = 100 * 12 * 64  # elements of q
    at = lambda e, **kw: heads(gca, FAKE + 2 * e, **kw)  # noqa: E731
    far = 1 << 30

    def forward(q, k, v, o, lse=FAKE + 8 * far, off=FAKE + 10 * far):
        st = L.gca_prompt_attention(q, k, v, gca.GCA_BF16, 100, 3, 12, 12, 64, off, 0, 0.125, o, lse, FAKE, 256, None)
        return st, L.gca_last_error_detail()
    q, k, v = at(0), at(far), at(2 * far)
    for o in (FAKE + 16, FAKE + 2 * n - 16, FAKE + 2 * far + 2048):
        assert forward(q, k, v, o) == (gca.GCA_ERR_INVALID_ARG, b"o and lse must not overlap an input"), o
    wide = at(0, ts=36 * 64)  # the queries of a fused projection: o lies in the first of them, or over several tokens
    assert forward(wide, k, v, FAKE + 2 * 36 * 64 * 50)[0] == gca.GCA_ERR_INVALID_ARG
    assert forward(wide, k, v, FAKE + 2 * 12 * 64)[0] == gca.GCA_ERR_INVALID_ARG
    turned = at(0, ts=64, hs=100 * 64)  # heads first
    assert forward(turned, k, v, FAKE + 2 * 11 * 100 * 64)[0] == gca.GCA_ERR_INVALID_ARG
    o = FAKE + 6 * far
    for kw in (dict(lse=o + 2 * n - 4), dict(lse=FAKE + 4), dict(off=o + 16), dict(off=FAKE + 8 * far + 4)):
        assert forward(q, k, v, o, **kw)[0] == gca.GCA_ERR_INVALID_ARG, kw

    def backward(dq, dk, dv, q=q, Hkv=12):
        st = L.gca_prompt_attention_backward(q, k, v, o, at(7 * far), FAKE + 8 * far, gca.GCA_BF16, 100, 3, 12, Hkv, 64, FAKE + 10 * far, 0, 0.125,
                                             dq, dk, dv, FAKE, 256, FAKE, 1 << 30, None)
        return st, L.gca_last_error_detail()
    a, b, c = at(11 * far), at(12 * far), at(13 * far)
    for x in (at(8), at(far + n - 8), at(2 * far + 64), at(3 * far + 8), at(7 * far - 8 + n), at(4 * far), at(5 * far)):
        for g in ((x, b, c), (a, x, c), (a, b, x)):
            assert backward(*g) == (gca.GCA_ERR_INVALID_ARG, b"a gradient must not overlap an input")
    for g in ((a, at(11 * far + n - 8), c), (a, b, at(11 * far + 8)), (a, b, at(12 * far + 64 * 3))):
        assert backward(*g)[0] == gca.GCA_ERR_INVALID_ARG and b"two gradients" in L.gca_last_error_detail()
    # Views of one tensor [N, 12 + 2 + 2, 64]: the values' gradients begin a head, or half a one, too soon.
    view = lambda h: at(11 * far + h * 64, ts=16 * 64)  # noqa: E731
    for first in (13, 13.5):
        assert backward(view(0), view(12), at(11 * far + int(first * 64), ts=16 * 64), Hkv=2)[0] == gca.GCA_ERR_INVALID_ARG
        assert b"two gradients" in L.gca_last_error_detail()


def test_norm_outputs_that_overlap_are_refused(gca):
    """Shifted, in another order, inside the other side's, or the other side's itself; each output."""
    L, far = gca.LIB, 1 << 30
    at = lambda e, **kw: heads(gca, FAKE + 2 * e, **kw)  # noqa: E731
    n = 2 * 64 * 12 * 64
    w = FAKE + 40 * far

    def forward(q, k, qo, ko, pos=None):
        st = L.gca_norm_rotary(q, k, qo, ko, gca.GCA_BF16, 2, 64, 12, 12, 64, 64, 0, 1e-6, w, w + 4096, w + 8192, pos, 64, 1.0, None)
        return st, L.gca_last_error_detail()
    q, k, a, b = at(0), at(far), at(2 * far), at(3 * far)
    for qo, ko, what in ((at(64), b, b"itself"), (a, at(far + n - 64), b"itself"), (k, b, b"itself"), (a, q, b"itself"), (k, q, b"itself"),
                         (a, at(2 * far + n - 64), b"two outputs"), (at(0, ts=64, hs=64 * 64), b, b"itself")):
        st, detail = forward(q, k, qo, ko)
        assert st == gca.GCA_ERR_INVALID_ARG and what in detail
    assert forward(q, k, at(20 * far), b)[1] == b"an output must not overlap an input"  # the weights
    assert forward(q, k, a, b, pos=FAKE + 4 * far)[0] == gca.GCA_ERR_INVALID_ARG

    def backward(dq, dk, dqw=w + 16384, dkw=w + 20480):
        size = L.gca_norm_rotary_backward_scratch_size(64)
        st = L.gca_norm_rotary_backward(q, k, at(4 * far), at(5 * far), dq, dk, gca.GCA_BF16, 2, 64, 12, 12, 64, 64, 0, 1e-6, w, w + 4096, w + 8192,
                                        None, 0, 1.0, dqw, dkw, FAKE + 60 * far, size, None)
        return st, L.gca_last_error_detail()
    for x in ((at(4 * far + 64), b), (at(5 * far), b), (k, b), (a, q), (a, at(4 * far)), (a, at(5 * far + 8)), (a, at(2 * far + 64)), (at(64), b)):
        assert backward(*x)[0] == gca.GCA_ERR_INVALID_ARG
    for kw in (dict(dqw=FAKE + 4 * far + 4), dict(dkw=w + 16384 + 252)):
        assert backward(a, b, **kw)[0] == gca.GCA_ERR_INVALID_ARG


# ------------------------------------------------------------------ the oracle
def test_oracle_attention_is_softmax_attention():
    """Against torch's own attention in float64 on one dense sequence, and packed sequences against each by itself."""
    r = np.random.default_rng(1)
    q, k, v = r.standard_normal((3, 20, 4, 8))
    o = orc.prompt_attention(q, k, v, [0, 20])["o"]
    t = [torch.from_numpy(x.transpose(1, 0, 2)[None].copy()) for x in (q, k, v)]
    ref = torch.nn.functional.scaled_dot_product_attention(*t, is_causal=True)[0].numpy().transpose(1, 0, 2)
    assert np.abs(o - ref).max() < 1e-13
    packed = orc.prompt_attention(q, k, v, [0, 7, 7, 20], window=3)
    for a, z in ((0, 7), (7, 20)):
        one = orc.prompt_attention(q[a:z], k[a:z], v[a:z], [0, z - a], window=3)
        assert np.array_equal(packed["o"][a:z], one["o"]) and np.array_equal(packed["lse"][a:z], one["lse"])


def test_oracle_gradients_against_differences():
    r = np.random.default_rng(2)
    x = [r.standard_normal((9, h, 4)) for h in (4, 2, 2)]
    do = r.standard_normal((9, 4, 4))
    f = lambda y: (orc.prompt_attention(*y, [0, 4, 9], window=3)["o"] * do).sum()  # noqa: E731
    g = orc.prompt_attention(*x, [0, 4, 9], window=3, dout=do)
    for i, name in enumerate(("dq", "dk", "dv")):
        d = r.standard_normal(x[i].shape)
        up, down = ([t + s * 1e-5 * d if j == i else t for j, t in enumerate(x)] for s in (1, -1))
        assert abs((f(up) - f(down)) / 2e-5 - (g[name] * d).sum()) < 1e-7
    y, w, pos = r.standard_normal((2, 3, 2, 8)), r.standard_normal(8), r.integers(0, 100, (2, 3))
    speeds, dy = dorc.speeds(6), r.standard_normal((2, 3, 2, 8))
    h = lambda a, b: (orc.norm_rotary(a, b, pos, speeds, 1e-3, True, 1.3) * dy).sum()  # noqa: E731
    dx, dw = orc.norm_rotary_backward(y, dy, w, pos, speeds, 1e-3, True, 1.3)
    d, e = r.standard_normal(y.shape), r.standard_normal(8)
    assert abs((h(y + 1e-5 * d, w) - h(y - 1e-5 * d, w)) / 2e-5 - (dx * d).sum()) < 1e-7
    assert abs((h(y, w + 1e-5 * e) - h(y, w - 1e-5 * e)) / 2e-5 - (dw * e).sum()) < 1e-7


def test_oracle_numbers_are_e4m3():
    """Every number is torch's e4m3 rounding of the scaled value, within half a step, and the scale the least."""
    r = np.random.default_rng(3)
    x = (r.standard_normal((50, 64)) * 2.0 ** r.integers(-30, 30, (50, 1))).astype(np.float32)
    x[0], x[1, 0] = 0.0, 448.0
    y, e = orc.quantise(x)
    scaled = torch.from_numpy(x.astype(np.float64) / 2.0 ** e[:, None]).float()
    assert np.array_equal(scaled.to(torch.float8_e4m3fn).double().numpy(), y)
    back = y * 2.0 ** e[:, None]
    assert (np.abs(back - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** (e[:, None] - 10.0))).all()
    big = np.abs(x).max(1)
    assert (big <= 448 * 2.0 ** e).all() and ((big > 224 * 2.0 ** e) | (e == -120)).all()
