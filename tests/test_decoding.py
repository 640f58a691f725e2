"""CPU tests of the decoding operators: refusals before anything is launched, the rotary
frequency table, and the page oracle's own rules."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle.decode_oracle as orc

FAKE = 0x100000  # 16-byte aligned, never dereferenced: every call below fails validation


@pytest.fixture(scope="module")
def gca():
    import __graft_entry__
    __graft_entry__.build()
    import retrieval_sparse_attention_causal_gb300 as m
    return m


def heads(g, data=FAKE, bs=64 * 12 * 64, ts=12 * 64, hs=64):
    return ctypes.byref(g.Heads(data, bs, ts, hs))


def pool(g, **kw):
    a = dict(k_pages=FAKE, v_pages=FAKE, dtype=g.GCA_BF16, heads=4, dh=64, pages=100, table=FAKE, slots=8, width=10,
             lengths=FAKE, refs=FAKE)
    a.update(kw)
    return ctypes.byref(g.Cache(**a))


def test_rotary_refusals(gca):
    L = gca.LIB

    def call(q=None, k=None, qo=None, ko=None, dt=gca.GCA_BF16, B=2, n=64, H=12, Hkv=12, dh=64, rot=64, freq=FAKE, pbs=0, nok=False):
        h = lambda x: x if x is not None else heads(gca)  # noqa: E731
        return L.gca_rotary(h(q), None if nok else h(k), h(qo), None if nok else h(ko), dt, B, n, H, Hkv, dh, rot, 0, 0,
                            freq, None, pbs, 1.0, None)
    assert call(dt=5) == gca.GCA_ERR_INVALID_ARG
    assert call(q=heads(gca, 0)) == gca.GCA_ERR_INVALID_ARG
    assert call(ko=heads(gca, 0)) == gca.GCA_ERR_INVALID_ARG
    assert call(B=0) == gca.GCA_ERR_INVALID_ARG
    assert call(Hkv=0) == gca.GCA_ERR_INVALID_ARG
    assert call(nok=True) == gca.GCA_ERR_INVALID_ARG  # Hkv without k
    assert call(n=1 << 30) == gca.GCA_ERR_INVALID_ARG
    assert call(B=65536, n=1) == gca.GCA_ERR_INVALID_ARG
    assert call(dh=300) == gca.GCA_ERR_UNSUPPORTED
    assert call(rot=63) == gca.GCA_ERR_INVALID_ARG
    assert call(rot=66) == gca.GCA_ERR_INVALID_ARG
    assert call(rot=0) == gca.GCA_ERR_INVALID_ARG
    assert call(freq=0) == gca.GCA_ERR_INVALID_ARG
    assert call(freq=FAKE + 4) == gca.GCA_ERR_INVALID_ARG
    assert call(pbs=-1) == gca.GCA_ERR_INVALID_ARG
    assert call(q=heads(gca, FAKE + 1)) == gca.GCA_ERR_INVALID_ARG
    assert call(q=heads(gca, ts=-64)) == gca.GCA_ERR_INVALID_ARG
    assert call(qo=heads(gca, hs=32)) == gca.GCA_ERR_INVALID_ARG  # heads overlap
    assert call(qo=heads(gca, ts=64, hs=64)) == gca.GCA_ERR_INVALID_ARG
    assert call(ko=heads(gca, bs=0)) == gca.GCA_ERR_INVALID_ARG
    assert b"overlap" in L.gca_last_error_detail()


def test_rotary_frequencies(gca):
    for rot, kw in ((64, {}), (2, {}), (40, dict(scaling="linear", factor=16.0)), (64, dict(scaling="ntk", factor=4.0, base=5e5)),
                    (2, dict(scaling="ntk", factor=4.0)), (128, dict(scaling="parts", factor=8.0, context=2048.0)),
                    (32, dict(scaling="parts", factor=8.0, context=8192.0, low=1.0, high=4.0))):
        got = gca.rotary_frequencies(rot, device="cpu", **kw).numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64 * 2 * math.pi
        want = orc.speeds(rot, **kw)
        # pow, a few products and the rounding to 2^-64 turns (6.3 2^-65 radians)
        assert np.all(np.abs(got - want) <= 16 * 2.0 ** -53 * want + 2.0 ** -62)
    for bad in (dict(rot=3), dict(rot=0), dict(rot=258), dict(rot=8, base=0.5), dict(rot=8, base=float("nan")),
                dict(rot=8, scaling="linear", factor=0.0), dict(rot=8, scaling="linear", factor=float("inf")),
                dict(rot=8, scaling="parts", factor=2.0, context=0.0), dict(rot=8, scaling="parts", factor=2.0, context=9.0, low=4.0, high=4.0)):
        with pytest.raises(gca.GCAError):
            gca.rotary_frequencies(device="cpu", **bad)
    with pytest.raises(ValueError):
        gca.rotary_frequencies(8, scaling="dynamic", device="cpu")


def test_cache_refusals(gca):
    L, E, U, W = gca.LIB, gca.GCA_ERR_INVALID_ARG, gca.GCA_ERR_UNSUPPORTED, gca.GCA_ERR_WORKSPACE

    def append(c=None, k=None, v=None, n=8, T=5, slots=None, counts=FAKE, ws=FAKE, wsb=256, sc=FAKE, scb=1 << 20):
        h = lambda x: x if x is not None else heads(gca, ts=256, bs=5 * 256)  # noqa: E731
        return L.gca_cache_append(c if c is not None else pool(gca), h(k), h(v), n, T, slots, counts, None, ws, wsb, sc, scb, None)
    for kw in (dict(k_pages=0), dict(v_pages=FAKE + 8), dict(dtype=9), dict(heads=0), dict(dh=0), dict(pages=0), dict(table=0),
               dict(slots=0), dict(width=0), dict(width=1 << 25), dict(lengths=0), dict(refs=0), dict(heads=1, dh=4)):
        assert append(c=pool(gca, **kw)) == E, kw
    assert append(n=0) == E and append(n=9) == E and append(n=1025, slots=FAKE) == E
    assert append(T=0) == E and append(counts=0) == E and append(n=1024, slots=FAKE, T=1 << 28) == E
    assert append(k=heads(gca, FAKE + 8)) == E and append(v=heads(gca, ts=257)) == E and append(k=heads(gca, hs=72)) == E
    assert append(ws=0) == W and append(wsb=8) == W and append(sc=0) == W and append(sc=FAKE + 16) == W
    assert append(scb=L.gca_cache_append_scratch_size(8, 5) - 1) == W
    assert L.gca_cache_fork(pool(gca), 2, None, FAKE, FAKE, 256, None) == E
    assert L.gca_cache_fork(pool(gca), 0, FAKE, FAKE, FAKE, 256, None) == E
    assert L.gca_cache_fork(pool(gca), 2, FAKE, FAKE, FAKE, 0, None) == W
    assert L.gca_cache_trim(pool(gca), 9, None, None, None, 0, FAKE, 256, None) == E
    assert L.gca_cache_trim(pool(gca, refs=0), 8, None, None, None, 0, FAKE, 256, None) == E
    assert L.gca_cache_compact(pool(gca), None, FAKE, 256, FAKE, 1 << 20, None) == E
    assert L.gca_cache_compact(pool(gca), FAKE, FAKE, 256, FAKE, 1024, None) == W
    assert L.gca_cache_lookup(pool(gca), 8, 0, None, FAKE, FAKE, FAKE, 256, None) == E
    assert L.gca_cache_lookup(pool(gca), 8, 4, None, None, FAKE, FAKE, 256, None) == E

    def attend(c=None, q=None, k=None, v=None, B=2, T=5, H=8, mask=None, window=0, scale=0.125, o=FAKE, lse=FAKE, wsb=256, scb=1 << 30):
        h = lambda x: x if x is not None else heads(gca)  # noqa: E731
        return L.gca_tree_attention(h(q), h(k), h(v), c if c is not None else pool(gca), B, T, H, mask, None, window, scale, o,
                                    lse, FAKE, wsb, FAKE, scb, None)
    assert attend(c=pool(gca, dh=96)) == U and attend(T=257) == U and attend(T=0) == U
    assert attend(B=0) == E and attend(B=9) == E and attend(H=6) == E and attend(H=2) == E
    assert attend(window=-1) == E and attend(scale=0.0) == E and attend(scale=-1.0) == E
    assert attend(scale=float("inf")) == E and attend(scale=float("nan")) == E
    assert attend(mask=FAKE + 4) == E and attend(o=0) == E and attend(o=FAKE + 4) == E and attend(lse=0) == E
    assert attend(q=heads(gca, FAKE + 2)) == E and attend(k=heads(gca, bs=4)) == E and attend(v=heads(gca, 0)) == E
    assert attend(k=heads(gca, ts=0)) == U and attend(v=heads(gca, ts=0)) == U  # one token repeated
    assert attend(c=pool(gca, heads=65535, width=1 << 24), H=65535) == U
    assert attend(wsb=0) == W and attend(scb=100) == W
    assert L.gca_tree_plan(FAKE, FAKE, 2, 257, FAKE, FAKE, FAKE, 256, None) == U
    assert L.gca_tree_plan(FAKE, FAKE, 0, 5, FAKE, FAKE, FAKE, 256, None) == E
    assert L.gca_tree_plan(0, FAKE, 2, 5, FAKE, FAKE, FAKE, 256, None) == E
    assert L.gca_tree_plan(FAKE, FAKE, 2, 5, FAKE + 4, FAKE, FAKE, 256, None) == E
    assert L.gca_status_string(gca.GCA_ERR_CACHE_FULL) == b"GCA_ERR_CACHE_FULL"


def test_binding_refuses_tensors_that_are_not_on_a_gpu(gca):
    x = torch.zeros(1, 1, 2, 64)
    with pytest.raises(ValueError):
        gca.rotary(x, None, torch.zeros(32, dtype=torch.int64))
    with pytest.raises(TypeError):
        gca.rotary(x.half(), None, torch.zeros(32, dtype=torch.int64))
    with pytest.raises(ValueError):
        gca.rotary(x, None, torch.zeros(32))
    pages, i = torch.zeros(4, 64, 2, 64), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        gca.PagedCache(pages, pages, torch.zeros(4, 2, dtype=torch.int32), i, i)
    with pytest.raises(ValueError):
        gca.PagedCache(pages[:, :32], pages, torch.zeros(4, 2, dtype=torch.int32), i, i)
    with pytest.raises(ValueError):
        gca.tree_attention(x, x, x, pages, pages, torch.zeros(4, 2, dtype=torch.int32), i)


def test_oracle_pages_keep_their_tokens():
    """The model's own rule: a slot's tokens are what was appended to it, whatever is forked,
    trimmed, freed or compacted around it."""
    rng = np.random.default_rng(0)
    m = orc.Pages(np.zeros((40, 64, 1, 1)), np.zeros((40, 64, 1, 1)), np.full((4, 6), -1), np.zeros(4, int), np.zeros(40, int))
    held = [[], [], [], []]
    for step in range(80):
        s = int(rng.integers(4))
        kind = rng.integers(4)
        if kind < 2:
            T = int(rng.integers(1, 60))
            counts = [int(min(rng.integers(0, T + 1), 384 - len(h))) if i == s else 0 for i, h in enumerate(held)]
            rows = rng.normal(size=(4, T, 1, 1))
            m.append(rows, rows, counts)
            if not m.full:
                held[s] += list(rows[s, :counts[s], 0, 0])
        elif kind == 2:
            cut = int(rng.integers(0, len(held[s]) + 1))
            m.trim(end=[cut], slots=[s])
            held[s] = held[s][:cut]
            m.compact()
        else:
            d = int(rng.integers(4))
            if d != s and not held[d]:
                m.fork([s], [d])
                held[d] = list(held[s])
        assert not m.flagged and not m.full
        for i in range(4):
            assert list(m.tokens(i).reshape(-1)) == held[i]
        counted = np.bincount(m.table[m.table >= 0], minlength=40)
        assert np.array_equal(counted, m.refs)


def test_oracle_attention_is_the_softmax_of_what_is_seen():
    rng = np.random.default_rng(1)
    see, pos = orc.tree([-1, 0, 0, -2, 2], 70)
    assert pos.tolist() == [70, 71, 71, -1, 72] and see[4].tolist() == [True, False, True, False, True]
    assert orc.pack_mask(see[None])[0, :, 0].tolist() == [1, 3, 5, 0, 21]
    k, v, q = rng.normal(size=(3, 64, 1, 4)), rng.normal(size=(3, 64, 1, 4)), rng.normal(size=(1, 5, 2, 4))
    kn, vn = rng.normal(size=(1, 5, 1, 4)), rng.normal(size=(1, 5, 1, 4))
    o, lse, *_ = orc.tree_attention(q, kn, vn, k, v, np.array([[2, 0]]), [70], see[None], pos[None], window=4)
    keys = np.concatenate([k[0, 5:6, 0], kn[0, [0, 2, 4], 0]])  # token 72 sees positions 69 to 72
    vals = np.concatenate([v[0, 5:6, 0], vn[0, [0, 2, 4], 0]])
    e = np.exp(keys @ q[0, 4, 1] / 2)
    assert np.allclose(o[0, 4, 1], e @ vals / e.sum()) and np.isclose(lse[0, 4, 1], np.log(e.sum()))
    assert not o[0, 3].any() and np.all(lse[0, 3] == -np.inf)


def test_oracle_rotary():
    x = np.random.default_rng(2).normal(size=(1, 2, 1, 6))
    w = orc.speeds(4)
    y = orc.rotary(x, np.array([[0, 7]]), w, gain=2.0)
    assert np.allclose(y[0, 0, 0, :4], 2 * x[0, 0, 0, :4]) and np.array_equal(y[..., 4:], x[..., 4:])
    z = (x[0, 1, 0, 1] + 1j * x[0, 1, 0, 3]) * np.exp(7j * w[1]) * 2
    assert np.allclose([y[0, 1, 0, 1], y[0, 1, 0, 3]], [z.real, z.imag])
    back = orc.rotary(y, np.array([[0, 7]]), w, gain=0.5, backward=True)
    assert np.allclose(back, x)


class Recorder:
    """Stands in for the native binding: keeps the arguments of the last call."""

    def __getattr__(self, name):
        def call(*args):
            self.__dict__["last"] = args
            return b"kept"
        return call


def test_paged_cache_hands_over_the_tensors_that_it_shows(gca, monkeypatch):
    """Every call gets the cache's tensors as they are at that call: of a deep copy or an unpickled
    cache its own, after an assignment the new one.  (Addresses kept from an earlier time would be
    those of another cache, or of memory that was given back.)"""
    import copy
    import pickle
    from retrieval_sparse_attention_causal_gb300 import decoding
    rec = Recorder()
    monkeypatch.setattr(decoding, "EXT", rec)
    names = ("k_pages", "v_pages", "table", "lengths", "refs")
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    pages = torch.zeros(4, 64, 2, 64)
    cache = gca.PagedCache(pages, pages.clone(), i(3, 2), i(3), i(4))
    x = torch.zeros(3, 1, 2, 64)

    def handed_over(c):
        for call, at in ((lambda: c.append(x, x, i(3)), 0), (lambda: c.fork(i(1), i(1)), 0), (lambda: c.trim(end=i(3)), 0),
                         (c.free, 0), (c.compact, 0), (lambda: c.lookup(i(3, 1)), 0), (lambda: c.attention(x, x, x), 3)):
            call()
            for n, t in zip(names, rec.last[at:at + 5]):
                assert t is getattr(c, n), n

    handed_over(cache)
    for twin in (copy.deepcopy(cache), pickle.loads(pickle.dumps(cache))):
        assert all(getattr(twin, n).data_ptr() != getattr(cache, n).data_ptr() for n in names)
        handed_over(twin)
    cache.table, cache.k_pages, cache.v_pages, cache.refs = i(3, 9), torch.zeros(8, 64, 2, 64), torch.zeros(8, 64, 2, 64), i(8)
    handed_over(cache)


def test_oracle_compact_clears_entries_that_name_free_pages():
    m = orc.Pages(np.arange(6.0).reshape(6, 1, 1, 1) * np.ones((6, 64, 1, 1)), np.zeros((6, 64, 1, 1)),
                  np.array([[5, 1, -1], [3, 0, 9]]), np.array([128, 64]), np.array([0, 1, 0, 1, 0, 1]))
    assert m.compact() == 3  # pages 3 and 5 move to 0 and 2; the entry with 0 named a free page, 9 no page
    assert m.flagged and m.table.tolist() == [[2, 1, -1], [0, -1, -1]] and m.refs.tolist() == [1, 1, 1, 0, 0, 0]
    assert m.k[:3, 0, 0, 0].tolist() == [3.0, 1.0, 5.0]


def test_the_extension_is_built_again_for_another_torch(gca, monkeypatch, tmp_path):
    """An extension fits the torch and the Python that it was compiled for; where one of them changed,
    build() compiles it again, and the C library is linked before a compiler's failure there is raised."""
    import os
    import subprocess
    from retrieval_sparse_attention_causal_gb300 import build as b
    out, torch_dir = tmp_path / "_build", tmp_path / "torch"
    out.mkdir(), torch_dir.mkdir()
    (torch_dir / "version.py").write_text("__version__ = '1'\n")
    fake = lambda name: type("Spec", (), {"submodule_search_locations": [str(torch_dir)]})()  # noqa: E731
    monkeypatch.setattr(b.importlib.util, "find_spec", fake)
    for n, f in (("BUILD", out), ("LIB", out / "libgca.so"), ("EXT", out / "_gca_decoding.so")):
        monkeypatch.setattr(b, n, str(f))
    made, broken = [], []

    def run(cmd, **kw):
        target = os.path.basename(cmd[cmd.index("-o") + 1])
        made.append(target)
        if target in broken:
            return subprocess.CompletedProcess(cmd, 1, "", "")
        (out / target).write_text("")
        return subprocess.CompletedProcess(cmd, 0, "", "")
    monkeypatch.setattr(b.subprocess, "run", run)
    b.build()
    assert sorted(made) == sorted([s.replace(".cu", ".o") for s in b.SOURCES] + ["binding.o", "libgca.so", "_gca_decoding.so"])
    made.clear()
    b.build()
    assert made == []
    (torch_dir / "version.py").write_text("__version__ = '2'\n")
    b.build()
    assert made == ["binding.o", "_gca_decoding.so"]
    made.clear()
    (torch_dir / "version.py").write_text("__version__ = '3'\n")
    (out / "libgca.so").unlink()
    broken.append("binding.o")
    with pytest.raises(RuntimeError):
        b.build()
    assert "libgca.so" in made and "_gca_decoding.so" not in made
    broken.clear(), made.clear()
    b.build()
    assert made == ["binding.o", "_gca_decoding.so"]


def test_a_link_that_failed_is_made_up_for(gca, monkeypatch, tmp_path):
    """An extension whose source was compiled anew but not linked is not taken for a current one."""
    import os
    import subprocess
    from retrieval_sparse_attention_causal_gb300 import build as b
    monkeypatch.setattr(b, "BUILD", str(tmp_path))
    for n in ("libgca.so", "_gca_decoding.so"):
        monkeypatch.setattr(b, {"libgca.so": "LIB"}.get(n, "EXT"), str(tmp_path / n))
    made, broken = [], []

    def run(cmd, **kw):
        target = os.path.basename(cmd[cmd.index("-o") + 1])
        made.append(target)
        if target not in broken:
            (tmp_path / target).write_text("")
        return subprocess.CompletedProcess(cmd, int(target in broken), "", "")
    monkeypatch.setattr(b.subprocess, "run", run)
    b.build()
    os.utime(tmp_path / "binding.o", (0, 0))  # as after a change of the source
    broken.append("_gca_decoding.so")
    with pytest.raises(RuntimeError):
        b.build()
    broken.clear(), made.clear()
    b.build()
    assert "_gca_decoding.so" in made


@pytest.mark.parametrize("broken", [False, True])
def test_the_library_imports_without_the_extension(gca, broken, tmp_path):
    """Without the extension (or with one that does not load) everything but the decoding operators is
    there, and those say what is missing."""
    import os
    import shutil
    import subprocess
    import sys
    src = os.path.dirname(gca.__file__)
    pkg = tmp_path / os.path.basename(src)
    shutil.copytree(src, pkg, ignore=shutil.ignore_patterns("_build", "csrc", "__pycache__"))
    (pkg / "_build").mkdir()
    (pkg / "_build" / "libgca.so").symlink_to(gca.LIB_PATH)
    if broken:
        (pkg / "_build" / "_gca_decoding.so").write_text("not a library")
    code = ("import torch, %s as g\n"
            "assert g.LIB.gca_forward_workspace_size() == 256 and g.gca_forward and g.retrieve_topk\n"
            "assert g.rotary_frequencies(8, device='cpu').shape == (4,)\n"
            "try:\n g.tree_plan(torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))\n"
            "except ImportError as e:\n assert '_gca_decoding' in str(e)\n"
            "else:\n raise SystemExit('no error')\n" % pkg.name)
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


@pytest.mark.parametrize("rot,kw", [(64, {}), (128, dict(base=5e5)), (128, dict(scaling="linear", factor=16.0)),
                                    (64, dict(scaling="ntk", factor=4.0)), (4, dict(scaling="ntk", factor=32.0, base=1e6)),
                                    (128, dict(scaling="parts", factor=8.0, context=8192.0)),
                                    (256, dict(scaling="parts", factor=32.0, context=2048.0, low=1.0, high=4.0))])
def test_rotary_frequencies_against_many_digits(gca, rot, kw):
    """Each speed is within 2^-49 radians a position of its value, as documented.  In units of 2^-53, with
    x = 2i / rot and w = base^-x <= 1: the rounding of x in the power w x ln(base) <= 1/e, pow itself 2 w; of
    an NTK base its own error (its power of factor: (ln factor e + 3)) times w x, at most 10 for what is below;
    by parts c is off by (4 high + low) / (high - low) <= 6, of which 1 - 1 / factor counts, and three products
    and a sum round; the division by 2 pi and its own rounding 3 w.  Together below 16.  The integer is off by a half, 2^-65
    turns."""
    mp = pytest.importorskip("mpmath")
    with mp.workdps(60):
        f = lambda x: mp.mpf(float(x))  # noqa: E731
        base, factor = f(kw.get("base", 10000.0)), f(kw.get("factor", 1.0))
        scaling = kw.get("scaling")
        got = gca.rotary_frequencies(rot, device="cpu", **kw).tolist()
        if scaling == "ntk":
            base *= factor ** (mp.mpf(rot) / (rot - 2))
        for i in range(rot // 2):
            w = base ** (-2 * mp.mpf(i) / rot)
            if scaling == "linear":
                w /= factor
            if scaling == "parts":
                low, high = f(kw.get("low", 1.0)), f(kw.get("high", 32.0))
                c = min(mp.mpf(1), max(mp.mpf(0), (f(kw["context"]) * w / (2 * mp.pi) - low) / (high - low)))
                w = c * w + (1 - c) * w / factor
            assert abs(mp.mpf(got[i]) * 2 * mp.pi / 2 ** 64 - w) <= mp.mpf(2) ** -49, (i, w)


def test_attention_refuses_tables_whose_positions_pass_31_bits(gca):
    """A draft behind a full table of 2^25 - 1 pages would lie at positions above 2^31 - 1."""
    def attend(width):
        return gca.LIB.gca_tree_attention(heads(gca), heads(gca), heads(gca), pool(gca, width=width), 2, 5, 8, None, None, 0, 0.125,
                                          FAKE, FAKE, FAKE, 256, FAKE, 0, None)  # no scratch: nothing is launched
    assert attend((1 << 25) - 1) == gca.GCA_ERR_UNSUPPORTED and attend((1 << 25) - 4) == gca.GCA_ERR_UNSUPPORTED
    assert attend((1 << 25) - 5) == gca.GCA_ERR_WORKSPACE
