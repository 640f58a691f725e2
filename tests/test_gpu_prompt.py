"""GPU parity of a prompt's operators (attention over packed sequences with its gradients, norms with
rotary positions, the quantised cache) against the float64 oracle, and their use together.

Tolerances count roundings.  u = 2^-24 is float32's half step, h the output type's (bf16 2^-8,
float32 2^-24); bf16 operands of a product that were rounded for it (P and dS) are off by 2^-8 of
themselves.
"""
import numpy as np
import pytest
import torch

import oracle.decode_oracle as dorc
import oracle.prompt_oracle as orc
from retrieval_sparse_attention_causal_gb300 import pipeline, synth
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


def offsets_of(lengths, first=0):
    return np.concatenate([[first], first + np.cumsum(lengths)]).astype(np.int64)


def within(got, ref, lim, what):
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    there = ~np.isnan(ref)
    assert not np.isnan(got[there]).any(), f"{what}: NaN"
    over = np.abs(got[there] - ref[there]) - np.broadcast_to(lim, ref.shape)[there]
    assert over.size == 0 or over.max() <= 0, f"{what}: {int((over > 0).sum())} of {over.size} beyond the bound by {over.max():.3g}"


# ------------------------------------------------------------------ packed sequences
def prompt_bounds(r, dtype, dh, longest, g, scale=None):
    """What the outputs of a call may be off.  A logit: dh + 8 roundings of its products' sum, the scale
    and the reference, all relative to scale sum |q||k| (s_abs).  An exponential: 2^-22 of itself from
    the hardware's, and what its argument is off.  So p is off by c of itself: its own logit and the
    sum's, the sum's n roundings.  Then o: bf16 rounds p for the product (2^-8), n + 16 roundings of the
    sum, and the output's rounding; D = <do, o> takes o as it was rounded.  The gradients: c for p, dh
    roundings of <do, v> and of D, bf16 rounds P or dS for the product, n g roundings of the sum (dq
    and dk have the scale's too), and the output's rounding."""
    h, p8 = HALF[dtype], 1.02 * (2.0 ** -8 if dtype == "bf16" else 0.0)
    # (a bound for all rows: the largest logit's)
    ds = (dh + 8) * U * np.nanmax(r["s_abs"]) + 8 * U
    c = 2 * ds + (longest + 16) * U
    lim = dict(lse=ds + (longest + 16) * U + 4 * U * np.abs(r["lse"]),
               o=h * np.abs(r["o"]) + r["o_abs"] * (p8 + 1.02 * c))
    if "dq" in r:
        e = 2 * c + (longest * g + 4 * dh + 32) * U
        for name, extra in (("dq", 1.02 * h), ("dk", 1.02 * h), ("dv", 0.0)):
            lim[name] = h * np.abs(r[name]) + r[name + "_abs"] * (p8 + 1.02 * e + extra) + 1e-30
    return lim


CASES = [  # lengths, H, Hkv, dh, window, dtype
    ((1,), 1, 1, 64, 0, "bf16"),
    ((77,), 12, 12, 64, 0, "bf16"),
    ((128,), 2, 1, 64, 0, "bf16"),
    ((129, 0, 1, 64), 2, 2, 64, 0, "bf16"),
    ((256, 255, 257), 3, 1, 64, 0, "bf16"),
    ((300, 5, 0, 641), 4, 2, 128, 0, "bf16"),
    ((130, 700), 3, 3, 128, 0, "bf16"),
    ((60, 200), 8, 2, 32, 0, "bf16"),
    ((900,), 5, 1, 32, 100, "bf16"),
    ((1000, 30), 4, 4, 64, 1, "bf16"),
    ((513, 640), 4, 1, 64, 128, "bf16"),
    ((777,), 2, 2, 64, 129, "bf16"),
    ((600, 600), 6, 3, 128, 300, "bf16"),
    ((1500,), 2, 1, 64, 1000, "bf16"),
    (tuple([3, 70] * 40), 2, 2, 64, 0, "bf16"),
    (tuple([130, 0, 1, 260] * 17), 2, 1, 64, 50, "bf16"),
    (tuple([100, 300, 20] * 20), 5, 5, 64, 0, "bf16"),
    (tuple([300, 40] * 40), 3, 1, 128, 60, "bf16"),
    (tuple([400, 128] * 30), 7, 7, 32, 200, "bf16"),
    ((1,), 1, 1, 32, 0, "f32"),
    ((64, 65, 0, 63), 2, 1, 64, 0, "f32"),
    ((200, 3), 6, 2, 32, 0, "f32"),
    ((150, 90), 3, 3, 128, 40, "f32"),
    (tuple([5, 66] * 20), 2, 1, 64, 7, "f32"),
]


@pytest.mark.parametrize("lengths,H,Hkv,dh,window,dtype", CASES)
def test_prompt_attention_against_oracle(lengths, H, Hkv, dh, window, dtype):
    """Outputs, log-sum-exps and gradients; rows in front of the first sequence and behind the last, which
    hold NaN, reach nothing and stay as they were."""
    g = _g()
    off = offsets_of(lengths, 3)
    N = int(off[-1]) + 5
    q, k, v, do = (synth.normal(21, s, (N, h, dh), 1.0, dtype) for s, h in ((0, H), (1, Hkv), (2, Hkv), (3, H)))
    r = orc.prompt_attention(q, k, v, off, window, dout=do)
    for x in (q, k, v, do):
        x[:3] = x[off[-1]:] = np.nan
    qd, kd, vd, dod = (dev(x, dtype) for x in (q, k, v, do))
    o = torch.full((N, H, dh), 7.0, dtype=TORCH[dtype], device="cuda")
    lse = torch.full((N, H), 7.0, device="cuda")
    got = dict(zip(("o", "lse"), g.prompt_attention(qd, kd, vd, ints(off), window=window, out=o, lse=lse)))
    grads = [torch.full_like(x, 7.0) for x in (qd, kd, vd)]
    got.update(zip(("dq", "dk", "dv"), g.prompt_attention_backward(qd, kd, vd, o, dod, lse, ints(off), window=window,
                                                                   dq=grads[0], dk=grads[1], dv=grads[2])))
    lim = prompt_bounds(r, dtype, dh, max(lengths), H // Hkv)
    for name, x in got.items():
        x = host(x)
        within(x, r[name], lim[name], name)
        assert (x[:3] == 7).all() and (x[off[-1]:] == 7).all(), f"{name}: rows of no sequence were written"


@pytest.mark.parametrize("dtype,dh", [("bf16", 64), ("bf16", 128), ("bf16", 32), ("f32", 64)])
def test_prompt_sequences_do_not_reach_each_other(dtype, dh):
    """NaN and infinities in one sequence leave the others' results as they were, to the bit."""
    g = _g()
    lengths = (130, 60, 300, 1, 90)
    off = offsets_of(lengths)
    N, H = int(off[-1]), 2
    x = [dev(synth.normal(22, s, (N, H, dh), 1.0, dtype), dtype) for s in range(4)]
    run = lambda q, k, v, do: (lambda o, lse: (o, lse) + g.prompt_attention_backward(q, k, v, o, do, lse, ints(off)))(  # noqa: E731
        *g.prompt_attention(q, k, v, ints(off)))
    want = run(*x)
    for b in (0, 2, 4):
        bad = [t.clone() for t in x]
        for t, value in zip(bad, (float("nan"), float("inf"), float("nan"), float("-inf"))):
            t[off[b]:off[b + 1]] = value
        for w, got in zip(want, run(*bad)):
            rest = torch.ones(N, dtype=torch.bool)
            rest[off[b]:off[b + 1]] = False
            assert torch.equal(w[rest], got[rest])


@pytest.mark.parametrize("dtype,dh", [("bf16", 64), ("bf16", 128), ("f32", 32)])
def test_prompt_large_logits(dtype, dh):
    """Logits that grow by hundreds along a sequence, and fall again: references that are outgrown."""
    g = _g()
    n, H = 700, 2
    q, k, v, do = (synth.normal(23, s, (n, H, dh), 1.0, dtype) for s in range(4))
    k = k * np.concatenate([np.linspace(0.1, 12, n // 2), np.linspace(12, 0.01, n - n // 2)])[:, None, None]
    k = host(dev(k, dtype))
    q[:, :, 0] = 4.0
    k[::-1, :, 0] += np.linspace(0, 60, n)[:, None] * (np.arange(n)[:, None] % 97 == 0)
    k = host(dev(k, dtype))
    off = offsets_of((n,))
    r = orc.prompt_attention(q, k, v, off, 0, dout=do)
    d = [dev(x, dtype) for x in (q, k, v, do)]
    o, lse = g.prompt_attention(*d[:3], ints(off))
    dq, dk, dv = g.prompt_attention_backward(*d[:3], o, d[3], lse, ints(off))
    lim = prompt_bounds(r, dtype, dh, n, 1)
    for name, x in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk), ("dv", dv)):
        within(host(x), r[name], lim[name], name)


@pytest.mark.parametrize("dtype,dh", [("bf16", 64), ("bf16", 128), ("f32", 64)])
def test_prompt_single_tokens_have_no_gradient(dtype, dh):
    """A row that sees itself alone has dS = 0.  What is left: P = 1 to a logit's roundings, 2 (dh + 8) u |s| <= 5e-4
    for |s| <= 30, times <do, v> - D with D of the rounded output, 2^-8 dh |do v| <= 4, times scale |k| <= 1 / 2."""
    g = _g()
    N, H = 70, 3
    q, k, v, do = (torch.randn(N, H, dh, device="cuda").to(TORCH[dtype]) for _ in range(4))
    off = ints(np.arange(N + 1))
    o, lse = g.prompt_attention(q, k, v, off)
    assert torch.equal(o, v)
    dq, dk, dv = g.prompt_attention_backward(q, k, v, o, do, lse, off)
    assert float(dq.abs().max()) <= 1e-3 and float(dk.abs().max()) <= 1e-3
    assert float((dv.float() - do.float()).abs().max()) <= 2 * HALF[dtype] * float(do.abs().max()) + 1e-6


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_views_scale_and_gradients_into_views(dtype):
    """Views of a fused projection, heads-first storage, one key head repeated, a scale of its own, and
    gradients into the views of one tensor give what contiguous tensors give."""
    g = _g()
    lengths = (140, 33)
    off, H, Hkv, dh = offsets_of(lengths), 4, 2, 64
    N = int(off[-1])
    qkv = torch.randn(N, H + 2 * Hkv, dh, device="cuda").to(TORCH[dtype])
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    do = torch.randn(N, H, dh, device="cuda").to(TORCH[dtype])
    c = [x.contiguous() for x in (q, k, v)]
    want = g.prompt_attention(*c, ints(off), scale=0.3)
    gwant = g.prompt_attention_backward(*c, want[0], do, want[1], ints(off), scale=0.3)
    got = g.prompt_attention(q, k, v, ints(off), scale=0.3)
    dqkv = torch.zeros_like(qkv)
    g.prompt_attention_backward(q, k, v, got[0], do.transpose(0, 1).contiguous().transpose(0, 1), got[1], ints(off), scale=0.3,
                                dq=dqkv[:, :H], dk=dqkv[:, H:H + Hkv], dv=dqkv[:, H + Hkv:])
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    assert torch.equal(dqkv, torch.cat(gwant, dim=1))
    turned = [x.transpose(0, 1).contiguous().transpose(0, 1) for x in c]
    assert torch.equal(g.prompt_attention(*turned, ints(off), scale=0.3)[0], want[0])
    one = [x[:, :1].expand(N, H, dh) for x in c[1:]]
    a, _ = g.prompt_attention(c[0], *one, ints(off))
    b, _ = g.prompt_attention(c[0], *(x.contiguous() for x in one), ints(off))
    assert torch.equal(a, b)


def test_prompt_outputs_between_and_over_others():
    """Outputs in the gaps of a tensor's rows are taken, those that share an element with an input or with another
    output are refused, and nothing of such a call is written."""
    g = _g()
    N, H, Hkv, dh = 70, 4, 2, 64
    off = ints([0, 30, 70])
    room = torch.randn(N, H + 2 * Hkv + H + 2 * Hkv, dh, device="cuda").bfloat16()  # inputs and gradients in turn, token by token
    at = np.cumsum([0, H, Hkv, Hkv, H, Hkv, Hkv])
    q, k, v, dq, dk, dv = (room[:, a:z] for a, z in zip(at, at[1:]))
    do = torch.randn(N, H, dh, device="cuda").bfloat16()
    c = [x.clone() for x in (q, k, v)]
    o, lse = g.prompt_attention(*c, off)
    want = g.prompt_attention_backward(*c, o, do, lse, off)
    got = g.prompt_attention_backward(q, k, v, o, do, lse, off, dq=dq, dk=dk, dv=dv)
    assert all(torch.equal(a, b) for a, b in zip(want, got)) and all(torch.equal(a, b) for a, b in zip(c, (q, k, v)))
    first = torch.randn(H + 2 * Hkv, N, dh, device="cuda").bfloat16().transpose(0, 1)  # heads first: each tensor a block
    for x, y in zip((first[:, :H], first[:, H:H + Hkv], first[:, H + Hkv:]), want):
        x.copy_(y + 1)
    grads = (first[:, :H], first[:, H:H + Hkv], first[:, H + Hkv:])
    assert all(torch.equal(a, b) for a, b in zip(want, g.prompt_attention_backward(*c, o, do, lse, off, dq=grads[0], dk=grads[1], dv=grads[2])))
    line = torch.randn(3 * N * H * dh, device="cuda").bfloat16()
    piece = lambda e, h=H: line[e:e + N * h * dh].view(N, h, dh)  # noqa: E731
    n = N * H * dh
    assert torch.equal(g.prompt_attention(piece(0), *c[1:], off, out=piece(n))[0], g.prompt_attention(piece(0).clone(), *c[1:], off)[0])
    before = line.clone(), room.clone(), o.clone(), lse.clone()
    for call in (lambda: g.prompt_attention(piece(0), *c[1:], off, out=piece(64)), lambda: g.prompt_attention(piece(n), *c[1:], off, out=piece(8)),
                 lambda: g.prompt_attention(c[0], piece(n - 8, Hkv), c[2], off, out=piece(0)),
                 lambda: g.prompt_attention(*c, off, out=piece(0), lse=line[n - 2:n - 2 + 2 * N * H].view(torch.float32).view(N, H)),
                 lambda: g.prompt_attention_backward(*c, o, do, lse, off, dq=piece(0), dk=piece(n - 64, Hkv)),
                 lambda: g.prompt_attention_backward(*c, o, do, lse, off, dq=room[:, :H], dv=room[:, H - 1:H - 1 + Hkv]),
                 lambda: g.prompt_attention_backward(q, k, v, o, do, lse, off, dk=room[:, 1:1 + Hkv]),
                 lambda: g.prompt_attention_backward(*c, piece(0), do, lse, off, dv=piece(n - 8, Hkv)),
                 lambda: g.prompt_attention_backward(*c, o, do, lse, off, dk=do[:, 1:1 + Hkv])):
        with pytest.raises(g.GCAError) as e:
            call()
        assert e.value.status == g.GCA_ERR_INVALID_ARG
    assert all(torch.equal(a, b) for a, b in zip(before, (line, room, o, lse)))


def test_prompt_calls_are_equal_and_follow_the_device():
    """Equal calls give equal bits; on another stream too; and a captured pass follows offsets and inputs that
    change behind it."""
    g = _g()
    H, Hkv, dh, N = 4, 2, 64, 900
    q, k, v, do = (torch.randn(N, h, dh, device="cuda").bfloat16() for h in (H, Hkv, Hkv, H))
    off = ints([0, 400, 400, 900])

    def step():
        o, lse = g.prompt_attention(q, k, v, off, window=200)
        return (o, lse) + g.prompt_attention_backward(q, k, v, o, do, lse, off, window=200)
    want = step()
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(want, step()))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    graphs = []
    for _ in range(2):  # two graphs share no scratch
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        graphs.append((graph, out))
    off.copy_(ints([0, 1, 877, 900]))
    q.copy_(torch.randn_like(q))
    want = step()
    for graph, _ in graphs:
        graph.replay()
    for _, out in graphs:
        assert all(torch.equal(a, b) for a, b in zip(want, out))


def test_prompt_gradient_against_differences():
    """(f(x + e d) - f(x - e d)) / 2e against <gradient, d>, f = <dout, o>, float32, e = 2^-6.  The difference's
    truncation is e^2 / 6 of a third derivative of order |f|; rounding leaves 2^-24 n dh |f| / e.  Both are
    far below 1e-2 of |f| here."""
    g = _g()
    off = ints([0, 30, 75])
    x = [torch.from_numpy(synth.normal(24, s, (75, h, 32))).float().cuda() for s, h in ((0, 4), (1, 2), (2, 2))]
    do = torch.from_numpy(synth.normal(24, 3, (75, 4, 32))).float().cuda()
    o, lse = g.prompt_attention(*x, off, window=20)
    grads = g.prompt_attention_backward(*x, o, do, lse, off, window=20)
    f = lambda y: (g.prompt_attention(*y, off, window=20)[0].double() * do.double()).sum()  # noqa: E731
    e = 2.0 ** -6
    size = (o.double() * do.double()).abs().sum()
    for i in range(3):
        d = torch.from_numpy(synth.normal(25, i, x[i].shape)).float().cuda()
        up, down = ([t + s * e * d if j == i else t for j, t in enumerate(x)] for s in (1, -1))
        left, right = (f(up) - f(down)) / (2 * e), (grads[i].double() * d.double()).sum()
        assert abs(float(left - right)) <= 1e-2 * float(size) * e + 1e-3 * abs(float(right)), (i, float(left), float(right))


@flags
def test_prompt_bad_offsets_are_flagged():
    """A sequence whose offsets are out of order or of range is left out; the others are right."""
    g = _g()
    q, k, v = (torch.randn(300, 2, 64, device="cuda").bfloat16() for _ in range(3))
    want, _ = g.prompt_attention(q, k, v, ints([100, 200]))
    for off in ([0, -5, 100, 200], [100, 200, 301], [100, 200, 150], [100, 200, 2 ** 31 - 1]):
        got, _ = g.prompt_attention(q, k, v, ints(off))
        assert torch.equal(got[100:200], want[100:200]), off
        with pytest.raises(g.GCAError) as e:
            g.cache_workspace("cuda").check()
        assert e.value.status == g.GCA_ERR_DEVICE_INDEX
    g.cache_workspace("cuda").check()


@flags
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_gradients_beside_bad_offsets(dtype):
    """Sequences beside those that are left out have their gradients, wherever the bad offsets lie."""
    g = _g()
    q, k, v, do = (torch.randn(300, 2, 64, device="cuda").to(TORCH[dtype]) for _ in range(4))

    def step(off):
        o, lse = torch.zeros_like(q), torch.zeros(300, 2, device="cuda")
        g.prompt_attention(q, k, v, ints(off), out=o, lse=lse)
        grads = [torch.zeros_like(q) for _ in range(3)]
        g.prompt_attention_backward(q, k, v, o, do, lse, ints(off), dq=grads[0], dk=grads[1], dv=grads[2])
        return [o, lse] + grads
    for off, there in (([0, 100, 400, 200, 300], [[0, 100], [200, 300]]), ([0, 70, -1, 50, 70, 300], [[70, 300]]),
                       ([250, 300, 0, 120, 120, 200], [[250, 300], [0, 120], [120, 200]])):
        got = step(off)
        with pytest.raises(g.GCAError):
            g.cache_workspace("cuda").check()
        for a, z in there:
            assert all(torch.equal(x[a:z], y[a:z]) for x, y in zip(got, step([a, z]))), (off, a, z)
    g.cache_workspace("cuda").check()


@flags
@pytest.mark.parametrize("dtype,dh", [("bf16", 64), ("bf16", 128), ("f32", 64)])
def test_prompt_gradients_of_sequences_out_of_order(dtype, dh):
    """Where offsets fall, the sequences on either side of the fall are right if they share no row, although
    those behind it start before the others: short and long ones, at even and odd rows."""
    g = _g()
    N, H = 700, 2
    q, k, v, do = (torch.randn(N, H, dh, device="cuda").to(TORCH[dtype]) for _ in range(4))

    def step(off):
        o, lse = torch.zeros_like(q), torch.zeros(N, H, device="cuda")
        g.prompt_attention(q, k, v, ints(off), out=o, lse=lse)
        grads = [torch.zeros_like(q) for _ in range(3)]
        g.prompt_attention_backward(q, k, v, o, do, lse, ints(off), dq=grads[0], dk=grads[1], dv=grads[2])
        return [o, lse] + grads
    for off in ([8, 12, 0, 4], [40, 60, 0, 0, 0, 20, 40], [9, 12, 5, 8, 1, 4], [401, 700, 2, 200, 203, 401], [403, 404, 400, 403, 130, 399],
                [600, 601, 300, 597, 1, 2, 300]):
        there = [(a, z) for a, z in zip(off, off[1:]) if a < z]
        for _ in range(2):
            got = step(off)
            with pytest.raises(g.GCAError):
                g.cache_workspace("cuda").check()
            rest = torch.ones(N, dtype=torch.bool, device="cuda")
            for a, z in there:
                rest[a:z] = False
                assert all(torch.equal(x[a:z], y[a:z]) for x, y in zip(got, step([a, z]))), (off, a, z)
            assert all((x[rest] == 0).all() for x in got), off
    g.cache_workspace("cuda").check()


@pytest.mark.parametrize("lengths,window,H,Hkv,dh", [
    ((2,) * 200, 0, 4, 4, 64), ((3, 5) * 60, 0, 4, 2, 64), ((17,) * 40, 0, 6, 2, 128), ((40, 90), 0, 8, 8, 32),
    ((700,), 2, 4, 4, 64), ((520, 300), 3, 6, 2, 128), ((700,), 4, 4, 1, 64), ((900,), 8, 4, 4, 64), ((640, 260), 16, 8, 2, 32)])
def test_prompt_gradients_of_rows_that_see_few_keys(lengths, window, H, Hkv, dh):
    """dS is rounded for its products and dq, dk as outputs, which leaves a relative error e; D from the rounded output
    instead of the right one makes it r (2.5 and 4.0e-3 with two keys, 2.36 and 2.50e-3 with sixteen).  Both by the formula
    in float64 with these roundings, on the same inputs; what the kernels add in float32 is 1e-5 of them, so they
    lie nearer to e than to r, over all rows and over those behind the first 128 of a sequence."""
    g = _g()
    off = offsets_of(lengths)
    N, rep, scale = int(off[-1]), H // Hkv, dh ** -0.5
    x = [dev(synth.normal(27, s, (N, h, dh), 1.0, "bf16"), "bf16") for s, h in ((0, H), (1, Hkv), (2, Hkv), (3, H))]
    o, lse = g.prompt_attention(*x[:3], ints(off), window=window)
    dq, dk, _ = g.prompt_attention_backward(*x[:3], o, x[3], lse, ints(off), window=window)
    b16 = lambda t: t.bfloat16().double()  # noqa: E731
    fold = lambda t, n: t.view(Hkv, rep, n, dh).sum(1)  # noqa: E731
    found = {}  # what: [got, right, raw], each with squares of (error, reference)
    for a, z in zip(off, off[1:]):
        n = int(z - a)
        q, k, v, do = (t[a:z].double().cpu().transpose(0, 1) for t in x)
        k, v = k.repeat_interleave(rep, 0), v.repeat_interleave(rep, 0)
        t = torch.arange(n)
        see = (t[None] <= t[:, None]) & ((t[None] > t[:, None] - window) if window else True)
        p = torch.softmax((q @ k.transpose(1, 2) * scale).masked_fill(~see, -float("inf")), 2)
        out, dp = p @ v, do @ v.transpose(1, 2)
        D = [(do * y).sum(2, keepdim=True) for y in (out, b16(out))]
        dS = [p * (dp - d) * scale for d in D]
        want = dS[0] @ k, fold(dS[0].transpose(1, 2) @ q, n)
        sides = [[(s[a:z].double().cpu().transpose(0, 1)) for s in (dq, dk)]]
        sides += [[b16(b16(s) @ k), b16(fold(b16(s).transpose(1, 2) @ q, n))] for s in dS]
        for name, i, first in (("dq", 0, 0), ("dk", 1, 0), ("dq behind", 0, 128), ("dk behind", 1, 128)):
            if n <= first:
                continue
            sums = found.setdefault(name, [[0.0, 0.0] for _ in range(3)])
            for s, side in zip(sums, sides):
                s[0] += float(((side[i] - want[i])[:, first:] ** 2).sum())
                s[1] += float((want[i][:, first:] ** 2).sum())
    for name, sums in found.items():
        got, right, raw = ((s / t) ** 0.5 for s, t in sums)
        assert got <= (right + raw) / 2, f"{name}: {got:.3e}, {right:.3e} with the right D, {raw:.3e} with the rounded output's"


def test_prompt_nothing_to_do():
    """No rows at all, and sequences that are all empty."""
    g = _g()
    q = torch.empty(0, 4, 64, device="cuda").bfloat16()
    o, lse = g.prompt_attention(q, q[:, :2], q[:, :2], ints([0, 0, 0]))
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    assert [x.shape[0] for x in g.prompt_attention_backward(q, q[:, :2], q[:, :2], o, q, lse, ints([0, 0]))] == [0, 0, 0]
    x = torch.ones(7, 4, 64, device="cuda").bfloat16()
    out, lse = torch.full_like(x, 3.0), torch.full((7, 4), 3.0, device="cuda")
    g.prompt_attention(x, x, x, ints([2, 2, 2]), out=out, lse=lse)
    assert (out == 3).all() and (lse == 3).all()
    grads = [torch.full_like(x, 3.0) for _ in range(3)]
    g.prompt_attention_backward(x, x, x, out, x, lse, ints([2, 2, 2]), dq=grads[0], dk=grads[1], dv=grads[2])
    assert all((t == 3).all() for t in grads)


def test_prompt_many_sequences_match_single_ones():
    """1024 sequences (the most) give what each gives by itself."""
    g = _g()
    rng = np.random.default_rng(5)
    lengths = rng.integers(0, 40, 1024)
    off = offsets_of(lengths)
    q, k, v = (torch.randn(int(off[-1]), h, 64, device="cuda").bfloat16() for h in (4, 2, 2))
    o, lse = g.prompt_attention(q, k, v, ints(off))
    for b in (0, 1, 31, 32, 511, 1022, 1023):
        a, z = int(off[b]), int(off[b + 1])
        if a == z:
            continue
        one, l1 = g.prompt_attention(q[a:z], k[a:z], v[a:z], ints([0, z - a]))
        assert torch.equal(one, o[a:z]) and torch.equal(l1, lse[a:z])


@pytest.mark.parametrize("B", [31, 32, 33, 128, 129, 1024])
@pytest.mark.parametrize("H,Hkv,dh,dtype", [(3, 1, 64, "bf16"), (5, 5, 128, "bf16"), (4, 2, 32, "bf16"), (2, 1, 64, "f32")])
def test_prompt_gradients_of_many_sequences_match_single_ones(B, H, Hkv, dh, dtype):
    """As many sequences as a warp has lanes, one more, and so on up to the most: outputs and gradients of each
    are those that it has by itself; a few are longer than a tile and some are empty.  (Float32's dk and dv are
    sums of parts whose number goes by the call's size: they are left to the tests against the oracle.)"""
    g = _g()
    lengths = np.random.default_rng(B).integers(0, 60, B)
    lengths[::9] *= 7
    off = offsets_of(lengths)
    N = int(off[-1])
    q, k, v, do = (torch.randn(N, h, dh, device="cuda").to(TORCH[dtype]) for h in (H, Hkv, Hkv, H))

    def step(q, k, v, do, off):
        o, lse = g.prompt_attention(q, k, v, off)
        return (o, lse) + g.prompt_attention_backward(q, k, v, o, do, lse, off)[:3 if dtype == "bf16" else 1]
    got = step(q, k, v, do, ints(off))
    for b in sorted({0, 1, 9, 27, 30, 31, 32, 33, 63, 64, 127, 128, B // 2, B - 2, B - 1}):
        if b >= B or lengths[b] == 0:
            continue
        a, z = int(off[b]), int(off[b + 1])
        for x, y in zip(got, step(q[a:z], k[a:z], v[a:z], do[a:z], ints([0, z - a]))):
            assert torch.equal(x[a:z], y), (b, z - a)


@pytest.mark.parametrize("H,Hkv,dtype,long", [(2, 2, "bf16", 33000), (2, 1, "bf16", 32640), (1, 1, "f32", 16400)])
def test_prompt_long_sequences_among_many(H, Hkv, dtype, long):
    """Sequences of 255 tiles and more behind the first 32, which a byte does not count, are what they are alone."""
    g = _g()
    lengths = np.full(70, 5)
    lengths[[34, 69]] = long, long - 200
    off = offsets_of(lengths)
    q, k, v, do = (torch.randn(int(off[-1]), h, 64, device="cuda").to(TORCH[dtype]) for h in (H, Hkv, Hkv, H))

    def step(q, k, v, do, off):
        o, lse = g.prompt_attention(q, k, v, off)
        return (o, lse) + g.prompt_attention_backward(q, k, v, o, do, lse, off)[:3 if dtype == "bf16" else 1]
    got = step(q, k, v, do, ints(off))
    for b in (0, 33, 34, 35, 68, 69):
        a, z = int(off[b]), int(off[b + 1])
        for x, y in zip(got, step(q[a:z], k[a:z], v[a:z], do[a:z], ints([0, z - a]))):
            assert torch.equal(x[a:z], y), b


# ------------------------------------------------------------------ norms with rotary positions
NORM = [  # B, L, H, Hkv, dh, rot, dtype, interleaved, eps
    (1, 1, 1, 1, 2, 2, "f32", False, 1e-6),
    (2, 5, 3, 1, 64, 64, "bf16", False, 1e-6),
    (1, 33, 12, 12, 64, 32, "bf16", True, 1e-5),
    (3, 17, 5, 1, 72, 40, "f32", False, 1e-6),
    (2, 9, 4, 2, 40, 6, "bf16", True, 1e-6),
    (1, 7, 2, 2, 50, 34, "bf16", False, 1e-6),
    (2, 3, 6, 3, 256, 256, "f32", True, 1e-6),
    (2, 3, 3, 1, 255, 2, "bf16", False, 1e-6),
    (2, 3, 3, 1, 256, 8, "bf16", True, 1e-6),
    (1, 700, 16, 4, 128, 96, "bf16", False, 0.0),
    (4, 1, 12, 12, 64, 64, "bf16", True, 1e-6),
    (2, 1500, 4, 2, 64, 64, "f32", False, 1e-6),
]


@pytest.mark.parametrize("B,L,H,Hkv,dh,rot,dtype,interleaved,eps", NORM)
def test_norm_rotary_against_oracle(B, L, H, Hkv, dh, rot, dtype, interleaved, eps):
    """The norm: dh + 8 roundings of the sum of squares halve through the root, its reciprocal 2 u, three
    products: (dh / 2 + 12) u of each element.  The rotation as in rotary's own test, relative to the pair's
    length r; bf16's rounding last.  Backward, mean(w u x r) sums dh terms more.  A weight's gradient sums
    n = B L heads terms, each off by as much, with n roundings (of a tree and short runs) at most."""
    g = _g()
    q, k = synth.normal(1, 0, (B, L, H, dh), 1.0, dtype), synth.normal(1, 1, (B, L, Hkv, dh), 1.0, dtype)
    dy = [synth.normal(1, 2 + i, x.shape, 1.0, dtype) for i, x in enumerate((q, k))]
    wt = [synth.normal(1, 4 + i, (dh,), 0.3, "f32") + 1.0 for i in range(2)]
    wt = [np.float32(x).astype(np.float64) for x in wt]
    pos = np.random.default_rng(3).integers(0, 1 << 24, (B, L))
    pos[0, 0] = (1 << 31) - 1
    w, gain = dorc.speeds(rot), 1.25
    args = (dev(wt[0], "f32"), dev(wt[1], "f32"), g.rotary_frequencies(rot))
    how = dict(positions=ints(pos), interleaved=interleaved, gain=gain, eps=eps)
    got = g.norm_rotary(dev(q, dtype), dev(k, dtype), *args, **how)
    back = g.norm_rotary_backward(dev(q, dtype), dev(k, dtype), dev(dy[0], dtype), dev(dy[1], dtype), *args, **how)
    i1 = np.arange(rot // 2) * 2 if interleaved else np.arange(rot // 2)
    i2 = i1 + 1 if interleaved else i1 + rot // 2
    ang = np.sqrt(2) * (np.pi * U / 2 + 6 * U + pos[:, :, None, None] * w * 2.0 ** -51)
    h = HALF[dtype]
    for i, (x, what) in enumerate(((q, "q"), (k, "k"))):
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + np.float64(np.float32(eps)))

        def turned(y):  # what the rotation adds to an element's error, and its size
            size, more = np.abs(y), np.zeros_like(y)
            pair = np.hypot(y[..., i1], y[..., i2])
            for at in (i1, i2):
                more[..., at] = gain * pair * ang
                size[..., at] = gain * pair
            return size, more
        ref = orc.norm_rotary(x, wt[i], pos, w, np.float64(np.float32(eps)), interleaved, gain)
        size, more = turned(x * r * wt[i])
        within(host(got[i]), ref, h * np.abs(ref) + (1 + h) * (more + 1.02 * (dh / 2 + 12) * U * size) + 1e-40, what)
        dref, dw = orc.norm_rotary_backward(x, dy[i], wt[i], pos, w, np.float64(np.float32(eps)), interleaved, gain)
        usize, umore = turned(dy[i])
        terms = r * np.abs(wt[i]) * usize
        dots = r * np.abs(x * r) * (np.abs(wt[i]) * usize * np.abs(x * r)).mean(-1, keepdims=True)
        e = 1.02 * (2 * dh + 30) * U
        extra = r * np.abs(wt[i]) * umore + r * np.abs(x * r) * (np.abs(wt[i]) * umore * np.abs(x * r)).mean(-1, keepdims=True)
        within(host(back[i]), dref, h * np.abs(dref) + (1 + h) * (extra + e * (terms + dots)) + 1e-40, "d" + what)
        n = B * L * x.shape[2]
        lim = (np.abs(x * r) * (umore + usize * 1.02 * (dh / 2 + 16 + n) * U)).sum((0, 1, 2))
        within(host(back[2 + i]), dw, lim + 1e-40, f"d{what}_weight")


@pytest.mark.parametrize("dtype,offset", [("bf16", 0), ("bf16", 1), ("f32", 0), ("f32", 1)])
def test_norm_rotary_views_and_in_place(dtype, offset):
    """Views of a fused projection (also at odd addresses), a broadcast key head, default and shared
    positions, no k, and the in-place forms give what contiguous tensors give; what lies around the views
    stays as it was.  (At an odd address sums run in another order: an ulp of float32, so bf16 may differ by
    one rounding and float32 by a few u.)"""
    g = _g()
    B, L, H, Hkv, dh, rot = 2, 11, 4, 2, 64, 48
    n = (H + 2 * Hkv) * dh
    raw = torch.randn(B * L * n + 8, device="cuda").to(TORCH[dtype])
    qkv = raw[offset:offset + B * L * n].view(B, L, H + 2 * Hkv, dh)
    q, k = qkv[:, :, :H], qkv[:, :, H:H + Hkv]
    freq, wt = g.rotary_frequencies(rot), [1 + 0.1 * torch.randn(dh, device="cuda") for _ in range(2)]
    same = lambda a, b: torch.allclose(a.float(), b.float(), rtol=2 * HALF[dtype] if offset == 1 else 0,  # noqa: E731
                                       atol=64 * U if offset == 1 else 0)
    want = g.norm_rotary(q.contiguous(), k.contiguous(), *wt, freq, positions=torch.arange(L, dtype=torch.int32, device="cuda"))
    got = g.norm_rotary(q, k, *wt, freq)
    assert same(got[0], want[0]) and same(got[1], want[1])
    assert same(g.norm_rotary(q, None, wt[0], None, freq)[0], want[0])
    one = k[:, :, :1].expand(B, L, 3, dh)
    assert same(g.norm_rotary(q, one, *wt, freq)[1], want[1][:, :, :1].expand(B, L, 3, dh))
    dy = [torch.randn_like(x) for x in want]
    grads = g.norm_rotary_backward(q.contiguous(), k.contiguous(), *dy, *wt, freq)
    mine = [x.clone() for x in dy]
    again = g.norm_rotary_backward(q.contiguous(), k.contiguous(), *mine, *wt, freq, dq=mine[0], dk=mine[1])
    assert all(torch.equal(a, b) for a, b in zip(grads, again)) and torch.equal(mine[0], grads[0])
    alone = g.norm_rotary_backward(q.contiguous(), None, dy[0], None, wt[0], None, freq)
    assert torch.equal(alone[0], grads[0]) and alone[1] is None and alone[3] is None
    before = raw.clone()
    g.norm_rotary(q, k, *wt, freq, q_out=q, k_out=k)
    assert torch.equal(q, got[0]) and torch.equal(k, got[1])
    rest = qkv[:, :, H + Hkv:]
    assert torch.equal(rest, before[offset:offset + B * L * n].view(B, L, -1, dh)[:, :, H + Hkv:])
    assert torch.equal(raw[:offset], before[:offset]) and torch.equal(raw[offset + B * L * n:], before[offset + B * L * n:])


def test_norm_rotary_outputs_between_and_over_others():
    """Outputs in the gaps of the inputs' rows and in place of the inputs (in the backward pass of either) are taken; each
    other's places, and shifted ones, are refused, and nothing is written."""
    g = _g()
    B, L, H, dh = 2, 9, 3, 64
    wt, freq = [torch.rand(dh, device="cuda") for _ in range(2)], g.rotary_frequencies(dh)
    room = torch.randn(B, L, 4 * H, dh, device="cuda").bfloat16()
    q, k, qo, ko = (room[:, :, i * H:(i + 1) * H] for i in range(4))
    c, dy = [q.clone(), k.clone()], [torch.randn(B, L, H, dh, device="cuda").bfloat16() for _ in range(2)]
    want, back = g.norm_rotary(*c, *wt, freq), g.norm_rotary_backward(*c, *dy, *wt, freq)
    assert all(torch.equal(a, b) for a, b in zip(want, g.norm_rotary(q, k, *wt, freq, q_out=qo, k_out=ko)))
    assert all(torch.equal(a, b) for a, b in zip(back, g.norm_rotary_backward(q, k, *dy, *wt, freq, dq=qo, dk=ko)))
    assert all(torch.equal(a, b) for a, b in zip(c, (q, k)))
    for i in range(2):  # in place of q and k, or of the gradients
        own = [x.clone() for x in c + dy]
        assert all(torch.equal(a, b) for a, b in zip(back, g.norm_rotary_backward(*own, *wt, freq, dq=own[2 * i], dk=own[2 * i + 1])))
    line = torch.randn(3 * B * L * H * dh, device="cuda").bfloat16()
    piece = lambda e: line[e:e + B * L * H * dh].view(B, L, H, dh)  # noqa: E731
    before = line.clone(), room.clone()
    for call in (lambda: g.norm_rotary(q, k, *wt, freq, q_out=k, k_out=q), lambda: g.norm_rotary(q, k, *wt, freq, k_out=q),
                 lambda: g.norm_rotary(piece(0), k, *wt, freq, q_out=piece(64)), lambda: g.norm_rotary(piece(64), None, wt[0], None, freq, q_out=piece(0)),
                 lambda: g.norm_rotary(q, k, *wt, freq, q_out=piece(0), k_out=piece(64)),
                 lambda: g.norm_rotary(q, k, *wt, freq, q_out=room[:, :, 1:1 + H]),
                 lambda: g.norm_rotary_backward(q, k, *dy, *wt, freq, dq=dy[1]), lambda: g.norm_rotary_backward(q, k, *dy, *wt, freq, dk=q),
                 lambda: g.norm_rotary_backward(q, k, piece(0), dy[1], *wt, freq, dq=piece(8))):
        with pytest.raises(g.GCAError) as e:
            call()
        assert e.value.status == g.GCA_ERR_INVALID_ARG
    assert all(torch.equal(a, b) for a, b in zip(before, (line, room)))


def test_norm_rotary_zero_rows():
    """A row of zeros: eps keeps it finite, and its gradient too."""
    g = _g()
    x = torch.zeros(1, 3, 2, 64, device="cuda").bfloat16()
    wt, freq = torch.ones(64, device="cuda"), g.rotary_frequencies(64)
    assert (g.norm_rotary(x, None, wt, None, freq)[0] == 0).all()
    dq, _, dw, _ = g.norm_rotary_backward(x, None, torch.ones_like(x), None, wt, None, freq)
    assert torch.isfinite(dq.float()).all() and (dw == 0).all()


# ------------------------------------------------------------------ the quantised cache
def numbers(cache):
    """Values of the cache's pages in float64, from their bytes."""
    k, v, ke, ve = cache.numbers()
    return [x.double().cpu().numpy() * 2.0 ** (e.long().cpu().numpy()[..., None] - 127.0) for x, e in ((k, ke), (v, ve))]


def expected(x):
    y, e = orc.quantise(x)
    return y * 2.0 ** e[..., None]


@pytest.mark.parametrize("heads,dh,dtype", [(12, 64, "bf16"), (1, 32, "f32"), (3, 128, "bf16"), (17, 32, "bf16"), (4, 64, "f32")])
def test_quantised_append_and_read(heads, dh, dtype):
    """Appends in pieces, a fork whose shared last page is copied, an accepted path, and what is read back:
    exactly the numbers of the definition."""
    g = _g()
    rng = np.random.default_rng(6)
    cache = g.QuantisedCache.empty(40, 5, 6, heads, dh)
    for p in (cache.k_pages, cache.v_pages):
        p.fill_(0x7f)
    rows = [[], [], [], [], []]
    for step, T in enumerate((70, 5, 1, 64)):
        k, v = (synth.normal(30 + step, s, (3, T, heads, dh), 1.0, dtype) * 2.0 ** rng.integers(-9, 9, (3, T, heads, 1)) for s in (0, 1))
        k[0, 0, 0] = 0.0
        counts = rng.integers(0, T + 1, 3)
        counts[0] = T
        path = np.stack([np.sort(rng.permutation(T)) for _ in range(3)]) if step == 1 else None
        cache.append(dev(k, dtype), dev(v, dtype), ints(counts), path=None if path is None else ints(path))
        for b in range(3):
            at = list(range(T)) if path is None else path[b]
            rows[b] += [(k[b, at[t]], v[b, at[t]]) for t in range(counts[b])]
        if step == 0:
            cache.fork(ints([0]), ints([3]))
            rows[3] = list(rows[0])
    one = synth.normal(40, 0, (1, 3, heads, dh), 1.0, dtype)
    cache.append(dev(one, dtype), dev(one, dtype), ints([3]), slots=ints([3]))
    rows[3] += [(one[0, t], one[0, t]) for t in range(3)]
    cache.check()
    assert cache.lengths.tolist() == [len(r) for r in rows]
    pool, table = numbers(cache), cache.table.cpu().numpy()
    for b, r in enumerate(rows):
        for t, pair in enumerate(r):
            for p, x in zip(pool, pair):
                assert np.array_equal(p[table[b, t // 64], t % 64], expected(x)), (b, t)
    idx = np.array([[0, 1, -1], [1, 0, 0], [0, 5, 0], [1, -1, 0], [0, 0, 0]])
    for out in (torch.bfloat16, torch.float32):
        k, v, local = cache.read(ints(idx), dtype=out)
        for b in range(5):
            for e in range(3):
                held = idx[b, e] >= 0 and table[b, idx[b, e]] >= 0
                assert int(local[b, e]) == (e if held else -1)
                n = min(64, max(0, len(rows[b]) - 64 * idx[b, e])) if held else 0
                for i, x in enumerate((k, v)):
                    x = host(x[b, 64 * e:64 * e + 64])
                    assert (x[n:] == 0).all()
                    for t in range(n):
                        assert np.array_equal(x[t], expected(rows[b][64 * idx[b, e] + t][i]))


def test_quantised_numbers_at_the_edges():
    """Ties, the largest and smallest numbers, subnormal ones, powers of two and their neighbours, infinities and
    NaN, in both input types."""
    g = _g()
    dh = 64
    x = np.zeros((8, dh))
    x[0] = np.linspace(-448, 448, dh)
    x[1, :8] = [448, 447.9, 432, 416, 208, 1.0625, 1.1875, 2.0 ** -10]
    x[2, :6] = [449, 2.0 ** -9, 3 * 2.0 ** -10, 2.0 ** -8, 17.0, 19.0]
    x[3, :4] = [2.0 ** 127, -(2.0 ** 127) * 1.9, 2.0 ** 110, 1.0]
    x[4, :4] = [2.0 ** -126, 2.0 ** -120, -(2.0 ** -125), 2.0 ** -130]
    x[5] = 2.0 ** np.linspace(-20, 20, dh)
    x[6, :4] = [1.0, np.inf, -np.inf, np.nan]
    for dtype in ("bf16", "f32"):
        y = x.astype(np.float32)
        t = torch.from_numpy(y).cuda().to(TORCH[dtype]).view(1, 8, 1, dh)
        cache = g.QuantisedCache.empty(1, 1, 1, 1, dh)
        cache.append(t, t, ints([8]))
        ref = expected(host(t)[0])
        k, v, _ = cache.read(ints([[0]]), dtype=torch.float32)
        for out in (k, v, cache.read(ints([[0]]))[0]):
            assert np.array_equal(host(out)[0, :8], ref, equal_nan=True)
        assert (host(k)[0, 8:] == 0).all()


def test_quantised_append_packed():
    """Packed prompts into slots in another order: what entry by entry gives; rows around them are not read."""
    g = _g()
    lengths, heads, dh = (130, 0, 64, 1, 300), 3, 64
    off = offsets_of(lengths, 2)
    k, v = (torch.randn(int(off[-1]) + 3, heads, dh, device="cuda").bfloat16() for _ in range(2))
    slots = [4, 1, 0, 3, 2]
    a, b = (g.QuantisedCache.empty(12, 5, 5, heads, dh) for _ in range(2))
    for c in (a, b):
        c.k_pages.zero_()
        c.v_pages.zero_()
    a.append_packed(k, v, ints(off), slots=ints(slots))
    for i, n in enumerate(lengths):
        if n:
            s = slice(int(off[i]), int(off[i + 1]))
            b.append(k[None, s], v[None, s], ints([n]), slots=ints([slots[i]]))
    for x, y in ((a.table, b.table), (a.lengths, b.lengths), (a.refs, b.refs), (a.k_pages, b.k_pages), (a.v_pages, b.v_pages)):
        assert torch.equal(x, y)
    a.append_packed(k[:0], v[:0], ints([0, 0]))
    a.check()


@flags
def test_quantised_refusals_on_the_device():
    """Offsets out of order, bad slots, chunks out of range and a pool without room are flagged, and nothing of
    what is refused is written."""
    g = _g()
    cache = g.QuantisedCache.empty(4, 2, 3, 1, 64)
    k = torch.randn(200, 1, 64, device="cuda").bfloat16()
    state = lambda: [x.clone() for x in (cache.table, cache.lengths, cache.refs)]  # noqa: E731
    before = state()
    for off in ([0, 200, 100], [0, 201, 201], [-1, 5, 9], [100, 50, 200]):
        cache.append_packed(k, k, ints(off))
        with pytest.raises(g.GCAError) as e:
            cache.check()
        assert e.value.status == g.GCA_ERR_DEVICE_INDEX
        assert all(torch.equal(x, y) for x, y in zip(before, state()))
    cache.append_packed(k, k, ints([0, 190]), slots=ints([7]))
    with pytest.raises(g.GCAError):
        cache.check()
    cache.append_packed(k, k, ints([0, 190, 200]))  # four pages for 200 tokens: 3 + 1
    cache.check()
    cache.append_packed(k, k, ints([0, 100]), slots=ints([1]))
    with pytest.raises(g.GCAError) as e:
        cache.check()
    assert e.value.status == g.GCA_ERR_CACHE_FULL and cache.lengths.tolist() == [190, 10]
    for idx in ([[0, 3]], [[-2, 0]]):
        out, _, local = cache.read(ints(idx))
        with pytest.raises(g.GCAError):
            cache.check()
        assert sorted(local[0].tolist()) == sorted([idx[0].index(0), -1])
        bad = 1 - idx[0].index(0)
        assert (out[0, 64 * bad:64 * bad + 64] == 0).all()
    cache.table[0, 0] = 99
    assert cache.read(ints([[0]]))[2].tolist() == [[-1]]
    with pytest.raises(g.GCAError):
        cache.check()


def test_quantised_page_operations():
    """fork, trim, compact and free move quantised rows as they are."""
    g = _g()
    cache = g.QuantisedCache.empty(30, 4, 8, 2, 32)
    x = torch.randn(3, 200, 2, 32, device="cuda").bfloat16()
    cache.append(x, -x, ints([200, 130, 64]))
    cache.free(ints([0]))
    cache.fork(ints([1]), ints([3]))
    cache.append(x[:1, :10], x[:1, :10], ints([10]), slots=ints([3]))
    idx = ints([[0, 1, 2], [0, 1, 2], [0, 0, 0], [0, 1, 2]])
    want = cache.read(idx)
    live = cache.compact()
    cache.check()
    assert int(live[0]) == int((cache.refs > 0).sum()) and int(cache.table.max()) < int(live[0])
    assert all(torch.equal(a, b) for a, b in zip(want, cache.read(idx)))
    cache.trim(begin=ints([0, 64, 0, 0]))
    assert cache.read(ints([[0], [0], [0], [0]]))[2].tolist() == [[-1], [-1], [0], [0]]
    with pytest.raises(TypeError):
        cache.store()
    with pytest.raises(TypeError):
        cache.attention(None, None, None)
    cache.check()


def test_quantised_page_operations_on_wide_rows():
    """Rows of more than 65536 bytes: appended, forked, trimmed, compacted, looked up and read like others."""
    g = _g()
    heads, dh = 520, 128
    cache = g.QuantisedCache.empty(8, 3, 3, heads, dh)
    x = torch.randn(2, 70, heads, dh, device="cuda").bfloat16()
    cache.append(x, -x, ints([70, 64]))
    want = cache.read(ints([[0, 1]]))
    cache.fork(ints([0]), ints([2]))
    cache.append(x[:1, :3], x[:1, :3], ints([3]), slots=ints([2]))
    cache.trim(end=ints([70, 0, 73]))
    assert int(cache.compact()[0]) == 3 and cache.lengths.tolist() == [70, 0, 73]
    assert cache.lookup(ints([[0, 1, 2]])).flatten().tolist() == cache.table[0].tolist()
    assert all(torch.equal(a, b) for a, b in zip(want, cache.read(ints([[0, 1]]))))
    tail = cache.read(ints([[1]]), slots=ints([2]))[0][0]
    assert torch.equal(tail[:6], want[0][0, 64:70]) and torch.equal(tail[6:9], want[0][0, :3])
    cache.check()


@pytest.mark.parametrize("H,Hkv,dh,window", [(12, 12, 64, 0), (10, 2, 128, 0), (24, 4, 64, 300), (12, 4, 32, 0), (8, 8, 128, 700)])
def test_prompt_many_tiles_a_cta(H, Hkv, dh, window):
    """Long sequences whose last tile has no neighbour among others that have, several work items a CTA: against
    the formulas in float64 on the GPU."""
    g = _g()
    lengths = (1400, 2300, 130, 1153, 900, 385, 2049, 60)
    off = offsets_of(lengths)
    N, dev_ = int(off[-1]), "cuda"
    gen = torch.Generator(device=dev_)
    gen.manual_seed(3)
    q, k, v, do = (torch.randn(N, h, dh, device=dev_, generator=gen).bfloat16() for h in (H, Hkv, Hkv, H))
    o, lse = g.prompt_attention(q, k, v, ints(off), window=window)
    grads = g.prompt_attention_backward(q, k, v, o, do, lse, ints(off), window=window)
    for a, z in zip(off, off[1:]):
        n, rep = int(z - a), H // Hkv
        qs, ks, vs, ds_ = (x[a:z].double().transpose(0, 1) for x in (q, k, v, do))
        ks, vs = ks.repeat_interleave(rep, 0), vs.repeat_interleave(rep, 0)
        t = torch.arange(n, device=dev_)
        see = (t[None] <= t[:, None]) & ((t[None] > t[:, None] - window) if window else True)
        s = (qs @ ks.transpose(1, 2) * dh ** -0.5).masked_fill(~see, -float("inf"))
        L = torch.logsumexp(s, 2)
        p = torch.exp(s - L[..., None])
        ref = p @ vs
        dS = p * (ds_ @ vs.transpose(1, 2) - (ds_ * ref).sum(2, keepdim=True)) * dh ** -0.5
        mag = p * (ds_.abs() @ vs.abs().transpose(1, 2) + (ds_.abs() * (p @ vs.abs())).sum(2, keepdim=True)) * dh ** -0.5
        fold = lambda x: x.view(Hkv, rep, n, dh).sum(1)  # noqa: E731
        # One rounding of the output, 2^-8 for the operand (P or dS), D's from the rounded output, and float32's sums.
        e = 2.0 ** -8 * 1.05
        for got, want, size in ((o, ref, p @ vs.abs()), (grads[0], dS @ ks, 2 * (mag @ ks.abs())),
                                (grads[1], fold(dS.transpose(1, 2) @ qs), 2 * fold(mag.transpose(1, 2) @ qs.abs())),
                                (grads[2], fold(p.transpose(1, 2) @ ds_), fold(p.transpose(1, 2) @ ds_.abs()))):
            err = (got[a:z].double().transpose(0, 1) - want).abs()
            assert bool((err <= 2.0 ** -8 * want.abs() + e * size + 1e-30).all()), (n, float((err - e * size).max()))
        assert float((lse[a:z].double().transpose(0, 1) - L).abs().max()) <= 2e-5


@pytest.mark.parametrize("dtype,dh", [("bf16", 64), ("bf16", 128), ("f32", 64)])
def test_prompt_widest_window_and_repeated_heads(dtype, dh):
    """A window as wide as an int is none; heads and gradients that repeat one (a stride of 0) are as their copies."""
    g = _g()
    off, N, H, Hkv = ints([0, 300, 301, 700]), 700, 4, 2
    q, k, v, do = (torch.randn(N, h, dh, device="cuda").to(TORCH[dtype]) for h in (H, Hkv, Hkv, H))

    def step(q, k, v, do, window=0):
        o, lse = g.prompt_attention(q, k, v, off, window=window)
        return (o, lse) + g.prompt_attention_backward(q, k, v, o, do, lse, off, window=window)
    assert all(torch.equal(a, b) for a, b in zip(step(q, k, v, do), step(q, k, v, do, 2 ** 31 - 1)))
    one = [x[:, :1].expand(N, x.shape[1], dh) for x in (q, k, v, do)]
    assert all(torch.equal(a, b) for a, b in zip(step(*one), step(*(x.contiguous() for x in one))))


def test_calls_at_once_share_the_error_word_alone():
    """Steps on two streams that overlap, with scratch of their own, give what they give one after another."""
    g = _g()
    off, N = ints([0, 900, 2000]), 2000
    sets = [[torch.randn(N, h, 64, device="cuda").bfloat16() for h in (8, 2, 2, 8)] for _ in range(2)]
    wt, freq = torch.rand(64, device="cuda"), g.rotary_frequencies(64)
    caches = [g.QuantisedCache.empty(40, 2, 20, 2, 64) for _ in range(4)]

    def step(x, cache):
        q, k = g.norm_rotary(x[0][None], x[1][None], wt, wt, freq)
        o, lse = g.prompt_attention(q[0], k[0], x[2], off)
        grads = g.prompt_attention_backward(q[0], k[0], x[2], o, x[3], lse, off)
        dq, dk, dwq, dwk = g.norm_rotary_backward(x[0][None], x[1][None], grads[0][None], grads[1][None], wt, wt, freq)
        cache.append_packed(k[0], x[2], off)
        return [o, lse, dq, dk, grads[2], dwq, dwk] + list(cache.read(ints([[0, 13], [3, -1]])))
    want = [step(x, c) for x, c in zip(sets, caches)]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [None, None]
    for _ in range(3):
        for c in caches[2:]:
            c.trim(end=ints([0, 0]))
        torch.cuda.synchronize()
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = step(sets[i], caches[2 + i])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for w, r in zip(want, got) for a, b in zip(w, r))


def test_norms_and_cache_in_a_graph():
    """A captured norm with its gradients, append and read follow the inputs, positions and state that change
    behind them."""
    g = _g()
    q, k, v = (torch.randn(3, 70, h, 64, device="cuda").bfloat16() for h in (4, 2, 2))
    wt, freq, pos, counts = torch.rand(64, device="cuda"), g.rotary_frequencies(64), ints([range(70)] * 3), ints([70, 1, 0])
    caches = [g.QuantisedCache.empty(20, 3, 6, 2, 64) for _ in range(2)]
    idx = ints([[0, 1, 2], [0, 1, -1], [0, 0, 0]])

    def step(cache):
        a, b = g.norm_rotary(q, k, wt, wt, freq, positions=pos)
        grads = g.norm_rotary_backward(q, k, a, b, wt, wt, freq, positions=pos)
        cache.append(b, v, counts)
        return [a, b] + list(grads) + list(cache.read(idx))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(caches[0])
    for turn in range(3):
        q.copy_(torch.randn_like(q))
        v.copy_(torch.randn_like(v))
        pos.copy_(pos + 70)
        counts.copy_(ints([[70, 1, 0], [0, 64, 3], [35, 0, 61]][turn]))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, step(caches[1])))
    caches[0].check()
    assert caches[0].lengths.tolist() == [105, 65, 64]


def test_quantised_chunks_and_slots_named_twice():
    """read() takes a chunk, and a slot, as often as it is named."""
    g = _g()
    cache = g.QuantisedCache.empty(8, 3, 4, 2, 64)
    x = torch.randn(2, 130, 2, 64, device="cuda").bfloat16()
    cache.append(x, -x, ints([130, 100]), slots=ints([2, 1]))
    one = cache.read(ints([[0, 1, 2]]), slots=ints([2]))
    two = cache.read(ints([[2, 2, 0], [1, 0, 1], [1, 1, -1]]), slots=ints([2, 2, 1]))
    split = lambda t: t.unflatten(1, (3, 64))  # noqa: E731
    for a, b in zip(one[:2], two[:2]):
        a, b = split(a)[0], split(b)
        assert torch.equal(b[0], a[[2, 2, 0]]) and torch.equal(b[1], a[[1, 0, 1]]) and torch.equal(b[2, 0], b[2, 1]) and (b[2, 2] == 0).all()
    assert two[2].tolist() == [[0, 1, 2], [0, 1, 2], [0, 1, -1]]


def test_more_elements_than_an_int_counts():
    """Tensors of more than 2^31 elements: the last rows are what they are in small tensors."""
    g = _g()
    n, L, H, dh = 530, 1000, 64, 64  # 2.17e9 elements
    N, last = n * L, (n - 1) * L
    q, k, v = (torch.randn(N, h, dh, device="cuda", dtype=torch.bfloat16) for h in (H, 1, 1))
    off, one = ints(np.arange(n + 1) * L), ints([0, L])
    o, lse = g.prompt_attention(q, k, v, off)
    grads = g.prompt_attention_backward(q, k, v, o, q, lse, off)
    s = [x[last:].contiguous() for x in (q, k, v)]
    o1, l1 = g.prompt_attention(*s, one)
    assert torch.equal(o[last:], o1) and torch.equal(lse[last:], l1)
    for x, y in zip(grads, g.prompt_attention_backward(*s, o1, s[0], l1, one)):
        assert torch.equal(x[last:], y)
    del o, grads
    wt, freq, pos = torch.rand(dh, device="cuda"), g.rotary_frequencies(dh), ints(np.arange(last, N))
    assert torch.equal(g.norm_rotary(q[None], None, wt, None, freq)[0][0, last:], g.norm_rotary(s[0][None], None, wt, None, freq, positions=pos)[0][0])
    dx = g.norm_rotary_backward(q[None], None, q[None], None, wt, None, freq)[0]
    assert torch.equal(dx[0, last:], g.norm_rotary_backward(s[0][None], None, s[0][None], None, wt, None, freq, positions=pos)[0][0])
    del dx
    pages, tail = -(-N // 64), N - N // 64 * 64
    cache, small = (g.QuantisedCache.empty(p, 1, p, H, dh) for p in (pages, 1))
    cache.append_packed(q, q, ints([0, N]))
    small.append_packed(q[N - tail:], q[N - tail:], ints([0, tail]))
    assert all(torch.equal(x, y) for x, y in zip(cache.read(ints([[pages - 1]]))[:2], small.read(ints([[0]]))[:2]))


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_step_against_oracle(dtype):
    """A packed training step: norms with rotary, attention, and the gradients of all of it, against the oracle's
    composition; in a captured graph too.  Tolerance: the repository's for its attention block, per element of
    max(1, |x|), bf16 2e-2 and float32 1e-5 times what the norms' and sums' sizes are here (10)."""
    g = _g()
    lengths, H, Hkv, dh = (150, 0, 61, 200), 4, 2, 64
    off = offsets_of(lengths)
    N = int(off[-1])
    q, k, v, do = (synth.normal(51, s, (N, h, dh), 1.0, dtype) for s, h in ((0, H), (1, Hkv), (2, Hkv), (3, H)))
    wt = [np.float32(1 + 0.2 * synth.normal(51, 4 + i, (dh,))).astype(np.float64) for i in range(2)]
    pos = np.concatenate([np.arange(n) for n in lengths])
    w = dorc.speeds(dh)
    args = [dev(x, dtype) for x in (q, k, v, do)] + [ints(off), dev(wt[0], "f32"), dev(wt[1], "f32"), g.rotary_frequencies(dh), ints(pos)]
    r = pipeline.prompt_step(*args, window=100)
    qr, kr = (orc.norm_rotary(x[None], y, pos[None], w, 1e-6)[0] for x, y in zip((q, k), wt))
    ref = orc.prompt_attention(qr, kr, v, off, 100, dout=do)
    dq, dqw = orc.norm_rotary_backward(q[None], ref["dq"][None], wt[0], pos[None], w, 1e-6)
    dk, dkw = orc.norm_rotary_backward(k[None], ref["dk"][None], wt[1], pos[None], w, 1e-6)
    tol = 2e-2 if dtype == "bf16" else 1e-4
    for name, want in (("o", ref["o"]), ("lse", ref["lse"]), ("dq", dq[0]), ("dk", dk[0]), ("dv", ref["dv"])):
        within(host(r[name]), want, 2 * tol * np.maximum(1, np.abs(want)), name)
    for name, want, terms in (("dq_weight", dqw, ref["dq"]), ("dk_weight", dkw, ref["dk"])):
        # a sum of N heads terms, each off by the rounding of the gradient that it takes: of random sign
        lim = tol * np.sqrt((terms ** 2).sum((0, 1))).max() * 4
        within(host(r[name]), want, lim, name)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = pipeline.prompt_step(*args, window=100)
    graph.replay()
    assert all(torch.equal(out[n], r[n]) for n in r)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompt_step_of_a_padded_batch(dtype):
    """Rows in front of the first sequence and behind the last change nothing, and have gradients of 0."""
    g = _g()
    off, H, Hkv, dh, lo, hi, N = [5, 140, 140, 333], 4, 2, 64, 5, 333, 400
    q, k, v, do = (torch.randn(N, h, dh, device="cuda").to(TORCH[dtype]) for h in (H, Hkv, Hkv, H))
    wt, freq, pos = torch.rand(dh, device="cuda"), g.rotary_frequencies(dh), torch.arange(N, dtype=torch.int32, device="cuda")
    r = pipeline.prompt_step(q, k, v, do, ints(off), wt, wt, freq, pos)
    cut = [x[lo:hi].contiguous() for x in (q, k, v, do)]
    want = pipeline.prompt_step(*cut, ints([0, 135, 135, 328]), wt, wt, freq, pos[lo:hi].contiguous())
    for n in ("o", "lse", "dq", "dk", "dv"):
        assert torch.equal(r[n][lo:hi], want[n]), n
    for n in ("dq", "dk", "dv"):
        assert (r[n][:lo] == 0).all() and (r[n][hi:] == 0).all(), n
    for n in ("dq_weight", "dk_weight"):
        # The same terms in another order, of N heads: a few roundings of sums of random sign.
        assert torch.allclose(r[n], want[n], rtol=0, atol=float(N * H * U * want[n].abs().max())), n


def test_prompt_to_quantised_decode():
    """Packed prompts into a quantised cache, then decoding over the chunks that retrieval names: the same as GCA's
    forward over the pages' values."""
    g = _g()
    lengths, H, dh, D = (640, 1280, 900), 4, 64, 256
    off = offsets_of(lengths)
    N = int(off[-1])
    q, k, v = (torch.randn(N, H, dh, device="cuda").bfloat16() for _ in range(3))
    pos = ints(np.concatenate([np.arange(n) for n in lengths]))
    wt, freq = torch.ones(dh, device="cuda"), g.rotary_frequencies(dh)
    cache = g.QuantisedCache.empty(60, 3, 25, H, dh)
    p = pipeline.prompt_forward(q, k, v, ints(off), wt, wt, freq, pos, cache=cache, slots=ints([2, 0, 1]))
    cache.check()
    assert cache.lengths.tolist() == [1280, 900, 640]
    nC = 10  # full chunks of the shortest
    lmk = torch.randn(3, nC, D, device="cuda").bfloat16()
    q_new, q_lmk = torch.randn(3, 64, H, dh, device="cuda").bfloat16(), torch.randn(3, 1, D, device="cuda").bfloat16()
    r = pipeline.decode_quantised(q_new, cache, q_lmk, lmk, topk=4)
    kn, vn, ke, ve = cache.numbers()
    wide = [x.float().mul(torch.exp2(e.float() - 127)[..., None]).bfloat16() for x, e in ((kn, ke), (vn, ve))]
    pages = cache.lookup(r["idx"])
    o, lse = g.gca_forward(q_new, wide[0].flatten(0, 1), wide[1].flatten(0, 1), pages, r["scores"], shift=0, kv_shared=True)
    assert torch.equal(o, r["o"]) and torch.equal(lse, r["lse"])
    # And the pages hold the prompt's keys, each within half a step of e4m3.
    a, z = int(off[1]), int(off[2])
    rows = wide[0][cache.table[0, :20].long()].flatten(0, 1)[:z - a].float()
    turned = p["k"][a:z].float()
    step = torch.exp2(torch.ceil(torch.log2(turned.abs().amax(-1, keepdim=True) / 448)) - 10)
    assert bool(((rows - turned).abs() <= torch.maximum(turned.abs() * 2.0 ** -4, step)).all())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        again = pipeline.decode_quantised(q_new, cache, q_lmk, lmk, topk=4)
    graph.replay()
    assert torch.equal(again["o"], r["o"])
