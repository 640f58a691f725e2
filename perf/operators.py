"""Cases of the decoding operators: rotary positions, attention of drafted tokens over a
paged cache, and the page operations of that cache.

`run` computes each of them in elementary torch operations (`own` false) or through the
library's calls (`own` true).  Pages hold 64 tokens; a cache is a pool of K and V pages
[pages, 64, Hkv, dh], a table [slots, width] of page numbers (-1: none), the slots' lengths
and the pages' reference counts.
"""
import functools
import math
import random

import torch

own = False

PAGE = 64
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------ cases
def _rotary(name, **kw):
    case = dict(name=name, op="rotary", dtype="bf16", B=1, L=1, H=12, Hkv=12, dh=64, rot=64, interleaved=False,
                backward=False, fused=False, base=10000.0, scaling="none", factor=1.0, context=0, gain=1.0, start=0)
    case.update(kw)
    return case


def _tree(name, **kw):
    case = dict(name=name, op="tree", dtype="bf16", B=1, T=1, H=12, Hkv=12, dh=64, ctx=4000, ragged=False, window=0,
                masked=False)
    case.update(kw)
    return case


def _pages(name, op, **kw):
    case = dict(name=name, op=op, dtype="bf16", B=4, T=1, Hkv=12, dh=64, ctx=1000, window=0)
    case.update(kw)
    return case


def listed():
    return [
        # The queries and keys of one layer of the 128M-model training step.
        _rotary("rotary, training", B=4, L=16384, H=12, Hkv=12, fused=True),
        # Their gradients with shared key heads, half of each head turned, pairs side by side.
        _rotary("rotary, gradients", B=8, L=16384, H=16, Hkv=4, rot=32, interleaved=True, backward=True,
                scaling="parts", factor=8.0, context=2048, gain=1.2),
        # One new token of 16 sequences at 16M context.
        _rotary("rotary, one token", B=16, L=1, start=1 << 24, scaling="ntk", factor=4.0),
        # The exact path: float32, odd lengths, a head that is turned in part.
        _rotary("rotary, float32", dtype="f32", B=3, L=1009, H=5, Hkv=1, dh=72, rot=40, scaling="linear", factor=16.0,
                start=100000),
        # Ordinary decoding of one sequence: latency.
        _tree("attention, one token", ctx=4000),
        # A ragged batch of single tokens over long caches, four queries to a key head.
        _tree("attention, ragged batch", B=32, H=16, Hkv=4, dh=128, ctx=65536, ragged=True),
        # Trees of drafted tokens beside retrieval: the 512-token window of the attention block.
        _tree("attention, trees in a window", B=16, T=48, ctx=16384, ragged=True, window=512, masked=True),
        # A full chunk of drafted tokens over two long contexts.
        _tree("attention, trees over 256K", B=2, T=64, H=16, Hkv=4, ctx=262144, masked=True),
        # The exact path: float32 and small heads.
        _tree("attention, float32", dtype="f32", B=3, T=13, H=6, Hkv=2, dh=32, ctx=1500, ragged=True, masked=True),
        # A prompt's keys and values go into fresh pages.
        _pages("pages, prompt", "append", B=4, T=16384, ctx=300),
        # One decoding step of 32 sequences, each forked once: the accepted tokens of a draft, then the window.
        _pages("pages, step", "step", B=32, T=12, ctx=4096, window=512),
        # A pool with half of its pages given back is compacted.
        _pages("pages, compact", "compact", B=16, ctx=65536),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "rotary", "tree", "tree", "tree", "append", "step", "compact"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    size = 2 if dtype == "bf16" else 4
    if op == "rotary":
        dh = rng.choice([32, 40, 64, 64, 72, 128])
        Hkv = rng.choice([1, 2, 4, 6, 8])
        H = Hkv * rng.choice([1, 1, 2, 4])
        rot = rng.choice([dh, dh, dh // 2 // 2 * 2, rng.randrange(2, dh + 1, 2)])
        B = _log(rng, 1, 16)
        L = _log(rng, 1, max(1, min(16384, 200_000_000 // (B * (H + Hkv) * dh * size))))
        case = _rotary("", dtype=dtype, B=B, L=L, H=H, Hkv=Hkv, dh=dh, rot=rot, interleaved=rng.random() < 0.5,
                       backward=rng.random() < 0.5, fused=rng.random() < 0.5, base=rng.choice([10000.0, 500000.0]),
                       scaling=rng.choice(["none", "linear", "ntk", "parts"]), factor=rng.choice([2.0, 8.0, 32.0]),
                       context=rng.choice([2048, 8192]), gain=rng.choice([1.0, 1.1]), start=_log(rng, 1, 1 << 24))
    elif op == "tree":
        Hkv = rng.choice([1, 2, 4, 6, 12])
        g = rng.choice([1, 1, 2, 3, 4, 8])
        dh = rng.choice([32, 64, 64, 128])
        B = _log(rng, 1, 32)
        T = rng.choice([1, _log(rng, 1, 200)])
        most = min(262144, (1 << 28) // (B * Hkv * dh), (1 << 28) // (B * Hkv * g * T))
        case = _tree("", dtype=dtype, B=B, T=T, H=Hkv * g, Hkv=Hkv, dh=dh, ctx=_log(rng, 1, max(1, most)),
                     ragged=rng.random() < 0.6, window=rng.choice([0, 0, rng.randrange(1, 1000)]),
                     masked=rng.random() < 0.7)
    else:
        Hkv, dh = rng.choice([1, 4, 12]), rng.choice([32, 64, 128])
        B = rng.randrange(1, 33)
        token = 2 * Hkv * dh * size
        case = _pages("", op, dtype=dtype, B=B, Hkv=Hkv, dh=dh, ctx=_log(rng, 1, min(16384, 400_000_000 // (B * token))),
                      window=rng.randrange(1, 2000) if op == "step" else 0,
                      T=_log(rng, 1, 64 if op == "step" else min(16384, 150_000_000 // (B * token))))
    del case["name"]
    return case


# ------------------------------------------------------------------------------ inputs
def _lengths(case):
    """The sequences' lengths: a fixed draw of the case's sizes, so that its work is known."""
    r = random.Random(case["B"] * 1_000_003 + case["ctx"])
    if not case.get("ragged", True):
        return [case["ctx"]] * case["B"]
    return [case["ctx"]] + [r.randrange(0, case["ctx"] + 1) for _ in range(case["B"] - 1)]


def _counts(case):
    """Tokens that each sequence takes: all T, or one to T of them where a draft is accepted in part."""
    r = random.Random(case["B"] * 7919 + case["T"])
    return [r.randrange(1, case["T"] + 1) if case["op"] == "step" else case["T"] for _ in range(case["B"])]


def _drafts(case):
    """Drafted tokens of each sequence (the others of its T are padding)."""
    r = random.Random(case["B"] * 104729 + case["T"])
    return [case["T"]] + [r.randrange(max(1, case["T"] // 2), case["T"] + 1) for _ in range(case["B"] - 1)]


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype) if math.prod(shape) < 1 << 27 \
        else torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def _inverse_frequencies(case):
    """Angle per position of each pair, in 64 bits, with the case's scaling for long contexts."""
    rot, base, factor = case["rot"], case["base"], case["factor"]
    if case["scaling"] == "ntk" and rot > 2:
        base *= factor ** (rot / (rot - 2))
    inv = torch.tensor([base ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64)
    if case["scaling"] == "linear":
        inv = inv / factor
    if case["scaling"] == "parts":  # pairs that turn often in the trained context keep their speed
        keep = ((case["context"] * inv / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        inv = inv * keep + inv / factor * (1 - keep)
    return inv


def _tree_mask(case, lengths, rng):
    """Random trees: mask words [B, T, W] (bit u of row t: t sees u) and positions [B, T]; padding at position -1."""
    B, T = case["B"], case["T"]
    words = (T + 63) // 64
    mask, pos = [[[0] * words for _ in range(T)] for _ in range(B)], [[-1] * T for _ in range(B)]
    for b, n in enumerate(_drafts(case)):
        seen, depth = [], []
        for t in range(n):
            p = rng.randrange(-1, t) if t else -1
            p = max(p, rng.randrange(-1, t)) if t else -1
            seen.append((seen[p] if p >= 0 else 0) | (1 << t))
            depth.append(depth[p] + 1 if p >= 0 else 0)
            pos[b][t] = lengths[b] + depth[t]
            for w in range(words):
                v = (seen[t] >> (64 * w)) & (2 ** 64 - 1)
                mask[b][t][w] = v - 2 ** 64 if v >> 63 else v
    return torch.tensor(mask, dtype=torch.int64, device="cuda"), torch.tensor(pos, dtype=torch.int32, device="cuda")


def _cache(case, gen, rng, slots, lengths, spare, used=None):
    """A pool whose pages lie in random order, and its state in one buffer: table, lengths, reference counts."""
    held = [(n + PAGE - 1) // PAGE for n in lengths]
    width = max(1, max(held) + (max(case.get("T", 1), 1) + PAGE - 1) // PAGE + 1)
    pages = sum(held) + spare
    order = list(range(pages))
    rng.shuffle(order)
    table = torch.full((slots, width), -1, dtype=torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32)
    at = 0
    for b, n in enumerate(held):
        if used is None or used[b]:
            table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            refs[order[at:at + n]] = 1
        at += n
    lens = torch.zeros(slots, dtype=torch.int32)
    lens[:len(lengths)] = torch.tensor([n if used is None or used[b] else 0 for b, n in enumerate(lengths)], dtype=torch.int32)
    first = torch.cat([table.reshape(-1), lens, refs]).cuda()
    meta = first.clone()
    shape = (pages, PAGE, case["Hkv"], case["dh"])
    n = slots * width
    return dict(first=first, meta=meta, table=meta[:n].view(slots, width), lengths=meta[n:n + slots], refs=meta[n + slots:],
                k_pages=_normal(gen, shape, DTYPES[case["dtype"]]), v_pages=_normal(gen, shape, DTYPES[case["dtype"]]))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = random.Random(seed)
    dtype = DTYPES[case["dtype"]]
    s = dict(case=case, op=case["op"])
    B, dh = case["B"], case["dh"]
    if case["op"] == "rotary":
        L, H, Hkv = case["L"], case["H"], case["Hkv"]
        if case["fused"]:  # views of one projection's output
            qkv = _normal(gen, (B, L, H + 2 * Hkv, dh), dtype)
            s["q"], s["k"] = qkv[:, :, :H], qkv[:, :, H:H + Hkv]
        else:
            s["q"], s["k"] = _normal(gen, (B, L, H, dh), dtype), _normal(gen, (B, L, Hkv, dh), dtype)
        start = torch.tensor([rng.randrange(0, case["start"] + 1) for _ in range(B)], dtype=torch.int32)
        s["positions"] = (start[:, None] + torch.arange(L, dtype=torch.int32)).cuda()
        s["inv"] = _inverse_frequencies(case).cuda()
        return s
    lengths = _lengths(case)
    if case["op"] == "tree":
        T, H, Hkv = case["T"], case["H"], case["Hkv"]
        s.update(_cache(case, gen, rng, B, lengths, 3))
        s["q"] = _normal(gen, (B, T, H, dh), dtype)
        s["k_new"], s["v_new"] = _normal(gen, (B, T, Hkv, dh), dtype), _normal(gen, (B, T, Hkv, dh), dtype)
        s["mask"], s["positions"] = _tree_mask(case, lengths, rng) if case["masked"] else (None, None)
        return s
    T, Hkv = case["T"], case["Hkv"]
    if case["op"] == "compact":  # half of the sequences have ended
        gone = rng.sample(range(B), B // 2)
        s.update(_cache(case, gen, rng, B, lengths, 5, used=[b not in gone for b in range(B)]))
        return s
    fresh = B * ((T + PAGE - 1) // PAGE + 2)
    slots = 2 * B if case["op"] == "step" else B
    s.update(_cache(case, gen, rng, slots, lengths, 2 * fresh if case["op"] == "step" else fresh))
    s["k_new"], s["v_new"] = _normal(gen, (slots, T, Hkv, dh), dtype), _normal(gen, (slots, T, Hkv, dh), dtype)
    counts = _counts(case)
    if case["op"] == "step":  # the second half of the slots are forks of the first
        s["src"] = torch.arange(B, dtype=torch.int32, device="cuda")
        s["dst"] = torch.arange(B, 2 * B, dtype=torch.int32, device="cuda")
        counts = counts + counts
        paths = [sorted(rng.sample(range(T), n)) for n in counts]  # the accepted nodes of each draft, in order
        s["path"] = torch.tensor([p + [0] * (T - len(p)) for p in paths], dtype=torch.int32, device="cuda")
        s["begin"] = torch.tensor([max(0, n + c - case["window"] + 1) for n, c in zip(lengths + lengths, counts)],
                                  dtype=torch.int32, device="cuda")
    s["counts"] = torch.tensor(counts, dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------------------ plain forms
def _plain_rotate(x, cos, sin, rot, interleaved):
    a = x[..., :rot].float()
    x1, x2 = (a[..., 0::2], a[..., 1::2]) if interleaved else (a[..., :rot // 2], a[..., rot // 2:])
    y1, y2 = x1 * cos - x2 * sin, x1 * sin + x2 * cos
    y = torch.stack([y1, y2], dim=-1).flatten(-2) if interleaved else torch.cat([y1, y2], dim=-1)
    return torch.cat([y.to(x.dtype), x[..., rot:]], dim=-1)


def _plain_rotary(s):
    c = s["case"]
    angle = s["positions"].double()[:, :, None, None] * s["inv"]
    cos = (c["gain"] * torch.cos(angle)).float()
    sin = (c["gain"] * torch.sin(angle)).float()
    sin = -sin if c["backward"] else sin
    return tuple(_plain_rotate(x, cos, sin, c["rot"], c["interleaved"]) for x in (s["q"], s["k"]))


def _plain_tree(s):
    c = s["case"]
    B, T, H, Hkv, dh = c["B"], c["T"], c["H"], c["Hkv"], c["dh"]
    g, width, dev = H // Hkv, s["table"].shape[1], s["q"].device
    lengths = s["lengths"].long()
    u = torch.arange(T, device=dev)
    if s["mask"] is None:
        tree = (u[None, :] <= u[:, None]).expand(B, T, T)
        pos = lengths[:, None] + u
    else:
        tree = ((s["mask"][..., None] >> torch.arange(64, device=dev)) & 1).bool().flatten(2)[:, :, :T]
        pos = s["positions"].long()
    j = torch.arange(width * PAGE, device=dev)
    past = (j < lengths[:, None])[:, None, :].expand(B, T, -1)
    if c["window"]:
        past = past & (j > pos[:, :, None] - c["window"])
        tree = tree & (pos[:, None, :] > pos[:, :, None] - c["window"])
    seen = torch.cat([past & (pos >= 0)[:, :, None], tree & (pos >= 0)[:, :, None]], dim=2)[:, None, None]
    pages = s["table"].clamp(min=0).long()
    k = torch.cat([s["k_pages"][pages].flatten(1, 2), s["k_new"]], dim=1).permute(0, 2, 1, 3).float()
    q = s["q"].float().view(B, T, Hkv, g, dh).permute(0, 2, 3, 1, 4).reshape(B, Hkv, g * T, dh)
    logits = torch.matmul(q, k.transpose(2, 3)).div_(math.sqrt(dh)).view(B, Hkv, g, T, -1)
    del k
    logits.masked_fill_(~seen, -math.inf)
    top = logits.amax(-1, keepdim=True).clamp(min=-3e38)
    p = logits.sub_(top).exp_()
    total = p.sum(-1, dtype=torch.float64)
    v = torch.cat([s["v_pages"][pages].flatten(1, 2), s["v_new"]], dim=1).permute(0, 2, 1, 3).float()
    o = torch.matmul(p.view(B, Hkv, g * T, -1), v).view(B, Hkv, g, T, dh)
    o = o / torch.where(total > 0, total, 1.0)[..., None].float()
    lse = (top[..., 0].double() + total.log()).float()
    return (o.to(s["q"].dtype).permute(0, 3, 1, 2, 4).reshape(B, T, H, dh), lse.permute(0, 3, 1, 2).reshape(B, T, H))


def _plain_append(s):
    table, lengths, refs, counts = s["table"], s["lengths"], s["refs"], s["counts"]
    T, dev = s["k_new"].shape[1], table.device
    slots = torch.arange(table.shape[0], device=dev)
    old, new = lengths.long(), (lengths + counts).long()
    # A last page that several slots hold is copied for each that writes to it.
    last = torch.where((old % PAGE > 0) & (counts > 0), table[slots, old // PAGE], -1).long()
    copied = (last >= 0) & (refs[last.clamp(min=0)] > 1)
    first = torch.where(copied, old // PAGE, (old + PAGE - 1) // PAGE)
    need = (new + PAGE - 1) // PAGE - first
    start = need.cumsum(0) - need
    free = torch.nonzero(refs == 0)[:, 0]
    p = torch.arange(table.shape[1], device=dev)
    fresh = (p >= first[:, None]) & (p < (first + need)[:, None])
    given = free[(start[:, None] + p - first[:, None])[fresh]]
    table[fresh] = given.int()
    refs[given] = 1
    refs.index_add_(0, last.clamp(min=0), -copied.int())
    t = torch.arange(T, device=dev)
    a, r = torch.nonzero((torch.arange(PAGE, device=dev) < (old % PAGE)[:, None]) & copied[:, None], as_tuple=True)
    to = table[a, old[a] // PAGE].long()
    b, i = torch.nonzero(t < counts[:, None], as_tuple=True)
    at = old[b] + i
    page, row = table[b, at // PAGE].long(), at % PAGE
    i = s["path"][b, i].long() if "path" in s else i
    for pool, rows in ((s["k_pages"], s["k_new"]), (s["v_pages"], s["v_new"])):
        pool[to, r] = pool[last[a], r]
        pool[page, row] = rows[b, i]
    lengths += counts


def _plain_fork(s):
    src, dst = s["src"].long(), s["dst"].long()
    rows = s["table"][src]
    s["table"][dst] = rows
    s["lengths"][dst] = s["lengths"][src]
    held = rows[rows >= 0].long()
    s["refs"].index_add_(0, held, torch.ones_like(held, dtype=torch.int32))


def _plain_trim(s):
    p = torch.arange(s["table"].shape[1], device=s["table"].device)
    gone = (s["table"] >= 0) & ((p + 1) * PAGE <= torch.minimum(s["begin"], s["lengths"])[:, None])
    held = s["table"][gone].long()
    s["refs"].index_add_(0, held, torch.full_like(held, -1, dtype=torch.int32))
    s["table"][gone] = -1


def _plain_compact(s):
    refs, table = s["refs"], s["table"]
    live = refs > 0
    n = live.sum()
    index = torch.arange(refs.shape[0], device=refs.device)
    moved, holes = torch.nonzero(live & (index >= n))[:, 0], torch.nonzero(~live & (index < n))[:, 0]
    to = index.int()
    to[moved] = holes.int()
    s["k_pages"][holes] = s["k_pages"][moved]
    s["v_pages"][holes] = s["v_pages"][moved]
    refs[holes] = refs[moved]
    refs[moved] = 0
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], -1))
    return n.int().view(1)


# ------------------------------------------------------------------------------ a pass
@functools.lru_cache(maxsize=None)
def _frequencies(rot, base, scaling, factor, context):
    import retrieval_sparse_attention_causal_gb300 as gca
    return gca.rotary_frequencies(rot, base=base, scaling=scaling, factor=factor, context=context)


def run(s):
    c = s["case"]
    if s["op"] == "rotary":
        if not own:
            return _plain_rotary(s)
        import retrieval_sparse_attention_causal_gb300 as gca
        turn = gca.rotary_backward if c["backward"] else gca.rotary
        return turn(s["q"], s["k"], _frequencies(c["rot"], c["base"], c["scaling"], c["factor"], c["context"]),
                    positions=s["positions"], interleaved=c["interleaved"], gain=c["gain"])
    if s["op"] == "tree":
        if not own:
            return _plain_tree(s)
        import retrieval_sparse_attention_causal_gb300 as gca
        return gca.tree_attention(s["q"], s["k_new"], s["v_new"], s["k_pages"], s["v_pages"], s["table"], s["lengths"],
                                  mask=s["mask"], positions=s["positions"], window=c["window"])
    s["meta"].copy_(s["first"])  # the cache as it was before the step
    out = dict(k_pages=s["k_pages"], v_pages=s["v_pages"], table=s["table"], lengths=s["lengths"], refs=s["refs"])
    if own:
        import retrieval_sparse_attention_causal_gb300 as gca
        cache = gca.PagedCache(s["k_pages"], s["v_pages"], s["table"], s["lengths"], s["refs"])
        if s["op"] == "compact":
            out["live"] = cache.compact()
        elif s["op"] == "append":
            cache.append(s["k_new"], s["v_new"], s["counts"])
        else:
            cache.fork(s["src"], s["dst"])
            cache.append(s["k_new"], s["v_new"], s["counts"], path=s["path"])
            cache.trim(begin=s["begin"])
    elif s["op"] == "compact":
        out["live"] = _plain_compact(s)
    elif s["op"] == "append":
        _plain_append(s)
    else:
        _plain_fork(s)
        _plain_append(s)
        _plain_trim(s)
    return out


# ------------------------------------------------------------------------------ work
def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    B, dh = case["B"], case["dh"]
    if case["op"] == "rotary":
        heads = case["H"] + case["Hkv"]
        values = B * case["L"] * heads * dh
        return dict(bytes=2 * values * size + 4 * B * case["L"], flops=3 * B * case["L"] * heads * case["rot"])
    if case["op"] == "tree":
        T, H, Hkv = case["T"], case["H"], case["Hkv"]
        keys = pairs = 0
        drafts = _drafts(case) if case["masked"] else [T] * B
        for n, d in zip(_lengths(case), drafts):
            past = min(n, case["window"] - 1) if case["window"] else n
            keys += past + d
            pairs += d * past + d * (d + 1) // 2
        return dict(bytes=2 * keys * Hkv * dh * size + 2 * sum(drafts) * H * dh * size + 4 * B * T * H, flops=4 * pairs * H * dh)
    token = 2 * case["Hkv"] * dh * size
    lengths = _lengths(case)
    held = [(n + PAGE - 1) // PAGE for n in lengths]
    if case["op"] == "compact":  # about half of the pages are held, and half of those lie behind them
        return dict(bytes=2 * (sum(held) // 4) * PAGE * token + 8 * sum(held), flops=0)
    counts = _counts(case)
    if case["op"] == "append":
        return dict(bytes=2 * sum(counts) * token + 8 * sum(held), flops=0)
    shared = 2 * sum(n % PAGE for n in lengths)  # rows of shared last pages that are copied
    return dict(bytes=2 * (2 * sum(counts) + shared) * token + 24 * sum(held), flops=0)


# ------------------------------------------------------------------------------ exact
def _exact_rotary(case, s):
    inv = _inverse_frequencies(case).cuda()
    turn = torch.polar(torch.full_like(inv, case["gain"]).expand(s["positions"].shape + inv.shape),
                       s["positions"].double()[..., None] * inv)
    turn = (turn.conj() if case["backward"] else turn)[:, :, None, :]
    outs = []
    for x in (s["q"], s["k"]):
        y = x.double()
        rot = case["rot"]
        if case["interleaved"]:
            z = torch.view_as_complex(y[..., :rot].reshape(y.shape[:-1] + (rot // 2, 2)))
            y[..., :rot] = torch.view_as_real(z * turn).flatten(-2)
        else:
            z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * turn
            y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
        outs.append(y)
    return tuple(outs)


def _exact_tree(case, s):
    B, T, H, Hkv, dh = case["B"], case["T"], case["H"], case["Hkv"], case["dh"]
    g = H // Hkv
    o = torch.zeros(B, T, H, dh, dtype=torch.float64, device="cuda")
    lse = torch.full((B, T, H), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lengths(case)):
        held = s["table"][b, :(n + PAGE - 1) // PAGE].long()
        sees = torch.zeros(T, n + T, dtype=torch.bool)
        words = s["mask"][b].tolist() if case["masked"] else None
        where = s["positions"][b].tolist() if case["masked"] else [n + t for t in range(T)]
        for t in range(T):
            if where[t] < 0:
                continue
            low = max(0, where[t] - case["window"] + 1) if case["window"] else 0
            sees[t, low:n] = True
            for u in range(T):
                bit = (words[t][u // 64] >> (u % 64)) & 1 if words else u <= t
                if bit and (not case["window"] or where[t] - where[u] < case["window"]):
                    sees[t, n + u] = True
        hidden = ~sees.cuda()
        rows = torch.tensor([w >= 0 for w in where], device="cuda")
        for m in range(Hkv):
            k = torch.cat([s["k_pages"][held, :, m].reshape(-1, dh)[:n], s["k_new"][b, :, m]]).double()
            v = torch.cat([s["v_pages"][held, :, m].reshape(-1, dh)[:n], s["v_new"][b, :, m]]).double()
            for h in range(m * g, m * g + g):
                a = (s["q"][b, :, h].double() @ k.T) / dh ** 0.5
                a.masked_fill_(hidden, -math.inf)
                z = torch.logsumexp(a, dim=1)
                y = torch.exp(a - z[:, None]) @ v
                o[b, rows, h], lse[b, rows, h] = y[rows], z[rows]
    return o, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(case, s)
    if case["op"] == "tree":
        return _exact_tree(case, s)
    return None
