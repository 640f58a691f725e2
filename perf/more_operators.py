"""Cases of a prompt's operators: attention over packed sequences with its gradients, norms of queries
and keys with the rotary positions in the same pass, and a cache that holds its keys and values in 8 bits.

`run` computes each of them in elementary torch operations (`own` false) or through the library's
calls (`own` true).  Packed sequences are the rows offsets[b] .. offsets[b + 1] - 1 of one tensor.
A quantised token is a row of bytes: heads x dh values in e4m3, then one exponent a head (biased by
127, filled up to a multiple of 16 bytes); a value is its e4m3 number times two to the exponent.
"""
import functools
import math
import random

import torch

own = False

PAGE = 64
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
MOST_PAIRS = 4 * 12 * 16384 ** 2  # (query, key) pairs of the largest attention


# ------------------------------------------------------------------------------ cases
def _attention(name, **kw):
    case = dict(name=name, op="attention", dtype="bf16", B=1, longest=100, ragged=True, H=12, Hkv=12, dh=64, window=0,
                fused=False, backward=False)
    case.update(kw)
    return case


def _norm(name, **kw):
    case = dict(name=name, op="norm", dtype="bf16", B=1, L=1, H=12, Hkv=12, dh=64, rot=64, interleaved=False,
                backward=False, fused=False, base=10000.0, eps=1e-6, gain=1.0, start=0)
    case.update(kw)
    return case


def _cached(name, op, **kw):
    case = dict(name=name, op=op, dtype="bf16", B=4, T=1, Hkv=12, dh=64, ctx=1000, per=0)
    case.update(kw)
    return case


def listed():
    return [
        # One layer of the 128M-model training step on documents packed into a batch, forward and backward.
        _attention("attention, training", B=4, longest=16384, fused=True, backward=True),
        # Serving: one long prompt, four query heads to a key head.
        _attention("attention, long prompt", longest=32768, H=16, Hkv=4, dh=128),
        # Serving: a batch of short prompts of different lengths.
        _attention("attention, short prompts", B=48, longest=300, fused=True),
        # One short prompt: latency.
        _attention("attention, one prompt", longest=77),
        # Training of the window sublayer on packed documents, with shared key heads.
        _attention("attention, window training", B=24, longest=4096, H=16, Hkv=4, window=512, backward=True),
        # The exact path: float32, small heads, odd lengths, with gradients.
        _attention("attention, float32", dtype="f32", B=3, longest=517, H=6, Hkv=2, dh=32, backward=True),
        # The queries and keys of one layer of the 128M-model training step.
        _norm("norm, training", B=4, L=16384, fused=True),
        # Their gradients with shared key heads, half of each head turned, pairs side by side.
        _norm("norm, gradients", B=8, L=16384, H=16, Hkv=4, rot=32, interleaved=True, backward=True),
        # One new token of 16 sequences at 16M context: latency.
        _norm("norm, one token", B=16, start=1 << 24),
        # Prompts of different lengths go into fresh pages, from the packed tensor.
        _cached("quantised, prompts", "write", B=8, T=16384),
        # A decoding step's tokens of 32 sequences, behind what the cache holds.
        _cached("quantised, step", "write", B=32, T=4, ctx=4096),
        # The chunks that 16 sequences retrieved, for the attention over them.
        _cached("quantised, retrieved", "read", B=16, ctx=16384, per=8),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "norm", "norm", "write", "read"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    size = 2 if dtype == "bf16" else 4
    if op == "attention":
        Hkv = rng.choice([1, 2, 4, 6, 8])
        H = Hkv * rng.choice([1, 1, 2, 3, 4, 8])
        B = _log(rng, 1, 64)
        most = min(16384, int(math.sqrt(MOST_PAIRS / (4 if dtype == "bf16" else 64) / (B * H))))
        backward = rng.random() < 0.5
        least = 8 if backward else 1  # a token that sees itself alone has no gradient but what rounding leaves
        case = _attention("", dtype=dtype, B=B, longest=_log(rng, least, max(2 * least, most)), ragged=rng.random() < 0.8, H=H,
                          Hkv=Hkv, dh=rng.choice([32, 64, 64, 128]), window=rng.choice([0, 0, rng.randrange(least, 1500)]),
                          fused=rng.random() < 0.5, backward=backward)
    elif op == "norm":
        dh = rng.choice([32, 40, 64, 64, 72, 128])
        Hkv = rng.choice([1, 2, 4, 6, 8])
        H = Hkv * rng.choice([1, 1, 2, 4])
        rot = rng.choice([dh, dh, dh // 2 // 2 * 2, rng.randrange(2, dh + 1, 2)])
        B = _log(rng, 1, 16)
        L = _log(rng, 1, max(1, min(16384, 150_000_000 // (B * (H + Hkv) * dh * size))))
        case = _norm("", dtype=dtype, B=B, L=L, H=H, Hkv=Hkv, dh=dh, rot=rot, interleaved=rng.random() < 0.5,
                     backward=rng.random() < 0.5, fused=rng.random() < 0.5, base=rng.choice([10000.0, 500000.0]),
                     eps=rng.choice([1e-6, 1e-5]), gain=rng.choice([1.0, 1.1]), start=_log(rng, 1, 1 << 24))
    else:
        Hkv, dh, B = rng.choice([1, 3, 4, 12]), rng.choice([32, 64, 128]), rng.randrange(1, 33)
        token = 2 * Hkv * dh * size
        case = _cached("", op, dtype=dtype, B=B, Hkv=Hkv, dh=dh, ctx=_log(rng, 64, min(16384, 200_000_000 // (B * token))),
                       T=_log(rng, 1, min(16384, 100_000_000 // (B * token))) if op == "write" else 1,
                       per=rng.randrange(1, 33) if op == "read" else 0)
    del case["name"]
    return case


# ------------------------------------------------------------------------------ inputs
def _lengths(case):
    """The sequences' lengths: a fixed draw of the case's sizes, so that its work is known."""
    r = random.Random(case["B"] * 1_000_003 + case["longest"])
    if not case["ragged"]:
        return [case["longest"]] * case["B"]
    return [case["longest"]] + [r.randrange(0, case["longest"] + 1) for _ in range(case["B"] - 1)]


def _held(case):
    """Tokens that the cache holds of each sequence: none before a prompt goes in."""
    r = random.Random(case["B"] * 15485863 + case["ctx"])
    if case["op"] == "write" and case["T"] > 64:
        return [0] * case["B"]
    return [case["ctx"]] + [r.randrange(0, case["ctx"] + 1) for _ in range(case["B"] - 1)]


def _counts(case):
    """Tokens that each sequence takes."""
    r = random.Random(case["B"] * 7919 + case["T"])
    return [case["T"]] + [r.randrange(0, case["T"] + 1) for _ in range(case["B"] - 1)]


def _offsets(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return at


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype) if math.prod(shape) < 1 << 27 \
        else torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def _row(case):
    """Bytes of a quantised token: its values, and its heads' exponents up to a multiple of 16 bytes."""
    return case["Hkv"] * case["dh"] + (case["Hkv"] + 15) // 16 * 16


def _pool(case, gen, pages):
    """A pool with e4m3 numbers in every row (no NaN) and exponents as activations have them."""
    values = case["Hkv"] * case["dh"]
    pool = torch.zeros((pages, PAGE, _row(case)), dtype=torch.uint8, device="cuda")
    bits = torch.randint(0, 254, (pages, PAGE, values), generator=gen, device="cuda", dtype=torch.int16)
    pool[..., :values] = torch.where(bits >= 127, bits + 1, bits).to(torch.uint8)
    pool[..., values:values + case["Hkv"]] = torch.randint(117, 122, (pages, PAGE, case["Hkv"]), generator=gen, device="cuda",
                                                           dtype=torch.int16).to(torch.uint8)
    return pool


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = random.Random(seed)
    dtype, dh = DTYPES[case["dtype"]], case["dh"]
    s = dict(case=case, op=case["op"])
    if case["op"] == "attention":
        lengths, H, Hkv = _lengths(case), case["H"], case["Hkv"]
        N = max(1, sum(lengths))
        if case["fused"]:  # views of one projection's output
            qkv = _normal(gen, (N, H + 2 * Hkv, dh), dtype)
            s["q"], s["k"], s["v"] = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
        else:
            s["q"], s["k"], s["v"] = (_normal(gen, (N, h, dh), dtype) for h in (H, Hkv, Hkv))
        if case["backward"]:
            s["dout"] = _normal(gen, (N, H, dh), dtype)
        s["offsets"] = torch.tensor(_offsets(lengths), dtype=torch.int32, device="cuda")
        s["padded"] = max(lengths)
        return s
    if case["op"] == "norm":
        B, L, H, Hkv = case["B"], case["L"], case["H"], case["Hkv"]
        if case["fused"]:
            qkv = _normal(gen, (B, L, H + 2 * Hkv, dh), dtype)
            s["q"], s["k"] = qkv[:, :, :H], qkv[:, :, H:H + Hkv]
        else:
            s["q"], s["k"] = _normal(gen, (B, L, H, dh), dtype), _normal(gen, (B, L, Hkv, dh), dtype)
        if case["backward"]:
            s["dq_out"], s["dk_out"] = _normal(gen, (B, L, H, dh), dtype), _normal(gen, (B, L, Hkv, dh), dtype)
        for name in ("q_weight", "k_weight"):
            s[name] = 1.0 + 0.2 * torch.randn(dh, generator=gen, device="cuda")
        start = torch.tensor([rng.randrange(0, case["start"] + 1) for _ in range(B)], dtype=torch.int32)
        s["positions"] = (start[:, None] + torch.arange(L, dtype=torch.int32)).cuda()
        s["inv"] = torch.tensor([case["base"] ** (-2.0 * i / case["rot"]) for i in range(case["rot"] // 2)],
                                dtype=torch.float64, device="cuda")
        return s
    # A pool whose pages lie in random order, and its state in one buffer: table, lengths, reference counts.
    B, Hkv, held = case["B"], case["Hkv"], _held(case)
    counts = _counts(case) if case["op"] == "write" else [0] * B
    here = [(n + PAGE - 1) // PAGE for n in held]
    fresh = sum((n + c + PAGE - 1) // PAGE for n, c in zip(held, counts)) - sum(here)
    width = max(1, max((n + c + PAGE - 1) // PAGE for n, c in zip(held, counts)))
    pages = sum(here) + fresh + 3
    order = list(range(pages))
    rng.shuffle(order)
    table = torch.full((B, width), -1, dtype=torch.int32)
    refs = torch.zeros(pages, dtype=torch.int32)
    at = 0
    for b, n in enumerate(here):
        table[b, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        refs[order[at:at + n]] = 1
        at += n
    first = torch.cat([table.reshape(-1), torch.tensor(held, dtype=torch.int32), refs]).cuda()
    meta = first.clone()
    n = B * width
    s.update(first=first, meta=meta, table=meta[:n].view(B, width), lengths=meta[n:n + B], refs=meta[n + B:],
             k_pages=_pool(case, gen, pages), v_pages=_pool(case, gen, pages))
    if case["op"] == "read":
        idx = [[rng.randrange(0, n // PAGE) if n >= PAGE else -1 for _ in range(case["per"])] for n in held]
        for row in idx[1::3]:  # some rows retrieve fewer
            row[-1] = -1
        s["idx"] = torch.tensor(idx, dtype=torch.int32, device="cuda").view(B, 1, case["per"])
        return s
    # Activations differ in size from token to token.
    N = max(1, sum(counts))
    size = torch.exp2(4 * torch.rand((N, 1, 1), generator=gen, device="cuda") - 2)
    s["k_new"], s["v_new"] = ((_normal(gen, (N, Hkv, dh), torch.float32) * size).to(dtype) for _ in range(2))
    s["offsets"] = torch.tensor(_offsets(counts), dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------------------ plain forms
def _plain_attention(s):
    c = s["case"]
    H, Hkv, dh, L = c["H"], c["Hkv"], c["dh"], s["padded"]
    g, offsets, dev = H // Hkv, s["offsets"].long(), s["q"].device
    lengths = offsets[1:] - offsets[:-1]
    B = lengths.shape[0]
    t = torch.arange(L, device=dev)
    there = t < lengths[:, None]
    rows = (offsets[:-1, None] + t).clamp(max=s["q"].shape[0] - 1)
    seen = t[None, :] <= t[:, None]
    if c["window"]:
        seen = seen & (t[None, :] > t[:, None] - c["window"])
    hidden = ~seen

    def heads(x, first, count):  # [B, count, L, dh]; what lies behind a sequence counts as zeros
        x = x[:, first:first + count][rows].float()
        return x.masked_fill_(~there[..., None, None], 0.0).permute(0, 2, 1, 3)

    outs = []
    step = max(1, min(Hkv, (1 << 31) // (B * g * L * L)))  # key heads at a time, as memory allows
    for m in range(0, Hkv, step):
        n = min(step, Hkv - m)
        q = heads(s["q"], m * g, n * g).reshape(B, n, g * L, dh)
        k, v = heads(s["k"], m, n), heads(s["v"], m, n)
        p = torch.matmul(q, k.transpose(2, 3)).div_(math.sqrt(dh)).view(B, n, g, L, L)
        p.masked_fill_(hidden, -math.inf)
        top = p.amax(-1, keepdim=True)
        p.sub_(top).exp_()
        total = p.sum(-1, keepdim=True, dtype=torch.float64)
        lse = (top.double() + total.log()).float().view(B, n * g, L)
        p.div_(total.float())
        p = p.view(B, n, g * L, L)
        o = torch.matmul(p, v)
        outs.append([o.view(B, n * g, L, dh), lse])
        if not c["backward"]:
            continue
        do = heads(s["dout"], m * g, n * g).reshape(B, n, g * L, dh)
        dv = torch.matmul(p.transpose(2, 3), do)
        ds = torch.matmul(do, v.transpose(2, 3)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).div_(math.sqrt(dh))
        dq, dk = torch.matmul(ds, k), torch.matmul(ds.transpose(2, 3), q)
        outs[-1] += [dq.view(B, n * g, L, dh), dk, dv]
        del ds
    outs = [torch.cat(x, dim=1) for x in zip(*outs)]
    o, lse, *grads = [x.transpose(1, 2)[there] for x in outs]
    return tuple([o.to(s["q"].dtype), lse] + [x.to(s["q"].dtype) for x in grads])


def _turned(x, cos, sin, rot, interleaved):
    a = x[..., :rot]
    x1, x2 = (a[..., 0::2], a[..., 1::2]) if interleaved else (a[..., :rot // 2], a[..., rot // 2:])
    y1, y2 = x1 * cos - x2 * sin, x1 * sin + x2 * cos
    y = torch.stack([y1, y2], dim=-1).flatten(-2) if interleaved else torch.cat([y1, y2], dim=-1)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _plain_norm(s):
    c = s["case"]
    angle = s["positions"].double()[:, :, None, None] * s["inv"]
    cos, sin = (c["gain"] * torch.cos(angle)).float(), (c["gain"] * torch.sin(angle)).float()
    outs, sums = [], []
    for x, dy, w in ((s["q"], s.get("dq_out"), s["q_weight"]), (s["k"], s.get("dk_out"), s["k_weight"])):
        a = x.float()
        r = torch.rsqrt(a.square().mean(-1, keepdim=True) + c["eps"])
        if not c["backward"]:
            outs.append(_turned(a * r * w, cos, sin, c["rot"], c["interleaved"]).to(x.dtype))
            continue
        u = _turned(dy.float(), cos, -sin, c["rot"], c["interleaved"])
        n = a * r
        sums.append((u * n).sum((0, 1, 2), dtype=torch.float64).float())
        u = u * w
        outs.append(((u - n * (u * n).mean(-1, keepdim=True)) * r).to(x.dtype))
    return tuple(outs + sums)


def _two_to(e):
    """Two to a whole power, from its bits: exact, which a power function need not be."""
    return ((e + 127).int() << 23).view(torch.float32)


def _plain_quantised(x):
    """Rows of bytes of x [N, heads, dh]: e4m3 numbers and exponents."""
    a = x.float()
    m, e = torch.frexp(a.abs().amax(-1))  # the least exponent by which the largest is 448 at most
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(-120, 127)
    e = torch.where(m == 0, -120, e)
    values = (a * _two_to(-e)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).flatten(1)
    fill = torch.zeros((x.shape[0], -x.shape[1] % 16), dtype=torch.uint8, device=x.device)
    return torch.cat([values, (e + 127).to(torch.uint8), fill], dim=1)


def _plain_write(s):
    table, lengths, refs, offsets = s["table"], s["lengths"], s["refs"], s["offsets"].long()
    dev = table.device
    counts = offsets[1:] - offsets[:-1]
    old, new = lengths.long(), lengths + counts
    first = (old + PAGE - 1) // PAGE
    need = (new + PAGE - 1) // PAGE - first
    start = need.cumsum(0) - need
    free = torch.nonzero(refs == 0)[:, 0]
    p = torch.arange(table.shape[1], device=dev)
    fresh = (p >= first[:, None]) & (p < (first + need)[:, None])
    given = free[(start[:, None] + p - first[:, None])[fresh]]
    table[fresh] = given.int()
    refs[given] = 1
    r = torch.arange(s["k_new"].shape[0], device=dev)
    b = (torch.bucketize(r, offsets, right=True) - 1).clamp(max=counts.shape[0] - 1)
    r, b = r[r < offsets[-1]], b[r < offsets[-1]]
    at = old[b] + r - offsets[b]
    page, row = table[b, at // PAGE].long(), at % PAGE
    for pool, x in ((s["k_pages"], s["k_new"]), (s["v_pages"], s["v_new"])):
        pool[page, row] = _plain_quantised(x[r])
    lengths += counts.int()


def _plain_read(s):
    c = s["case"]
    B, Hkv, dh, per = c["B"], c["Hkv"], c["dh"], c["per"]
    idx = s["idx"].view(B, per).long()
    page = s["table"].gather(1, idx.clamp(min=0)).long()
    there = idx >= 0
    outs = []
    for pool in (s["k_pages"], s["v_pages"]):
        x = pool[page.clamp(min=0)]
        values = x[..., :Hkv * dh].contiguous().view(torch.float8_e4m3fn).float().view(B, per, PAGE, Hkv, dh)
        e = x[..., Hkv * dh:Hkv * dh + Hkv].int() - 127
        y = (values * _two_to(e)[..., None]).to(DTYPES[c["dtype"]])
        outs.append(y.masked_fill_(~there[:, :, None, None, None], 0.0).view(B, per * PAGE, Hkv, dh))
    local = torch.where(there, torch.arange(per, device=idx.device), -1).int().view(B, 1, per)
    return tuple(outs + [local])


# ------------------------------------------------------------------------------ a pass
@functools.lru_cache(maxsize=None)
def _frequencies(rot, base):
    import retrieval_sparse_attention_causal_gb300 as gca
    return gca.rotary_frequencies(rot, base=base)


def _own(s):
    import retrieval_sparse_attention_causal_gb300 as gca
    c = s["case"]
    if s["op"] == "attention":
        o, lse = gca.prompt_attention(s["q"], s["k"], s["v"], s["offsets"], window=c["window"])
        if not c["backward"]:
            return o, lse
        return (o, lse) + gca.prompt_attention_backward(s["q"], s["k"], s["v"], o, s["dout"], lse, s["offsets"],
                                                        window=c["window"])
    if s["op"] == "norm":
        freq = _frequencies(c["rot"], c["base"])
        how = dict(positions=s["positions"], interleaved=c["interleaved"], gain=c["gain"], eps=c["eps"])
        if not c["backward"]:
            return gca.norm_rotary(s["q"], s["k"], s["q_weight"], s["k_weight"], freq, **how)
        return gca.norm_rotary_backward(s["q"], s["k"], s["dq_out"], s["dk_out"], s["q_weight"], s["k_weight"], freq, **how)
    cache = gca.QuantisedCache(s["k_pages"], s["v_pages"], s["table"], s["lengths"], s["refs"], c["Hkv"], c["dh"])
    if s["op"] == "read":
        return cache.read(s["idx"], dtype=DTYPES[c["dtype"]])
    return cache.append_packed(s["k_new"], s["v_new"], s["offsets"])


def run(s):
    c = s["case"]
    if s["op"] == "attention":
        return _own(s) if own else _plain_attention(s)
    if s["op"] == "norm":
        return _own(s) if own else _plain_norm(s)
    if s["op"] == "read":
        return _own(s) if own else _plain_read(s)
    s["meta"].copy_(s["first"])  # the cache as it was before the step
    if own:
        _own(s)
    else:
        _plain_write(s)
    n = c["Hkv"] * c["dh"]
    return dict(k=s["k_pages"].view(torch.float8_e4m3fn)[..., :n], v=s["v_pages"].view(torch.float8_e4m3fn)[..., :n],
                k_exponents=s["k_pages"][..., n:n + c["Hkv"]], v_exponents=s["v_pages"][..., n:n + c["Hkv"]],
                table=s["table"], lengths=s["lengths"], refs=s["refs"])


# ------------------------------------------------------------------------------ work
def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    dh = case["dh"]
    if case["op"] == "attention":
        lengths, H, Hkv, w = _lengths(case), case["H"], case["Hkv"], case["window"]
        pairs = sum(n * (n + 1) // 2 - (max(0, n - w) * (max(0, n - w) + 1) // 2 if w else 0) for n in lengths)
        N = sum(lengths)
        moved = N * (2 * H + 2 * Hkv) * dh * size + 4 * N * H
        if case["backward"]:  # the output's gradient in; those of q, k and v out
            moved += N * (2 * H + 2 * Hkv) * dh * size
        return dict(bytes=moved, flops=(14 if case["backward"] else 4) * pairs * H * dh)
    if case["op"] == "norm":
        heads = case["H"] + case["Hkv"]
        values = case["B"] * case["L"] * heads * dh
        return dict(bytes=(3 if case["backward"] else 2) * values * size + 4 * case["B"] * case["L"],
                    flops=(12 if case["backward"] else 7) * values)
    token = 2 * case["Hkv"] * dh * size
    if case["op"] == "read":
        chunks = sum(case["per"] - (1 if b % 3 == 1 else 0) for b, n in enumerate(_held(case)) if n >= PAGE)
        zeros = case["B"] * case["per"] - chunks
        return dict(bytes=PAGE * (chunks * (2 * (_row(case)) + token) + zeros * token), flops=0)
    counts = _counts(case)
    return dict(bytes=sum(counts) * (token + 2 * _row(case)) + 8 * sum((n + c) // PAGE for n, c in zip(_held(case), counts)),
                flops=0)


# ------------------------------------------------------------------------------ exact
def _exact_attention(case, s):
    H, dh, w = case["H"], case["dh"], case["window"]
    g, N = H // case["Hkv"], s["q"].shape[0]
    like = dict(dtype=torch.float64, device="cuda")
    o, lse = torch.zeros(N, H, dh, **like), torch.zeros(N, H, **like)
    dq, dk, dv = torch.zeros_like(o), torch.zeros(N, H // g, dh, **like), torch.zeros(N, H // g, dh, **like)
    scale = dh ** -0.5
    for a, z in zip(_offsets(_lengths(case)), _offsets(_lengths(case))[1:]):
        for h in range(H):
            k, v = s["k"][a:z, h // g].double(), s["v"][a:z, h // g].double()
            for i in range(0, z - a, 2048):  # 2048 queries at a time, and the keys that they can see
                j = min(i + 2048, z - a)
                lo = max(0, i - w + 1) if w else 0
                q = s["q"][a + i:a + j, h].double()
                x, y = torch.arange(i, j, device="cuda")[:, None], torch.arange(lo, j, device="cuda")
                sees = (y <= x) & (y > x - w) if w else y <= x
                logits = (q @ k[lo:j].T).mul_(scale).masked_fill_(~sees, -math.inf)
                z_ = torch.logsumexp(logits, dim=1)
                p = logits.sub_(z_[:, None]).exp_()
                out = p @ v[lo:j]
                o[a + i:a + j, h], lse[a + i:a + j, h] = out, z_
                if case["backward"]:
                    do = s["dout"][a + i:a + j, h].double()
                    dv[a + lo:a + j, h // g] += p.T @ do
                    ds = (do @ v[lo:j].T).sub_((do * out).sum(1, keepdim=True)).mul_(p).mul_(scale)
                    dq[a + i:a + j, h] = ds @ k[lo:j]
                    dk[a + lo:a + j, h // g] += ds.T @ q
    n = sum(_lengths(case))
    return (o[:n], lse[:n], dq[:n], dk[:n], dv[:n]) if case["backward"] else (o[:n], lse[:n])


def _exact_norm(case, s):
    rot, sides = case["rot"], []
    turn = torch.polar(torch.full_like(s["inv"], case["gain"]).expand(s["positions"].shape + s["inv"].shape),
                       s["positions"].double()[..., None] * s["inv"])[:, :, None, :]

    def rotate(y, by):
        y = y.clone()
        if case["interleaved"]:
            z = torch.view_as_complex(y[..., :rot].reshape(y.shape[:-1] + (rot // 2, 2))) * by
            y[..., :rot] = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(y[..., :rot // 2].contiguous(), y[..., rot // 2:rot].contiguous()) * by
            y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
        return y

    for name in ("q", "k"):
        x, w = s[name].double(), s[name + "_weight"].double()
        length = torch.linalg.vector_norm(x, dim=-1, keepdim=True)
        rms = torch.sqrt(length ** 2 / case["dh"] + case["eps"])
        if not case["backward"]:
            sides.append((rotate(x / rms * w, turn),))
            continue
        # y = R diag(w) x / rms(x): the Jacobian's transpose, term by term.
        back = rotate(s["d" + name + "_out"].double(), turn.conj())
        dw = torch.einsum("blhd,blhd->d", back, x / rms)
        c = torch.einsum("blhd,blhd->blh", back * w, x)[..., None]
        sides.append((back * w / rms - x * c / (case["dh"] * rms ** 3), dw))
    return tuple(side[i] for i in range(len(sides[0])) for side in sides)


def _e4m3(y):
    """The nearest e4m3 number, ties to the even one, of numbers up to 448."""
    _, x = torch.frexp(y)
    step = torch.exp2((x - 1).clamp(min=-6).double() - 3)
    return torch.round(y / step) * step


def _exact_write(case, s):
    n, Hkv, dh = case["Hkv"] * case["dh"], case["Hkv"], case["dh"]
    state = [t.tolist() for t in (s["table"], s["lengths"], s["refs"])]
    table, lengths, refs = state
    pools = [p.view(torch.float8_e4m3fn)[..., :n].double() for p in (s["k_pages"], s["v_pages"])]
    scales = [p[..., n:n + Hkv].long() for p in (s["k_pages"], s["v_pages"])]
    free = iter([p for p, r in enumerate(refs) if r == 0])
    to, rows = [], []
    for b, (a, z) in enumerate(zip(_offsets(_counts(case)), _offsets(_counts(case))[1:])):
        for r in range(a, z):
            at = lengths[b]
            if at % PAGE == 0:
                table[b][at // PAGE] = next(free)
                refs[table[b][at // PAGE]] = 1
            to.append(table[b][at // PAGE] * PAGE + at % PAGE)
            rows.append(r)
            lengths[b] += 1
    to, rows = torch.tensor(to, device="cuda", dtype=torch.long), torch.tensor(rows, device="cuda", dtype=torch.long)
    for pool, scale, x in zip(pools, scales, (s["k_new"], s["v_new"])):
        x = x[rows].double()
        most = x.abs().amax(-1)
        e = torch.ceil(torch.log2(most / 448)).clamp(min=-120)
        e = e + (most > 448 * torch.exp2(e)) - (most <= 448 * torch.exp2(e - 1)).double()  # what the logarithm rounds
        e = e.clamp(min=-120)
        pool.view(-1, n)[to] = _e4m3(x / torch.exp2(e)[..., None]).flatten(1)
        scale.reshape(-1, Hkv)[to] = (e + 127).long()
    like = dict(dtype=torch.int32)
    return dict(k=pools[0], v=pools[1], k_exponents=None, v_exponents=None, table=torch.tensor(table, **like),
                lengths=torch.tensor(lengths, **like), refs=torch.tensor(refs, **like))


def _exact_read(case, s):
    B, per, Hkv, dh = case["B"], case["per"], case["Hkv"], case["dh"]
    outs = [torch.zeros(B, per * PAGE, Hkv, dh, dtype=torch.float64, device="cuda") for _ in range(2)]
    for b, chunks in enumerate(s["idx"].view(B, per).tolist()):
        for i, j in enumerate(chunks):
            if j < 0:
                continue
            for out, pool in zip(outs, (s["k_pages"], s["v_pages"])):
                x = pool[int(s["table"][b, j])].long()
                bits, e = x[:, :Hkv * dh].view(PAGE, Hkv, dh), x[:, Hkv * dh:Hkv * dh + Hkv, None] - 127
                high, low = (bits >> 3) & 15, bits & 7
                size = torch.where(high > 0, (8 + low).double() * torch.exp2(high.double() - 10), low.double() * 2.0 ** -9)
                out[b, i * PAGE:(i + 1) * PAGE] = torch.where(bits >= 128, -size, size) * torch.exp2(e.double())
    return outs[0], outs[1], None


def exact(case, seed):
    s = prepare(case, seed)
    return {"attention": _exact_attention, "norm": _exact_norm, "write": _exact_write, "read": _exact_read}[case["op"]](case, s)
