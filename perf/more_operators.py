"""What the attention half of a layer costs: rotary positions, the store that
rotates and quantizes new keys and values into a cache of 4-bit blocks (read
back through the load), and attention over that cache, for single tokens, a
few of them and whole prompts.

``listed()`` names the measured cases, ``draw(rng)`` gives further ones of the
same ranges, ``prepare`` makes a case's inputs, ``run`` is one call and
``work`` what that call cannot do without.  With ``own`` false ``run`` computes
the operator from elementary torch operations in f32; with ``own`` true it
calls this package's kernels.  ``exact`` evaluates the definition in 64 bits.

The head layouts are the 7B ones the benchmark runs (28 query heads and 4
key/value heads of 128: the grouped q|k|v of 4608) and the 8B-like ones (32 and
8 heads of 128), with generic ones beside them.

A batch is ragged: sequence b has ``rows`` new rows, which are the last of its
``len`` tokens.  The cache is paged: token t of a sequence is in page
``table[b, t // page]``.
"""

import math
import random

import torch

own = False

DTYPE = {"f16": torch.float16, "f32": torch.float32}
SIZE = {"f16": 2, "f32": 4}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _rope(name, M, H, D, n_rot, layout="half", x="f16", far=0, factor=1.0, pad=0):
    return {"name": name, "op": "rope", "M": M, "H": H, "D": D, "n_rot": n_rot, "layout": layout,
            "x": x, "far": far, "factor": factor, "pad": pad}


def _store(name, B, rows, past, H, Hkv, D, page, layout="half", x="f16", far=0, ragged=False):
    return {"name": name, "op": "store", "B": B, "rows": rows, "past": past, "H": H, "Hkv": Hkv,
            "D": D, "page": page, "layout": layout, "x": x, "far": far, "ragged": ragged}


def _attn(name, B, rows, past, H, Hkv, D, page, x="f16", ragged=False, causal=True, window=0,
          cap=0.0, slopes=False, prefix=False):
    return {"name": name, "op": "attention", "B": B, "rows": rows, "past": past, "H": H,
            "Hkv": Hkv, "D": D, "page": page, "x": x, "ragged": ragged, "causal": causal,
            "window": window, "cap": cap, "slopes": slopes, "prefix": prefix}


def listed():
    return [
        # one generated token: q and k of the grouped q|k|v row, rotated in one call
        _rope("rope f16 m1", 1, 32, 128, 128, far=20000, pad=512),
        # a full prompt far into a long context, half of each head rotated, pairs side by side
        _rope("rope f32 partial m2048", 2048, 40, 128, 64, layout="interleaved", x="f32",
              far=1000000, factor=4.0),
        # sixteen sequences decoded together: each stores one token and rotates its q
        _store("store m16", 16, 1, 1000, 28, 4, 128, 32, ragged=True),
        # prompts of several lengths, f32 activations, ends and starts inside pages
        _store("store ragged prompts", 3, 1000, 100, 32, 8, 128, 64, layout="interleaved",
               x="f32", ragged=True),
        # one token of a small model at the start of a conversation: latency is all
        _attn("attention m1 short", 1, 1, 36, 8, 8, 64, 64),
        # one generated token of a 7B model in a middling context
        _attn("attention m1 4k", 1, 1, 4095, 28, 4, 128, 64),
        # one generated token in a very long context
        _attn("attention m1 131k", 1, 1, 131071, 32, 8, 128, 256),
        # a server's batch: one token each, contexts of all lengths
        _attn("attention batch", 64, 1, 8000, 28, 4, 128, 64, ragged=True),
        # a few drafted tokens each, heads of 256 with capped scores and a window
        _attn("attention drafts", 8, 5, 3000, 16, 8, 256, 32, ragged=True, window=1024, cap=50.0),
        # a full prompt
        _attn("attention prompt", 1, 2048, 0, 28, 4, 128, 64),
        # prompts of several lengths with a shared readable start and a distance bias, f32 q
        _attn("attention ragged prompts", 5, 777, 90, 10, 10, 96, 32, x="f32", ragged=True,
              slopes=True, prefix=True),
        # a piece of a prompt on a long context
        _attn("attention piece", 1, 512, 16000, 32, 8, 128, 128, cap=30.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = ((28, 4), (32, 8), (8, 8), (16, 2), (10, 10), (16, 1), (40, 8), (32, 2), (6, 2))


def draw(rng):
    op = rng.choice(("rope", "store", "attention", "attention", "attention"))
    D = rng.choice((64, 96, 128, 128, 128, 256))
    H, Hkv = rng.choice(HEADS)
    layout = rng.choice(("half", "interleaved"))
    x = rng.choice(("f16", "f16", "f32"))
    page = rng.choice((32, 64, 96, 256))
    ragged = rng.random() < 0.5
    if op == "rope":
        M = _log(rng, 1, 4096)
        while M * H * D > 2048 * 40 * 128:
            M //= 2
        return {"op": op, "M": M, "H": H, "D": D, "n_rot": rng.choice((D, D, D // 2, D // 4 + 2)),
                "layout": layout, "x": x, "far": rng.choice((0, 5000, 1000000)),
                "factor": rng.choice((1.0, 4.0)), "pad": rng.choice((0, 1, 512))}
    if op == "store":
        B = _log(rng, 1, 32)
        rows = rng.choice((1, _log(rng, 1, 2048)))
        while B * rows * Hkv * D > 2048 * 8 * 128 or B * rows * H * D > 2048 * 32 * 128:
            rows = max(1, rows // 2)
            B = max(1, B // 2) if rows == 1 else B
        return {"op": op, "B": B, "rows": rows, "past": _log(rng, 1, 4000), "H": H, "Hkv": Hkv,
                "D": D, "page": page, "layout": layout, "x": x,
                "far": rng.choice((0, 0, 500000)), "ragged": ragged}
    if rng.random() < 0.6:                         # single tokens and drafts
        rows = rng.choice((1, 1, 1, 2, 4, 8))
        B = _log(rng, 1, 64)
        past = _log(rng, 8, 131072)
        while B * past * Hkv * D > 64 * 8000 * 4 * 128 or B * rows * H * past > 1 << 26:
            past = past // 2
    else:                                          # prompts and pieces of them
        B = _log(rng, 1, 6)
        rows = _log(rng, 9, 2048)
        past = rng.choice((0, _log(rng, 1, 16000)))
        while B * rows * H * (past + rows) * D > 512 * 32 * 16512 * 128:
            rows, past = max(1, rows // 2), past // 2
    c = {"op": op, "B": B, "rows": rows, "past": past, "H": H, "Hkv": Hkv, "D": D, "page": page,
         "x": x, "ragged": ragged, "causal": rng.random() < 0.85,
         "window": rng.choice((0, 0, _log(rng, 16, 2048))), "cap": rng.choice((0.0, 0.0, 20.0)),
         "slopes": rng.random() < 0.25, "prefix": rng.random() < 0.25}
    return c


def _batch(case):
    """Rows and lengths of each sequence: of the case alone, not of the seed."""
    B, rows, past = case["B"], case["rows"], case["past"]
    r, n = [], []
    for b in range(B):
        u = math.fmod((b + 1) * 0.6180339887, 1.0) if case["ragged"] else 1.0
        v = math.fmod((b + 1) * 0.7548776662, 1.0) if case["ragged"] else 1.0
        r.append(max(1, int(round(rows * u))))
        n.append(r[-1] + int(round(past * v)))
    return r, n


def _prefix(case, n):
    """How many first tokens every row of the sequence may read."""
    return [(7 * b + 13) % (k + 1) for b, k in enumerate(n)]


def work(case):
    """Every input read once, every output written once; two operations per
    multiply-add."""
    e = SIZE[case["x"]]
    if case["op"] == "rope":
        n = case["M"] * case["H"] * case["D"]
        return {"bytes": 2 * n * e + 4 * case["M"] + 4 * case["n_rot"], "flops": 3 * n}
    r, n = _batch(case)
    T, H, Hkv, D = sum(r), case["H"], case["Hkv"], case["D"]
    row = D // 2 + D // 16                          # bytes of a key or value in the cache
    if case["op"] == "store":
        # k, v and q read; the cache rows and q written; the rows read back as f16
        b = T * (2 * Hkv * D * e + H * D * (e + 2) + 2 * Hkv * row + 2 * Hkv * D * 2)
        return {"bytes": b, "flops": T * (3 * (H + Hkv) * D + 4 * 2 * Hkv * D)}
    pairs, read = 0, 0
    pre = _prefix(case, n) if case["prefix"] else [0] * len(n)
    w = case["window"]
    for rb, nb, pb in zip(r, n, pre):
        first = nb - rb                             # position of the first row
        i = torch.arange(first, nb, dtype=torch.float64)
        hi = torch.clamp(i + 1, max=nb) if case["causal"] else torch.full_like(i, nb)
        if w and not case["causal"]:
            hi = torch.clamp(i + w, max=nb)
        lo = torch.clamp(i - w + 1, min=0) if w else torch.zeros_like(i)
        # the visible range [lo, hi) and the prefix [0, pb)
        seen = torch.where(lo > pb, hi - lo + pb, torch.clamp(hi, min=pb))
        pairs += int(seen.sum())
        low = int(lo.min())
        read += nb - low + pb if low > pb else nb
    return {"bytes": T * H * D * (e + 2) + read * Hkv * 2 * row, "flops": 4 * D * H * pairs}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _freqs(n_rot, factor, device):
    """Rotation per position of each pair, in f64: base 10000, every pair
    slowed down by `factor`."""
    j = torch.arange(n_rot // 2, dtype=torch.float64, device=device)
    return 10000.0 ** (-2 * j / n_rot) / factor


def _rows(g, M, H, D, dtype, device, pad=0, gain=1.0):
    """Activations of H heads, a few channels of each twice the others' size."""
    big = 1 + (torch.rand(H * D + pad, generator=g, device=device) < 0.05).float()
    x = torch.randn(M, H * D + pad, generator=g, device=device) * (gain * big)
    return x.to(dtype)[:, :H * D]


def _quantize(x):
    """(codes 0..15, scales f16) of 4-bit blocks along the last axis."""
    b = x.float().unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    first = (b.abs() == top).to(torch.uint8).argmax(-1, keepdim=True)
    d = (b.gather(-1, first) / -8).half()
    df = d.float()
    q = torch.floor(b / torch.where(df == 0, torch.ones_like(df), df) + 8.5)
    q = torch.where(df == 0, torch.full_like(q, 8), torch.clamp(q, 0, 15))
    return q.to(torch.uint8).flatten(-2), d[..., 0]


def _pack(q):
    """Two codes in a byte: element j of 32 low, element j + 16 high."""
    q = q.unflatten(-1, (-1, 2, 16))
    return (q[..., 0, :] | (q[..., 1, :] << 4)).flatten(-2)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    s = dict(case)
    xt = DTYPE[case["x"]]
    if case["op"] == "rope":
        M = case["M"]
        s["xt"] = _rows(g, M, case["H"], case["D"], xt, dev, case["pad"])
        start = torch.randint(0, case["far"] + 1, (1,), generator=g, device=dev)
        s["pos"] = (start + torch.arange(M, device=dev)).to(torch.int32)
        s["freqs"] = _freqs(case["n_rot"], case["factor"], dev)
        s["mscale"] = 1.0 + 0.1 * math.log(case["factor"])
        return s
    r, n = _batch(case)
    B, T, D, H, Hkv, page = case["B"], sum(r), case["D"], case["H"], case["Hkv"], case["page"]
    width = -(-max(n) // page)
    need = [-(-k // page) for k in n]
    pages = sum(need) + 3
    # every sequence's pages lie anywhere in the cache
    order = random.Random(seed).sample(range(pages), sum(need))
    table = torch.full((B, width), pages - 1, dtype=torch.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = torch.tensor(order[at:at + k], dtype=torch.int32)
        at += k
    s["table"] = table.to(dev)
    s["lens"] = torch.tensor(n, dtype=torch.int32, device=dev)
    cu = [0]
    for k in r:
        cu.append(cu[-1] + k)
    s["cu"] = torch.tensor(cu, dtype=torch.int32, device=dev) if case["ragged"] else None
    # sequence and row within it of each row of the batch
    s["seq"] = torch.repeat_interleave(torch.arange(B, device=dev), torch.tensor(r, device=dev))
    s["row"] = torch.arange(T, device=dev) - torch.tensor(cu, device=dev)[s["seq"]]
    s["rmax"], s["nmax"], s["T"] = max(r), max(n), T
    s["nrows"] = torch.tensor(r, device=dev)
    s["q"] = _rows(g, T, H, D, xt, dev, gain=2.0 if case["op"] == "attention" else 1.0)
    if case["op"] == "store":
        s["k"] = _rows(g, T, Hkv, D, xt, dev)
        s["v"] = _rows(g, T, Hkv, D, xt, dev)
        s["freqs"] = _freqs(D, 1.0, dev)
        s["shift"] = case["far"]
        s["pos"] = (s["lens"].long() - s["nrows"])[s["seq"]] + s["row"] + case["far"]
        s["pos32"] = s["pos"].to(torch.int32)
        if own:
            import quantized_weight_prefill_q4_amd as mq
            s["cache"] = mq.kv_cache_q4(pages, Hkv, page, D, device=dev)
        return s
    # the cache's contents, token by token of each sequence
    total = sum(n)
    k, v = (_rows(g, total, Hkv, D, torch.float16, dev) for _ in range(2))
    seq = torch.repeat_interleave(torch.arange(B, device=dev), s["lens"].long())
    ends = torch.cumsum(s["lens"].long(), 0)
    tok = torch.arange(total, device=dev) - (ends - s["lens"])[seq]
    place = s["table"].long()[seq, tok // page] * page + tok % page
    for name, t in (("kc", k), ("vc", v)):
        codes, d = _quantize(t.unflatten(-1, (Hkv, D)))
        packed = torch.zeros(pages * page, Hkv, D // 2, dtype=torch.uint8, device=dev)
        scales = torch.zeros(pages * page, Hkv, D // 32, dtype=torch.float16, device=dev)
        packed[place], scales[place] = _pack(codes), d
        s[name], s[name + "_d"] = packed, scales
    s["slopes"] = s["prefix"] = None
    if case["slopes"]:
        s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)],
                                   dtype=torch.float32, device=dev)
    if case["prefix"]:
        s["prefix"] = torch.tensor(_prefix(case, n), dtype=torch.int32, device=dev)
    if own:
        import quantized_weight_prefill_q4_amd as mq
        s["cache"] = mq.kv_cache_q4(pages, Hkv, page, D, device=dev)
        all_cu = torch.nn.functional.pad(ends, (1, 0)).to(torch.int32)
        mq.kv_store_q4(k, v, s["cache"], s["table"], s["lens"], cu_rows=all_cu)
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

def _rotate(x, pos, freqs, mscale, layout):
    """x [T, H, D] in f32 with the first 2·len(freqs) elements of each head
    rotated; the angles in f64."""
    a = pos.double().unsqueeze(-1) * freqs
    c = (torch.cos(a) * mscale).float().unsqueeze(1)
    s = (torch.sin(a) * mscale).float().unsqueeze(1)
    n = freqs.numel()
    if layout == "half":
        x0, x1, rest = x[..., :n], x[..., n:2 * n], x[..., 2 * n:]
        return torch.cat((x0 * c - x1 * s, x1 * c + x0 * s, rest), -1)
    x0, x1, rest = x[..., :2 * n:2], x[..., 1:2 * n:2], x[..., 2 * n:]
    y = torch.stack((x0 * c - x1 * s, x1 * c + x0 * s), -1).flatten(-2)
    return torch.cat((y, rest), -1)


def _value(codes, d):
    """What codes and scales stand for, in f32."""
    return ((codes.float() - 8).unflatten(-1, (-1, 32)) * d.float().unsqueeze(-1)).flatten(-2)


def _plain_store(s):
    H, Hkv, D = s["H"], s["Hkv"], s["D"]
    rot = [_rotate(s[n].float().unflatten(-1, (h, D)), s["pos"], s["freqs"], 1.0, s["layout"])
           for n, h in (("q", H), ("k", Hkv))]
    k = _value(*_quantize(rot[1]))
    v = _value(*_quantize(s["v"].float().unflatten(-1, (Hkv, D))))
    return {"q": rot[0].flatten(1).half(), "k": k.flatten(1).half(), "v": v.flatten(1).half()}


def _gather(packed, d, place):
    """The cache rows at `place` [B, L], as f32 [B, Hkv, L, D]."""
    b = packed[place].unflatten(-1, (-1, 16))
    q = torch.cat((b & 15, b >> 4), -1).flatten(-2)
    return _value(q, d[place]).transpose(1, 2).contiguous()


def _plain_attention(s):
    B, H, Hkv, D, page, R, L = s["B"], s["H"], s["Hkv"], s["D"], s["page"], s["rmax"], s["nmax"]
    dev, G = s["q"].device, s["H"] // s["Hkv"]
    tok = torch.arange(L, device=dev)
    place = s["table"].long()[:, tok // page] * page + tok % page
    k, v = _gather(s["kc"], s["kc_d"], place), _gather(s["vc"], s["vc_d"], place)
    # the rows of each sequence, padded to the longest
    q = torch.zeros(B * R, H, D, device=dev)
    flat = s["seq"] * R + s["row"]
    q[flat] = s["q"].float().unflatten(-1, (H, D))
    q = q.view(B, R, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * R, D)
    w = torch.matmul(q, k.transpose(2, 3).contiguous()) * (1 / math.sqrt(D))
    w = w.view(B, H, R, L)
    if s["cap"]:
        w = s["cap"] * torch.tanh(w / s["cap"])
    n = s["lens"].long().view(B, 1, 1)
    at = n - s["nrows"].view(B, 1, 1) + torch.arange(R, device=dev).view(1, R, 1)
    if s["slopes"] is not None:
        w = w - s["slopes"].view(1, H, 1, 1) * (at - tok).abs().unsqueeze(1)
    seen = torch.ones(B, R, L, dtype=torch.bool, device=dev)
    if s["causal"]:
        seen = tok <= at
    if s["window"]:
        seen = seen & ((at - tok).abs() < s["window"])
    if s["prefix"] is not None:
        seen = seen | (tok < s["prefix"].view(B, 1, 1))
    seen = (seen & (tok < n)).unsqueeze(1)
    w = w.masked_fill(~seen, -math.inf)
    top = w.amax(-1, keepdim=True)
    p = torch.exp(w - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, torch.ones_like(total), total)
    y = torch.matmul(p.view(B, Hkv, G * R, L), v)
    y = y.view(B, H, R, D).transpose(1, 2).reshape(B * R, H * D)
    return {"y": y[flat].half()}


def run(state):
    s = state
    if own:
        return _run_own(s)
    if s["op"] == "rope":
        x = s["xt"].float().unflatten(-1, (s["H"], s["D"]))
        y = _rotate(x, s["pos"], s["freqs"], s["mscale"], s["layout"])
        return {"y": y.flatten(1).to(s["xt"].dtype)}
    return _plain_store(s) if s["op"] == "store" else _plain_attention(s)


# ---------------------------------------------------------------------------
# The package's operators
# ---------------------------------------------------------------------------

def _run_own(s):
    import quantized_weight_prefill_q4_amd as mq

    if s["op"] == "rope":
        return {"y": mq.rope(s["xt"], s["pos"], s["freqs"], s["D"], layout=s["layout"],
                             mscale=s["mscale"])}
    if s["op"] == "store":
        q = mq.kv_store_q4(s["k"], s["v"], s["cache"], s["table"], s["lens"], cu_rows=s["cu"],
                           freqs=s["freqs"], layout=s["layout"],
                           positions=s["pos32"] if s["shift"] else None, q=s["q"])
        k, v = mq.kv_load_q4(s["cache"], s["table"], s["lens"], s["T"], cu_rows=s["cu"])
        return {"q": q, "k": k, "v": v}
    return {"y": mq.attention_q4(s["q"], s["cache"], s["table"], s["lens"], cu_rows=s["cu"],
                                 causal=s["causal"], window=s["window"], cap=s["cap"],
                                 slopes=s["slopes"], prefix=s["prefix"])}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_rotate(x, pos, freqs, mscale, layout):
    """One pair after the other as a complex number times mscale·e^(i·angle)."""
    n, y = freqs.numel(), x.double().clone()
    turn = torch.polar(torch.full_like(freqs, mscale).expand(len(pos), n).contiguous(),
                       pos.double().view(-1, 1) * freqs.view(1, -1))
    for j in range(n):
        a, b = (j, j + n) if layout == "half" else (2 * j, 2 * j + 1)
        z = torch.complex(x[..., a].double(), x[..., b].double()) * turn[:, j:j + 1]
        y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_blocks(x):
    """The value each element has in the cache, block by block."""
    y = torch.empty_like(x)
    for g in range(x.shape[-1] // 32):
        b = x[..., 32 * g:32 * g + 32]
        hi, lo = b.max(-1).values, b.min(-1).values
        at_hi = (b == hi.unsqueeze(-1)).double().argmax(-1)
        at_lo = (b == lo.unsqueeze(-1)).double().argmax(-1)
        pos = (hi > -lo) | ((hi == -lo) & (at_hi < at_lo))
        d = (torch.where(pos, hi, lo) / -8).half().double().unsqueeze(-1)
        q = torch.floor(b / torch.where(d == 0, torch.ones_like(d), d) + 8.5).clamp(0, 15)
        y[..., 32 * g:32 * g + 32] = (q - 8) * d
    return y


def exact(case, seed):
    s = prepare(case, seed)
    H, D = case["H"], case["D"]
    if case["op"] == "rope":
        y = _exact_rotate(s["xt"].unflatten(-1, (H, D)), s["pos"], s["freqs"], s["mscale"],
                          case["layout"])
        return {"y": y.flatten(1)}
    Hkv = case["Hkv"]
    if case["op"] == "store":
        q, k = (_exact_rotate(s[n].unflatten(-1, (h, D)), s["pos"], s["freqs"], 1.0, case["layout"])
                for n, h in (("q", H), ("k", Hkv)))
        v = _exact_blocks(s["v"].unflatten(-1, (Hkv, D)).double())
        return {"q": q.flatten(1), "k": _exact_blocks(k).flatten(1), "v": v.flatten(1)}
    r, n = _batch(case)
    pre = _prefix(case, n) if case["prefix"] else [0] * len(n)
    out, at, page = torch.zeros(sum(r), H, D, dtype=torch.float64, device=s["q"].device), 0, case["page"]

    def rows(packed, d, places, h):
        e = torch.arange(D, device=packed.device)
        byte = packed[places, h][:, 16 * (e // 32) + e % 16].int()
        code = (byte >> (4 * ((e % 32) // 16))) & 15
        return (code - 8).double() * d[places, h][:, e // 32].double()

    for b in range(len(n)):
        places = torch.cat([torch.arange(page, device=out.device) + int(p) * page
                            for p in s["table"][b, :-(-n[b] // page)].tolist()])[:n[b]]
        j = torch.arange(n[b], device=out.device).view(1, -1)
        i = torch.arange(n[b] - r[b], n[b], device=out.device).view(-1, 1)
        see = (j <= i) if case["causal"] else (j >= 0).expand(r[b], -1)
        if case["window"]:
            see = see & (j > i - case["window"]) & (j < i + case["window"])
        see = see | (j < pre[b])
        for h in range(Hkv):
            k, v = rows(s["kc"], s["kc_d"], places, h), rows(s["vc"], s["vc_d"], places, h)
            for a in range(h * (H // Hkv), (h + 1) * (H // Hkv)):
                q = s["q"][at:at + r[b], a * D:(a + 1) * D].double()
                w = torch.mm(q, k.t().contiguous()) / math.sqrt(D)
                if case["cap"]:
                    w = torch.tanh(w / case["cap"]) * case["cap"]
                if case["slopes"]:
                    w = w - 2.0 ** (-8.0 * (a + 1) / H) * (i - j).abs().double()
                w = torch.where(see, w, torch.full_like(w, -math.inf))
                out[at:at + r[b], a] = torch.mm(torch.softmax(w, -1), v)
        at += r[b]
    return {"y": out.flatten(1)}
