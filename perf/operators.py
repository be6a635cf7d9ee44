"""What the fused operators around the quantized products cost: a linear layer
with its epilogue (bias, activation, residual), a gated pair of them, and the
norm that feeds both (residual addition, RMS norm, f16 or Q8_1 output).

``listed()`` names the measured cases, ``draw(rng)`` gives further ones of the
same ranges, ``prepare`` makes a case's inputs, ``run`` is one call and
``work`` what that call cannot do without.  With ``own`` false ``run`` computes
the operator from elementary torch operations in f32; with ``own`` true it
calls this package's kernels.  ``exact`` evaluates the definition in 64 bits.

The layer sizes are the 7B shapes the benchmark runs (hidden 3584, feed-forward
18944, grouped q|k|v 4608) and the 8B-like ones (4096, 14336), with generic odd
sizes beside them.
"""

import math

import torch

own = False

EPS = 1e-6
FORMATS = ("q4_0", "q5_0", "q5_1", "q8_0", "q4_k", "q5_k", "q6_k")
# elements and bytes of a weight block
BLOCK = {"q4_0": (32, 18), "q5_0": (32, 22), "q5_1": (32, 24), "q8_0": (32, 34),
         "q4_k": (256, 144), "q5_k": (256, 176), "q6_k": (256, 210)}
DTYPE = {"f16": torch.float16, "f32": torch.float32}
SIZE = {"f16": 2, "f32": 4}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def _linear(name, w, M, N, K, x="f16", bias=False, act="none", residual="none", y="f32"):
    return {"name": name, "op": "linear", "w": w, "M": M, "N": N, "K": K, "x": x, "bias": bias,
            "act": act, "residual": residual, "y": y}


def _glu(name, w, M, N, K, x="f16", bias=False, act="silu", y="f16"):
    return {"name": name, "op": "glu", "w": w, "M": M, "N": N, "K": K, "x": x, "bias": bias,
            "act": act, "y": y}


def _norm(name, M, K, x="f32", residual="f32", y="f16", pad=0):
    return {"name": name, "op": "norm", "M": M, "K": K, "x": x, "residual": residual, "y": y,
            "pad": pad}


def listed():
    return [
        # one generated token: the attention output projection onto the residual stream
        _linear("linear f16 o m1", "f16", 1, 3584, 3584, residual="f32"),
        # one generated token: the down projection straight from its blocks, the long K
        _linear("linear q6_k down m1", "q6_k", 1, 3584, 18944, residual="f32"),
        # a few sequences decoded together: q|k|v with its bias, f32 activations in
        _linear("linear q4_k qkv m13", "q4_k", 13, 4608, 3584, x="f32", bias=True, y="f16"),
        # a ragged projection of a classifier or adapter head, no size a multiple of a tile
        _linear("linear f16 ragged m333", "f16", 333, 1000, 1048, bias=True, act="gelu", y="f16"),
        # a prompt of middling length through the up half of an ungated feed-forward
        _linear("linear q8_0 up m512", "q8_0", 512, 14336, 4096, bias=True, act="gelu_tanh",
                y="f16"),
        # a full prompt: the down projection from the resident cache onto the residual stream
        _linear("linear f16 down m2048", "f16", 2048, 3584, 18944, residual="f32"),
        # one generated token: gate and up from their blocks
        _glu("glu q4_k m1", "q4_k", 1, 14336, 4096),
        # a short prompt through a small model's gated layer, odd sizes
        _glu("glu q5_k ragged m100", "q5_k", 100, 2730, 1024, bias=True, act="gelu"),
        # a full prompt: gate and up from the resident cache, the largest product of a layer
        _glu("glu f16 m2048", "f16", 2048, 18944, 3584),
        # one generated token: the norm between two layers, where latency is all
        _norm("norm f16 m1", 1, 3584),
        # a full prompt on the int8 path: the norm writes the codes its product reads
        _norm("norm q8_1 m2048", 2048, 3584, y="q8_1"),
        # many rows of an odd width inside a wider buffer, f16 in
        _norm("norm odd f16 m4099", 4099, 1001, x="f16", residual="f16", y="f16", pad=7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "linear", "glu", "norm"))
    if op == "norm":
        M = _log(rng, 1, 16384)
        y = rng.choice(("f16", "f16", "f32", "q8_1"))
        K = _log(rng, 64, min(18944, max(64, (1 << 26) // M)))
        pad = rng.choice((0, 0, 1, 8, 24))
        if y == "q8_1":
            K = max(32, K // 32 * 32)
        return {"op": op, "M": M, "K": K, "x": rng.choice(("f32", "f32", "f16")),
                "residual": rng.choice(("f32", "f32", "f16", "none")), "y": y, "pad": pad}
    w = rng.choice(("f16", "f16", "f16") + FORMATS)
    step = 8 if w == "f16" else BLOCK[w][0]
    M = rng.choice((_log(rng, 1, 64), _log(rng, 1, 2048)))
    while True:
        N, K = _log(rng, 40, 18944), max(step, _log(rng, 256, 18944) // step * step)
        if N * K <= 3584 * 18944:
            break
    c = {"op": op, "w": w, "M": M, "N": N, "K": K, "x": rng.choice(("f16", "f16", "f32")),
         "bias": rng.random() < 0.5, "y": rng.choice(("f16", "f32"))}
    if op == "glu":
        c["act"] = rng.choice(("silu", "silu", "gelu", "gelu_tanh", "relu", "none"))
    else:
        c["act"] = rng.choice(("none", "none", "silu", "gelu", "gelu_tanh", "relu"))
        c["residual"] = rng.choice(("none", "f32", "f32", "f16"))
    return c


def work(case):
    """Every input read once, every output written once; two operations per
    multiply-add."""
    M, K = case["M"], case["K"]
    if case["op"] == "norm":
        b = M * K * SIZE[case["x"]] + 4 * K
        if case["residual"] != "none":
            b += 2 * M * K * SIZE[case["residual"]]      # read, and the sum written
        b += M * K + M * K // 4 if case["y"] == "q8_1" else M * K * SIZE[case["y"]]
        return {"bytes": b, "flops": 5 * M * K}
    N = case["N"]
    rows = 2 * N if case["op"] == "glu" else N
    if case["w"] == "f16":
        wb = rows * K * 2
    else:
        be, bb = BLOCK[case["w"]]
        wb = rows * (K // be) * bb
    b = wb + M * K * SIZE[case["x"]] + M * N * SIZE[case["y"]]
    b += 4 * rows if case["bias"] else 0
    if case.get("residual", "none") != "none":
        b += M * N * SIZE[case["residual"]]
    return {"bytes": b, "flops": 2 * M * rows * K}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _cache_ld(K):
    """Row stride of the f16 cache: one 128-byte line more where the row is a
    multiple of 2048 bytes."""
    return K + 64 if (2 * K) % 2048 == 0 else K


def _scale(g, shape, lo, device):
    """f16 block scales in [lo, 2·lo), as their two bytes."""
    s = (lo * (1 + torch.rand(shape, generator=g, device=device))).half()
    return s.unsqueeze(-1).view(torch.uint8)


def _blocks(g, fmt, N, K, device):
    """A quantized N×K weight with uniform codes and scales that give weights of
    a trained layer's size (about 0.02)."""
    be, bb = BLOCK[fmt]
    nb = K // be
    w = torch.randint(0, 256, (N, nb, bb), generator=g, device=device, dtype=torch.uint8)
    if fmt in ("q4_k", "q5_k"):
        lo = 6e-5 if fmt == "q4_k" else 3e-5
        w[..., 0:2] = _scale(g, (N, nb), lo, device)
        w[..., 2:4] = _scale(g, (N, nb), 7.6 * 6e-5, device)
    elif fmt == "q6_k":
        sc = torch.randint(-32, 33, (N, nb, 16), generator=g, device=device)
        w[..., 192:208] = sc.to(torch.int8).view(torch.uint8)
        w[..., 208:210] = _scale(g, (N, nb), 6e-5, device)
    elif fmt == "q5_1":
        w[..., 0:2] = _scale(g, (N, nb), 1.5e-3, device)
        w[..., 2:4] = (-_scale(g, (N, nb), 2.3e-2, device).view(torch.float16)).view(torch.uint8)
    else:
        lo = {"q4_0": 3e-3, "q5_0": 1.5e-3, "q8_0": 2e-4}[fmt]
        w[..., 0:2] = _scale(g, (N, nb), lo, device)
    return w.view(-1)


def _activations(g, M, K, dtype, device, pad=0):
    """Normal activations with a few large channels, as a transformer's are."""
    big = 1 + 9 * (torch.rand(K + pad, generator=g, device=device) < 0.01).float()
    x = torch.randn(M, K + pad, generator=g, device=device) * big
    return x.to(dtype)[:, :K]


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    M, K = case["M"], case["K"]
    s = dict(case)
    if case["op"] == "norm":
        s["xt"] = _activations(g, M, K, DTYPE[case["x"]], dev, case["pad"])
        s["weight"] = 1 + 0.2 * torch.randn(K, generator=g, device=dev)
        s["rt"] = None
        if case["residual"] != "none":
            s["rt"] = 4 * _activations(g, M, K, torch.float32, dev, case["pad"])
            s["rt"] = s["rt"].to(DTYPE[case["residual"]])
        return s
    N = case["N"]
    rows = 2 * N if case["op"] == "glu" else N
    s["xt"] = _activations(g, M, K, DTYPE[case["x"]], dev)
    if case["w"] == "f16":
        w = torch.zeros(rows, _cache_ld(K), dtype=torch.float16, device=dev)
        w[:, :K] = torch.randn(rows, K, generator=g, device=dev, dtype=torch.float16) * 0.02
        s["wt"] = w
    else:
        s["wt"] = _blocks(g, case["w"], rows, K, dev)
    s["bt"] = torch.randn(rows, generator=g, device=dev) if case["bias"] else None
    s["rt"] = None
    if case.get("residual", "none") != "none":
        r = 4 * torch.randn(M, N, generator=g, device=dev)
        s["rt"] = r.to(DTYPE[case["residual"]])
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

def _f16(b):
    """The f16 value of two bytes (last axis), in f32, the axis kept as 1."""
    return b.contiguous().view(torch.float16).float()


def _nibbles(q):
    """Low nibbles then high nibbles of the last axis, as f32."""
    return torch.cat((q & 15, q >> 4), -1).float()


def _bits(qh, n):
    """The bits of little-endian bytes (last axis), lowest first: n of them."""
    k = torch.arange(8, device=qh.device, dtype=torch.uint8)
    return ((qh.unsqueeze(-1) >> k) & 1).flatten(-2)[..., :n].float()


def _k_scales(s):
    """The eight 6-bit scales and eight 6-bit mins packed into 12 bytes."""
    a, b, c = s[..., 0:4], s[..., 4:8], s[..., 8:12]
    sc = torch.cat((a & 63, (c & 15) | ((a >> 6) << 4)), -1)
    mn = torch.cat((b & 63, (c >> 4) | ((b >> 6) << 4)), -1)
    return sc.float(), mn.float()


def _dequant(w, fmt, N, K):
    """The weight's values: each computed in f32 and rounded once to f16."""
    be, bb = BLOCK[fmt]
    w = w.view(N, K // be, bb)
    if fmt == "q8_0":
        v = _f16(w[..., 0:2]) * w[..., 2:].view(torch.int8).float()
    elif fmt == "q4_0":
        v = _f16(w[..., 0:2]) * (_nibbles(w[..., 2:]) - 8)
    elif fmt == "q5_0":
        v = _f16(w[..., 0:2]) * (_nibbles(w[..., 6:]) + 16 * _bits(w[..., 2:6], 32) - 16)
    elif fmt == "q5_1":
        v = _f16(w[..., 0:2]) * (_nibbles(w[..., 8:]) + 16 * _bits(w[..., 4:8], 32))
        v = v + _f16(w[..., 2:4])
    elif fmt == "q6_k":
        ql = w[..., 0:128].unflatten(-1, (2, 1, 64))
        qh = w[..., 128:192].unflatten(-1, (2, 1, 32))
        low = torch.cat((ql & 15, ql >> 4), -2).unflatten(-1, (2, 32)).flatten(-3, -2)
        high = torch.cat([(qh >> s) & 3 for s in (0, 2, 4, 6)], -2)
        q = (low | (high << 4)).float().flatten(-3).unflatten(-1, (16, 16)) - 32
        sc = w[..., 192:208].view(torch.int8).float().unsqueeze(-1)
        v = ((_f16(w[..., 208:210]).unsqueeze(-1) * sc) * q).flatten(-2)
    else:
        sc, mn = _k_scales(w[..., 4:16])
        q0 = 48 if fmt == "q5_k" else 16
        q = _nibbles(w[..., q0:].unflatten(-1, (4, 32))).unflatten(-1, (2, 32)).flatten(-3, -2)
        if fmt == "q5_k":
            k = torch.arange(8, device=w.device, dtype=torch.uint8).unsqueeze(-1)
            q = q + 16 * ((w[..., 16:48].unsqueeze(-2) >> k) & 1).float()
        v = (_f16(w[..., 0:2]) * sc).unsqueeze(-1) * q - (_f16(w[..., 2:4]) * mn).unsqueeze(-1)
        v = v.flatten(-2)
    return v.reshape(N, K).half().float()


def _act(v, act):
    if act == "relu":
        return torch.clamp(v, min=0)
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _plain_product(s, rows):
    K = s["K"]
    w = s["wt"][:, :K].float() if s["w"] == "f16" else _dequant(s["wt"], s["w"], rows, K)
    y = s["xt"].half().float() @ w.t()
    return y if s["bt"] is None else y + s["bt"]


def _plain_norm(s):
    h = s["xt"].float()
    if s["rt"] is not None:
        h = h + s["rt"].float()
        h16 = h.to(s["rt"].dtype)
        h = h16.float()                       # the norm is of the stream as stored
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["weight"]
    out = {} if s["rt"] is None else {"h": h16}
    if s["y"] != "q8_1":
        out["y"] = y.to(DTYPE[s["y"]])
        return out
    b = y.unflatten(-1, (-1, 32))
    d = b.abs().amax(-1, keepdim=True) / 127
    t = torch.where(d > 0, b / d, torch.zeros_like(b))
    q = torch.trunc(t)
    q = q + torch.sign(t) * ((t - q).abs() >= 0.5)      # halves away from zero
    return out | {"d": d[..., 0], "s": (d[..., 0] * q.sum(-1)).half(), "y": (q * d).half()}


def run(state):
    s = state
    if own:
        return _run_own(s)
    if s["op"] == "norm":
        return _plain_norm(s)
    N = s["N"]
    if s["op"] == "glu":
        v = _plain_product(s, 2 * N)
        return {"y": (_act(v[:, :N], s["act"]) * v[:, N:]).to(DTYPE[s["y"]])}
    v = _act(_plain_product(s, N), s["act"])
    if s["rt"] is not None:
        v = v + s["rt"].float()
    return {"y": v.to(DTYPE[s["y"]])}


# ---------------------------------------------------------------------------
# The package's operators
# ---------------------------------------------------------------------------

def _run_own(s):
    import quantized_weight_prefill_q4_amd as mq

    if s["op"] == "norm":
        if s["y"] != "q8_1":
            y, h = mq.add_rms_norm(s["xt"], s["weight"], residual=s["rt"], eps=EPS,
                                   out_dtype=DTYPE[s["y"]])
            return {"y": y} if h is None else {"h": h, "y": y}
        xq, ds, h = mq.add_rms_norm_q8_1(s["xt"], s["weight"], residual=s["rt"], eps=EPS)
        # the codes as the values they stand for
        M, K = s["M"], s["K"]
        d = ds[..., 0]
        y = torch.empty(M, K // 32, 32, dtype=torch.float16, device=xq.device)
        torch.mul(xq[:, :K].unflatten(-1, (-1, 32)), d.unsqueeze(-1), out=y)
        out = {"d": d, "s": ds[..., 1].half(), "y": y}
        return out if h is None else out | {"h": h}
    N, K, act = s["N"], s["K"], s["act"]
    y = DTYPE[s["y"]]
    if s["op"] == "glu":
        if s["w"] == "f16":
            return {"y": mq.glu_f16cache(s["xt"], s["wt"], K, act=act, bias=s["bt"], out_dtype=y)}
        return {"y": mq.glu_fused(s["xt"], s["wt"], s["w"], N, K, act=act, bias=s["bt"],
                                  out_dtype=y)}
    if s["w"] == "f16":
        return {"y": mq.linear_f16cache(s["xt"], s["wt"], K, bias=s["bt"], act=act,
                                        residual=s["rt"], out_dtype=y)}
    return {"y": mq.linear_fused(s["xt"], s["wt"], s["w"], N, K, bias=s["bt"], act=act,
                                 residual=s["rt"], out_dtype=y)}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _half_at(raw, at):
    """The f16 at byte `at` of every block, in f64."""
    bits = raw[:, :, at].int() | (raw[:, :, at + 1].int() << 8)
    e, m = (bits >> 10) & 31, (bits & 1023).double()
    v = torch.where(e > 0, (1 + m / 1024) * torch.exp2(e.double() - 15), m * 2.0 ** -24)
    return torch.where(bits >= 32768, -v, v)


def _exact_weight(raw, fmt, N, K):
    """Element by element from the block layouts: the place of element e of a
    block is looked up for all blocks at once."""
    be, bb = BLOCK[fmt]
    raw = raw.view(N, K // be, bb)
    e = torch.arange(be, device=raw.device)

    def byte(at):
        return raw[:, :, at].int()

    if be == 32:
        d = _half_at(raw, 0).unsqueeze(-1)
        if fmt == "q8_0":
            b = byte(2 + e)
            v = d * (b - 256 * (b > 127)).double()
        else:
            q0 = {"q4_0": 2, "q5_0": 6, "q5_1": 8}[fmt]
            q = (byte(q0 + e % 16) >> (4 * (e // 16))) & 15
            if fmt != "q4_0":
                q = q + 16 * ((byte((2 if fmt == "q5_0" else 4) + e // 8) >> (e % 8)) & 1)
            if fmt == "q5_1":
                v = d * q.double() + _half_at(raw, 2).unsqueeze(-1)
            else:
                v = d * (q - (8 if fmt == "q4_0" else 16)).double()
    elif fmt == "q6_k":
        half, grp, l = e // 128, (e % 128) // 32, e % 32
        lo = (byte(64 * half + 32 * (grp % 2) + l) >> (4 * (grp // 2))) & 15
        hi = (byte(128 + 32 * half + l) >> (2 * grp)) & 3
        s = byte(192 + e // 16)
        v = _half_at(raw, 208).unsqueeze(-1) * ((s - 256 * (s > 127)) * (lo + 16 * hi - 32)).double()
    else:
        sub, l = e // 32, e % 32
        j = sub % 4
        first, lo_s, lo_m, top = sub < 4, byte(4 + j), byte(8 + j), byte(12 + j)
        sc = torch.where(first, lo_s & 63, (top & 15) + 16 * (lo_s >> 6))
        mn = torch.where(first, lo_m & 63, (top >> 4) + 16 * (lo_m >> 6))
        q = (byte((48 if fmt == "q5_k" else 16) + 32 * (sub // 2) + l) >> (4 * (sub % 2))) & 15
        if fmt == "q5_k":
            q = q + 16 * ((byte(16 + l) >> sub) & 1)
        v = _half_at(raw, 0).unsqueeze(-1) * (sc * q).double()
        v = v - _half_at(raw, 2).unsqueeze(-1) * mn.double()
    # the weights are f16 by definition: f32 first, then f16
    return v.reshape(N, K).float().half().double()


def _exact_act(v, act):
    if act == "relu":
        return v * (v > 0)
    if act == "silu":
        return v * torch.special.expit(v)
    if act == "gelu":
        return 0.5 * v * torch.special.erfc(-v / math.sqrt(2))
    if act == "gelu_tanh":
        return v * torch.special.expit(2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3))
    return v


def exact(case, seed):
    s = prepare(case, seed)
    K = case["K"]
    if case["op"] == "norm":
        h = s["xt"].double()
        out = {}
        if s["rt"] is not None:
            h = h + s["rt"].double()
            out["h"] = h
            h = h.to(DTYPE[case["residual"]]).double()
        y = h / torch.sqrt(h.pow(2).sum(-1, keepdim=True) / K + EPS) * s["weight"].double()
        if case["y"] != "q8_1":
            return out | {"y": y}
        b = y.view(case["M"], K // 32, 32)
        d = b.abs().max(-1).values / 127
        q = torch.floor(b.abs() / d.clamp(min=1e-300).unsqueeze(-1) + 0.5) * torch.sign(b)
        return out | {"d": d, "s": d * q.sum(-1), "y": q * d.unsqueeze(-1)}
    N = case["N"]
    rows = 2 * N if case["op"] == "glu" else N
    w = s["wt"][:, :K].double() if case["w"] == "f16" else _exact_weight(s["wt"], case["w"], rows, K)
    v = torch.mm(s["xt"].half().double(), w.t().contiguous())
    if s["bt"] is not None:
        v += s["bt"].double()
    if case["op"] == "glu":
        return {"y": _exact_act(v[:, :N], case["act"]) * v[:, N:]}
    v = _exact_act(v, case["act"])
    if s["rt"] is not None:
        v = v + s["rt"].double()
    return {"y": v}
