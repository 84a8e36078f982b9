"""What the operators around the quantised products are measured on: the
residual add with RMS norm into 8-bit activations, the append of rotated keys
and values to a paged 4-bit cache, and the attention over that cache.

`run` computes them in plain torch operations, or with `own` through the
library.  The two agree on the layouts that the library documents
(include/qmv.h): Q8_0 / Q8_K blocks, and the 4-bit pages below.

A page holds `page` tokens; for each key/value head it is page * 36 * nb bytes
(nb = head_dim / 32): the K codes, the V codes, the K scales, the V scales.
  K codes  [token][g 0..3][b][4 bytes]: the 8 nibbles (low first) of the four
           bytes are elements 0, 2, 4, 6, 1, 3, 5, 7 of 32b + 8g + ...
  V codes  [token / 4][m 0..15][b][token % 4]: low nibble element 32b + 2m,
           high nibble 32b + 2m + 1
  scales   [token][b] fp16; the value is d * (nibble - 8)
"""
import math

import torch

own = False

EPS = 1e-5
# nibble j of a K word holds element NIB[j] of its eight
NIB = (0, 2, 4, 6, 1, 3, 5, 7)


# --------------------------------------------------------------- the cases --

def listed():
    big = dict(hq=32, hkv=8, d=128, rot=128, halves=False)    # the 8B-class layer of the benchmark (4096 q, 1024 k/v rows)
    small = dict(hq=14, hkv=2, d=64, rot=64, halves=True)     # the 896-wide layer of the benchmark (896 q, 128 k/v rows)
    return [
        # one token through the 8B-class layer: latency
        dict(name="norm_q8_0_1x4096", op="norm", fmt="q8_0", rows=1, k=4096, res=True),
        # a decode batch on the Q8_K path
        dict(name="norm_q8_k_16x4096", op="norm", fmt="q8_k", rows=16, k=4096, res=True),
        # a prefill of 2048 tokens
        dict(name="norm_q8_0_2048x4096", op="norm", fmt="q8_0", rows=2048, k=4096, res=True),
        # one token appended: latency
        dict(name="append_1_token", op="append", b=1, n_lo=1, n_hi=1, l_lo=777, l_hi=777, page=64, **big),
        # a decode batch of the small model, rotation by halves
        dict(name="append_64_tokens", op="append", b=64, n_lo=1, n_hi=1, l_lo=1, l_hi=2000, page=16, **small),
        # ragged prompts appended in one call
        dict(name="append_prompts", op="append", b=8, n_lo=33, n_hi=1023, l_lo=1023, l_hi=1500, page=64, **big),
        # a short chat of the small model: latency
        dict(name="attn_1x500", op="attn", b=1, n_lo=1, n_hi=1, l_lo=500, l_hi=500, page=64, window=0, **small),
        # one sequence of some thousand tokens
        dict(name="attn_1x4097", op="attn", b=1, n_lo=1, n_hi=1, l_lo=4097, l_hi=4097, page=64, window=0, **big),
        # a serving batch of ragged lengths
        dict(name="attn_32x8191", op="attn", b=32, n_lo=1, n_hi=1, l_lo=301, l_hi=8191, page=32, window=0, **big),
        # one very long context
        dict(name="attn_1x131072", op="attn", b=1, n_lo=1, n_hi=1, l_lo=131072, l_hi=131072, page=256, window=0, **big),
        # a prompt's chunks of 256 tokens behind cached prefixes
        dict(name="attn_chunks", op="attn", b=4, n_lo=250, n_hi=256, l_lo=256, l_hi=4000, page=64, window=0, **big),
        # a whole prompt with a sliding window
        dict(name="attn_prompt_window", op="attn", b=1, n_lo=2048, n_hi=2048, l_lo=2048, l_hi=2048, page=64, window=1024, **big),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "append", "attn", "attn"))
    if op == "norm":
        fmt = rng.choice(("q8_0", "q8_k"))
        unit = 32 if fmt == "q8_0" else 256
        k = unit * max(1, _log(rng, 256, 16384) // unit)
        rows = min(_log(rng, 1, 2048), max(1, 2048 * 4096 // k))
        return dict(op="norm", fmt=fmt, rows=rows, k=k, res=rng.random() < 0.75)
    d = rng.choice((64, 96, 128, 256))
    hkv = rng.choice((1, 2, 3, 4, 8))
    g = rng.choice((1, 2, 4, 5, 7, 8, 16))
    c = dict(op=op, hq=g * hkv, hkv=hkv, d=d, rot=rng.choice((d, d, d // 2)), halves=rng.random() < 0.5,
             page=rng.choice((16, 32, 64, 128, 256)))
    if op == "append":
        b = _log(rng, 1, 64)
        n = _log(rng, 1, 512) if rng.random() < 0.5 else 1
        n = max(1, min(n, 4096 * 48 * 128 // (b * (g + 2) * hkv * d)))
        lo = n + rng.randrange(0, 500)
        return dict(c, b=b, n_lo=max(1, n // 2), n_hi=n, l_lo=lo, l_hi=lo + rng.randrange(0, 1500))
    c["window"] = rng.choice((0, 0, 0, 100, 512, 1000))
    if rng.random() < 0.65:
        b = _log(rng, 1, 64)
        most = max(64, 131072 * 8 * 128 // (b * hkv * d))
        hi = _log(rng, 1, min(most, 65536))
        return dict(c, b=b, n_lo=1, n_hi=1, l_lo=max(1, hi // 7), l_hi=hi)
    n = _log(rng, 2, 1024)
    b = rng.choice((1, 2, 3))
    hi = n + _log(rng, 1, 4096)
    while b * n * hi * g * hkv * d > 2048 * 2048 * 32 * 128:
        n, hi = n // 2 + 1, hi // 2 + 1
    return dict(c, b=b, n_lo=max(1, n // 3), n_hi=n, l_lo=max(n, hi // 3), l_hi=max(n, hi))


def _spread(lo, hi, b):
    """b whole numbers from lo to hi, unevenly spread, the same for every seed."""
    if b == 1:
        return [hi]
    return [lo + (hi - lo) * ((i * 7919) % b) // (b - 1) for i in range(b)]


def _seqs(case):
    """New tokens and length (with them) of each sequence."""
    n = _spread(case["n_lo"], case["n_hi"], case["b"])
    return n, [max(a, b) for a, b in zip(n, _spread(case["l_lo"], case["l_hi"], case["b"]))]


def _pairs(n, length, window):
    """(visible (query, key) pairs, keys that any query sees) of one sequence."""
    first = length - n
    if not window:
        return n * first + n * (n + 1) // 2, length
    see = [min(p + 1, window) for p in range(first, length)]
    return sum(see), length - max(0, first + 1 - window)


def work(case):
    if case["op"] == "norm":
        rows, k = case["rows"], case["k"]
        held = 34 / 32 if case["fmt"] == "q8_0" else 292 / 256
        return {"bytes": rows * k * (4 + (8 if case["res"] else 0) + held) + 4 * k, "flops": rows * k * 8}
    n, length = _seqs(case)
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "append":
        t = sum(n)
        return {"bytes": t * d * (8 * hq + 2 * hkv * (4 + 18 / 32)), "flops": t * d * (3 * hq + 9 * hkv)}
    both = [_pairs(a, b, case["window"]) for a, b in zip(n, length)]
    return {"bytes": sum(k for _, k in both) * hkv * d * 2 * 18 / 32 + 8 * sum(n) * hq * d,
            "flops": 4 * hq * d * sum(p for p, _ in both)}


# -------------------------------------------------------------- the inputs --

def _rand(gen, *shape, scale=1.0):
    return torch.randn(*shape, generator=gen, device="cuda") * scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 2 + 1)
    s = {"case": dict(case)}
    if case["op"] == "norm":
        rows, k = case["rows"], case["k"]
        # a residual stream with some channels much larger than the rest
        wide = 1 + 20 * (torch.rand(k, generator=gen, device="cuda") < 0.01)
        s["x"] = _rand(gen, rows, k, scale=0.3)
        s["res"] = _rand(gen, rows, k) * wide if case["res"] else None
        s["w"] = 1 + _rand(gen, k, scale=0.2)
        return s
    n, length = _seqs(case)
    b, page, hq, hkv, d = case["b"], case["page"], case["hq"], case["hkv"], case["d"]
    nb, t = d // 32, sum(n)
    per = [-(-x // page) for x in length]
    pages = sum(per)
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)  # pages in no order
    table = torch.zeros(b, max(per), dtype=torch.int32, device="cuda")
    at = 0
    for i, m in enumerate(per):
        table[i, :m] = order[at:at + m]
        at += m
    starts = [sum(n[:i]) for i in range(b + 1)]
    one = case["n_hi"] == 1
    s.update(table=table, lens=torch.tensor(length, dtype=torch.int32, device="cuda"), t=t,
             start=None if one else torch.tensor(starts, dtype=torch.int32, device="cuda"),
             max_len=max(length), max_n=max(n), scale=1 / math.sqrt(d))
    s["seq"] = torch.repeat_interleave(torch.arange(b, device="cuda"), torch.tensor(n, device="cuda"))
    s["pos"] = torch.cat([torch.arange(x - m, x, device="cuda") for m, x in zip(n, length)])
    if case["op"] == "append":
        s["pages"] = torch.zeros(pages * hkv * page * 36 * nb, dtype=torch.uint8, device="cuda")
        s["q"], s["k"], s["v"] = _rand(gen, t, hq * d), _rand(gen, t, hkv * d, scale=2.0), _rand(gen, t, hkv * d)
        s["freq"] = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, device="cuda") / case["rot"])
        return s
    s["q"] = _rand(gen, t, hq * d, scale=2.0)
    cells = torch.empty(pages, hkv, page * 36 * nb, dtype=torch.uint8, device="cuda")
    step = max(1, (64 << 20) // (hkv * page * d))
    for i in range(0, pages, step):
        m = min(step, pages - i)
        k = _q4_0(_rand(gen, m, hkv, page, nb, 32))
        v = _q4_0(_rand(gen, m, hkv, page, nb, 32))
        cells[i:i + m, :, :page * 16 * nb] = _pack_k(k[0]).reshape(m, hkv, -1)
        cells[i:i + m, :, page * 16 * nb:page * 32 * nb] = _pack_v(v[0]).reshape(m, hkv, page // 4, 4, 16, nb).permute(0, 1, 2, 4, 5, 3).reshape(m, hkv, -1)
        cells[i:i + m, :, page * 32 * nb:page * 34 * nb] = k[1].view(torch.uint8).reshape(m, hkv, -1)
        cells[i:i + m, :, page * 34 * nb:] = v[1].view(torch.uint8).reshape(m, hkv, -1)
    s["pages"] = cells.reshape(-1)
    return s


# --------------------------------------------------------- the plain forms --

def _q4_0(x):
    """x [..., 32] f32 -> codes 0..15 (uint8) and fp16 scales [...] of Q4_0.
    The first value of the largest magnitude gives d = value / -8."""
    top = x.gather(-1, x.abs().argmax(-1, keepdim=True))
    d = top / -8
    inv = (1.0 / d.double()).float()
    inv = torch.where(torch.isfinite(inv), inv, 0.0)
    return (x * inv + 8.5).clamp(0, 15).to(torch.uint8), d.squeeze(-1).half()


def _pack_k(code):
    """[..., nb, 32] codes -> [..., 4, nb, 4] bytes."""
    c = code.unflatten(-1, (4, 8))[..., list(NIB)].transpose(-3, -2)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _pack_v(code):
    """[..., nb, 32] codes -> [..., 16, nb] bytes."""
    c = code.transpose(-2, -1)
    return c[..., 0::2, :] | (c[..., 1::2, :] << 4)


def _plain_norm(s):
    x, res, w, case = s["x"], s["res"], s["w"], s["case"]
    h = x if res is None else x + res
    hd = h.double()  # codes next to a border: 64 bits up to the value that is quantised
    y = (hd * torch.rsqrt(hd.square().mean(-1, keepdim=True) + EPS) * w).float()
    out = {} if res is None else {"h": h}
    size = 32 if case["fmt"] == "q8_0" else 256
    yb = y.unflatten(-1, (-1, size))
    d = (yb.abs().amax(-1, keepdim=True).double() / 127).float()  # torch divides f32 by a number as a product: not the rounded quotient
    inv = (1.0 / d.double()).float()
    t = yb * torch.where(torch.isfinite(inv), inv, 0.0)
    code = torch.trunc(t) + torch.sign(t) * ((t - torch.trunc(t)).abs() >= 0.5)  # halves away from zero
    if case["fmt"] == "q8_0":
        return {**out, "values": code * d.half().float()}
    return {**out, "values": code * d, "sums": code.unflatten(-1, (16, 16)).sum(-1).to(torch.int16)}


def _rotate(x, pos, freq, rot, halves):
    """x [T, heads, D] f32 rotated at the positions, in 64 bits (angles of far positions), rounded once."""
    a = pos.double()[:, None] * freq
    cos, sin = torch.cos(a)[:, None], torch.sin(a)[:, None]
    y = x.double()
    x0, x1 = (y[..., :rot // 2], y[..., rot // 2:rot]) if halves else (y[..., 0:rot:2], y[..., 1:rot:2])
    y0, y1 = x0 * cos - x1 * sin, x0 * sin + x1 * cos
    turned = torch.cat((y0, y1), -1) if halves else torch.stack((y0, y1), -1).flatten(-2)
    return torch.cat((turned.float(), x[..., rot:]), -1)


def _plain_append(s):
    c = s["case"]
    page, hkv, d = c["page"], c["hkv"], c["d"]
    nb, t = d // 32, s["t"]
    q = _rotate(s["q"].view(t, c["hq"], d), s["pos"], s["freq"], c["rot"], c["halves"])
    k = _rotate(s["k"].view(t, hkv, d), s["pos"], s["freq"], c["rot"], c["halves"])
    kc, kd = _q4_0(k.unflatten(-1, (nb, 32)))
    vc, vd = _q4_0(s["v"].view(t, hkv, nb, 32))
    cells = s["pages"].view(-1, hkv, page * 36 * nb)
    at, off = s["table"][s["seq"], s["pos"] // page].long(), s["pos"] % page
    cells[:, :, :page * 16 * nb].unflatten(-1, (page, 4, nb, 4))[at, :, off] = _pack_k(kc)
    cells[:, :, page * 16 * nb:page * 32 * nb].unflatten(-1, (page // 4, 16, nb, 4))[at, :, off // 4, :, :, off % 4] = _pack_v(vc)
    cells[:, :, page * 32 * nb:page * 34 * nb].unflatten(-1, (page, 2 * nb))[at, :, off] = kd.view(torch.uint8)
    cells[:, :, page * 34 * nb:].unflatten(-1, (page, 2 * nb))[at, :, off] = vd.view(torch.uint8)
    value = lambda code, scale: ((code.float() - 8) * scale.float()[..., None]).view(t, hkv * d)  # noqa: E731
    return {"q": q.reshape(t, -1), "k": value(kc, kd), "v": value(vc, vd)}


def _plain_attn(s):
    c = s["case"]
    page, hq, hkv, d, b = c["page"], c["hq"], c["hkv"], c["d"], c["b"]
    nb, g, t = d // 32, hq // hkv, s["t"]
    cells = s["pages"].view(-1, hkv, page * 36 * nb)[s["table"].long()]  # [b, pages, hkv, bytes]
    m = cells.shape[1] * page
    raw = cells[..., :page * 16 * nb].reshape(b, -1, hkv, page, 4, nb, 4)
    k = torch.stack((raw & 15, raw >> 4), -1).flatten(-2)[..., [NIB.index(e) for e in range(8)]]
    k = k.permute(0, 2, 1, 3, 5, 4, 6).reshape(b, hkv, m, nb, 32).float() - 8
    raw = cells[..., page * 16 * nb:page * 32 * nb].reshape(b, -1, hkv, page // 4, 16, nb, 4)
    v = torch.stack((raw & 15, raw >> 4), -1).permute(0, 2, 1, 3, 6, 5, 4, 7).reshape(b, hkv, m, nb, 32).float() - 8
    scale = lambda lo: cells[..., page * lo * nb:page * (lo + 2) * nb].contiguous().view(torch.float16).view(  # noqa: E731
        b, -1, hkv, page, nb).transpose(1, 2).reshape(b, hkv, m, nb, 1).float()
    k = (k * scale(32)).view(b, hkv, m, d)
    v = (v * scale(34)).view(b, hkv, m, d)
    n = s["max_n"]
    if s["start"] is None:
        row = torch.arange(t, device="cuda")
    else:
        row = s["seq"] * n + torch.arange(t, device="cuda") - s["start"].long()[s["seq"]]
    q = torch.zeros(b * n, hkv, g, d, device="cuda")
    q[row] = s["q"].view(t, hkv, g, d)
    pos = torch.full((b * n,), -1, device="cuda")
    pos[row] = s["pos"]
    q = q.view(b, n, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * n, d)
    score = torch.matmul(q, k.transpose(-1, -2)).view(b, hkv, g, n, m) * s["scale"]
    key, pos = torch.arange(m, device="cuda"), pos.view(b, 1, 1, n, 1)
    seen = key <= pos
    if c["window"]:
        seen = seen & (key > pos - c["window"])
    score = score.masked_fill(~seen, -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True).clamp(min=-3e38))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-38)
    out = torch.matmul(p.view(b, hkv, g * n, m), v).view(b, hkv, g, n, d).permute(0, 3, 1, 2, 4)
    return out.reshape(b * n, hq * d)[row]


# ------------------------------------------------------------ the library --

def _own_norm(s):
    import gguf_quantized_matvec_amd as lib
    rows, k = s["case"]["rows"], s["case"]["k"]
    if s["case"]["fmt"] == "q8_0":
        h, xq = lib.add_rmsnorm(s["x"], s["w"], EPS, res=s["res"])
        blocks = xq[:rows * (k // 32) * 34].view(rows, k // 32, 34)
        out = {"values": blocks[..., 2:].view(torch.int8) * blocks[..., :2].view(torch.float16).float()}
    else:
        h, xq = lib.add_rmsnorm_q8k(s["x"], s["w"], EPS, res=s["res"])
        blocks = xq[:rows * (k // 256) * 292].view(rows, k // 256, 292)
        out = {"values": blocks[..., 4:260].view(torch.int8) * blocks[..., :4].view(torch.float32),
               "sums": blocks[..., 260:].view(torch.int16)}
    return out if s["res"] is None else {"h": h, **out}


def _own_append(s):
    import gguf_quantized_matvec_amd as lib
    c = s["case"]
    cache = lib.KVCache(s["pages"], c["page"], c["hkv"], c["d"])
    batch = lib.KVBatch(s["table"], s["lens"], s["start"], s["t"], s["max_len"])
    q = lib.kv_append(cache, batch, s["q"], s["k"], s["v"], s["freq"], halves=c["halves"])
    k, v = lib.kv_read(cache, batch)
    return {"q": q, "k": k, "v": v}


def _own_attn(s):
    import gguf_quantized_matvec_amd as lib
    c = s["case"]
    cache = lib.KVCache(s["pages"], c["page"], c["hkv"], c["d"])
    batch = lib.KVBatch(s["table"], s["lens"], s["start"], s["t"], s["max_len"])
    return lib.kv_attention(cache, batch, s["q"], s["scale"], window=c["window"])


def run(state):
    if own:
        return {"norm": _own_norm, "append": _own_append, "attn": _own_attn}[state["case"]["op"]](state)
    return {"norm": _plain_norm, "append": _plain_append, "attn": _plain_attn}[state["case"]["op"]](state)


# ------------------------------------------------- the definitions, 64 bits --

def _f32(x):
    """x (64 bits) rounded to 32 bits where the definition rounds, and held in 64 again."""
    return x.float().double()


def _exact_norm(s):
    case = s["case"]
    x, w = s["x"].double(), s["w"].double()
    h = x if s["res"] is None else _f32(x + s["res"].double())
    rows, k = h.shape
    norm = torch.sqrt((h * h).sum(1) / k + EPS)
    y = _f32(h * (w[None, :] / norm[:, None]))
    size = 32 if case["fmt"] == "q8_0" else 256
    y = y.reshape(rows * (k // size), size)
    d = _f32(y.abs().max(1, keepdim=True).values / 127)
    inv = _f32(1 / d)
    inv[torch.isinf(inv)] = 0
    t = _f32(y * inv)
    code = torch.floor(t.abs() + 0.5) * torch.sign(t)
    held = d.half().double() if size == 32 else d
    out = {"values": (code * held).view(rows, -1, size)}
    if size == 256:
        out["sums"] = None
    return out if s["res"] is None else {"h": h, **out}


def _exact_turn(x, s):
    """x [T, heads, D]: the rotation as a product of complex numbers."""
    c = s["case"]
    half, y = c["rot"] // 2, x.double()
    z = torch.complex(y[..., :half], y[..., half:2 * half]) if c["halves"] else torch.view_as_complex(y[..., :c["rot"]].reshape(*y.shape[:2], half, 2).contiguous())
    turn = s["pos"].double()[:, None, None] * s["freq"]
    z = z * torch.polar(torch.ones_like(turn), turn)
    out = y.clone()
    if c["halves"]:
        out[..., :half], out[..., half:2 * half] = z.real, z.imag
    else:
        out[..., 0:c["rot"]:2], out[..., 1:c["rot"]:2] = z.real, z.imag
    return out


def _exact_q4(y):
    """y [T, heads * D] (64 bits, already rounded to 32) -> the values of its Q4_0 blocks."""
    x = y.reshape(-1, 32)
    up, down = x.max(1).values, x.min(1).values
    where = (x == up[:, None]).int().argmax(1) < (x == down[:, None]).int().argmax(1)
    top = torch.where(up > -down, up, torch.where(up < -down, down, torch.where(where, up, down)))
    d = top / -8
    inv = _f32(1 / d)
    inv[torch.isinf(inv)] = 0
    code = torch.floor(_f32(_f32(x * inv[:, None]) + 8.5)).clamp(max=15)
    return ((code - 8) * d.half().double()[:, None]).reshape(y.shape)


def _exact_append(s):
    c = s["case"]
    t = s["t"]
    k = _f32(_exact_turn(s["k"].view(t, c["hkv"], -1), s)).reshape(t, -1)
    q = _exact_turn(s["q"].view(t, c["hq"], -1), s).reshape(t, -1)
    return {"q": q, "k": _exact_q4(k), "v": _exact_q4(s["v"].double())}


def _exact_attn(s):
    """One sequence and one key/value head at a time, the codes read nibble by nibble."""
    c = s["case"]
    page, hkv, d = c["page"], c["hkv"], c["d"]
    nb, g = d // 32, c["hq"] // hkv
    n, length = _seqs(c)
    e = torch.arange(d, device="cuda")
    b, i = e // 32, e % 32
    spot = torch.tensor([0, 4, 1, 5, 2, 6, 3, 7], device="cuda")[i % 8]  # the nibble of element i % 8
    k_byte, k_up = (i // 8) * 4 * nb + b * 4 + spot // 2, spot % 2
    v_byte, v_up = (i // 2) * 4 * nb + b * 4, i % 2
    out = torch.empty(s["t"], c["hq"] * d, dtype=torch.float64, device="cuda")
    flat, size = s["pages"], page * 36 * nb
    at = 0
    for j in range(c["b"]):
        low = 0 if not c["window"] else max(0, length[j] - n[j] + 1 - c["window"])
        key = torch.arange(low, length[j], device="cuda")
        pos = torch.arange(length[j] - n[j], length[j], device="cuda").repeat_interleave(g)
        for head in range(hkv):
            base = (s["table"][j].long()[key // page] * hkv + head) * size
            off = key % page
            kc = (flat[base[:, None] + off[:, None] * 16 * nb + k_byte] >> (4 * k_up).to(torch.uint8)) & 15
            vc = (flat[base[:, None] + page * 16 * nb + (off // 4)[:, None] * 64 * nb + (off % 4)[:, None] + v_byte] >> (4 * v_up).to(torch.uint8)) & 15
            half = flat.view(torch.float16)
            kd = half[base[:, None] // 2 + (page * 32 * nb // 2) + off[:, None] * nb + b].double()
            vd = half[base[:, None] // 2 + (page * 34 * nb // 2) + off[:, None] * nb + b].double()
            k, v = kd * (kc.double() - 8), vd * (vc.double() - 8)
            q = s["q"][at:at + n[j], head * g * d:(head + 1) * g * d].double().reshape(n[j] * g, d)
            z = (q @ k.T) * s["scale"]
            z[key[None, :] > pos[:, None]] = -math.inf
            if c["window"]:
                z[key[None, :] <= pos[:, None] - c["window"]] = -math.inf
            p = torch.softmax(z, 1)
            out[at:at + n[j], head * g * d:(head + 1) * g * d] = (p @ v).reshape(n[j], g * d)
        at += n[j]
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "append": _exact_append, "attn": _exact_attn}[case["op"]](s)
