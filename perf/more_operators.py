"""What the mixture-of-experts operators are measured on: the routing of tokens
to experts, the experts' gate and up products with the SwiGLU, and the experts'
down products with the weighted sum over a token's experts, all on GGUF block
weights and activations quantised on the fly to Q8_0.

`run` computes them in plain torch operations, or with `own` through the
library.  An expert tensor is `experts` matrices of n rows and k elements one
after another, each in GGUF block layout; pair p = token * top + slot.
"""
import math

import torch

own = False

# elements and bytes of a block
BLOCK = {"q8_0": (32, 34), "q4_0": (32, 18), "q5_0": (32, 22), "q4_1": (32, 20), "q5_1": (32, 24), "q8_1": (32, 36),
         "q4_k": (256, 144), "q6_k": (256, 210)}


# --------------------------------------------------------------- the cases --

def listed():
    big = dict(experts=8, top=2)      # eight experts of the 8B-class feed-forward of the benchmark (14336 x 4096), two a token
    fine = dict(experts=64, top=8)    # many narrow experts
    plain = dict(op="route", score="softmax", bias=False, groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0)
    return [
        # one token: latency
        dict(plain, name="route_1x64", t=1, experts=64, top=8),
        # a decode batch, sigmoid scores with a balancing bias and groups
        dict(plain, name="route_64x256_groups", t=64, experts=256, top=8, score="sigmoid", bias=True, groups=8, top_groups=4,
             group_top=2, scale=2.5),
        # a prompt's tokens
        dict(plain, name="route_8192x128", t=8192, experts=128, top=8),
        # one token through two large experts: the weights' bytes
        dict(big, name="gateup_1_8b", op="gateup", fmt="q4_k", t=1, n=14336, k=4096, drop=False),
        # a few tokens, small odd experts of the 896-wide model: latency
        dict(name="gateup_5_odd", op="gateup", fmt="q8_0", experts=32, top=4, t=5, n=1217, k=896, drop=True),
        # a decode batch over many narrow experts, four tokens each
        dict(fine, name="gateup_32_fine", op="gateup", fmt="q4_0", t=32, n=1024, k=2048, drop=False),
        # a prompt of 2048 tokens
        dict(big, name="gateup_2048_8b", op="gateup", fmt="q4_k", t=2048, n=14336, k=4096, drop=False),
        # one token, the way down
        dict(big, name="down_1_8b", op="down", fmt="q6_k", t=1, n=4096, k=14336, drop=False),
        # a decode batch: four rows an expert
        dict(big, name="down_16_8b", op="down", fmt="q4_k", t=16, n=4096, k=14336, drop=False),
        # a short prompt of the 896-wide model, some slots without an expert
        dict(name="down_300_896", op="down", fmt="q5_0", experts=16, top=4, t=300, n=896, k=4864, drop=True),
        # a prompt of 2048 tokens, the way down
        dict(big, name="down_2048_8b", op="down", fmt="q6_k", t=2048, n=4096, k=14336, drop=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("route", "gateup", "gateup", "down", "down"))
    if op == "route":
        groups = rng.choice((1, 1, 2, 4, 8))
        experts = groups * max(4, _log(rng, 8, 512) // groups)
        top_groups = rng.randint(max(1, groups // 2), groups)
        top = rng.randint(1, min(16, top_groups * (experts // groups)))
        return dict(op="route", t=min(_log(rng, 1, 8192), 8192 * 256 // experts), experts=experts, top=top,
                    score=rng.choice(("softmax", "sigmoid")), bias=rng.random() < 0.5, groups=groups, top_groups=top_groups,
                    group_top=rng.choice((1, 2)), renorm=rng.random() < 0.7, scale=rng.choice((1.0, 2.5)))
    fmt = rng.choice(tuple(BLOCK))
    unit = BLOCK[fmt][0]
    experts = rng.choice((4, 8, 16, 30, 64, 128))
    top = rng.choice([x for x in (1, 2, 4, 6, 8) if x <= experts])
    t = _log(rng, 1, 2048)
    k = unit * max(1, _log(rng, 256, 14336) // unit)
    n = _log(rng, 64, 14336)
    most = 2048 * 2 * 14336 * 4096 // (2 if op == "gateup" else 1)
    while t * top * n * k > most // 2 or experts * n * k > 8 * 14336 * 4096:
        n, t = n // 2 + 1, t // 2 + 1
    return dict(op=op, fmt=fmt, experts=experts, top=top, t=t, n=n, k=k, drop=rng.random() < 0.3)


def work(case):
    t, e, top = case["t"], case["experts"], case["top"]
    if case["op"] == "route":
        return {"bytes": 4 * t * e + 8 * t * top + (4 * e if case["bias"] else 0), "flops": t * e * 8}
    n, k = case["n"], case["k"]
    elements, size = BLOCK[case["fmt"]]
    used = e * (1 - (1 - top / e) ** t)   # experts that a call of this shape meets
    pair = 2 if case["op"] == "gateup" else 1
    rows = t * k + t * top * n if case["op"] == "gateup" else t * top * k + t * n
    return {"bytes": pair * used * n * (k // elements) * size + 4 * rows, "flops": 2 * pair * t * top * n * k}


# -------------------------------------------------------------- the inputs --

def _rand(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _weights(gen, fmt, rows, k):
    """rows x k weights of about 2 / sqrt(k), as the bytes of their blocks: random codes, scales of the right size."""
    elements, size = BLOCK[fmt]
    blocks = k // elements
    raw = torch.randint(0, 256, (rows * blocks, size), generator=gen, device="cuda", dtype=torch.uint8)

    def put(at, value):
        raw[:, at:at + 2] = value.half().view(torch.uint8).view(-1, 2)

    size_of = {"q8_0": 73.9, "q8_1": 73.9, "q4_0": 4.6, "q4_1": 4.6, "q5_0": 9.2, "q5_1": 9.2, "q4_k": 165.0, "q6_k": 680.0}[fmt]
    d = (0.3 + torch.rand(rows * blocks, generator=gen, device="cuda")) * (2.0 / math.sqrt(k) / size_of)
    if fmt == "q6_k":
        raw[:, 192:208] = torch.randint(0, 128, (rows * blocks, 16), generator=gen, device="cuda", dtype=torch.uint8) - 64
        put(208, d)
        return raw.view(-1)
    put(0, d)
    if fmt == "q4_k":        # mins that stand in the middle of their sub-block's codes
        raw[:, 8:12] = raw[:, 4:8]
        raw[:, 12:16] = (raw[:, 12:16] & 15) * 17
        put(2, d * 7.5)
    elif fmt in ("q4_1", "q5_1"):
        put(2, d * (-7.5 if fmt == "q4_1" else -15.5))
    return raw.view(-1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed * 2 + 1)
    t, e, top = case["t"], case["experts"], case["top"]
    s = {"case": dict(case)}
    logits = _rand(gen, t, e) * 1.5 + _rand(gen, e) * 0.5    # some experts are liked better
    if case["op"] == "route":
        s["logits"] = logits
        s["bias"] = _rand(gen, e) * 0.1 if case["bias"] else None
        return s
    n, k = case["n"], case["k"]
    order = logits.sort(-1, descending=True)
    idx = order.indices[:, :top].to(torch.int32)
    s["weight"] = torch.softmax(order.values[:, :top], -1)
    if case["drop"]:         # slots over an expert's capacity, or padded tokens
        lost = torch.rand(t, top, generator=gen, device="cuda") < 0.1
        idx = idx.masked_fill(lost, -1)
        s["weight"] = s["weight"].masked_fill(lost, 0.0)
    s["idx"] = idx.contiguous()
    # what the plain form asks the host for: the experts in use and the most rows of one
    count = torch.bincount(idx.flatten().long() + 1, minlength=e + 1)[1:]
    s["used"] = count.nonzero().flatten() if int(count.sum()) else torch.zeros(1, dtype=torch.long, device="cuda")
    s["cap"] = max(1, int(count.max()))
    if case["op"] == "gateup":
        wide = 1 + 6 * (torch.rand(k, generator=gen, device="cuda") < 0.01)   # a norm's output with some wide channels
        s["x"] = _rand(gen, t, k) * wide
        s["w_gate"], s["w_up"] = _weights(gen, case["fmt"], e * n, k), _weights(gen, case["fmt"], e * n, k)
    else:
        g, u = _rand(gen, t, top, k) * 2, _rand(gen, t, top, k)
        s["h"] = g * torch.sigmoid(g) * u
        s["w"] = _weights(gen, case["fmt"], e * n, k)
    return s


# --------------------------------------------------------- the plain forms --

def _plain_route(s):
    c = s["case"]
    t, e, k, groups = c["t"], c["experts"], c["top"], c["groups"]
    logit, bias = s["logits"], s["bias"]
    x = logit.double()                  # choices next to each other: 64 bits up to the value that is compared
    if c["score"] == "softmax":
        p = torch.exp(x - x.amax(-1, keepdim=True))
        p = p / p.sum(-1, keepdim=True)
    else:
        p = 1 / (1 + torch.exp(-x))
    alive = logit > -math.inf
    if c["score"] == "softmax" and bias is None and (groups == 1 or c["group_top"] == 1):
        choice = logit                  # the softmax keeps the logits' order
    else:
        choice = p.float() if bias is None else p.float() + bias
    choice = choice.masked_fill(~alive, -math.inf)
    if groups > 1:
        best = choice.view(t, groups, -1).sort(-1, descending=True).values
        rank = best[..., 0]
        if c["group_top"] == 2:
            rank = torch.where(best[..., 1] > -math.inf, best[..., 0] + best[..., 1], best[..., 0])
        keep = rank.sort(dim=-1, descending=True, stable=True).indices[:, :c["top_groups"]]
        stay = torch.zeros(t, groups, dtype=torch.bool, device=logit.device).scatter(1, keep, True)
        choice = choice.masked_fill(~stay.repeat_interleave(e // groups, 1), -math.inf)
    order = choice.sort(dim=-1, descending=True, stable=True)
    there = order.values[:, :k] > -math.inf
    chosen = order.indices[:, :k]
    w = p.gather(1, chosen).masked_fill(~there, 0.0)
    if c["renorm"]:
        total = w.sum(-1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return {"idx": chosen.masked_fill(~there, -1).to(torch.int32), "weight": (w * c["scale"]).float()}


def _f16(raw, at):
    return raw[..., at:at + 2].contiguous().view(torch.float16).float()


def _nibbles(raw):
    """[..., 16] bytes -> [..., 32]: the low nibbles, then the high ones."""
    return torch.cat((raw & 15, raw >> 4), -1)


def _fifth(raw):
    """[..., 4] bytes -> [..., 32]: bit e of the word, as 16."""
    bit = torch.arange(8, device=raw.device, dtype=torch.uint8)
    return (((raw[..., None] >> bit) & 1) << 4).flatten(-2)


def _values(fmt, raw, n, k):
    """Bytes of [U, n rows] -> [U, n, k] f32."""
    u = raw.shape[0]
    raw = raw.view(u, n, k // BLOCK[fmt][0], BLOCK[fmt][1])
    if fmt == "q4_k":
        a, b, m = raw[..., 4:8], raw[..., 8:12], raw[..., 12:16]
        sc = torch.cat((a & 63, (m & 15) | ((a >> 6) << 4)), -1).float()
        mn = torch.cat((b & 63, (m >> 4) | ((b >> 6) << 4)), -1).float()
        q = raw[..., 16:].unflatten(-1, (4, 32))
        q = torch.stack((q & 15, q >> 4), -2).flatten(-3, -2).float()     # [..., 8, 32]
        return (q * (_f16(raw, 0) * sc)[..., None] - (_f16(raw, 2) * mn)[..., None]).view(u, n, k)
    if fmt == "q6_k":
        low = raw[..., :128].unflatten(-1, (2, 2, 32))                    # half, which 32 bytes
        low = torch.stack((low & 15, low >> 4), -3)                       # half, nibble, which, 32
        high = raw[..., 128:192].unflatten(-1, (2, 1, 32))
        high = torch.cat((high & 3, (high >> 2) & 3, (high >> 4) & 3, high >> 6), -2)
        q = (low.flatten(-3, -2) | (high << 4)).flatten(-3).unflatten(-1, (16, 16)).float() - 32
        sc = raw[..., 192:208].contiguous().view(torch.int8).float()
        return (q * (_f16(raw, 208) * sc)[..., None]).view(u, n, k)
    d = _f16(raw, 0)
    if fmt in ("q8_0", "q8_1"):
        value = raw[..., _codes_at(fmt):].contiguous().view(torch.int8).float() * d
    elif fmt == "q4_0":
        value = (_nibbles(raw[..., 2:]).float() - 8) * d
    elif fmt == "q5_0":
        value = ((_nibbles(raw[..., 6:]) | _fifth(raw[..., 2:6])).float() - 16) * d
    elif fmt == "q4_1":
        value = _nibbles(raw[..., 4:]).float() * d + _f16(raw, 2)
    else:
        value = (_nibbles(raw[..., 8:]) | _fifth(raw[..., 4:8])).float() * d + _f16(raw, 2)
    return value.view(u, n, k)


def _codes_at(fmt):
    """Where the codes of an 8-bit block begin."""
    return 2 if fmt == "q8_0" else 4


def _q8_0(x):
    """[rows, K] -> the values of its Q8_0 blocks, f32."""
    y = x.unflatten(-1, (-1, 32))
    d = (y.abs().amax(-1, keepdim=True).double() / 127).float()
    inv = (1.0 / d.double()).float()
    t = y * torch.where(torch.isfinite(inv), inv, 0.0)
    code = torch.trunc(t) + torch.sign(t) * ((t - torch.trunc(t)).abs() >= 0.5)   # halves away from zero
    return (code * d.half().float()).flatten(-2)


def _spread(s, rows):
    """Each expert's rows side by side: ([U, cap, K], the place of each pair, whether it has an expert)."""
    used, cap = s["used"], s["cap"]
    e = s["idx"].flatten().long()
    there = e >= 0
    u = used.numel()
    slot = torch.where(there, torch.searchsorted(used, e), u)
    rank = ((slot[:, None] == torch.arange(u, device=e.device)).cumsum(0) - 1).gather(1, slot.clamp(max=u - 1)[:, None])[:, 0]
    rank = torch.where(there, rank, 0)
    x = torch.zeros(u + 1, cap, rows.shape[1], device=rows.device)
    x[slot, rank] = rows
    return x[:u], (slot.clamp(max=u - 1), rank), there


def _product(s, w, x):
    c = s["case"]
    value = _values(c["fmt"], w.view(c["experts"], -1)[s["used"]], c["n"], c["k"])
    return torch.matmul(x, value.transpose(1, 2))


def _plain_gateup(s):
    c = s["case"]
    x, place, there = _spread(s, _q8_0(s["x"]).repeat_interleave(c["top"], 0))
    g, u = _product(s, s["w_gate"], x)[place], _product(s, s["w_up"], x)[place]
    h = g / (1 + torch.exp(-g)) * u
    return torch.where(there[:, None], h, 0.0).view(c["t"], c["top"], c["n"])


def _plain_down(s):
    c = s["case"]
    x, place, there = _spread(s, _q8_0(s["h"].flatten(0, 1)))
    y = torch.where(there[:, None], _product(s, s["w"], x)[place], 0.0).view(c["t"], c["top"], c["n"])
    return (y * s["weight"][..., None]).sum(1)


# ------------------------------------------------------------ the library --

def _own_route(s):
    import gguf_quantized_matvec_amd as lib
    c = s["case"]
    idx, weight = lib.moe_route(s["logits"], c["top"], score=c["score"], bias=s["bias"], groups=c["groups"],
                                top_groups=c["top_groups"], group_top=c["group_top"], renorm=c["renorm"], scale=c["scale"])
    return {"idx": idx, "weight": weight}


def _own_gateup(s):
    import gguf_quantized_matvec_amd as lib
    c = s["case"]
    return lib.moe_gateup_swiglu(lib.TYPES[c["fmt"].upper()], s["w_gate"], s["w_up"], c["n"], c["k"], s["idx"], x=s["x"])


def _own_down(s):
    import gguf_quantized_matvec_amd as lib
    c = s["case"]
    return lib.moe_down(lib.TYPES[c["fmt"].upper()], s["w"], c["n"], c["k"], s["idx"], s["weight"], s["h"])


def run(state):
    if own:
        return {"route": _own_route, "gateup": _own_gateup, "down": _own_down}[state["case"]["op"]](state)
    return {"route": _plain_route, "gateup": _plain_gateup, "down": _plain_down}[state["case"]["op"]](state)


# ------------------------------------------------- the definitions, 64 bits --

def _exact_route(s):
    """The weights, from the sets that the definition chooses expert by expert: an expert is in a set when fewer than its
    size stand before it."""
    c = s["case"]
    k, groups = c["top"], c["groups"]
    x = s["logits"].double()
    if c["score"] == "softmax":
        p = torch.softmax(x, -1)
    else:
        p = torch.sigmoid(x)
    out = torch.zeros(c["t"], k, dtype=torch.float64, device=x.device)
    step = max(1, (1 << 26) // (c["experts"] ** 2))
    for at in range(0, c["t"], step):
        part, q = x[at:at + step], p[at:at + step]
        if not (c["score"] == "softmax" and s["bias"] is None and (groups == 1 or c["group_top"] == 1)):
            part = q.float().double()
            if s["bias"] is not None:
                part = (part + s["bias"].double()).float().double()
        if groups > 1:
            best = part.unflatten(1, (groups, -1)).topk(c["group_top"], -1).values
            rank = best.sum(-1).float().double()
            first = torch.arange(groups, device=x.device)
            before = (rank[:, None, :] > rank[:, :, None]) | ((rank[:, None, :] == rank[:, :, None]) & (first[None, None, :] < first[None, :, None]))
            out_of = before.sum(-1) >= c["top_groups"]
            part = part.masked_fill(out_of.repeat_interleave(c["experts"] // groups, 1), -math.inf)
        first = torch.arange(c["experts"], device=x.device)
        before = ((part[:, None, :] > part[:, :, None]) | ((part[:, None, :] == part[:, :, None]) & (first[None, None, :] < first[None, :, None]))).sum(-1)
        row, expert = (before < k).nonzero(as_tuple=True)
        out[at + row, before[row, expert]] = q[row, expert]
    if c["renorm"]:
        out = out / out.sum(1, keepdim=True)
    return {"idx": None, "weight": out * c["scale"]}


def _exact_values(fmt, raw, n, k):
    """One expert's bytes -> [n, k] f64: each element's byte, shift and scale by its number."""
    elements, size = BLOCK[fmt]
    raw = raw.view(n * (k // elements), size)
    i = torch.arange(elements, device=raw.device)
    half = lambda at: raw[:, at:at + 2].contiguous().view(torch.float16).double()  # noqa: E731
    if fmt in ("q8_0", "q8_1"):
        q = raw[:, i + (2 if fmt == "q8_0" else 4)].view(torch.int8).double()
        return (half(0) * q).view(n, k)
    if fmt == "q4_k":
        sub = i // 32
        q = (raw[:, 16 + 32 * (i // 64) + i % 32] >> (4 * (sub % 2)).to(torch.uint8)) & 15
        j = torch.arange(8, device=raw.device)
        a, b, m = raw[:, j].int(), raw[:, 4 + j].int(), raw[:, 8 + j].int()    # bytes 4 before, at and 4 after the sub-block's own
        sc = torch.where(j < 4, b & 63, (m & 15) | ((a >> 6) << 4))
        mn = torch.where(j < 4, m & 63, (m >> 4) | ((b >> 6) << 4))
        return (half(0) * sc.double()[:, sub] * q.double() - half(2) * mn.double()[:, sub]).view(n, k)
    if fmt == "q6_k":
        part = (i % 128) // 32
        low = raw[:, 64 * (i // 128) + 32 * (part % 2) + i % 32] >> (4 * (part // 2)).to(torch.uint8)
        high = raw[:, 128 + 32 * (i // 128) + i % 32] >> (2 * part).to(torch.uint8)
        q = (low & 15).double() + 16 * (high & 3).double() - 32
        return (half(208) * raw[:, 192 + i // 16].view(torch.int8).double() * q).view(n, k)
    at = {"q4_0": 2, "q5_0": 6, "q4_1": 4, "q5_1": 8}[fmt]
    q = ((raw[:, at + i % 16] >> (4 * (i // 16)).to(torch.uint8)) & 15).double()
    if fmt in ("q5_0", "q5_1"):
        q = q + 16 * ((raw[:, at - 4 + i // 8] >> (i % 8).to(torch.uint8)) & 1).double()
    if fmt in ("q4_1", "q5_1"):
        return (half(0) * q + half(2)).view(n, k)
    return (half(0) * (q - (8 if fmt == "q4_0" else 16))).view(n, k)


def _exact_q8_0(x):
    """[rows, K] f32 -> the values of its Q8_0 blocks, in 64 bits (each step that the format rounds to 32 is rounded)."""
    rows = x.shape[0]
    b = x.double().reshape(-1, 32)
    d = (b.abs().max(1, keepdim=True).values / 127).float().double()
    inv = (1 / d).float().double()
    inv[torch.isinf(inv)] = 0
    t = (b * inv).float().double()
    return (torch.floor(t.abs() + 0.5) * torch.sign(t) * d.half().double()).reshape(rows, -1)


def _exact_pairs(s, w, rows):
    """y[p] = W[expert of p] rows[p], one expert at a time; 0 without one."""
    c = s["case"]
    e, out = s["idx"].flatten(), torch.zeros(c["t"] * c["top"], c["n"], dtype=torch.float64, device="cuda")
    w = w.view(c["experts"], -1)
    for i in range(c["experts"]):
        p = (e == i).nonzero()[:, 0]
        if p.numel():
            out[p] = rows[p] @ _exact_values(c["fmt"], w[i], c["n"], c["k"]).T
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        return _exact_route(s)
    if case["op"] == "gateup":
        rows = _exact_q8_0(s["x"])[torch.arange(case["t"] * case["top"], device="cuda") // case["top"]]
        g = _exact_pairs(s, s["w_gate"], rows)
        return (g * torch.sigmoid(g) * _exact_pairs(s, s["w_up"], rows)).view(case["t"], case["top"], -1)
    y = _exact_pairs(s, s["w"], _exact_q8_0(s["h"].flatten(0, 1)))
    return (y.view(case["t"], case["top"], -1) * s["weight"].double()[..., None]).sum(1)
