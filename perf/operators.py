"""The cases on which rotary positions, span attention and shared-prefix attention are measured.

Three operators: `rope` (RMS norm of queries and keys with rotary positions on several axes), `span`
(attention whose query rows each see one interval of keys, with an optional tanh cap and distance
bias), `prefix` (the same for a batch whose sequences share a long prefix of keys).
"""

import math

import torch

own = False

# ------------------------------------------------------------------------------------------- cases


def listed():
    return [
        # every layer of a 720p video model: fused qkv projection, norm over the whole row
        dict(name="rope 720p layer", op="rope", B=1, N=75600, H=40, Hk=40, d=128, gf=21, gh=45, gw=80, start=0,
             norm="row", pairing="interleaved", dtype="bf16", pos="grid"),
        # the 480p latent at head dimension 64: norm of each head, fp32 projections, halves rotated against each other
        dict(name="rope 480p d64", op="rope", B=1, N=32760, H=40, Hk=40, d=64, gf=21, gh=30, gw=52, start=0,
             norm="head", pairing="half", dtype="fp32", pos="grid"),
        # one late frame of a long stream
        dict(name="rope stream frame", op="rope", B=2, N=1560, H=40, Hk=40, d=128, gf=100000, gh=30, gw=52,
             start=99990 * 1560, norm="head", pairing="interleaved", dtype="fp16", pos="grid"),
        # one token for each of a few streams, positions given
        dict(name="rope one token", op="rope", B=4, N=1, H=40, Hk=8, d=128, gf=0, gh=0, gw=0, start=0, norm="none",
             pairing="half", dtype="bf16", pos="given"),
        # frame-causal 480p layer: a token sees all tokens of its frame and of those before it
        dict(name="span 480p frame-causal", op="span", mask="frames", B=1, Nq=32760, Nk=32760, H=40, Hk=40, d=128,
             frame=1560, cap=0.0, bias=False),
        # videos of different lengths packed into one sequence, capped scores
        dict(name="span documents capped", op="span", mask="documents", B=1, Nq=23101, Nk=23101, H=20, Hk=20, d=128,
             docs=9, cap=30.0, bias=False),
        # text prefix and a causal rest, with a bias on the distance
        dict(name="span text prefix biased", op="span", mask="prefixed", B=2, Nq=8416, Nk=8416, H=16, Hk=16, d=64,
             lead=226, cap=0.0, bias=True),
        # one new token of each sequence of a padded batch against its cache, grouped heads
        dict(name="span one token", op="span", mask="padded", B=8, Nq=1, Nk=32760, H=40, Hk=8, d=128, cap=0.0,
             bias=False),
        # a tiny latent, where the time of the call itself counts
        dict(name="span tiny", op="span", mask="documents", B=1, Nq=1024, Nk=1024, H=1, Hk=1, d=64, docs=4, cap=0.0,
             bias=False),
        # sixteen variants drawn from one history, one token each
        dict(name="prefix one token", op="prefix", mask="padded", B=16, Nq=1, Nk=1560, Np=32760, H=40, Hk=40, d=128,
             cap=0.0, bias=False),
        # a pair of guidance branches: the next 720p frame against seven shared ones and itself
        dict(name="prefix 720p frame", op="prefix", mask="all", B=2, Nq=3600, Nk=3600, Np=25200, H=40, Hk=40, d=128,
             cap=0.0, bias=False),
        # a few image tokens of each sequence, shared text
        dict(name="prefix short", op="prefix", mask="causal", B=5, Nq=17, Nk=93, Np=512, H=12, Hk=12, d=64, cap=20.0,
             bias=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "span", "span", "prefix"])
    d = rng.choice([64, 128])
    Hk = rng.choice([1, 2, 3, 5, 8, 12])
    H = Hk * rng.choice([1, 1, 1, 2, 4, 5])
    if op == "rope":
        gh, gw = rng.randint(1, 45), rng.randint(1, 80)
        gf = _log(rng, 1, 100000)
        total = gf * gh * gw
        N = min(total, _log(rng, 1, 20000))
        return dict(op="rope", B=rng.choice([1, 1, 2]), N=N, H=H, Hk=Hk, d=d, gf=gf, gh=gh, gw=gw,
                    start=rng.randint(0, total - N), norm=rng.choice(["none", "head", "row"]),
                    pairing=rng.choice(["interleaved", "half"]), dtype=rng.choice(["bf16", "fp16", "fp32"]),
                    pos=rng.choice(["grid", "given"]))
    cap = rng.choice([0.0, 0.0, 15.0, 50.0])
    bias = rng.choice([False, False, True])
    if op == "prefix":
        B = rng.randint(1, 12)
        Nq = _log(rng, 1, 700)
        return dict(op="prefix", mask=rng.choice(["all", "causal", "padded"]), B=B, Nq=Nq, Nk=Nq + _log(rng, 1, 900),
                    Np=_log(rng, 1, 20000), H=H, Hk=Hk, d=d, cap=cap, bias=bias)
    kind = rng.choice(["frames", "documents", "prefixed", "padded"])
    if kind == "padded":
        return dict(op="span", mask=kind, B=rng.randint(1, 9), Nq=_log(rng, 1, 130), Nk=_log(rng, 1, 30000), H=H,
                    Hk=Hk, d=d, cap=cap, bias=bias)
    N = _log(rng, 1, 9000)
    c = dict(op="span", mask=kind, B=rng.choice([1, 2]), Nq=N, Nk=N, H=H, Hk=Hk, d=d, cap=cap, bias=bias)
    if kind == "frames":
        c["frame"] = rng.randint(1, min(N, 1560))
    elif kind == "documents":
        c["docs"] = rng.randint(1, min(N, 12))
    else:
        c["lead"] = rng.randint(0, min(N, 512))
    return c


# ---------------------------------------------------------------------------------------- geometry


def _axes(d):
    """Frame, row and column parts of a head dimension."""
    side = 2 * (d // 6)
    return d - 2 * side, side, side


def _spans(c):
    """[B, Nq, 2] on the CPU: the keys first .. end-1 that each query row sees."""
    B, Nq, Nk = c["B"], c["Nq"], c["Nk"]
    n = torch.arange(Nq)
    first = torch.zeros(B, Nq, dtype=torch.int64)
    if c["mask"] == "all":
        return torch.stack([first, first + Nk], -1)
    if c["mask"] == "frames":
        end = torch.clamp((n // c["frame"] + 1) * c["frame"], max=Nk).expand(B, Nq)
    elif c["mask"] == "documents":
        g = torch.Generator().manual_seed(Nq)
        cuts = torch.randperm(Nq - 1, generator=g)[: c["docs"] - 1].sort().values + 1 if Nq > 1 else torch.zeros(0, dtype=torch.int64)
        edge = torch.cat([torch.tensor([0]), cuts, torch.tensor([Nk])])
        at = torch.searchsorted(edge, n, right=True) - 1
        return torch.stack([edge[at], edge[at + 1]], -1).expand(B, Nq, 2).contiguous()
    elif c["mask"] == "prefixed":
        end = torch.clamp(n + 1, min=c["lead"]).expand(B, Nq)
    elif c["mask"] == "causal":
        end = (n + 1 + Nk - Nq).expand(B, Nq)
    else:  # padded: sequence b holds a part of the longest length
        part = torch.tensor([Nk - (Nk * b) // (2 * B) for b in range(B)])
        end = torch.clamp(part[:, None].expand(B, Nq), min=1)
    return torch.stack([first, end], -1)


def _pairs(c):
    s = _spans(c)
    return int((s[..., 1] - s[..., 0]).sum())


def work(case):
    c = case
    if c["op"] == "rope":
        el = c["B"] * c["N"] * (c["H"] + c["Hk"]) * c["d"]
        size = 4 if c["dtype"] == "fp32" else 2
        extra = 4 * 3 * c["B"] * c["N"] if c["pos"] == "given" else 0
        return {"bytes": el * (size + 2) + extra, "flops": 10 * el}
    rows = c["B"] * c["Nq"] * c["H"]
    s = _spans(c)
    # keys that some row of a batch entry sees
    lo, hi = s[..., 0].amin(1), s[..., 1].amax(1)
    keys = int((hi - lo).sum()) + c.get("Np", 0)
    visible = _pairs(c) + c["B"] * c["Nq"] * c.get("Np", 0)
    return {"bytes": rows * c["d"] * 4 + rows * 4 + keys * c["Hk"] * c["d"] * 4 + c["B"] * c["Nq"] * 8,
            "flops": 4 * c["d"] * c["H"] * visible}


# ------------------------------------------------------------------------------------------ inputs

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 13)

    def normal(*shape, dtype=torch.float32, gain=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * gain).to(dtype)

    s = {"case": c}
    d, B = c["d"], c["B"]
    if c["op"] == "rope":
        N, H, Hk = c["N"], c["H"], c["Hk"]
        # one projection gives queries, keys and values of a token side by side
        s["qkv"] = normal(B, N, H + 2 * Hk, d, dtype=_TYPES[c["dtype"]], gain=1.5)
        s["q"], s["k"] = s["qkv"][:, :, :H], s["qkv"][:, :, H : H + Hk]
        wide = {"none": None, "head": (d, d), "row": (H * d, Hk * d)}[c["norm"]]
        s["wq"] = s["wk"] = None
        if wide:
            s["wq"], s["wk"] = 1.0 + normal(wide[0], gain=0.2), 1.0 + normal(wide[1], gain=0.2)
        s["pos"] = None
        if c["pos"] == "given":
            # frames far into a stream, rows and columns of a resized image
            far = torch.rand((B, 3, N), generator=g, device="cuda")
            s["pos"] = far * torch.tensor([100000.0, 45.0, 80.0], device="cuda")[:, None]
        if own:
            from temporal_block_sparse_b200 import lite_attn as la

            s["plan"] = la.RopePlan(_axes(d), theta=10000.0, pairing=c["pairing"])
        return s
    Nq, Nk, H, Hk, Np = c["Nq"], c["Nk"], c["H"], c["Hk"], c.get("Np", 0)
    bf = torch.bfloat16
    s["q"] = normal(B, Nq, H, d, dtype=bf, gain=1.5)
    kv = normal(B, Nk, 2, Hk, d, dtype=bf)
    s["k"], s["v"] = kv[:, :, 0], kv[:, :, 1]
    if Np:
        s["kp"], s["vp"] = normal(Np, Hk, d, dtype=bf), normal(Np, Hk, d, dtype=bf)
    sp = _spans(c).to(torch.int32)
    s["spans"] = None if c["mask"] == "all" else (sp if c["mask"] == "padded" else sp[:1]).cuda().contiguous()
    s["slopes"] = None
    if c["bias"]:
        # a geometric series over the heads
        s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device="cuda")
    return s


# --------------------------------------------------------------------------------------------- run


def _frequencies(c, dtype):
    """Axis and frequency of each of the d/2 pairs."""
    parts = _axes(c["d"])
    axis = torch.cat([torch.full((p // 2,), a) for a, p in enumerate(parts)]).cuda()
    w = torch.cat([10000.0 ** (-2.0 * torch.arange(p // 2, dtype=torch.float64) / p) for p in parts]).cuda()
    return axis, w.to(dtype)


def _positions(s):
    """[B or 1, 3, N] in 64 bits."""
    c = s["case"]
    if s["pos"] is not None:
        return s["pos"].double()
    i = c["start"] + torch.arange(c["N"], device="cuda", dtype=torch.int64)
    return torch.stack([i // (c["gh"] * c["gw"]), (i // c["gw"]) % c["gh"], i % c["gw"]])[None].double()


def _rotate(x, weight, cos, sin, pairing):
    x = x.float()
    if weight is not None:
        if weight.numel() == x.shape[-1]:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * weight
        else:
            x = x * torch.rsqrt(x.square().mean((-2, -1), keepdim=True) + 1e-6) * weight.view(x.shape[-2:])
    if pairing == "interleaved":
        a, b = x[..., 0::2], x[..., 1::2]
        y = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x.chunk(2, -1)
        y = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return y.to(torch.bfloat16)


def _plain_rope(s):
    c = s["case"]
    axis, w = _frequencies(c, torch.float64)
    angle = _positions(s)[:, axis].transpose(1, 2) * w  # [B or 1, N, d/2], in 64 bits: positions reach 10^5
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]
    return (_rotate(s["q"], s["wq"], cos, sin, c["pairing"]), _rotate(s["k"], s["wk"], cos, sin, c["pairing"]))


def _plain_heads(s, h0, h1):
    """Output and log-sum-exp of the key heads h0 .. h1-1."""
    c = s["case"]
    B, Nq, Nk, H, Hk, d, Np = c["B"], c["Nq"], c["Nk"], c["H"], c["Hk"], c["d"], c.get("Np", 0)
    G, n = H // Hk, h1 - h0
    q = s["q"].view(B, Nq, Hk, G, d)[:, :, h0:h1].float().permute(2, 0, 3, 1, 4).reshape(n, B * G * Nq, d)
    k = s["k"][:, :, h0:h1].float().permute(2, 0, 1, 3)
    v = s["v"][:, :, h0:h1].float().permute(2, 0, 1, 3)
    x = (q.view(n, B, G * Nq, d) @ k.transpose(2, 3)).view(n, B, G, Nq, Nk)
    if Np:
        kp, vp = s["kp"][:, h0:h1].float().transpose(0, 1), s["vp"][:, h0:h1].float().transpose(0, 1)
        x = torch.cat([(q @ kp.transpose(1, 2)).view(n, B, G, Nq, Np), x], -1)
    x.mul_(1.0 / math.sqrt(d))
    if c["cap"]:
        x = x.div_(c["cap"]).tanh_().mul_(c["cap"])
    if c["bias"]:
        # queries are the last Nq of all positions
        far = (torch.arange(Np + Nk - Nq, Np + Nk, device="cuda")[:, None] - torch.arange(Np + Nk, device="cuda")).abs()
        x.sub_(s["slopes"].view(Hk, G)[h0:h1].view(n, 1, G, 1, 1) * far.float())
    if s["spans"] is not None:
        m = torch.arange(Nk, device="cuda")
        out = (m < s["spans"][..., :1]) | (m >= s["spans"][..., 1:])  # [B or 1, Nq, Nk]
        x[..., Np:].masked_fill_(out[None, :, None], float("-inf"))
    top = x.amax(-1, keepdim=True)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p[..., Np:].reshape(n, B, G * Nq, Nk) @ v).view(n, B, G, Nq, d)
    if Np:
        o = o + (p[..., :Np].reshape(n, B * G * Nq, Np) @ vp).view(n, B, G, Nq, d)
    return (o / total).to(torch.bfloat16), (top + total.log())[..., 0]


def _plain_attention(s):
    c = s["case"]
    B, Nq, H, Hk, d = c["B"], c["Nq"], c["H"], c["Hk"], c["d"]
    # as many heads at a time as have their scores within 8 GB
    step = max(1, min(Hk, (1 << 31) // (B * Nq * (c["Nk"] + c.get("Np", 0)) * (H // Hk))))
    parts = [_plain_heads(s, h, min(h + step, Hk)) for h in range(0, Hk, step)]
    o = torch.cat([p[0] for p in parts])  # [Hk, B, G, Nq, d]
    lse = torch.cat([p[1] for p in parts])
    return o.permute(1, 3, 0, 2, 4).reshape(B, Nq, H, d), lse.permute(1, 0, 2, 3).reshape(B, H, Nq)


def run(state):
    s, c = state, state["case"]
    if not own:
        return _plain_rope(s) if c["op"] == "rope" else _plain_attention(s)
    from temporal_block_sparse_b200 import lite_attn as la

    if c["op"] == "rope":
        grid = None if s["pos"] is not None else (c["gf"], c["gh"], c["gw"])
        return la.lite_qk_rope(s["q"], s["k"], s["plan"], grid=grid, start=c["start"] if grid else 0, pos=s["pos"],
                               q_weight=s["wq"], k_weight=s["wk"], eps=1e-6)
    if c["op"] == "span":
        return la.lite_attn_span(s["q"], s["k"], s["v"], s["spans"], cap=c["cap"], slopes=s["slopes"])
    return la.lite_attn_prefix(s["q"], s["kp"], s["vp"], s["k"], s["v"], s["spans"], cap=c["cap"], slopes=s["slopes"])


# ------------------------------------------------------------------------------------------- exact


def exact(case, seed):
    """The definition in 64 bits: one head (or one tensor) after the other."""
    c, s = case, prepare(case, seed)
    if c["op"] == "rope":
        return tuple(_exact_rope(c, s, x, w) for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])))
    B, Nq, Nk, H, d, Np = c["B"], c["Nq"], c["Nk"], c["H"], c["d"], c.get("Np", 0)
    o = torch.empty(B, Nq, H, d, dtype=torch.float64, device="cuda")
    lse = torch.empty(B, H, Nq, dtype=torch.float64, device="cuda")
    spans = _spans(c).cuda()
    key = torch.arange(Nk, device="cuda")
    where_q = torch.arange(Nq, device="cuda", dtype=torch.float64) + (Np + Nk - Nq)
    where_k = torch.arange(Np + Nk, device="cuda", dtype=torch.float64)
    for b in range(B):
        seen = (key >= spans[b, :, 0:1]) & (key < spans[b, :, 1:2])
        if Np:
            seen = torch.cat([torch.ones(Nq, Np, dtype=torch.bool, device="cuda"), seen], 1)
        for h in range(H):
            hk = h * c["Hk"] // H
            k, v = s["k"][b, :, hk].double(), s["v"][b, :, hk].double()
            if Np:
                k, v = torch.cat([s["kp"][:, hk].double(), k]), torch.cat([s["vp"][:, hk].double(), v])
            t = s["q"][b, :, h].double() @ k.T / math.sqrt(d)
            if c["cap"]:
                t = c["cap"] * torch.tanh(t / c["cap"])
            if c["bias"]:
                t = t - s["slopes"][h].double() * (where_q[:, None] - where_k[None]).abs()
            t = torch.where(seen, t, -math.inf)
            norm = torch.logsumexp(t, 1)
            lse[b, h] = norm
            o[b, :, h] = torch.exp(t - norm[:, None]) @ v
    return o, lse


def _exact_rope(c, s, x, weight):
    x = x.double()
    B, N, heads, d = x.shape
    if weight is not None:
        over = (3,) if weight.numel() == d else (2, 3)
        x = x / torch.sqrt((x * x).mean(over, keepdim=True) + 1e-6)
        x = x * (weight.double() if weight.numel() == d else weight.double().view(heads, d))
    index = torch.arange(c["start"], c["start"] + N, device="cuda")
    if s["pos"] is not None:
        places = [s["pos"][:, a].double() for a in range(3)]
    else:
        column = index % c["gw"]
        row = (index - column) // c["gw"] % c["gh"]
        frame = index // (c["gw"] * c["gh"])
        places = [p.double().expand(B, N) for p in (frame, row, column)]
    y = torch.empty_like(x)
    pair = 0
    for a, part in enumerate(_axes(d)):
        for i in range(part // 2):
            lo, hi = (2 * pair, 2 * pair + 1) if c["pairing"] == "interleaved" else (pair, pair + d // 2)
            turn = torch.polar(torch.ones_like(places[a]), places[a] * math.pow(10000.0, -2.0 * i / part))
            z = torch.complex(x[..., lo], x[..., hi]) * turn[:, :, None]
            y[..., lo], y[..., hi] = z.real, z.imag
            pair += 1
    return y
