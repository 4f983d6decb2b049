"""Cases and plain forms of the token operators around the attention: root-mean-square norm (with the
residual's addition and an 8-bit output), rotary positions of Q and K over several axes (with the
per-head norm in the same pass), and attention over packed whole prompts with grouped heads.

`run` computes an operator from elementary torch operations in binary32 (angles in binary64), or, with
`own`, by the calls a user of block_sparse_tiled_b200 makes.  Sizes are those of the video transformer
whose attention this package runs (56 heads, hidden 5376, the 480p- and 1344x768-shaped sequences) and of
the text model that feeds it (hidden 5120, grouped heads).
"""
import math

import torch

own = False

BF16, F32, F64, E4M3 = torch.bfloat16, torch.float32, torch.float64, torch.float8_e4m3fn
EPS = 1e-6


def _vsa():
    """The package, imported only where its own kernels are called."""
    import block_sparse_tiled_b200 as vsa

    return vsa


# ---------------------------------------------------------------------------------------------- cases


def _norm(name, rows, width, residual, out):
    """residual: "none", "bf16" or "f32" (the type of the residual stream); out: "bf16" or "e4m3"."""
    return {"name": name, "op": "norm", "rows": rows, "width": width, "residual": residual, "out": out}


def _rope(name, prefix, t, h, w, heads, kv_heads, dim, sections, interleaved, shared, norm, packed):
    """prefix text tokens, then a t x h x w grid; sections: rotated pairs per axis; packed: Q and K are
    views into one [tokens, (heads + 2 kv_heads) dim] projection, else two tensors."""
    return {"name": name, "op": "rope", "prefix": prefix, "t": t, "h": h, "w": w, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "sections": sections, "interleaved": interleaved,
            "shared": shared, "norm": norm, "packed": packed}


def _attn(name, lengths, heads, kv_heads, dim, causal):
    """lengths: the prompts' token counts, in order, as a text."""
    return {"name": name, "op": "attn", "lengths": lengths, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "causal": causal}


def listed():
    return [
        # the norm before a projection of a single text token: latency is all
        _norm("norm: one token", 1, 5120, "bf16", "bf16"),
        # a batch of packed prompts, odd token count, residual stream kept in binary32, 8-bit output
        _norm("norm: text, 8-bit", 1537, 5120, "f32", "e4m3"),
        # the 480p-shaped sequence, first norm of the model (no residual yet)
        _norm("norm: 480p", 14208, 5376, "none", "bf16"),
        # the 1344x768-shaped sequence inside the model, 8-bit input of the next projection
        _norm("norm: 1344x768, 8-bit", 75008, 5376, "bf16", "e4m3"),
        # a short prompt of the text model: grouped heads, one frequency ladder over the axes, no head norm
        _rope("rope: prompt", 77, 0, 0, 0, 40, 8, 128, "24,20,20", False, True, False, False),
        # the 480p-shaped sequence out of one QKV projection, the model's head dimension
        _rope("rope: 480p, packed qkv", 768, 8, 30, 56, 56, 56, 96, "16,16,16", False, False, True, True),
        # the 1344x768-shaped sequence, neighbouring pairs, some pairs not rotated
        _rope("rope: 1344x768", 1280, 24, 48, 64, 56, 56, 128, "16,22,22", True, False, True, False),
        # a few very short prompts, single tokens and an empty one among them: latency
        _attn("attn: tiny prompts", "1,9,33,0,17,1,64", 40, 8, 128, True),
        # a served batch of ordinary prompts of very different lengths
        _attn("attn: 24 prompts", "77,512,1,300,129,640,33,255,128,96,700,411,18,222,350,64,5,489,127,256,600,2,191,1000",
              40, 8, 128, True),
        # long documents and short ones together, narrow heads
        _attn("attn: ragged, D = 64", "4096,1,1023,2049,513,2800,65", 64, 8, 64, True),
        # reference segments encoded without a mask, the video model's heads
        _attn("attn: references, D = 96", "2048,1153,1536,700", 56, 56, 96, False),
        # one long prompt
        _attn("attn: one long prompt", "8192", 40, 8, 128, True),
    ]


def _spread(rng, lo, hi):
    """A whole number, its logarithm spread evenly over [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "rope", "attn", "attn"))
    if op == "norm":
        width = 8 * _spread(rng, 8, 1024)
        rows = _spread(rng, 1, 75008 * 5376 // max(width, 5376))
        c = _norm("", rows, width, rng.choice(("none", "bf16", "f32")), rng.choice(("bf16", "e4m3")))
        if c["residual"] == "f32" and c["out"] == "bf16":
            c["rows"] = max(1, c["rows"] // 2)
    elif op == "rope":
        dim = rng.choice((64, 96, 128))
        kv_heads = rng.choice((1, 2, 4, 8, 16, 56))
        heads = 56 if kv_heads == 56 else kv_heads * rng.choice((1, 2, 3, 5, 7))
        prefix = rng.choice((0, 1, 77, _spread(rng, 1, 2000)))
        t, h, w = rng.choice((0, rng.randint(1, 24))), rng.randint(1, 48), rng.randint(1, 64)
        if t * h * w == 0:
            t, h, w, prefix = 0, 0, 0, prefix + _spread(rng, 1, 8000)
        pairs = dim // 2
        a = rng.randint(0, pairs)
        b = rng.randint(0, pairs - a)
        c3 = rng.choice((pairs - a - b, rng.randint(0, pairs - a - b)))
        c = _rope("", prefix, t, h, w, heads, kv_heads, dim, "%d,%d,%d" % (a, b, c3), rng.random() < 0.5,
                  rng.random() < 0.5, rng.random() < 0.6, rng.random() < 0.5)
    else:
        dim = rng.choice((64, 96, 128))
        kv_heads = rng.choice((1, 2, 4, 8))
        heads = kv_heads * rng.choice((1, 2, 3, 4, 5, 7, 8))
        count, longest = _spread(rng, 1, 40), _spread(rng, 1, 6000)
        # the padded plain form's scores stay below those of the largest listed case
        while count * heads * longest * longest > 40 * 8192 * 8192:
            if count > 1:
                count //= 2
            else:
                longest = longest * 3 // 4
        lengths = [longest] + [rng.choice((1, rng.randint(1, longest), _spread(rng, 1, longest))) for _ in range(count - 1)]
        rng.shuffle(lengths)
        c = _attn("", ",".join(map(str, lengths)), heads, kv_heads, dim, rng.random() < 0.75)
    del c["name"]
    return c


# --------------------------------------------------------------------------------------------- inputs


def _ints(text):
    return [int(x) for x in text.split(",")]


def _positions(c, device):
    """[tokens, 3]: the prefix counts on all axes at once, the grid starts behind it."""
    p = torch.arange(c["prefix"], dtype=torch.int32, device=device)[:, None].expand(-1, 3)
    t, h, w = c["t"], c["h"], c["w"]
    if t * h * w == 0:
        return p.contiguous()
    at = [torch.arange(n, dtype=torch.int32, device=device) for n in (t, h, w)]
    grid = torch.stack(torch.meshgrid(*at, indexing="ij"), -1).reshape(-1, 3) + c["prefix"]
    return torch.cat((p, grid)).contiguous()


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=BF16):
        return (torch.randn(*shape, generator=g, device=dev, dtype=F32) * scale).to(dtype)

    s = {"case": c}
    if c["op"] == "norm":
        rows, width = c["rows"], c["width"]
        # a residual stream grows with depth and a few of its channels run far ahead of the others
        s["x"] = normal(rows, width)
        s["weight"] = (1.0 + 0.2 * torch.randn(width, generator=g, device=dev)).to(BF16)
        s["residual"] = None
        if c["residual"] != "none":
            r = normal(rows, width, scale=3.0, dtype=F32)
            r[:, :: max(1, width // 5)] *= 20.0
            s["residual"] = r.to(BF16 if c["residual"] == "bf16" else F32)
        s["out"] = torch.empty(rows, width, dtype=E4M3 if c["out"] == "e4m3" else BF16, device=dev)
        s["scale"] = torch.empty(rows, dtype=F32, device=dev) if c["out"] == "e4m3" else None
        s["residual_out"] = None if s["residual"] is None else torch.empty_like(s["residual"])
    elif c["op"] == "rope":
        s["positions"] = _positions(c, dev)
        n, hq, hk, d = s["positions"].shape[0], c["heads"], c["kv_heads"], c["dim"]
        if c["packed"]:
            qkv = normal(n, hq + 2 * hk, d, scale=2.0)
            s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        else:
            s["q"], s["k"] = normal(n, hq, d, scale=2.0), normal(n, hk, d, scale=2.0)
        s["q_weight"] = s["k_weight"] = None
        if c["norm"]:
            s["q_weight"] = (1.0 + 0.2 * torch.randn(d, generator=g, device=dev)).to(BF16)
            s["k_weight"] = (1.0 + 0.2 * torch.randn(d, generator=g, device=dev)).to(BF16)
        s["q_out"] = torch.empty(n, hq, d, dtype=BF16, device=dev)
        s["k_out"] = torch.empty(n, hk, d, dtype=BF16, device=dev)
        s["theta"] = 10000.0
        if own:
            s["rope"] = _vsa().vsa_rope_create(d, _ints(c["sections"]), theta=s["theta"], interleaved=c["interleaved"],
                                               shared_ladder=c["shared"])
    else:
        n, hq, hk, d = sum(_ints(c["lengths"])), c["heads"], c["kv_heads"], c["dim"]
        s["q"], s["k"], s["v"] = normal(n, hq, d), normal(n, hk, d), normal(n, hk, d)
        # some keys that many queries look at, so that a row's weights are not all alike
        s["k"][:: 61] *= 3.0
        s["out"] = torch.empty_like(s["q"])
        if own:
            s["plan"] = _vsa().vsa_packed_plan(_ints(c["lengths"]), heads=hq, kv_heads=hk, head_dim=d, causal=c["causal"])
    return s


# ------------------------------------------------------------------------------------- one pass, plain


def _plain_norm(s):
    x = s["x"].float()
    if s["residual"] is not None:
        x = x + s["residual"].float()
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    res = None if s["residual"] is None else x.to(s["residual"].dtype)
    if s["scale"] is None:
        return {"out": y.to(BF16), "residual": res}
    scale = y.abs().amax(-1) / 448.0
    codes = torch.where(scale[:, None] > 0, y / scale[:, None], torch.zeros_like(y)).to(E4M3)
    return {"out": codes, "scale": scale, "residual": res}


def _ladder(c, theta, device):
    """Each pair's angle per step and the axis whose position it follows (pairs behind the sections: none)."""
    half, parts = c["dim"] // 2, torch.tensor(_ints(c["sections"]), device=device)
    pair = torch.arange(half, device=device)
    ends = parts.cumsum(0)
    axis = (pair[:, None] >= ends[None, :]).sum(-1)
    rotated = axis < 3
    axis = axis.clamp(max=2)
    start, size = (ends - parts)[axis], parts[axis]
    share = pair.to(F64) / half if c["shared"] else (pair - start).to(F64) / size.clamp(min=1).to(F64)
    return torch.where(rotated, theta ** -share, torch.zeros_like(share)), axis


def _plain_turn(c, x, weight, cos, sin):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    if c["interleaved"]:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2).to(BF16)
    a, b = x.chunk(2, -1)
    return torch.cat((a * cos - b * sin, a * sin + b * cos), -1).to(BF16)


def _plain_rope(s):
    c = s["case"]
    freq, axis = _ladder(c, s["theta"], s["q"].device)
    angle = s["positions"].to(F64)[:, axis] * freq
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    return {"q": _plain_turn(c, s["q"], s["q_weight"], cos, sin), "k": _plain_turn(c, s["k"], s["k_weight"], cos, sin)}


def _plain_attn(s):
    c, q, k, v = s["case"], s["q"], s["k"], s["v"]
    hq, hk, d, dev = c["heads"], c["kv_heads"], c["dim"], q.device
    lens = torch.tensor(_ints(c["lengths"]), device=dev)
    longest = max(_ints(c["lengths"]))
    at = torch.arange(longest, device=dev)
    real = at[None, :] < lens[:, None]  # [prompts, longest]
    index = ((lens.cumsum(0) - lens)[:, None] + at[None, :]).clamp(max=q.shape[0] - 1)
    zero = torch.zeros((), device=dev)
    # padded to the longest prompt: [prompts, kv heads, queries of the group, longest, d]
    qp = q[index].float().view(-1, longest, hk, hq // hk, d).permute(0, 2, 3, 1, 4)
    kp = torch.where(real[:, :, None, None], k[index].float(), zero).permute(0, 2, 3, 1)[:, :, None]
    vp = torch.where(real[:, :, None, None], v[index].float(), zero).permute(0, 2, 1, 3)[:, :, None]
    scores = qp @ kp
    scores *= 1.0 / math.sqrt(d)
    seen = real[:, None, :].expand(-1, longest, -1)
    if c["causal"]:
        seen = seen & (at[None, None, :] <= at[None, :, None])
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    scores -= scores.amax(-1, keepdim=True)
    scores.exp_()
    out = (scores @ vp) / scores.sum(-1, keepdim=True)
    return out.permute(0, 3, 1, 2, 4).reshape(-1, longest, hq, d)[real].to(BF16)


# ------------------------------------------------------------------------------- one pass, this package


def _own_run(s):
    op, vsa = s["case"]["op"], _vsa()
    if op == "norm":
        out, scale, res = vsa.vsa_rms_norm(s["x"], s["weight"], EPS, residual=s["residual"], out=s["out"],
                                           residual_out=s["residual_out"], scale=s["scale"])
        return {"out": out, "residual": res} if scale is None else {"out": out, "scale": scale, "residual": res}
    if op == "rope":
        q, k = vsa.vsa_qk_rope(s["rope"], s["q"], s["k"], s["positions"], q_weight=s["q_weight"],
                               k_weight=s["k_weight"], eps=EPS, q_out=s["q_out"], k_out=s["k_out"])
        return {"q": q, "k": k}
    return vsa.vsa_packed_attn(s["plan"], s["q"], s["k"], s["v"], out=s["out"])


def run(state):
    if own:
        return _own_run(state)
    return {"norm": _plain_norm, "rope": _plain_rope, "attn": _plain_attn}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------------- what it costs


def _pairs(c):
    return sum(n * (n + 1) // 2 if c["causal"] else n * n for n in _ints(c["lengths"]))


def work(case):
    c = case
    if c["op"] == "norm":
        n = c["rows"] * c["width"]
        res = {"none": 0, "bf16": 4, "f32": 8}[c["residual"]]
        out = 2 if c["out"] == "bf16" else 1
        return {"bytes": n * (2 + res + out) + 2 * c["width"] + (4 * c["rows"] if out == 1 else 0), "flops": 5 * n}
    if c["op"] == "rope":
        tokens = c["prefix"] + c["t"] * c["h"] * c["w"]
        n = tokens * (c["heads"] + c["kv_heads"]) * c["dim"]
        return {"bytes": 4 * n + 12 * tokens + (4 * c["dim"] if c["norm"] else 0), "flops": (7 if c["norm"] else 3) * n}
    tokens = sum(_ints(c["lengths"]))
    return {"bytes": 2 * tokens * c["dim"] * (2 * c["heads"] + 2 * c["kv_heads"]),
            "flops": 4 * c["dim"] * c["heads"] * _pairs(c)}


# ------------------------------------------------------------------------------- the definition, 64 bits


def _e4m3_of(v):
    """The nearest E4M3 value (ties to even): 4 significant bits, steps of 2^-9 at the bottom, at most 448."""
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3.0)
    return (torch.round(v / step) * step).clamp(-448.0, 448.0)


def _exact_norm(s):
    t = s["x"].double() if s["residual"] is None else s["x"].double() + s["residual"].double()
    length = torch.linalg.vector_norm(t, dim=-1, keepdim=True)
    y = s["weight"].double() * t / torch.sqrt(length ** 2 / t.shape[-1] + EPS)
    res = None if s["residual"] is None else t
    if s["scale"] is None:
        return {"out": y, "residual": res}
    scale = torch.linalg.vector_norm(y, ord=math.inf, dim=-1) / 448.0
    codes = _e4m3_of(y / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None])
    return {"out": codes, "scale": scale, "residual": res}


def _exact_rope(s):
    c, n = s["case"], s["positions"].shape[0]
    half = c["dim"] // 2
    turn = torch.zeros(n, half, dtype=F64, device=s["q"].device)
    at = 0
    for axis, size in enumerate(_ints(c["sections"])):
        for i in range(size):
            exponent = (at + i) / half if c["shared"] else i / size
            turn[:, at + i] = s["positions"][:, axis].double() * math.exp(-exponent * math.log(s["theta"]))
        at += size
    turn = torch.polar(torch.ones_like(turn), turn)[:, None]
    out = {}
    for name in ("q", "k"):
        x, weight = s[name].double(), s[name + "_weight"]
        if weight is not None:
            rms = torch.linalg.vector_norm(x, dim=-1, keepdim=True) / math.sqrt(c["dim"])
            x = x / torch.sqrt(rms ** 2 + EPS) * weight.double()
        if c["interleaved"]:
            z = torch.view_as_complex(x.unflatten(-1, (half, 2)).contiguous()) * turn
            out[name] = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(x[..., :half], x[..., half:]) * turn
            out[name] = torch.cat((z.real, z.imag), -1)
    return out


def _exact_attn(s):
    c, out, at = s["case"], torch.empty_like(s["q"], dtype=F64), 0
    group = c["heads"] // c["kv_heads"]
    for n in _ints(c["lengths"]):
        rows = slice(at, at + n)
        hidden = torch.ones(n, n, dtype=torch.bool, device=out.device).triu(1) if c["causal"] else None
        for h in range(c["heads"]):
            logits = s["q"][rows, h].double() @ s["k"][rows, h // group].double().T / math.sqrt(c["dim"])
            if hidden is not None:
                logits = logits.masked_fill(hidden, -math.inf)
            weights = torch.exp(logits - torch.logsumexp(logits, -1, keepdim=True))
            out[rows, h] = weights @ s["v"][rows, h // group].double()
        at += n
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "rope": _exact_rope, "attn": _exact_attn}[case["op"]](s)
