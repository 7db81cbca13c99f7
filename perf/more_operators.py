"""Cases and timings of the operators around a packed KV cache that bring rows to it and read it whole.

  table    rows of cosines and sines for positions 0, 1, 2, ..., with the usual
           ways of stretching them over long contexts
  rope     rotary positions of query or key rows: half or interleaved pairs,
           all or part of the head, forward or transposed (the gradient)
  append   keys and values of a ragged batch's new tokens, straight from a
           projection's output: keys rotated, smoothed, Hadamard-transformed,
           both quantised and packed into a contiguous or paged cache
  cross    cross attention: ragged queries over all cached tokens of their
           sequence (an encoder's states, or a shared document)

With ``own`` false, ``run`` computes them in elementary torch operations; with
``own`` true it calls the library.
"""
import math
import random

import torch

own = False

D = 128   # head dimension

# name -> (library mode, codebook entries, channels per code, tokens and bytes per layout tile)
MODES = {"2": (0, 256, 4, 16, 512), "1.5": (1, 4096, 8, 64, 1536), "4": (2, 256, 2, 16, 1024),
         "3": (3, 4096, 4, 16, 768), "1.25": (4, 1024, 8, 16, 320)}
TYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
SCALINGS = ("none", "linear", "base", "wavelength", "ramp")   # in the library's numbering


# ---------------------------------------------------------------- cases

def _table(name=None, **kw):
    c = {"op": "table", "n": 4096, "rot": 128, "base": 10000.0, "scaling": "none", "factor": 1.0, "low": 1.0, "high": 4.0,
         "old": 4096, "amp": 1.0}
    return {**c, **kw, **({"name": name} if name else {})}


def _rope(name=None, **kw):
    c = {"op": "rope", "T": 1, "H": 32, "rot": 128, "inter": False, "back": False, "dt": "fp16", "far": 4096, "fused": False}
    return {**c, **kw, **({"name": name} if name else {})}


def _append(name=None, **kw):
    c = {"op": "append", "bits": "2", "B": 1, "Hq": 32, "Hkv": 8, "dt": "fp16", "new_lo": 1, "new_hi": 1, "ctx_lo": 0,
         "ctx_hi": 0, "page": 0, "rot": 128, "inter": False, "shift": 0, "fused": False, "pad": 0}
    return {**c, **kw, **({"name": name} if name else {})}


def _cross(name=None, **kw):
    c = {"op": "cross", "bits": "2", "B": 1, "Hq": 16, "Hkv": 16, "dt": "fp16", "q_lo": 1, "q_hi": 1, "lo": 1, "hi": 1,
         "page": 0, "pad": 0}
    return {**c, **kw, **({"name": name} if name else {})}


def listed():
    return [
        # start-up of a model with half of each head rotated, positions compressed four times
        _table("table_part", n=16384, rot=64, scaling="linear", factor=4.0),
        # start-up for the long context of the benchmark's default step, slow wavelengths stretched
        _table("table_196k", n=196608, base=500000.0, scaling="wavelength", factor=8.0, low=1.0, high=4.0, old=8192),
        # queries of one decode step of a batch, far into their contexts
        _rope("rope_step", T=64, H=40, far=65536, fused=True),
        # queries of a long prompt, interleaved pairs on half of the head
        _rope("rope_prompt", T=16384, H=32, rot=64, inter=True, dt="bf16", far=32768, fused=True),
        # gradient of the rotated rows of a training batch, odd token count
        _rope("rope_gradient", T=8191, H=40, rot=96, dt="fp32", back=True, far=8192),
        # one decode step of one long sequence
        _append("append_one", ctx_lo=196000, ctx_hi=196000, fused=True),
        # one decode step of a batch behind a block table, 1.5 bit; 200 tokens were evicted, so angles run ahead
        _append("append_step_paged", bits="1.5", B=64, Hq=40, new_lo=1, new_hi=1, ctx_lo=1000, ctx_hi=16000, page=256,
                shift=200, dt="bf16", fused=True),
        # ragged prompts of a batch into a paged 2-bit cache, a padded token buffer
        _append("append_prompts", B=6, new_lo=1001, new_hi=4500, ctx_lo=0, ctx_hi=2000, page=128, dt="bf16", fused=True,
                pad=57),
        # a prompt chunk at 3 bit, interleaved pairs on half of the head
        _append("append_chunk_3bit", bits="3", B=3, new_lo=150, new_hi=500, ctx_lo=3001, ctx_hi=7000, rot=64, inter=True),
        # one decoder token per sequence over an encoder's states
        _cross("cross_step", B=16, lo=700, hi=1500),
        # decoder prompts of a ragged batch over paged 4-bit encoder states, a padded token buffer
        _cross("cross_prompts_paged", bits="4", B=12, q_lo=33, q_hi=448, lo=600, hi=1500, page=64, dt="bf16", pad=13),
        # questions about a long document: 2,048 queries, four to a KV head
        _cross("cross_document", Hq=32, Hkv=8, q_lo=2048, q_hi=2048, lo=32768, hi=32768),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["table", "rope", "append", "cross"])
    if op == "table":
        rot = rng.choice([8, 32, 64, 80, 96, 128])
        scaling = rng.choice(SCALINGS)
        return _table(n=_log(rng, 1, 196608), rot=rot, base=rng.choice([10000.0, 500000.0, 1000000.0]), scaling=scaling,
                      factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 32.0]), low=1.0,
                      high=32.0 if scaling == "ramp" else 4.0, old=rng.choice([2048, 4096, 8192, 32768]),
                      amp=rng.choice([1.0, 1.0, 1.1386]))
    Hkv = rng.choice([1, 2, 4, 8])
    g = rng.randint(1, 8)
    rot = rng.choice([8, 32, 64, 96, 128, 128, 128])
    if op == "rope":
        H = rng.choice([1, 5, Hkv, Hkv * g, 40])
        T = _log(rng, 1, max(1, min(32768, 16384 * 32 // H)))
        return _rope(T=T, H=H, rot=rot, inter=rng.random() < 0.4, back=rng.random() < 0.3,
                     dt=rng.choice(["fp16", "bf16", "fp32"]) if T * H <= 8191 * 40 else rng.choice(["fp16", "bf16"]),
                     far=_log(rng, 2, 196608), fused=rng.random() < 0.5)
    bits = rng.choice(list(MODES))
    _, E, d, _, _ = MODES[bits]
    page = rng.choice([0, 0, 64, 128, 512])
    if op == "append":
        # distances to centroids at most those of the ragged prompts above
        room = (17000 * 8 * 32 * 256) // (Hkv * (D // d) * E)
        total = _log(rng, 1, max(2, min(16384, room)))
        B = _log(rng, 1, min(64, total))
        hi = max(1, total // B)
        ctx = _log(rng, 1, max(2, min(196608, 196608 * 8 // (B * Hkv))))
        return _append(bits=bits, B=B, Hq=Hkv * g, Hkv=Hkv, dt=rng.choice(["fp16", "bf16", "fp32"]),
                       new_lo=rng.choice([0, 1, max(1, hi // 3)]) if B > 1 else hi, new_hi=hi, ctx_lo=rng.randint(0, ctx),
                       ctx_hi=ctx, page=page, rot=rng.choice([0, rot, rot, rot]), inter=rng.random() < 0.4,
                       shift=rng.choice([0, 0, 1234]), fused=rng.random() < 0.5, pad=rng.choice([0, 0, 1, 40]))
    hi = _log(rng, 1, 32768)
    # scores at most those of the document above
    room = (2048 * 32 * 32768) // (hi * Hkv * g)
    B = _log(rng, 1, max(1, min(64, room)))
    q_hi = _log(rng, 1, max(1, min(4096, room // B)))
    return _cross(bits=bits, B=B, Hq=Hkv * g, Hkv=Hkv, dt=rng.choice(["fp16", "bf16"]),
                  q_lo=rng.choice([0, 1, max(1, q_hi // 3)]) if B > 1 else q_hi, q_hi=q_hi,
                  lo=rng.choice([0, max(1, hi // 3)]) if B > 1 else hi, hi=hi, page=page, pad=rng.choice([0, 0, 1, 19]))


# ---------------------------------------------------------------- packed layout (token r of a tile)

def _token_bytes(bits, role, r):
    """The bytes of a tile that token r owns, in an order that is the same for every token."""
    if bits == "2":
        if role == 0:
            return [16 * (4 * (r % 8) + j % 4) + 8 * (r // 8) + j // 4 for j in range(32)]
        return [16 * (4 * (j % 8) + (r % 8) // 2) + 4 * (j // 8) + 2 * (r // 8) + r % 2 for j in range(32)]
    if bits == "4":
        if role == 0:
            return [512 * (r // 8) + 16 * (4 * (r % 8) + j % 4) + 2 * (j // 8) + (j // 4) % 2 for j in range(64)]
        return [512 * (j // 32) + 16 * (4 * (j % 8) + (r % 8) // 2) + 4 * ((j // 8) % 4) + 2 * (r // 8) + r % 2
                for j in range(64)]
    if bits == "1.5":
        u, q = r // 16, r % 16
        if role == 0:
            return [48 * (4 * (q % 8) + p % 4) + 12 * u + 6 * (q // 8) + 3 * (p // 4) + k
                    for p in range(8) for k in range(3)]
        return [48 * (4 * p + (q % 8) // 2) + 12 * u + 3 * (q % 2 + 2 * (q // 8)) + k for p in range(8) for k in range(3)]
    if bits == "3":
        def at(lane, n):
            return 16 * lane + n if n < 16 else 512 + 8 * lane + n - 16
        if role == 0:
            return [at(4 * (r % 8) + p % 4, 12 * (r // 8) + 3 * (p // 4) + k) for p in range(16) for k in range(3)]
        return [at(4 * (p % 8) + (r % 8) // 2, 6 * (2 * (r // 8) + r % 2) + 3 * (p // 8) + k)
                for p in range(16) for k in range(3)]
    if role == 0:   # 1.25 bit: 5 bytes of each of four runs
        return [8 * L + n if n < 8 else 256 + 2 * L + n - 8
                for i in range(4) for L in [4 * (r % 8) + i] for n in range(5 * (r // 8), 5 * (r // 8) + 5)]
    slot = 2 * (r // 8) + r % 2
    return [16 * R + n if n < 16 else 256 + 4 * R + n - 16
            for i in range(4) for R in [4 * i + (r % 8) // 2] for n in range(5 * slot, 5 * slot + 5)]


def _code_at(bits, role, j):
    """(first byte, second byte, shift) of subvector j's code among a token's bytes."""
    if bits in ("2", "4"):
        return j, j, 0
    if bits in ("1.5", "3"):
        half = 8 if bits == "1.5" else 16
        p, high = j % half, j // half
        return 3 * p + high, 3 * p + high + 1, 4 * high
    if role == 0:
        i, bit = j % 4, 10 * (j // 4)
    else:
        i, bit = (j % 8) // 2, 10 * (j % 2 + 2 * (j // 8))
    return 5 * i + bit // 8, 5 * i + bit // 8 + 1, bit % 8


def _tables(bits, dev):
    """Per role: the token bytes [T][n] and each code's first and second byte [T][J] and shift [J]."""
    _, E, d, T, _ = MODES[bits]
    out = {}
    for role in (0, 1):
        tb = torch.tensor([_token_bytes(bits, role, r) for r in range(T)])
        at = [_code_at(bits, role, j) for j in range(D // d)]
        lo, hi = torch.tensor([a[0] for a in at]), torch.tensor([a[1] for a in at])
        sh = torch.tensor([a[2] for a in at], dtype=torch.int32)
        out[role] = {"bytes": tb.to(dev), "lo": tb[:, lo].to(dev), "hi": tb[:, hi].to(dev), "shift": sh.to(dev)}
    return out


def _pack(bits, role, codes):
    """The bytes of a token [...][n], in the order of _token_bytes, from its codes [...][J]."""
    if bits in ("2", "4"):
        return codes.to(torch.uint8)
    if bits in ("1.5", "3"):
        half = codes.shape[-1] // 2
        word = codes[..., :half] | (codes[..., half:] << 12)
        parts = [(word >> (8 * k)) & 255 for k in range(3)]
    else:
        pick = (lambda i: [i, i + 4, i + 8, i + 12]) if role == 0 else (lambda i: [2 * i, 2 * i + 1, 2 * i + 8, 2 * i + 9])
        at = torch.tensor([pick(i) for i in range(4)], device=codes.device)   # [run][slot]
        word = (codes[..., at] << (10 * torch.arange(4, device=codes.device))).sum(dim=-1)
        parts = [(word >> (8 * k)) & 255 for k in range(5)]
    return torch.stack(parts, dim=-1).flatten(-2).to(torch.uint8)


# ---------------------------------------------------------------- inputs

def _code_bytes(bits, tokens):
    _, _, _, T, tile = MODES[bits]
    return (tokens + T - 1) // T * tile


def _spread(lo, hi, n, rng):
    """n whole numbers spread over lo .. hi, the largest among them; the same ones for every seed, in another order."""
    x = [hi] + [lo + int((hi - lo + 1) * ((0.618034 * i) % 1.0)) for i in range(1, n)]
    rng.shuffle(x)
    return x


def _starts(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def _ints(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def _pools(c, tokens, gen, dev):
    """Packed K and V codes (every bit pattern is a valid code), contiguous or in shuffled blocks."""
    B, Hkv, page = c["B"], c["Hkv"], c["page"]
    cap = max(tokens, 1) if not page else (max(tokens, 1) + page - 1) // page * page
    shape = (B, Hkv, _code_bytes(c["bits"], cap))
    table, nblocks = None, 0
    if page:
        per = cap // page
        nblocks = B * per + 3
        shape = (nblocks, Hkv, _code_bytes(c["bits"], page))
        table = torch.randperm(nblocks, generator=gen, device=dev)[:B * per].view(B, per).to(torch.int32).contiguous()
    k = torch.randint(0, 256, shape, generator=gen, device=dev, dtype=torch.uint8)
    v = torch.randint(0, 256, shape, generator=gen, device=dev, dtype=torch.uint8)
    return k, v, table, nblocks, cap


def _hadamard(dev, dtype):
    i = torch.arange(D, device=dev)
    x = i[:, None] & i[None, :]
    par = torch.zeros_like(x)
    for b in range(7):
        par ^= (x >> b) & 1
    return (1 - 2 * par).to(dtype) / math.sqrt(D)


def _cos_sin(n, rot, dev):
    """fp32 rows [n][rot] for the plain frequencies 10000^(-2i/rot): cosines, then sines."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    a = torch.arange(n, dtype=torch.float64, device=dev)[:, None] * f
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rng = random.Random(seed)
    c = dict(case)
    st = {"c": c}
    if c["op"] == "table":
        # two models started after one another differ a little in their base
        st["base"] = c["base"] * (1.0 + rng.random() / 64)
        st["table"] = torch.zeros((c["n"], c["rot"]), device=dev)
        return st
    dt = TYPES[c["dt"]]
    if c["op"] == "rope":
        T, H = c["T"], c["H"]
        x = torch.randn((T, H + (16 if c["fused"] else 0), D), generator=gen, device=dev).to(dt)
        st["x"] = x[:, :H]      # fused: the queries of a projection that holds keys and values behind them
        st["out"] = torch.zeros((T, H, D), dtype=dt, device=dev)
        st["pos"] = torch.randint(0, c["far"], (T,), generator=gen, device=dev, dtype=torch.int32)
        st["table"] = _cos_sin(c["far"], c["rot"], dev)
        return st
    B, Hq, Hkv = c["B"], c["Hq"], c["Hkv"]
    _, E, d, _, _ = MODES[c["bits"]]
    st["tables"] = _tables(c["bits"], dev)
    if c["op"] == "append":
        new, ctx = _spread(c["new_lo"], c["new_hi"], B, rng), _spread(c["ctx_lo"], c["ctx_hi"], B, rng)
        st["n"] = n = sum(new)
        T = n + c["pad"]
        cap = c["new_hi"] + c["ctx_hi"]
        st["k"], st["v"], st["block_table"], st["nblocks"], st["cap"] = _pools(c, cap, gen, dev)
        st["row_start"], st["pos"] = _ints(_starts(new), dev), _ints(ctx, dev)
        # keys have a few large channels; the smoothing factors know them
        size = torch.ones((Hkv, D), device=dev)
        for h in range(Hkv):
            for ch in rng.sample(range(D), 4):
                size[h, ch] = rng.uniform(8.0, 20.0)
        extra = Hq if c["fused"] else 0
        qkv = torch.randn((T, extra + 2 * Hkv, D), generator=gen, device=dev)
        qkv[:, extra:extra + Hkv] *= size
        qkv = qkv.to(dt)
        st["xk"], st["xv"] = qkv[:, extra:extra + Hkv], qkv[:, extra + Hkv:]
        if not c["fused"]:
            st["xk"], st["xv"] = st["xk"].contiguous(), st["xv"].contiguous()
        st["s"] = (4.5 * size).sqrt()
        st["kcb"] = (0.55 * torch.randn((Hkv, E, d), generator=gen, device=dev)).half()
        st["vcb"] = torch.randn((Hkv, E, d), generator=gen, device=dev).half()
        st["had"] = _hadamard(dev, torch.float64)
        st["table"] = st["rope_pos"] = None
        if c["rot"]:
            st["table"] = _cos_sin(cap + c["shift"] + 1, c["rot"], dev)
            at = [p + i + c["shift"] for m, p in zip(new, ctx) for i in range(m)] + [0] * c["pad"]
            st["rope_pos"] = _ints(at, dev)
        return st
    queries, lens = _spread(c["q_lo"], c["q_hi"], B, rng), _spread(c["lo"], c["hi"], B, rng)
    st["n"], st["most"], st["longest"] = sum(queries), c["q_hi"], c["hi"]
    st["row_start"], st["lens"] = _ints(_starts(queries), dev), _ints(lens, dev)
    st["k"], st["v"], st["block_table"], st["nblocks"], st["cap"] = _pools(c, c["hi"], gen, dev)
    st["q"] = torch.randn((st["n"] + c["pad"], Hq, D), generator=gen, device=dev).to(dt)
    st["kcb"] = (0.6 * torch.randn((Hkv, E, d), generator=gen, device=dev)).half()
    st["vcb"] = torch.randn((Hkv, E, d), generator=gen, device=dev).half()
    st["s"] = 0.5 + 3.5 * torch.rand((Hkv, D), generator=gen, device=dev)
    st["out"] = torch.zeros((st["n"] + c["pad"], Hq, D), dtype=dt, device=dev)
    st["had"] = _hadamard(dev, torch.float32)
    return st


# ---------------------------------------------------------------- plain forms

def _frequencies(c, base, dev):
    """Radians per position of each pair, fp64."""
    i = torch.arange(0, c["rot"], 2, dtype=torch.float64, device=dev)
    if c["scaling"] == "base":
        base = base * c["factor"] ** (c["rot"] / (c["rot"] - 2))
    f = base ** (-i / c["rot"])
    if c["scaling"] == "linear":
        return f / c["factor"]
    if c["scaling"] == "wavelength":      # stretched below `low` turns over the old length, kept above `high`
        keep = ((c["old"] * f / (2 * math.pi) - c["low"]) / (c["high"] - c["low"])).clamp(0, 1)
        return f * (keep + (1 - keep) / c["factor"])
    if c["scaling"] == "ramp":            # the same two borders, a straight line over the pairs' numbers
        at = [c["rot"] * math.log(c["old"] / (2 * math.pi * turns)) / (2 * math.log(base)) for turns in (c["high"], c["low"])]
        a = max(math.floor(at[0]), 0)
        z = min(math.ceil(at[1]), c["rot"] - 1)
        stretch = ((i / 2 - a) / (z - a if z > a else 0.001)).clamp(0, 1)
        return f * (1 - stretch + stretch / c["factor"])
    return f


def _plain_table(st):
    c, t = st["c"], st["table"]
    a = torch.arange(c["n"], dtype=torch.float64, device=t.device)[:, None] * _frequencies(c, st["base"], t.device)
    t.copy_(torch.cat([a.cos(), a.sin()], dim=1) * c["amp"])
    return t


def _rotate(x, rows, inter, back):
    """Rotates x [T][H][128] by rows [T][rot] (cosines, sines) of the same type."""
    rot = rows.shape[1]
    cos, sin = rows[:, None, :rot // 2], rows[:, None, rot // 2:]
    if back:
        sin = -sin
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., :rot // 2], x[..., rot // 2:rot])
    y, z = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([y, z], dim=-1).flatten(-2) if inter else torch.cat([y, z], dim=-1)
    return torch.cat([turned, x[..., rot:]], dim=-1)


def _plain_rope(st):
    c = st["c"]
    rows = st["table"][st["pos"].long()]
    st["out"].copy_(_rotate(st["x"].float(), rows, c["inter"], c["back"]))
    return st["out"]


def _nearest(x, cb):
    """Codes [n][H][J] of fp32 rows [n][H][128]: the nearest centroid by fp32 squared distance, summed channel by channel
    with one rounding per product and sum; the lowest index where two are equal."""
    E, d = cb.shape[1:]
    sub = x.view(*x.shape[:2], D // d, 1, d)
    cent = cb.float()[None, :, None]                                   # [1][H][1][E][d]
    dist = None
    for i in range(d):
        u = sub[..., i] - cent[..., i]
        if dist is None:
            dist = u * u
        else:
            u = u.double()
            dist = u.mul_(u).add_(dist).float()
    return dist.argmin(dim=-1)


def _plain_append(st):
    c, n = st["c"], st["n"]
    B, Hkv, bits = c["B"], c["Hkv"], c["bits"]
    _, _, _, T, tile = MODES[bits]
    dev = st["pos"].device
    if not n:
        return st["k"], st["v"]
    t = torch.arange(n, device=dev)
    b = (t[:, None] >= st["row_start"].long()[None, 1:]).sum(dim=1)    # the sequence of each token
    at = st["pos"].long()[b] + t - st["row_start"].long()[b]
    key = st["xk"][:n].double()
    if c["rot"]:
        key = _rotate(key, st["table"][st["rope_pos"][:n].long()].double(), c["inter"], False).float().double()
    key = ((key / st["s"].double()) @ st["had"]).float()
    h = torch.arange(Hkv, device=dev)
    if st["block_table"] is None:
        base = (b[:, None] * Hkv + h) * st["k"].shape[2] + (at // T * tile)[:, None]
    else:
        page = c["page"]
        block = st["block_table"].long()[b, at // page]
        base = (block[:, None] * Hkv + h) * st["k"].shape[2] + (at % page // T * tile)[:, None]
    for role, name, rows, cb in ((0, "k", key, "kcb"), (1, "v", st["xv"][:n].float(), "vcb")):
        codes = _nearest(rows, st[cb])
        where = base[:, :, None] + st["tables"][role]["bytes"][at % T][:, None]
        st[name].view(-1).scatter_(0, where.flatten(), _pack(bits, role, codes).flatten())
    return st["k"], st["v"]


def _logical(pool, table):
    """A cache's streams [B][Hkv][bytes], through the block table where there is one."""
    if table is None:
        return pool
    x = pool[table.long()]                      # [B][blocks][Hkv][bytes]
    return x.permute(0, 2, 1, 3).reshape(x.shape[0], x.shape[2], -1)


def _dequant(bits, buf, tab, cb):
    """fp32 rows [B][Hkv][tokens][128] of a packed cache: each code's centroid."""
    _, E, d, T, tile = MODES[bits]
    B, Hkv = buf.shape[:2]
    x = buf.view(B, Hkv, -1, tile)
    codes = (x[..., tab["lo"]].int() | (x[..., tab["hi"]].int() << 8)) >> tab["shift"]
    codes = (codes & (E - 1)).view(B, Hkv, -1, D // d)
    head = torch.arange(Hkv, device=buf.device).view(1, Hkv, 1, 1)
    return cb.float()[head, codes.long()].view(B, Hkv, codes.shape[2], D)


def _plain_cross(st):
    c, n, M, S = st["c"], st["n"], st["most"], st["longest"]
    B, Hq, Hkv = c["B"], c["Hq"], c["Hkv"]
    g = Hq // Hkv
    dev = st["lens"].device
    if not n:
        return st["out"]
    start = st["row_start"].long()
    row = (start[:-1, None] + torch.arange(M, device=dev)).clamp(max=n - 1)       # [B][M], rows past a sequence's are not used
    q = (st["q"].float() * st["s"].repeat_interleave(g, dim=0)) @ st["had"]
    q = q[row].view(B, M, Hkv, g, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, M * g, D)
    k = _dequant(c["bits"], _logical(st["k"], st["block_table"]), st["tables"][0], st["kcb"])[:, :, :S]
    w = (q / math.sqrt(D)) @ k.transpose(2, 3)
    del k
    see = (torch.arange(S, device=dev) < st["lens"][:, None])[:, None, None]
    w.masked_fill_(~see, -math.inf)
    w.sub_(w.amax(dim=3, keepdim=True).clamp(min=-1e30)).exp_()
    total = w.sum(dim=3, keepdim=True)
    v = _dequant(c["bits"], _logical(st["v"], st["block_table"]), st["tables"][1], st["vcb"])[:, :, :S]
    o = (w @ v) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.view(B, Hkv, M, g, D).permute(0, 2, 1, 3, 4).reshape(B, M, Hq, D)
    t = torch.arange(n, device=dev)
    b = (t[:, None] >= start[None, 1:]).sum(dim=1)
    st["out"][:n] = o[b, t - start[b]].to(st["out"].dtype)
    return st["out"]


# ---------------------------------------------------------------- one pass

def _paged(st):
    c = st["c"]
    return {"block_table": st["block_table"], "block_tokens": c["page"], "num_blocks": st["nblocks"]} if c["page"] else {}


def _run_own(st):
    from vector_quantized_bit_gb300 import _lib
    c = st["c"]
    op = c["op"]
    if op == "table":
        _lib.vqkv_rope_table(st["table"], base=st["base"], scaling=SCALINGS.index(c["scaling"]), factor=c["factor"],
                             low_turns=c["low"], high_turns=c["high"], original_len=c["old"], amplitude=c["amp"])
        return st["table"]
    if op == "rope":
        _lib.vqkv_rope(st["x"], st["pos"], st["table"], st["out"], interleaved=c["inter"], transpose=c["back"])
        return st["out"]
    mode = MODES[c["bits"]][0]
    if op == "append":
        _lib.vqkv_append(mode, st["xk"], st["xv"], st["row_start"], st["pos"], st["s"], st["kcb"], st["vcb"], st["k"], st["v"],
                         st["cap"], rope_table=st["table"], rope_pos=st["rope_pos"], interleaved=c["inter"], **_paged(st))
        return st["k"], st["v"]
    if "ws" not in st:   # kept from step to step, as a serving loop does
        st["ws"] = _lib.cross_attn_workspace(mode, c["B"], c["Hq"], c["Hkv"], st["q"].shape[0], st["most"], st["cap"],
                                             st["longest"])
    _lib.vqkv_cross_attn(mode, st["q"], st["row_start"], st["k"], st["v"], st["lens"], st["kcb"], st["vcb"], st["s"],
                         st["out"], st["ws"], st["cap"], st["longest"], st["most"], **_paged(st))
    return st["out"]


def run(st):
    if own:
        return _run_own(st)
    return {"table": _plain_table, "rope": _plain_rope, "append": _plain_append, "cross": _plain_cross}[st["c"]["op"]](st)


# ---------------------------------------------------------------- work

def work(case):
    c = case
    if c["op"] == "table":
        return {"bytes": 4.0 * c["n"] * c["rot"], "flops": 0.0}
    e = 4.0 if c["dt"] == "fp32" else 2.0
    if c["op"] == "rope":
        rows = min(c["T"], c["far"])
        return {"bytes": c["T"] * (2 * e * c["H"] * D + 4) + 4.0 * rows * c["rot"], "flops": 3.0 * c["T"] * c["H"] * c["rot"]}
    B, Hq, Hkv = c["B"], c["Hq"], c["Hkv"]
    _, E, d, T, tile = MODES[c["bits"]]
    code = 2.0 * tile / T                                          # K + V bytes of one (token, KV head)
    books = 4.0 * Hkv * E * d + 4 * Hkv * D
    rng = random.Random(0)
    if c["op"] == "append":
        n = sum(_spread(c["new_lo"], c["new_hi"], B, rng))
        return {"bytes": n * (Hkv * (2 * e * D + code) + 4.0 * c["rot"] + (4 if c["rot"] else 0)) + books,
                "flops": 2.0 * n * Hkv * 2 * E * D}
    qs, lens = _spread(c["q_lo"], c["q_hi"], B, random.Random(0)), _spread(c["lo"], c["hi"], B, random.Random(0))
    pairs = sum(qs) * sum(lens) / B                                # expected (query, token) pairs
    return {"bytes": sum(lens) * Hkv * code + 2 * e * sum(qs) * Hq * D + books, "flops": 4.0 * D * Hq * pairs}


# ---------------------------------------------------------------- definition in 64 bits

def _exact_frequency(c, base, i):
    r, f = c["rot"], c["factor"]
    plain = math.exp(-2 * i / r * math.log(base))
    if c["scaling"] == "none":
        return plain
    if c["scaling"] == "linear":
        return plain / f
    if c["scaling"] == "base":
        return math.exp(-2 * i / r * (math.log(base) + r / (r - 2) * math.log(f)))
    if c["scaling"] == "wavelength":
        wave = 2 * math.pi / plain
        if wave < c["old"] / c["high"]:
            return plain
        if wave > c["old"] / c["low"]:
            return plain / f
        mix = (c["old"] / wave - c["low"]) / (c["high"] - c["low"])
        return (1 - mix) * plain / f + mix * plain

    def pair_of(turns):   # the (broken) pair number that makes that many turns over the old length
        return r / 2 * math.log(c["old"] / (turns * 2 * math.pi)) / math.log(base)
    first, last = max(math.floor(pair_of(c["high"])), 0), min(math.ceil(pair_of(c["low"])), r - 1)
    if last <= first:
        last = first + 0.001
    slow = min(1.0, max(0.0, (i - first) / (last - first)))
    return slow * plain / f + (1 - slow) * plain


def _exact_table(st):
    c = st["c"]
    p = torch.arange(c["n"], dtype=torch.float64, device=st["table"].device)
    out = torch.zeros((c["n"], c["rot"]), dtype=torch.float64, device=p.device)
    half = c["rot"] // 2
    for i in range(half):
        z = torch.polar(torch.full_like(p, c["amp"]), p * _exact_frequency(c, st["base"], i))
        out[:, i], out[:, half + i] = z.real, z.imag
    return out


def _exact_rope(st):
    c = st["c"]
    half = c["rot"] // 2
    rows = st["table"].double()[st["pos"].long()]
    turn = torch.complex(rows[:, :half], rows[:, half:])
    if c["back"]:
        turn = turn.conj()
    out = st["x"].double().clone()
    lo = slice(0, c["rot"], 2) if c["inter"] else slice(0, half)
    hi = slice(1, c["rot"], 2) if c["inter"] else slice(half, c["rot"])
    z = torch.complex(out[:, :, lo], out[:, :, hi]) * turn[:, None]
    out[:, :, lo], out[:, :, hi] = z.real, z.imag
    return out


def _exact_rows(bits, role, stream, n, cb):
    """fp64 rows [n][128] of one stream, each code taken from its bytes one by one."""
    _, E, d, T, tile = MODES[bits]
    dev = stream.device
    x = stream.view(-1, tile)[:(n + T - 1) // T].long()
    own_bytes = torch.tensor([_token_bytes(bits, role, r) for r in range(T)], device=dev)   # [T][n]
    tok = x[:, own_bytes].reshape(x.shape[0] * T, -1)
    rows = []
    for j in range(D // d):
        a, b, shift = _code_at(bits, role, j)
        word = tok[:, a] + 256 * tok[:, b] if b != a else tok[:, a]
        rows.append(cb.double()[torch.div(word, 1 << shift, rounding_mode="floor") % E])
    return torch.cat(rows, dim=1)[:n]


def _exact_cross(st):
    c = st["c"]
    Hq, Hkv = c["Hq"], c["Hkv"]
    g = Hq // Hkv
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=st["q"].device)
    one = torch.ones((1, 1), dtype=torch.float64, device=out.device)
    had = one
    for _ in range(7):
        had = torch.cat([torch.cat([had, had], 1), torch.cat([had, -had], 1)], 0)
    had = had / math.sqrt(D)
    starts = st["row_start"].tolist()
    for b, L in enumerate(st["lens"].tolist()):
        first, last = starts[b], starts[b + 1]
        if L == 0 or first == last:
            continue
        for h in range(Hkv):
            rows = []
            for name, role, cb in (("k", 0, "kcb"), ("v", 1, "vcb")):
                stream = st[name][b, h] if st["block_table"] is None else st[name][st["block_table"][b].long(), h].reshape(-1)
                rows.append(_exact_rows(c["bits"], role, stream, L, st[cb][h]))
            key = (rows[0] @ had.T) * st["s"][h].double()     # back to the unrotated, unsmoothed keys
            q = st["q"][first:last, h * g:(h + 1) * g].double().reshape(-1, D)
            o = torch.softmax(q @ key.T / D ** 0.5, dim=1) @ rows[1]
            out[first:last, h * g:(h + 1) * g] = o.view(last - first, g, D)
    return out


def exact(case, seed):
    st = prepare(dict(case), seed)
    op = st["c"]["op"]
    if op == "append":
        return None
    return {"table": _exact_table, "rope": _exact_rope, "cross": _exact_cross}[op](st)
