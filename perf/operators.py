"""Cases and timings of the cache-editing and draft-verification operators.

Four operators work on a packed vector-quantised KV cache that changes under a
running model:

  tree     attention of M drafted tokens per sequence over the cache; every
           draft sees the cached prefix and the drafts that its 64-bit mask
           names (its ancestors in the draft tree)
  mass     decode attention that also adds every cached token's attention
           weight (summed over the queries and query heads of its KV head) to
           a running fp32 sum
  select   the tokens a sequence keeps: its first and its most recent ones and
           those of the largest accumulated weight, as ascending positions
  compact  moves chosen tokens' codes (and accumulated weights) to the front
           of the cache, in place

With ``own`` false, ``run`` computes them in elementary torch operations; with
``own`` true it calls the library.
"""
import math

import torch

own = False

D = 128   # head dimension

# name -> (library mode, codebook entries, channels per code, tokens and bytes per layout tile)
MODES = {"2": (0, 256, 4, 16, 512), "1.5": (1, 4096, 8, 64, 1536), "4": (2, 256, 2, 16, 1024),
         "3": (3, 4096, 4, 16, 768), "1.25": (4, 1024, 8, 16, 320)}


# ---------------------------------------------------------------- cases

def _case(op, name=None, **kw):
    base = {"op": op, "bits": "2", "B": 1, "Hq": 32, "Hkv": 8, "lo": 1, "hi": 1, "page": 0}
    base.update(kw)
    if name:
        base["name"] = name
    return base


def listed():
    return [
        # the first verification after a short prompt: one small tree, latency counts
        _case("tree", "tree_short_prompt", lo=519, hi=519, M=8),
        # a draft tree over the long 2-bit context of the benchmark's default step
        _case("tree", "tree_196k", lo=196608, hi=196608, M=16),
        # a ragged batch behind a block table, 1.5 bit, five query heads per KV head, an odd draft count
        _case("tree", "tree_batch_paged", bits="1.5", B=8, Hq=40, lo=4097, hi=32768, M=27, page=256),
        # a wide tree (64 drafts, 256 softmax columns per KV head) over a 4-bit cache
        _case("tree", "tree_wide_32k", bits="4", lo=32768, hi=32768, M=64),
        # one decode step of a short sequence
        _case("mass", "mass_1k", lo=1000, hi=1000, M=1),
        # one decode step over the long 2-bit context
        _case("mass", "mass_196k", lo=196608, hi=196608, M=1),
        # the last 16 prompt tokens of a ragged 3-bit batch (an observation window)
        _case("mass", "mass_window_batch", bits="3", B=4, lo=2001, hi=16384, M=16),
        # which 8192 tokens of a ragged batch stay
        _case("select", "select_batch", B=32, lo=16384, hi=32768, keep=8192, sink=4, recent=1024),
        # which third of a 196k context stays
        _case("select", "select_196k", lo=196608, hi=196608, keep=65536, sink=64, recent=4096),
        # the accepted path of a draft tree moves up, same tokens for every head
        _case("compact", "compact_accepted_path", B=8, lo=4000, hi=8192, keep=16, tail=1),
        # a third of a 196k context stays, each head its own tokens, weights move along
        _case("compact", "compact_196k", lo=196608, hi=196608, keep=65536, tail=0),
        # a paged 1.25-bit batch down to half its capacity
        _case("compact", "compact_paged_batch", bits="1.25", B=16, lo=9000, hi=32768, keep=16384, tail=0, page=128),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tree", "mass", "select", "compact"])
    Hkv = rng.choice([1, 2, 4, 8])
    g = rng.randint(1, 8)
    # tokens x KV heads stay below those of the 196k cases
    hi = _log(rng, 65, 196608)
    most = max(1, (196608 * 8) // (hi * Hkv))
    B = _log(rng, 1, min(32, most))
    lo = rng.randint(max(1, hi // 3), hi)
    c = _case(op, bits=rng.choice(list(MODES)), B=B, Hq=Hkv * g, Hkv=Hkv, lo=lo, hi=hi,
              page=rng.choice([0, 0, 64, 128, 512]))
    if op == "tree":
        # columns x tokens x heads at most those of the 196k tree
        room = (196608 * 8 * 64) // (hi * Hkv * B * g)
        c["M"] = _log(rng, 1, max(1, min(64, room)))
    elif op == "mass":
        room = (196608 * 8 * 8) // (hi * Hkv * B * g)
        c["M"] = _log(rng, 1, max(1, min(64 // g, room)))
    elif op == "select":
        c["page"] = 0
        c["keep"] = _log(rng, 2, 9 * hi // 10)
        c["sink"] = rng.randint(0, min(64, c["keep"] // 4))
        c["recent"] = rng.randint(0, c["keep"] // 2)
    else:
        c["tail"] = rng.choice([0, 0, 1])
        c["keep"] = _log(rng, 1, min(hi, 64)) if c["tail"] else _log(rng, 1, hi)
    return c


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


# ---------------------------------------------------------------- inputs

def _code_bytes(bits, tokens):
    _, _, _, T, tile = MODES[bits]
    return (tokens + T - 1) // T * tile


def _lens(c, gen, dev):
    lens = torch.randint(c["lo"], c["hi"] + 1, (c["B"],), generator=gen, device=dev, dtype=torch.int32)
    lens[0] = c["hi"]   # the batch's longest sequence reaches the upper length
    return lens


def _capacity(c):
    return c["hi"] if not c["page"] else (c["hi"] + c["page"] - 1) // c["page"] * c["page"]


def _caches(c, gen, dev):
    """Packed K and V codes (every bit pattern is a valid code), contiguous or in shuffled blocks."""
    B, Hkv, page, cap = c["B"], c["Hkv"], c["page"], _capacity(c)
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


def _hadamard(dev):
    i = torch.arange(D, device=dev)
    x = i[:, None] & i[None, :]
    par = torch.zeros_like(x)
    for b in range(7):
        par ^= (x >> b) & 1
    return (1 - 2 * par).to(torch.float32) / math.sqrt(D)


def _weights(c, lens, cap, gen, dev):
    """Accumulated attention weights as they grow in use: skewed, with untouched (equal) tokens; 0 past the end."""
    B, Hkv = c["B"], c["Hkv"]
    x = torch.randn((B, Hkv, cap), generator=gen, device=dev).mul_(2.0).exp_()
    x[torch.rand((B, Hkv, cap), generator=gen, device=dev) < 0.1] = 0.0
    return torch.where(torch.arange(cap, device=dev) < lens[:, None, None], x, torch.zeros_like(x))


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    c = dict(case)
    B, Hq, Hkv = c["B"], c["Hq"], c["Hkv"]
    st = {"c": c, "lens": _lens(c, gen, dev)}
    if c["op"] == "select":
        st["cap"] = cap = c["hi"]
        st["weights"] = _weights(c, st["lens"], cap, gen, dev)
        st["keep"] = torch.full((B, Hkv, c["keep"]), -1, dtype=torch.int32, device=dev)
        st["keep_lens"] = torch.full((B,), -1, dtype=torch.int32, device=dev)
        return st
    st["k"], st["v"], st["table"], st["nblocks"], st["cap"] = _caches(c, gen, dev)
    st["tables"] = _tables(c["bits"], dev)
    cap = st["cap"]
    if c["op"] == "compact":
        n, lens = c["keep"], st["lens"]
        st["weights"] = _weights(c, lens, cap, gen, dev)
        if c["tail"]:   # the accepted drafts among the last `keep` tokens
            m = torch.clamp(lens, max=n)
            st["start"] = lens - m
            hit = torch.rand((B, 1, n), generator=gen, device=dev) < 0.4
            hit &= torch.arange(n, device=dev) < m[:, None, None]
            base = st["start"]
        else:           # `keep` of a sequence's tokens at random, each head its own
            st["start"] = None
            pick = torch.rand((B, Hkv, cap), generator=gen, device=dev)
            pick[:] = torch.where(torch.arange(cap, device=dev) < lens[:, None, None], pick, torch.full_like(pick, 2.0))
            kept = torch.zeros((B, Hkv, cap), dtype=torch.bool, device=dev)
            kept.scatter_(2, pick.topk(min(n, cap), dim=2, largest=False).indices, True)
            hit = kept & (torch.arange(cap, device=dev) < lens[:, None, None])
            base = torch.zeros_like(lens)
        t = torch.arange(hit.shape[2], device=dev)
        order = torch.where(hit, t, torch.full_like(t, 1 << 30)).sort(dim=2).values[:, :, :n]
        st["counts"] = hit[:, 0].sum(dim=1).to(torch.int32)
        live = torch.arange(order.shape[2], device=dev) < st["counts"][:, None, None]
        st["src"] = torch.where(live, order + base[:, None, None], torch.zeros_like(order)).to(torch.int32).contiguous()
        return st
    _, E, d, _, _ = MODES[c["bits"]]
    M = c["M"]
    st["q"] = torch.randn((B, M, Hq, D), generator=gen, device=dev).half()
    st["kcb"] = (0.6 * torch.randn((Hkv, E, d), generator=gen, device=dev)).half()
    st["vcb"] = torch.randn((Hkv, E, d), generator=gen, device=dev).half()
    st["s"] = 0.5 + 3.5 * torch.rand((Hkv, D), generator=gen, device=dev)
    st["out"] = torch.zeros((B, M, Hq, D), dtype=torch.float16, device=dev)
    st["had"] = _hadamard(dev)
    if c["op"] == "mass":
        # a few earlier steps' worth of weight on the tokens that were there before this call's
        st["weights"] = _weights(c, torch.clamp(st["lens"] - M, min=0), cap, gen, dev) * (Hq // Hkv * M / c["hi"])
    else:   # a random tree: draft 0 follows the prefix, draft m a random earlier one
        masks = torch.zeros((B, M), dtype=torch.int64, device=dev)
        parent = (torch.rand((B, M), generator=gen, device=dev) * torch.arange(0, M, device=dev)).long()
        one = torch.ones((B,), dtype=torch.int64, device=dev)
        for m in range(M):
            up = masks.gather(1, parent[:, m:m + 1])[:, 0] if m else torch.zeros_like(one)
            masks[:, m] = up | (one << m)
        st["tree"] = masks
    return st


# ---------------------------------------------------------------- plain forms

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


def _plain_attention(st, visible):
    """Softmax weights [B][Hkv][M*g][tokens] and O of the queries over the dequantised cache.

    visible: [B][M][tokens] truth values; a row that sees nothing gives zeros."""
    c = st["c"]
    B, Hq, Hkv, M = c["B"], c["Hq"], c["Hkv"], c["M"]
    g = Hq // Hkv
    s = st["s"].repeat_interleave(g, dim=0)
    q = (st["q"].float() * s) @ st["had"]                              # [B][M][Hq][128]
    q = q.view(B, M, Hkv, g, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, M * g, D)
    n = visible.shape[2]
    k = _dequant(c["bits"], _logical(st["k"], st["table"]), st["tables"][0], st["kcb"])[:, :, :n]
    w = (q / math.sqrt(D)) @ k.transpose(2, 3)
    del k
    see = visible.repeat_interleave(g, dim=1).unsqueeze(1)             # [B][1][M*g][tokens]
    w = w.masked_fill(~see, -math.inf)
    top = w.amax(dim=3, keepdim=True).clamp(min=-1e30)
    w = torch.exp(w - top)
    total = w.sum(dim=3, keepdim=True)
    w = w / torch.where(total > 0, total, torch.ones_like(total))
    v = _dequant(c["bits"], _logical(st["v"], st["table"]), st["tables"][1], st["vcb"])[:, :, :n]
    o = (w @ v).view(B, Hkv, M, g, D).permute(0, 2, 1, 3, 4).reshape(B, M, Hq, D)
    return w, o.half()


def _causal(st):
    c = st["c"]
    t = torch.arange(c["hi"], device=st["lens"].device)
    last = st["lens"].long()[:, None] - c["M"] + torch.arange(c["M"], device=t.device)
    return t <= last[:, :, None]


def _tree_visible(st):
    c = st["c"]
    t = torch.arange(c["hi"], device=st["lens"].device)
    lens = st["lens"].long()[:, None, None]
    j = t - (lens - c["M"])                                            # draft index of token t
    bit = (st["tree"][:, :, None] >> j.clamp(0, 63)) & 1
    return (t < lens) & ((j < 0) | (bit == 1))


def _plain_select(st):
    c, lens, w = st["c"], st["lens"].long()[:, None, None], st["weights"]
    t = torch.arange(w.shape[2], device=w.device)
    safe = (t < c["sink"]) | (t >= lens - c["recent"])
    rank = torch.where(safe, torch.full_like(w, math.inf), w)
    rank = torch.where(t < lens, rank, torch.full_like(w, -1.0))
    order = rank.sort(dim=2, descending=True, stable=True).indices
    n = torch.clamp(lens, max=c["keep"])
    live = torch.arange(w.shape[2], device=w.device) < n
    kept = torch.where(live, order, torch.full_like(order, 1 << 30)).sort(dim=2).values[:, :, :c["keep"]]
    m = kept.shape[2]
    st["keep"][:, :, :m] = torch.where(kept < (1 << 30), kept.int(), st["keep"][:, :, :m])
    st["keep_lens"].copy_(n.view(-1))
    return st["keep"], st["keep_lens"]


def _plain_move(buf, bits, tb, src, dst, live):
    """Token dst[b][h][i] of a stream takes token src[b][h][i]'s bytes, where live."""
    _, _, _, T, tile = MODES[bits]
    n = tb.shape[1]
    old = buf.clone()
    at_src = (src // T * tile).unsqueeze(3) + tb[src % T]
    at_dst = (dst // T * tile).unsqueeze(3) + tb[dst % T]
    moved = old.gather(2, at_src.flatten(2)).view(at_src.shape)
    stay = old.gather(2, at_dst.flatten(2)).view(at_dst.shape)
    buf.scatter_(2, at_dst.flatten(2), torch.where(live.unsqueeze(3).expand(-1, -1, -1, n), moved, stay).flatten(2))
    return buf


def _plain_compact(st):
    c = st["c"]
    B, Hkv, bits = c["B"], c["Hkv"], c["bits"]
    src = st["src"].long().expand(B, Hkv, -1)
    start = st["start"].long() if st["start"] is not None else torch.zeros((B,), dtype=torch.int64, device=src.device)
    i = torch.arange(src.shape[2], device=src.device)
    live = (i < st["counts"][:, None, None]).expand(B, Hkv, -1)
    dst = (start[:, None, None] + i).expand(B, Hkv, -1)   # entries past the count write their own bytes back
    for name, role in (("k", 0), ("v", 1)):
        x = _plain_move(_logical(st[name], st["table"]), bits, st["tables"][role]["bytes"], src, dst, live)
        if st["table"] is not None:
            per = st["table"].shape[1]
            st[name][st["table"].long()] = x.view(B, Hkv, per, -1).permute(0, 2, 1, 3)
    w = st["weights"]
    moved = torch.where(live, w.gather(2, src), w.gather(2, dst))
    w.scatter_(2, dst, moved)
    t = torch.arange(w.shape[2], device=w.device)
    end = (start + st["counts"].long())[:, None, None]
    w.masked_fill_((t >= end) & (t < st["lens"].long()[:, None, None]), 0.0)
    return st["k"], st["v"], w


# ---------------------------------------------------------------- one pass

def _paged(st):
    c = st["c"]
    return {"block_table": st["table"], "block_tokens": c["page"], "num_blocks": st["nblocks"]} if c["page"] else {}


def _run_own(st):
    from vector_quantized_bit_gb300 import _lib
    c = st["c"]
    op, mode, cap, hi = c["op"], MODES[c["bits"]][0], st["cap"], c["hi"]
    if op == "select":
        _lib.vqkv_evict_select(st["weights"], st["lens"], st["keep"], st["keep_lens"], n_sink=c["sink"],
                               n_recent=c["recent"], max_seq_len=hi)
        return st["keep"], st["keep_lens"]
    if op == "compact":
        _lib.vqkv_cache_compact(mode, st["k"], st["v"], st["lens"], st["src"], st["counts"], cap, start=st["start"],
                                mass=st["weights"], **_paged(st))
        return st["k"], st["v"], st["weights"]
    if "ws" not in st:   # kept from step to step, as a serving loop does
        make = _lib.decode_tree_workspace if op == "tree" else _lib.decode_mass_workspace
        st["ws"] = make(mode, c["B"], c["Hq"], c["Hkv"], c["M"], cap, hi)
    if op == "tree":
        _lib.vqkv_decode_attn_tree(mode, st["q"], st["tree"], st["k"], st["v"], st["lens"], st["kcb"], st["vcb"],
                                   st["s"], st["out"], st["ws"], cap, hi, **_paged(st))
        return st["out"]
    _lib.vqkv_decode_attn_mass(mode, st["q"], st["k"], st["v"], st["lens"], st["kcb"], st["vcb"], st["s"], st["out"],
                               st["weights"], st["ws"], cap, hi, **_paged(st))
    return st["out"], st["weights"]


def run(st):
    if own:
        return _run_own(st)
    op = st["c"]["op"]
    if op == "select":
        return _plain_select(st)
    if op == "compact":
        return _plain_compact(st)
    if op == "tree":
        st["out"].copy_(_plain_attention(st, _tree_visible(st))[1])
        return st["out"]
    w, o = _plain_attention(st, _causal(st))
    st["weights"][:, :, :w.shape[3]] += w.sum(dim=2)
    st["out"].copy_(o)
    return st["out"], st["weights"]


# ---------------------------------------------------------------- work

def work(case):
    c = case
    B, Hq, Hkv = c["B"], c["Hq"], c["Hkv"]
    rows = Hkv * (c["hi"] + (B - 1) * (c["lo"] + c["hi"]) // 2)   # expected (token, KV head) pairs
    kept = B * Hkv * min(c.get("keep", 0), c["hi"])
    _, E, d, T, tile = MODES[c["bits"]]
    code = 2.0 * tile / T                                          # K + V bytes of one pair
    if c["op"] == "select":
        return {"bytes": 4.0 * rows + 4.0 * min(kept, rows), "flops": 0.0}
    if c["op"] == "compact":
        kept = 0.4 * kept if c["tail"] else min(kept, rows)
        dropped = (B * Hkv * c["keep"] if c["tail"] else rows) - kept
        index = kept / Hkv if c["tail"] else kept
        return {"bytes": kept * (2 * code + 8) + 4 * index + 4 * max(0.0, dropped), "flops": 0.0}
    M = c["M"]
    io = 2.0 * 2 * B * M * Hq * D + 2 * 2 * Hkv * E * d + 4 * Hkv * D
    if c["op"] == "tree":
        io += 8 * B * M
    else:
        io += 8.0 * rows
    return {"bytes": rows * code + io, "flops": 4.0 * D * rows * (Hq // Hkv) * M}


# ---------------------------------------------------------------- definition in 64 bits

def _exact_places(bits, role):
    """The bit of a tile that holds bit b of the code of token t, subvector j, as [b][t][j]."""
    _, E, d, T, _ = MODES[bits]
    nbit = E.bit_length() - 1
    place = torch.zeros((nbit, T, D // d), dtype=torch.int64)
    for t in range(T):
        for j in range(D // d):
            for b in range(nbit):
                if bits == "2":
                    r = t
                    byte = (16 * (4 * (r % 8) + j % 4) + 8 * (r // 8) + j // 4 if role == 0 else
                            16 * (4 * (j % 8) + (r % 8) // 2) + 4 * (j // 8) + 2 * (r // 8) + r % 2)
                    bit = 8 * byte + b
                elif bits == "4":
                    r = t
                    byte = (512 * (r // 8) + 16 * (4 * (r % 8) + j % 4) + 2 * (j // 8) + (j // 4) % 2 if role == 0 else
                            512 * (j // 32) + 16 * (4 * (j % 8) + (r % 8) // 2) + 4 * ((j // 8) % 4) + 2 * (r // 8)
                            + r % 2)
                    bit = 8 * byte + b
                elif bits == "1.25":
                    r = t
                    if role == 0:
                        run, B = 4 * (r % 8) + j % 4, 40 * (r // 8) + 10 * (j // 4) + b
                        byte = 8 * run + B // 8 if B < 64 else 256 + 2 * run + B // 8 - 8
                    else:
                        run, B = 4 * ((j % 8) // 2) + (r % 8) // 2, 40 * (2 * (r // 8) + r % 2) + 10 * (j % 2 + 2 * (j // 8)) + b
                        byte = 16 * run + B // 8 if B < 128 else 256 + 4 * run + B // 8 - 16
                    bit = 8 * byte + B % 8
                else:   # 12-bit codes of subvectors p and p + half in 3 bytes
                    half = (D // d) // 2
                    p, r = j % half, t % 16
                    pairbit = b + 12 * (j // half)
                    if bits == "1.5":
                        u = t // 16
                        first = (48 * (4 * (r % 8) + p % 4) + 12 * u + 6 * (r // 8) + 3 * (p // 4) if role == 0 else
                                 48 * (4 * p + (r % 8) // 2) + 12 * u + 3 * (r % 2 + 2 * (r // 8)))
                        bit = 8 * first + pairbit
                    else:
                        lane, n0 = ((4 * (r % 8) + p % 4, 12 * (r // 8) + 3 * (p // 4)) if role == 0 else
                                    (4 * (p % 8) + (r % 8) // 2, 6 * (2 * (r // 8) + r % 2) + 3 * (p // 8)))
                        k = n0 + pairbit // 8
                        bit = 8 * (16 * lane + k if k < 16 else 512 + 8 * lane + k - 16) + pairbit % 8
                place[b, t, j] = bit
    return place


def _exact_rows(bits, place, stream, n, cb):
    """fp64 rows [n][128] of one stream, code bits picked one by one."""
    _, E, d, T, tile = MODES[bits]
    dev = stream.device
    x = stream.view(-1, tile)[:(n + T - 1) // T]
    nbit = place.shape[0]
    place = place.to(dev)
    code = torch.zeros((x.shape[0], T, D // d), dtype=torch.int64, device=dev)
    for b in range(nbit):
        code += ((x[:, place[b] // 8].long() >> (place[b] % 8)) & 1) << b
    return cb.double()[code].reshape(-1, D)[:n]


def _exact_attention(st):
    """O fp64 and the summed weights, one (sequence, KV head) after another, in the keys' own domain."""
    c = st["c"]
    B, Hq, Hkv, M = c["B"], c["Hq"], c["Hkv"], c["M"]
    g = Hq // Hkv
    dev = st["lens"].device
    out = torch.zeros((B, M, Hq, D), dtype=torch.float64, device=dev)
    acc = torch.zeros((B, Hkv, st["cap"]), dtype=torch.float64, device=dev)
    had = torch.ones((1, 1), dtype=torch.float64, device=dev)
    for _ in range(7):
        had = torch.cat([torch.cat([had, had], 1), torch.cat([had, -had], 1)], 0)
    had = had / math.sqrt(D)
    places = [_exact_places(c["bits"], role) for role in (0, 1)]
    for b in range(B):
        L = int(st["lens"][b])
        for h in range(Hkv):
            rows = []
            for name, role, cb in (("k", 0, "kcb"), ("v", 1, "vcb")):
                if st["table"] is None:
                    stream = st[name][b, h]
                else:
                    stream = st[name][st["table"][b].long(), h].reshape(-1)
                rows.append(_exact_rows(c["bits"], places[role], stream, L, st[cb][h]))
            key = (rows[0] @ had.T) * st["s"][h].double()     # back to the unrotated, unsmoothed keys
            t = torch.arange(L, device=dev)
            for m in range(M):
                if c["op"] == "tree":
                    pos = t - (L - M)
                    see = (pos < 0) | (((st["tree"][b, m] >> pos.clamp(min=0)) & 1) == 1)
                else:
                    see = t <= L - M + m
                if not bool(see.any()):
                    continue
                sc = (st["q"][b, m, h * g:(h + 1) * g].double() @ key.T) / D ** 0.5
                p = torch.softmax(sc.masked_fill(~see, -math.inf), dim=1)
                out[b, m, h * g:(h + 1) * g] = p @ rows[1]
                acc[b, h, :L] += p.sum(0)
    return out, acc


def exact(case, seed):
    c = dict(case)
    if c["op"] == "select":
        return None
    st = prepare(c, seed)
    if c["op"] == "compact":
        w, new = st["weights"].double(), st["weights"].double().clone()
        for b in range(c["B"]):
            a = int(st["start"][b]) if st["start"] is not None else 0
            n, L = int(st["counts"][b]), int(st["lens"][b])
            for h in range(c["Hkv"]):
                src = st["src"][b, h if st["src"].shape[1] > 1 else 0, :n].long()
                new[b, h, a:a + n] = w[b, h, src]
                new[b, h, a + n:L] = 0.0
        return None, None, new
    out, acc = _exact_attention(st)
    if c["op"] == "tree":
        return out
    return out, st["weights"].double() + acc
