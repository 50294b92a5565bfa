"""Cases of a decoder's self attention: rotary positions, appending keys and values to a paged cache
with the rotation on the way, and attention over the paged cache, where a batch may share a prefix.

Each case is one pass through one operator. ``run`` computes it either in its plain form
(elementary torch operations in 32 bits, angles in 64, rounded once at the end) or, with ``own``, through the
calls of ``vision_transformer_encoder_gb300.api``. ``exact`` gives the same outputs from the
definitions in 64 bits.

Definitions:
  frequencies  f_i = base^(-2 i / width), i < width / 2; where positions are stretched by `factor` past a
               trained length n: r = n f_i / 2 pi, w = clamp((r - 1) / 31, 0, 1), f_i (w + (1 - w) / factor)
  rotary       pair i of the first `width` columns of a head at position p turns by the angle p f_i, times `scale`:
               columns i and i + width / 2 ("half"), or 2 i and 2 i + 1 ("interleaved"); the others stay
  append       token t of sequence b has index u = starts[b] + t, position u + prefix; its rotated key and its value go
               to slot u % page of page table[b, u // page], for t < lens[b]; its rotated query is returned
  paged        query t of sequence b sees all keys of its group's prefix and its own keys u < kv_lens[b] - (q_lens[b] - 1 - t):
               softmax of scale * q k^T over both, times v; rows t >= q_lens[b] are zeros
"""
import math

import torch

own = False
DEVICE = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4}
TINY = 2.0 ** -126


def _rotary(B, T, H, dh, width, layout, x, far=0, factor=1.0, name=None):
    """far: the largest position."""
    return _case(name, op="rotary", B=B, T=T, H=H, dh=dh, width=width, layout=layout, x=x, far=max(far, T), factor=factor)


def _append(B, T, H, Hkv, dh, width, layout, x, page, held, ragged, prefix=0, name=None):
    """held: keys that a sequence has at most, the new ones among them."""
    return _case(name, op="append", B=B, T=T, H=H, Hkv=Hkv, dh=dh, width=width, layout=layout, x=x, page=page,
                 held=max(held, T), ragged=ragged, prefix=prefix)


def _paged(B, Tq, H, Hkv, dh, x, page, held, ragged, prefix=0, groups=1, name=None):
    return _case(name, op="paged", B=B, Tq=Tq, H=H, Hkv=Hkv, dh=dh, x=x, page=page, held=max(held, Tq), ragged=ragged,
                 prefix=prefix, groups=groups)


def _case(name, **kw):
    return dict(kw, name=name) if name else kw


def listed():
    return [
        # the queries of one decoding step of eight sequences
        _rotary(8, 1, 16, 64, 64, "half", "bf16", 577, name="rotary decode"),
        # long text kept in 32 bits, positions stretched eightfold past the trained length, half of each head turned
        _rotary(2, 8200, 12, 64, 32, "interleaved", "f32", 1000000, 8.0, name="rotary far"),
        # one decoding step of 32 captions behind their images' 577 states: queries, keys and values
        _append(32, 1, 16, 16, 64, 64, "half", "bf16", 16, 128, True, 577, name="append decode"),
        # prompts of different lengths taken in whole, eight query heads on each key head
        _append(4, 2048, 16, 2, 128, 128, "half", "bf16", 64, 2100, True, name="append prompts"),
        # one decoding step of 32 captions with caches of their own
        _paged(32, 1, 16, 16, 64, "bf16", 16, 577, True, name="paged decode"),
        # a few long texts, eight query heads on each key head
        _paged(8, 1, 16, 2, 128, "bf16", 64, 8200, True, name="paged decode long"),
        # 32 captions sampled for one image: its 1025 states are the prefix, a few own tokens behind them
        _paged(32, 1, 16, 16, 64, "bf16", 16, 64, True, 1025, name="shared decode"),
        # four samples of each of 16 long prompts, three drafted tokens checked at once
        _paged(64, 3, 16, 2, 128, "bf16", 64, 577, True, 8200, 16, name="shared drafts"),
        # questions of different lengths about one image, read whole behind its states, heads of 80
        _paged(8, 500, 16, 16, 80, "bf16", 32, 500, True, 1025, name="shared questions"),
        # the next part of long prompts behind what is cached already
        _paged(2, 1025, 12, 12, 64, "bf16", 128, 4100, False, name="paged prompt part"),
        # long texts read whole behind a long shared prefix, eight query heads on each key head
        _paged(4, 2048, 16, 2, 128, "bf16", 64, 2048, False, 8200, name="shared long"),
        # a decoding step in 32 bits at the size of the middle encoder
        _paged(8, 1, 12, 12, 64, "f32", 16, 577, True, 197, name="paged f32"),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "append", "paged", "paged", "paged"])
    x = "f32" if rng.random() < (0.4 if op == "rotary" else 0.2) else "bf16"
    H, Hkv = rng.choice([(12, 12), (16, 16), (16, 2), (12, 3), (16, 8), (15, 5)])
    dh = rng.choice([64, 64, 80, 96, 128])
    layout = rng.choice(["half", "interleaved"])
    width = dh if rng.random() < 0.6 else 8 * rng.randint(1, dh // 8)
    page = rng.choice([16, 16, 32, 64, 128, 256])
    if op == "rotary":
        T = rng.choice([1, _logint(rng, 1, 8200)])
        return _rotary(_logint(rng, 1, max(1, min(64, 16400 // T))), T, H, dh, width, layout, x,
                       _logint(rng, T, 1000000), rng.choice([1.0, 1.0, 8.0]))
    ragged = rng.random() < 0.7
    if op == "append":
        T = rng.choice([1, _logint(rng, 1, 2048)])
        B = _logint(rng, 1, max(1, min(64, 8192 // T)))
        return _append(B, T, H, Hkv, dh, width, layout, x, page, T + _logint(rng, 1, 577), ragged, rng.choice([0, 577]))
    if x == "f32":   # a step or a few tokens
        groups = rng.choice([1, 2])
        return _paged(groups * rng.randint(1, 4), rng.choice([1, 1, 2, 4]), H, Hkv, dh, x, page, _logint(rng, 1, 1100),
                      ragged, rng.choice([0, _logint(rng, 1, 1100)]), groups)
    prefix = rng.choice([0, _logint(rng, 1, 8200)])
    groups = rng.choice([1, 1, 2, 8]) if prefix else 1
    Tq = rng.choice([1, 1, rng.randint(2, 8), _logint(rng, 2, 2048)])
    held = max(Tq, _logint(rng, 1, 8200) if rng.random() < 0.5 else _logint(rng, 1, 577))
    B = groups * _logint(rng, 1, max(1, min(64, 60_000 // held) // groups))
    most = 4 * 2048 * 9000 * 16 * 128
    Tq = max(1, min(Tq, most // (B * (held + prefix) * H * dh)))
    return _paged(B, Tq, H, Hkv, dh, "bf16", page, held, ragged, prefix, groups)


def _spread(n, most, least):
    """n lengths, evenly spread from `most` down to `least`."""
    return [most - (most - least) * i // max(1, n - 1) for i in range(n)]


def _lens(c):
    """(keys, new tokens) of each sequence; the new ones are the last of the keys."""
    B, T = c["B"], c.get("T", c.get("Tq"))
    if not c["ragged"]:
        return [c["held"]] * B, [T] * B
    keys = _spread(B, c["held"], max(1, c["held"] // 2))
    return keys, [min(k, n) for k, n in zip(keys, _spread(B, T, max(1, T // 2)))]


def _prefixes(c):
    """Prefix length of each group."""
    return _spread(c["groups"], c["prefix"], max(1, c["prefix"] // 2)) if c["prefix"] else []


def work(c):
    e, dh, H = SIZE[c["x"]], c["dh"], c["H"]
    if c["op"] == "rotary":
        n = c["B"] * c["T"] * H
        return {"bytes": 2 * e * n * dh + 4 * c["B"] * c["T"], "flops": 3 * n * c["width"]}
    keys, new = _lens(c)
    Hkv = c["Hkv"]
    if c["op"] == "append":
        n = sum(new)
        # every query, padding too, is read, turned and written
        return {"bytes": 2 * e * dh * (n * 2 * Hkv + c["B"] * c["T"] * H) + 4 * n // c["page"] + 8 * c["B"],
                "flops": 3 * c["width"] * (n * Hkv + c["B"] * c["T"] * H)}
    S = c["B"] // c["groups"]
    before = [p for p in _prefixes(c) for _ in range(S)] or [0] * c["B"]
    # the keys that the new tokens of a sequence see, in all
    seen = sum(n * (p + k) - n * (n - 1) // 2 for k, n, p in zip(keys, new, before))
    return {"bytes": e * dh * (2 * Hkv * (sum(keys) + sum(_prefixes(c))) + H * (sum(new) + c["B"] * c["Tq"])),
            "flops": 4 * dh * H * seen}


# ------------------------------------------------------------------------------- inputs
def _frequencies(width, factor, base=10000.0, trained=2048):
    """One list of Python numbers, 64 bits each."""
    f = [base ** (-2 * i / width) for i in range(width // 2)]
    if factor != 1:
        w = [min(max((trained * x / (2 * math.pi) - 1) / 31, 0.0), 1.0) for x in f]
        f = [x * (y + (1 - y) / factor) for x, y in zip(f, w)]
    return f


def _scale(c):
    """What rotated columns are multiplied by: stretched positions sharpen their scores."""
    return 0.1 * math.log(c["factor"]) + 1 if c.get("factor", 1) != 1 else 1.0


def _table(g, lens, rows, page, first, pages):
    """Page table of sequences with room for `rows` keys each: pages in no order, -1 where nothing is held.
    first: the first of `pages`, the pool's pages in the order in which they are given out."""
    per = -(-rows // page)
    t = torch.full((len(lens), per), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        m = -(-n // page)
        t[b, :m] = pages[first:first + m]
        first += m
    return t.to(DEVICE), first


def prepare(c, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    gc = torch.Generator().manual_seed(seed)
    dt = TYPES[c["x"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEVICE).to(dt)

    def order(n):
        return torch.randperm(n, generator=gc)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=DEVICE)

    B, H, dh, s = c["B"], c["H"], c["dh"], {"c": c}
    if c["op"] != "paged":
        s["frequencies"] = torch.tensor(_frequencies(c["width"], c.get("factor", 1)), dtype=torch.float64).to(DEVICE)
    if c["op"] == "rotary":
        T = c["T"]
        s["x"] = normal(B, T, H, dh)
        ends = [c["far"] - (c["far"] - T) * i // (2 * B) for i in range(B)]
        s["positions"] = (ints(ends)[:, None] - T + torch.arange(T, device=DEVICE, dtype=torch.int32)).contiguous()
        return s
    page, Hkv = c["page"], c["Hkv"]
    keys, new = _lens(c)
    before = _prefixes(c) if c["op"] == "paged" else []
    count = sum(-(-n // page) for n in keys + before)
    pool = normal(2, count + count // 16 + 1, page, Hkv, dh)
    s["k_pages"], s["v_pages"] = pool[0], pool[1]
    pages = order(pool.shape[1]).int()
    at = order(B).tolist()
    keys, new = [keys[i] for i in at], [new[i] for i in at]
    s["table"], first = _table(g, keys, c["held"], page, 0, pages)
    if c["op"] == "append":
        # one projection leaves queries, keys and values side by side
        qkv = normal(B, c["T"], H + 2 * Hkv, dh)
        s["q"], s["k"], s["v"] = qkv[:, :, :H], qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:]
        s["starts"] = ints([k - n for k, n in zip(keys, new)])
        s["lens"] = ints(new)
        s["positions"] = (s["starts"][:, None] + c["prefix"] + torch.arange(c["T"], device=DEVICE)).int()
        return s
    s["q"] = normal(B, c["Tq"], H, dh)
    s["kv_lens"] = ints(keys)
    s["q_lens"] = ints(new) if c["ragged"] and c["Tq"] > 1 else None
    s["prefix_table"], _ = _table(g, before, c["prefix"], page, first, pages) if before else (None, 0)
    s["prefix_lens"] = ints(before) if before else None
    return s


# --------------------------------------------------------------------------- plain forms
def _turned(c, x, positions, f):
    """x (B, T, heads, dh) in 32 bits, rotated: angles in 64."""
    a = positions.double()[:, :, None, None] * f
    cos, sin = (torch.cos(a) * _scale(c)).float(), (torch.sin(a) * _scale(c)).float()
    n, x = c["width"], x.float()
    r = x[..., :n]
    if c["layout"] == "half":
        u, v = r[..., : n // 2], r[..., n // 2:]
        r = torch.cat([u * cos - v * sin, u * sin + v * cos], 3)
    else:
        u, v = r[..., 0::2], r[..., 1::2]
        r = torch.stack([u * cos - v * sin, u * sin + v * cos], 4).flatten(3)
    return torch.cat([r, x[..., n:]], 3)


def _held(pages, table):
    """The pages of a table in turn, in 32 bits: (sequences, heads, keys, dh)."""
    return pages[table.clamp_min(0).long()].flatten(1, 2).permute(0, 2, 1, 3).float()


def run(s):
    if own:
        return _run_own(s)
    c = s["c"]
    dt = TYPES[c["x"]]
    if c["op"] == "rotary":
        return [_turned(c, s["x"], s["positions"], s["frequencies"]).to(dt)]
    page = c["page"]
    if c["op"] == "append":
        t = torch.arange(c["T"], device=s["k"].device)
        live = t < s["lens"][:, None]
        u = (s["starts"][:, None] + t).clamp_max(s["table"].shape[1] * page - 1).long()
        at = (s["table"].long().gather(1, u // page) * page + u % page)[live]
        s["k_pages"].view(-1, c["Hkv"], c["dh"])[at] = _turned(c, s["k"], s["positions"], s["frequencies"]).to(dt)[live]
        s["v_pages"].view(-1, c["Hkv"], c["dh"])[at] = s["v"][live]
        return [s["k_pages"], s["v_pages"], _turned(c, s["q"], s["positions"], s["frequencies"]).to(dt)]
    B, Tq, H, Hkv, dh = (c[n] for n in ("B", "Tq", "H", "Hkv", "dh"))
    G = H // Hkv
    q = s["q"].float().view(B, Tq, Hkv, G, dh).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Tq, dh) * dh ** -0.5
    k, v = _held(s["k_pages"], s["table"]), _held(s["v_pages"], s["table"])
    t = torch.arange(Tq, device=q.device)
    ends = s["kv_lens"][:, None] - (s["q_lens"][:, None] if s["q_lens"] is not None else Tq) + 1 + t     # (B, Tq)
    gone = torch.arange(k.shape[2], device=q.device) >= ends.repeat(1, G)[:, None, :, None]
    x = (q @ k.transpose(2, 3)).masked_fill_(gone, -math.inf)
    n = 0
    if s["prefix_table"] is not None:
        n, groups = c["prefix"], c["groups"]
        kp, vp = _held(s["k_pages"], s["prefix_table"])[:, :, :n], _held(s["v_pages"], s["prefix_table"])[:, :, :n]
        # the rows of a group's sequences against its keys at once
        y = _regroup(q, groups) @ kp.transpose(2, 3)
        y.masked_fill_(torch.arange(n, device=q.device) >= s["prefix_lens"][:, None, None, None], -math.inf)
        x = torch.cat([_ungroup(y, B), x], 3)
    m = x.amax(3, keepdim=True).clamp_min(torch.finfo(torch.float32).min)
    p = torch.exp(x.sub_(m))
    z = p.sum(3, keepdim=True).clamp_min(TINY)
    o = p[..., n:] @ v
    if n:
        o = o + _ungroup(_regroup(p[..., :n], groups) @ vp, B)
    o = (o / z).view(B, Hkv, G, Tq, dh).permute(0, 3, 1, 2, 4).reshape(B, Tq, H, dh)
    if s["q_lens"] is not None:
        o = o.masked_fill((t >= s["q_lens"][:, None])[:, :, None, None], 0)
    return [o.to(dt)]


def _regroup(x, groups):
    """(B, heads, rows, n) -> (groups, heads, B / groups * rows, n)"""
    B, h, r, n = x.shape
    return x.reshape(groups, B // groups, h, r, n).transpose(1, 2).reshape(groups, h, -1, n)


def _ungroup(x, B):
    groups, h, r, n = x.shape
    return x.view(groups, h, B // groups, -1, n).transpose(1, 2).reshape(B, h, -1, n)


# ----------------------------------------------------------------------------- own calls
def _run_own(s):
    from vision_transformer_encoder_gb300 import api

    c = s["c"]
    layout = api.ROTARY_HALF if c.get("layout") == "half" else api.ROTARY_INTERLEAVED
    if c["op"] == "rotary":
        return [api.rotary(s["x"], s["frequencies"], positions=s["positions"], layout=layout, scale=_scale(c))]
    if c["op"] == "append":
        q = api.cache_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["starts"], lens=s["lens"], q=s["q"],
                             frequencies=s["frequencies"], positions=s["positions"], layout=layout)
        return [s["k_pages"], s["v_pages"], q]
    return [api.paged_attention(s["q"], s["k_pages"], s["v_pages"], s["table"], s["kv_lens"], q_lens=s["q_lens"],
                                prefix_table=s["prefix_table"], prefix_lens=s["prefix_lens"])]


# -------------------------------------------------------------------------- 64-bit values
def _turned_64(c, x, positions):
    """Pair by pair, as a product of complex numbers."""
    x = x.double().clone()
    half, n = c["width"] // 2, c["width"]
    for i, f in enumerate(_frequencies(n, c.get("factor", 1))):
        i, j = (i, i + half) if c["layout"] == "half" else (2 * i, 2 * i + 1)
        z = torch.complex(x[..., i], x[..., j]) * (torch.polar(torch.ones_like(f_p := positions.double() * f), f_p) * _scale(c))[:, :, None]
        x[..., i], x[..., j] = z.real, z.imag
    return x


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "rotary":
        return [_turned_64(c, s["x"], s["positions"])]
    table = s["table"].tolist()
    page = c["page"]
    if c["op"] == "append":
        kp, vp = s["k_pages"].double(), s["v_pages"].double()
        k = _turned_64(c, s["k"], s["positions"])
        for b, (start, n) in enumerate(zip(s["starts"].tolist(), s["lens"].tolist())):
            t = 0
            while t < n:   # page by page
                u = start + t
                m = min(n - t, page - u % page)
                kp[table[b][u // page], u % page:u % page + m] = k[b, t:t + m]
                vp[table[b][u // page], u % page:u % page + m] = s["v"][b, t:t + m].double()
                t += m
        return [kp, vp, _turned_64(c, s["q"], s["positions"])]
    B, Tq, H, dh = (c[n] for n in ("B", "Tq", "H", "dh"))
    G = H // c["Hkv"]
    o = torch.zeros(B, Tq, H, dh, dtype=torch.float64, device=DEVICE)

    def states(pages, row, n):
        at = torch.tensor(row[: -(-n // page)], device=DEVICE, dtype=torch.long)
        return pages[at].flatten(0, 1)[:n].double()

    lens = s["q_lens"].tolist() if s["q_lens"] is not None else [Tq] * B
    for b, (n, new) in enumerate(zip(s["kv_lens"].tolist(), lens)):
        k, v, L = states(s["k_pages"], table[b], n), states(s["v_pages"], table[b], n), 0
        if s["prefix_table"] is not None:
            j = b // (B // c["groups"])
            row, L = s["prefix_table"].tolist()[j], int(s["prefix_lens"][j])
            k = torch.cat([states(s["k_pages"], row, L), k])
            v = torch.cat([states(s["v_pages"], row, L), v])
        see = torch.arange(L + n, device=DEVICE) <= (L + n - new + torch.arange(new, device=DEVICE))[:, None]
        for h in range(H):
            x = s["q"][b, :new, h].double() @ k[:, h // G].t() / math.sqrt(dh)
            o[b, :new, h] = torch.softmax(x.masked_fill(~see, -math.inf), 1) @ v[:, h // G]
    return [o]
