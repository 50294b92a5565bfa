"""Cases of the serving operators: root-mean-square norm, 8-bit quantisation, the 8-bit matrix
product and cross attention.

Each case is one pass through one operator. ``run`` computes it either in its plain form
(elementary torch operations in 32 bits, rounded once at the end) or, with ``own``, through the
calls of ``vision_transformer_encoder_gb300.api``. ``exact`` gives the same outputs from the
definitions in 64 bits.

Definitions (s, y, z in the arithmetic of the form; B = 128 columns):
  norm      s = x + residual;  y = s / sqrt(mean(s^2) + eps) * gamma
  e4m3      per row and block of B columns: scale = max(max|y| / 448, 2^-126), q = e4m3(y / scale)
  weight    w (K, N) -> q (N, K), one scale for each B x B block
  linear    z[m, n] = sum_b a_scale[m, b] w_scale[n / B, b] sum_{k in b} a[m, k] w[n, k] (+ bias),
            then z, GELU_tanh(z) or residual + z
  cross     softmax over the first kv_len keys of scale * q k^T, times v; no keys: zeros
"""
import math

import torch

own = False
DEVICE = "cuda"
BLOCK = 128
E4M3_MAX = 448.0
TINY = 2.0 ** -126
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "f32": 4, "e4m3": 1, "": 0}


def _norm(rows, D, x, residual, out, name=None):
    return _case(name, op="norm", rows=rows, D=D, x=x, residual=residual, out=out)


def _quant(rows, K, x, name=None):
    return _case(name, op="quantize", rows=rows, K=K, x=x)


def _weight(K, N, x, name=None):
    return _case(name, op="weight", K=K, N=N, x=x)


def _linear(M, K, N, epilogue, out, residual="", bias=True, name=None):
    return _case(name, op="linear", M=M, K=K, N=N, epilogue=epilogue, out=out, residual=residual, bias=bias)


def _cross(B, Tq, Tk, H, Hkv, dh, x, ragged, name=None):
    return _case(name, op="cross", B=B, Tq=Tq, Tk=Tk, H=H, Hkv=Hkv, dh=dh, x=x, ragged=ragged)


def _case(name, **kw):
    return dict(kw, name=name) if name else kw


def listed():
    return [
        # one decoding step of eight sequences: the residual's addition, the norm and the 8-bit
        # input of the next product
        _norm(8, 1024, "bf16", "bf16", "e4m3", "norm decode"),
        # 16 images of 1025 tokens of the widest encoder, as they enter a product in 8 bits
        _norm(16400, 1280, "bf16", "bf16", "e4m3", "norm encoder"),
        # a residual stream kept in 32 bits over an odd number of rows
        _norm(2049, 5120, "bf16", "f32", "bf16", "norm f32 stream"),
        # attention outputs of 64 images on their way into an 8-bit output projection
        _quant(12608, 1024, "bf16", "quantize activations"),
        # a feed-forward weight, laid out once when a model is loaded
        _weight(1024, 4096, "bf16", "quantize weight"),
        # one decoding step: few rows against a whole weight, latency and the weight's bytes
        _linear(8, 1024, 4096, "gelu", "e4m3", name="linear decode"),
        # the tokens of three images: ragged rows, a residual, one wave of tiles
        _linear(1731, 1280, 1280, "residual", "bf16", "bf16", name="linear ragged"),
        # the first feed-forward product of 64 images of 577 tokens, its output in 8 bits again
        _linear(36928, 1024, 4096, "gelu", "e4m3", name="linear batch"),
        # a caption's next token against its image's states, sequences of different lengths
        _cross(32, 1, 577, 16, 16, 64, "bf16", True, "cross decode"),
        # captions read whole against 1025 states of heads of 80, some images with no states
        _cross(16, 500, 1025, 16, 16, 80, "bf16", True, "cross prefill"),
        # long text against many tiles' states, eight query heads on each key head
        _cross(4, 2048, 8200, 16, 2, 128, "bf16", False, "cross long"),
        # the same in 32 bits at the size of the middle encoder
        _cross(8, 197, 577, 12, 12, 64, "f32", True, "cross f32"),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "quantize", "weight", "linear", "linear", "cross", "cross", "cross"])
    if op == "norm":
        D = _logint(rng, 64, 8192)
        if rng.random() < 0.7:
            D = max(64, D // 64 * 64)
        rows = _logint(rng, 1, max(1, min(16400, 20_000_000 // D)))
        x, residual = rng.choice([("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("bf16", "")])
        out = rng.choice(["e4m3", "e4m3", "bf16", "f32"] if x == "f32" else ["e4m3", "e4m3", "bf16"])
        return _norm(rows, D, x, residual, out)
    if op == "quantize":
        K = _logint(rng, 64, 5120)
        if rng.random() < 0.7:
            K = max(64, K // 64 * 64)
        return _quant(_logint(rng, 1, max(1, min(12608, 13_000_000 // K))), K, rng.choice(["bf16", "f32"]))
    if op == "weight":
        return _weight(16 * rng.randint(4, 320), _logint(rng, 64, 4096), rng.choice(["bf16", "f32"]))
    if op == "linear":
        K, N = 16 * _logint(rng, 4, 320), _logint(rng, 64, 5120)
        if rng.random() < 0.75:
            N = max(64, N // 64 * 64)
        M = _logint(rng, 1, min(36928, 36928 * 1024 * 4096 // (K * N)))
        epilogue, out, residual = rng.choice([("store", "bf16", ""), ("store", "f32", ""), ("gelu", "e4m3", ""),
                                              ("gelu", "bf16", ""), ("residual", "bf16", "bf16"),
                                              ("residual", "f32", "f32"), ("store", "e4m3", "")])
        return _linear(M, K, N, epilogue, out, residual, rng.random() < 0.5)
    if rng.random() < 0.2:
        B, Tq, Tk, H = rng.randint(1, 8), _logint(rng, 1, 300), _logint(rng, 1, 1100), rng.choice([3, 12, 16])
        return _cross(B, Tq, Tk, H, H, rng.choice([64, 80]), "f32", rng.random() < 0.7)
    H, group = rng.choice([(12, 1), (16, 1), (16, 2), (12, 4), (16, 8), (15, 3)])
    dh = rng.choice([64, 64, 80, 96, 128])
    Tk = _logint(rng, 1, 8200)
    B = _logint(rng, 1, min(64, max(1, 60_000 // Tk)))
    Tq = rng.choice([1, _logint(rng, 1, 2048)])
    most = 4 * 2048 * 8200 * 16 * 128
    Tq = max(1, min(Tq, most // (B * Tk * H * dh)))
    return _cross(B, Tq, Tk, H, H // group, dh, "bf16", rng.random() < 0.7)


def _lens(c):
    """Key counts of a batch, evenly spread from half the keys to all of them; one image of a batch of eight or
    more has none."""
    B, Tk = c["B"], c["Tk"]
    if not c["ragged"]:
        return [Tk] * B
    lens = [Tk - (Tk // 2) * i // max(1, B - 1) for i in range(B)]
    if B >= 8:
        lens[-1] = 0
    return lens


def work(c):
    op = c["op"]
    if op == "norm":
        n, r = c["rows"] * c["D"], SIZE[c["residual"]]
        b = n * (SIZE[c["x"]] + 2 * r + SIZE[c["out"]]) + 4 * c["D"]
        if c["out"] == "e4m3":
            b += 4 * c["rows"] * -(-c["D"] // BLOCK)
        return {"bytes": b, "flops": 5 * n}
    if op == "quantize":
        n = c["rows"] * c["K"]
        return {"bytes": n * (SIZE[c["x"]] + 1) + 4 * c["rows"] * -(-c["K"] // BLOCK), "flops": 2 * n}
    if op == "weight":
        n = c["K"] * c["N"]
        return {"bytes": n * (SIZE[c["x"]] + 1) + 4 * -(-c["N"] // BLOCK) * -(-c["K"] // BLOCK), "flops": 2 * n}
    if op == "linear":
        M, K, N = c["M"], c["K"], c["N"]
        kb, nb = -(-K // BLOCK), -(-N // BLOCK)
        b = M * K + N * K + 4 * kb * (M + nb) + M * N * (SIZE[c["out"]] + SIZE[c["residual"]])
        if c["out"] == "e4m3":
            b += 4 * M * nb
        return {"bytes": b + (2 * N if c["bias"] else 0), "flops": 2 * M * N * K}
    keys, e = sum(_lens(c)), SIZE[c["x"]]
    return {"bytes": e * c["dh"] * (2 * keys * c["Hkv"] + 2 * c["B"] * c["Tq"] * c["H"]) + 4 * c["B"],
            "flops": 4 * c["dh"] * c["H"] * c["Tq"] * keys}


# ------------------------------------------------------------------------------- inputs
def _inputs(c, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device=DEVICE) * std

    def channels(n):  # activations: a few channels stand out, as they do behind an attention or feed-forward block
        return torch.exp(0.5 * torch.randn(n, generator=g, device=DEVICE))

    return g, normal, channels


def prepare(c, seed):
    g, normal, channels = _inputs(c, seed)
    op = c["op"]
    s = {"c": c}
    if op == "norm":
        s["x"] = (normal(c["rows"], c["D"]) * channels(c["D"])).to(TYPES[c["x"]])
        s["residual"] = (normal(c["rows"], c["D"]) * channels(c["D"])).to(TYPES[c["residual"]]) if c["residual"] else None
        s["gamma"] = (1 + normal(c["D"], std=0.1)).to(TYPES[c["x"]])
    elif op == "quantize":
        s["x"] = (normal(c["rows"], c["K"]) * channels(c["K"])).to(TYPES[c["x"]])
    elif op == "weight":
        s["w"] = normal(c["K"], c["N"], std=c["K"] ** -0.5).to(TYPES[c["x"]])
    elif op == "linear":
        s["a"], s["a_scales"] = _quantize_rows(normal(c["M"], c["K"]) * channels(c["K"]))
        s["w"], s["w_scales"] = _quantize_blocks(normal(c["N"], c["K"], std=c["K"] ** -0.5))
        s["bias"] = normal(c["N"], std=0.1).to(torch.bfloat16) if c["bias"] else None
        s["residual"] = normal(c["M"], c["N"]).to(TYPES[c["residual"]]) if c["residual"] else None
    else:
        dt = TYPES[c["x"]]
        s["q"] = normal(c["B"], c["Tq"], c["H"], c["dh"]).to(dt)
        # keys and values as one projection of the encoder's states leaves them, side by side
        kv = normal(c["B"], c["Tk"], 2, c["Hkv"], c["dh"]).to(dt)
        s["k"], s["v"] = kv[:, :, 0], kv[:, :, 1]
        lens = torch.tensor(_lens(c), dtype=torch.int32, device=DEVICE)
        s["lens"] = lens[torch.randperm(c["B"], generator=g, device=DEVICE)].contiguous() if c["ragged"] else None
    return s


# --------------------------------------------------------------------------- plain forms
def _blocks(y):
    """y (rows, n) cut into blocks of 128 columns, the last one filled up with zeros: (rows, blocks, 128)."""
    y = torch.nn.functional.pad(y, (0, -y.shape[1] % BLOCK))
    return y.view(y.shape[0], -1, BLOCK)


def _quantize_rows(y):
    b = _blocks(y)
    scales = (b.abs().amax(2) / E4M3_MAX).clamp_min(TINY)
    q = (b / scales[:, :, None]).reshape(y.shape[0], -1)[:, : y.shape[1]]
    return q.to(torch.float8_e4m3fn).contiguous(), scales


def _quantize_blocks(w):
    """w (N, K) with one scale for each 128 x 128 block."""
    N, K = w.shape
    t = torch.nn.functional.pad(w, (0, -K % BLOCK, 0, -N % BLOCK))
    t = t.view(t.shape[0] // BLOCK, BLOCK, -1, BLOCK)
    scales = (t.abs().amax((1, 3)) / E4M3_MAX).clamp_min(TINY)
    q = (t / scales[:, None, :, None]).reshape(t.shape[0] * BLOCK, -1)[:N, :K]
    return q.to(torch.float8_e4m3fn).contiguous(), scales


def _values(q, scales, rows_per_scale, dt):
    """The numbers that 8-bit values with scales stand for."""
    s = scales.to(dt)
    if rows_per_scale > 1:
        s = s.repeat_interleave(rows_per_scale, 0)[: q.shape[0]]
    return q.to(dt) * s.repeat_interleave(BLOCK, 1)[:, : q.shape[1]]


def _gelu(z):
    return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))


def run(s):
    if own:
        return _run_own(s)
    c = s["c"]
    op = c["op"]
    if op == "norm":
        t = s["x"].float()
        if s["residual"] is not None:
            t = t + s["residual"].float()
        y = t * torch.rsqrt(t.square().mean(1, keepdim=True) + EPS) * s["gamma"].float()
        got = list(_quantize_rows(y)) if c["out"] == "e4m3" else [y.to(TYPES[c["out"]])]
        return got + ([t.to(s["residual"].dtype)] if s["residual"] is not None else [])
    if op == "quantize":
        return list(_quantize_rows(s["x"].float()))
    if op == "weight":
        return list(_quantize_blocks(s["w"].float().t()))
    if op == "linear":
        z = _values(s["a"], s["a_scales"], 1, torch.float32) @ _values(s["w"], s["w_scales"], BLOCK, torch.float32).t()
        if s["bias"] is not None:
            z = z + s["bias"].float()
        if c["epilogue"] == "gelu":
            z = _gelu(z)
        elif c["epilogue"] == "residual":
            z = s["residual"].float() + z
        return list(_quantize_rows(z)) if c["out"] == "e4m3" else [z.to(TYPES[c["out"]])]
    o = _attend(s, torch.float32)
    return [o.to(s["q"].dtype)]


def _attend(s, dt):
    c = s["c"]
    B, Tq, Tk, H, Hkv, dh = (c[n] for n in ("B", "Tq", "Tk", "H", "Hkv", "dh"))
    q = s["q"].to(dt).view(B, Tq, Hkv, H // Hkv, dh).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, dh)
    k, v = s["k"].to(dt).permute(0, 2, 3, 1), s["v"].to(dt).permute(0, 2, 1, 3)
    x = (q @ k) * dh ** -0.5
    if s["lens"] is not None:
        gone = torch.arange(Tk, device=x.device) >= s["lens"][:, None, None, None]
        x = x.masked_fill(gone, -math.inf)
        m = x.amax(3, keepdim=True).clamp_min(torch.finfo(dt).min)
    else:
        m = x.amax(3, keepdim=True)
    p = torch.exp(x - m)
    o = (p @ v) / p.sum(3, keepdim=True).clamp_min(TINY)
    return o.view(B, Hkv, H // Hkv, Tq, dh).permute(0, 3, 1, 2, 4).reshape(B, Tq, H, dh)


# ----------------------------------------------------------------------------- own calls
def _run_own(s):
    from vision_transformer_encoder_gb300 import api

    c = s["c"]
    op = c["op"]
    if op == "norm":
        r = api.rmsnorm(s["x"], EPS, gamma=s["gamma"], residual=s["residual"], out_dtype=TYPES[c["out"]])
        return list(r) if isinstance(r, tuple) else [r]
    if op == "quantize":
        return list(api.quantize(s["x"]))
    if op == "weight":
        return list(api.quantize_weight(s["w"]))
    if op == "linear":
        epilogue = {"store": api.EPI_STORE, "gelu": api.EPI_GELU, "residual": api.EPI_RESIDUAL}[c["epilogue"]]
        r = api.linear_fp8(s["a"], s["a_scales"], s["w"], s["w_scales"], bias=s["bias"], residual=s["residual"],
                           epilogue=epilogue, out_dtype=TYPES[c["out"]])
        return list(r) if isinstance(r, tuple) else [r]
    return [api.cross_attention(s["q"], s["k"], s["v"], kv_lens=s["lens"])]


# -------------------------------------------------------------------------- 64-bit values
def _e4m3_64(y, scales):
    """y / scales on the grid of e4m3 (three bits behind the point, smallest step 2^-9), ties to even."""
    v = y / scales
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _rows_64(y):
    n = y.shape[1]
    blocks = torch.arange(n, device=y.device) // BLOCK
    top = torch.zeros(y.shape[0], -(-n // BLOCK), dtype=y.dtype, device=y.device)
    top = top.scatter_reduce(1, blocks.expand_as(y), y.abs(), "amax")
    scales = torch.clamp(top / E4M3_MAX, min=TINY)
    return [_e4m3_64(y, scales[:, blocks]), scales]


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    if op == "norm":
        t = s["x"].double() + (s["residual"].double() if c["residual"] else 0)
        y = t / torch.sqrt((t * t).sum(1) / c["D"] + EPS)[:, None] * s["gamma"].double()
        return (_rows_64(y) if c["out"] == "e4m3" else [y]) + ([t] if c["residual"] else [])
    if op == "quantize":
        return _rows_64(s["x"].double())
    if op == "weight":
        w = s["w"].double().t()
        scales = torch.stack([torch.stack([b.abs().max() for b in r.split(BLOCK, 1)]) for r in w.split(BLOCK, 0)])
        scales = torch.clamp(scales / E4M3_MAX, min=TINY)
        n, k = (torch.arange(m, device=w.device) // BLOCK for m in w.shape)
        return [_e4m3_64(w, scales[n][:, k]), scales]
    if op == "linear":
        a, w = s["a"].double(), s["w"].double()
        z = torch.zeros(c["M"], c["N"], dtype=torch.float64, device=a.device)
        n = torch.arange(c["N"], device=a.device) // BLOCK
        for b in range(-(-c["K"] // BLOCK)):
            at = slice(b * BLOCK, (b + 1) * BLOCK)
            z += (a[:, at] @ w[:, at].t()) * s["a_scales"][:, b, None].double() * s["w_scales"][n, b].double()
        if c["bias"]:
            z += s["bias"].double()
        if c["epilogue"] == "gelu":
            u = math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
            z = z * torch.sigmoid(2 * u)
        elif c["epilogue"] == "residual":
            z = z + s["residual"].double()
        return _rows_64(z) if c["out"] == "e4m3" else [z]
    o = torch.zeros(c["B"], c["Tq"], c["H"], c["dh"], dtype=torch.float64, device=s["q"].device)
    lens = s["lens"].tolist() if c["ragged"] else [c["Tk"]] * c["B"]
    for b, n in enumerate(lens):
        for h in range(c["H"] if n else 0):
            j = h // (c["H"] // c["Hkv"])
            x = s["q"][b, :, h].double() @ s["k"][b, :n, j].double().t() / math.sqrt(c["dh"])
            o[b, :, h] = torch.softmax(x, 1) @ s["v"][b, :n, j].double()
    return [o]
