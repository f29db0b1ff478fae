"""More of the text-side operators: what a layer of a text encoder, or of a decoder that rewrites its
prompts, runs between the ones of operators.py.

  norm    the residual's addition and the RMSNorm behind it, to bf16 or to e4m3 with a scale per 128
          values of a row
  linear  a bf16 product with bias, activation and residual in its epilogue
  cache   new keys and values appended to a paged 4-bit cache, and the whole sequences read back in
          bf16 (what the next chunk of a long prompt attends to)
  attn4   attention of new tokens over the 4-bit cache
"""
import math
import random

import torch

own = False

DEV = "cuda"
ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
EPS = 1e-6


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of a batch of seven: the smallest call, latency counts
        {"name": "norm_7", "op": "norm", "rows": 7, "cols": 2560, "res": True, "out": "e4m3", "offset": 0.0},
        # a batch of prompts, rows and columns off every power of two, gains stored as w - 1
        {"name": "norm_1777_ragged", "op": "norm", "rows": 1777, "cols": 2576, "res": True, "out": "bf16", "offset": 1.0},
        # the widest hidden state over many prompts, both outputs
        {"name": "norm_16384", "op": "norm", "rows": 16384, "cols": 4096, "res": True, "out": "both", "offset": 0.0},
        # the attention's output projection of one new token, added to the residual
        {"name": "linear_1", "op": "linear", "m": 1, "n": 2560, "k": 4096, "act": "none", "bias": False, "res": True, "f32": False},
        # scores over an odd number of classes for 33 rows, kept in 32 bits
        {"name": "linear_33_odd", "op": "linear", "m": 33, "n": 10007, "k": 2568, "act": "none", "bias": True, "res": False,
         "f32": True},
        # an encoder's second MLP product over a few prompts, ragged in all three sizes
        {"name": "linear_777_ragged", "op": "linear", "m": 777, "n": 1544, "k": 5160, "act": "gelu_tanh", "bias": True, "res": True,
         "f32": False},
        # an encoder's first MLP product over a batch of prompts
        {"name": "linear_8192", "op": "linear", "m": 8192, "n": 12288, "k": 4096, "act": "gelu", "bias": True, "res": False,
         "f32": False},
        # one decoding step of a batch of eight short chats, in small pages
        {"name": "cache_8_short", "op": "cache", "seqs": 8, "new": 1, "lo": 20, "hi": 300, "hk": 8, "d": 128, "page": 16, "lens": 1},
        # the next 512 tokens of sixteen long prompts
        {"name": "cache_16_long", "op": "cache", "seqs": 16, "new": 512, "lo": 700, "hi": 8192, "hk": 8, "d": 128, "page": 64,
         "lens": 2},
        # one new token over one chat of a thousand
        {"name": "attn4_1", "op": "attn4", "seqs": 1, "new": 1, "lo": 1000, "hi": 1000, "hq": 32, "hk": 8, "d": 128, "page": 64,
         "lens": 3},
        # five new tokens each (a draft to be checked) of nine sequences, heads of 64, small pages
        {"name": "attn4_draft_64", "op": "attn4", "seqs": 9, "new": 5, "lo": 333, "hi": 5001, "hq": 24, "hk": 8, "d": 64,
         "page": 16, "lens": 4},
        # one new token for each of 48 sequences over caches of 100 to 32768 tokens
        {"name": "attn4_48", "op": "attn4", "seqs": 48, "new": 1, "lo": 100, "hi": 32768, "hq": 32, "hk": 8, "d": 128, "page": 64,
         "lens": 7},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "cache", "attn4", "attn4"])
    if op == "norm":
        while True:
            c = {"op": op, "rows": _log_int(rng, 1, 16384), "cols": 16 * _log_int(rng, 16, 1024), "res": rng.random() < 0.8,
                 "out": rng.choice(["bf16", "e4m3", "both"]), "offset": rng.choice([0.0, 0.0, 1.0])}
            if c["rows"] * c["cols"] <= 16384 * 4096:
                return c
    if op == "linear":
        while True:
            c = {"op": op, "m": _log_int(rng, 1, 8192), "n": _log_int(rng, 128, 12288), "k": 8 * _log_int(rng, 16, 1280),
                 "act": rng.choice(ACTS), "bias": rng.random() < 0.7, "res": rng.random() < 0.5, "f32": rng.random() < 0.15}
            if c["m"] * c["n"] * c["k"] <= 8192 * 12288 * 4096:
                return c
    while True:
        hi = _log_int(rng, 2, 32768)
        c = {"op": op, "seqs": _log_int(rng, 1, 64), "new": rng.choice([1, 1, 1, 2, 3, 4, 5, 8, _log_int(rng, 1, 600)]),
             "lo": rng.randint(max(1, hi // 20), hi), "hi": hi, "hk": rng.randint(1, 8), "d": rng.choice([64, 128]),
             "page": rng.choice([16, 32, 64, 128, 256]), "lens": rng.randint(0, 10**6)}
        total = sum(_lengths(c)) * c["hk"] * c["d"]
        if op == "cache" and total <= 70000 * 8 * 128:
            return c
        c["hq"] = c["hk"] * rng.choice([1, 2, 3, 4, 5, 8, 12])
        if c["new"] <= 64 and total <= 700000 * 8 * 128 and c["seqs"] * hi * c["hq"] * c["new"] <= 1 << 29 and \
                c["seqs"] * hi * c["hk"] * c["d"] <= 48 * 32768 * 8 * 128:
            return c


def _lengths(c):
    """Tokens of each sequence, the new ones among them."""
    r = random.Random(c["lens"])
    n = [r.randint(c["lo"], c["hi"]) for _ in range(c["seqs"])]
    n[r.randrange(len(n))] = c["hi"]
    return n


def _news(c):
    return [min(c["new"], n) for n in _lengths(c)]


# ------------------------------------------------------------------------------- the 4-bit cache
# A page of one head holds, for `page` tokens: codes of the keys, their scales, codes of the values, their
# scales.  32 neighbouring values of a token share a bf16 scale; a code is value / scale + 8, 1 to 15.  A
# row of key codes is 32-bit words of 8 values, word t * (d / 32) + j holding values 32 j + 8 t onwards; a
# row of value codes is 16-bit words of 4, word g * (d / 32) + j holding values 32 j + 4 g onwards.
def _quantise(x):
    """Codes [..., d / 32, 32] and scales [..., d / 32] of bf16 values [..., d]."""
    x = x.float().unflatten(-1, (-1, 32))
    scale = (x.abs().amax(-1).clamp(min=7.0 * 2.0 ** -118) / 7.0).to(torch.bfloat16)
    return (torch.round(x * (1.0 / scale.float())[..., None]).clamp(-7, 7) + 8).to(torch.uint8), scale


def _pack(code, key):
    """Bytes [..., d / 2] of codes [..., d / 32, 32]."""
    c = code.unflatten(-1, (4, 8) if key else (8, 4)).transpose(-3, -2).flatten(-3)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def _unpack(row, key):
    """Codes [..., d / 32, 32] of bytes [..., d / 2]."""
    c = torch.stack([row & 15, row >> 4], -1).flatten(-2)
    return c.unflatten(-1, (4, -1, 8) if key else (8, -1, 4)).transpose(-3, -2).flatten(-2)


def _parts(cache, page, d):
    """Views of the four parts of every (page, head): key codes and scales, value codes and scales."""
    c, s = page * d // 2, page * d // 16
    at = (0, c, c + s, 2 * c + s, 2 * c + 2 * s)
    raw = [cache[..., a:b] for a, b in zip(at, at[1:])]
    codes = lambda t: t.unflatten(-1, (page, d // 2))  # noqa: E731
    scales = lambda t: t.view(torch.bfloat16).unflatten(-1, (page, d // 32))  # noqa: E731
    return codes(raw[0]), scales(raw[1]), codes(raw[2]), scales(raw[3])


def _slab(c):
    return c["page"] * c["d"] * 9 // 8


# ------------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=DEV).mul_(std).to(dtype)

    op = case["op"]
    st = {"case": case}
    if op == "norm":
        rows, cols = case["rows"], case["cols"]
        # a sub-layer's output, and a residual stream with a few columns that have grown large
        st["x"] = normal(rows, cols, std=0.5)
        grown = 1 + 20 * (torch.rand(cols, generator=g, device=DEV) < 0.01).float()
        st["r"] = (torch.randn(rows, cols, generator=g, device=DEV) * grown).to(torch.bfloat16) if case["res"] else None
        st["w"] = normal(cols, std=0.1, dtype=torch.float32).add_(1 - case["offset"]).to(torch.bfloat16)
        st["sum"] = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV) if case["res"] else None
        st["y"] = torch.zeros(rows, cols, dtype=torch.bfloat16, device=DEV) if case["out"] != "e4m3" else None
        st["q"] = torch.zeros(rows, cols, dtype=torch.uint8, device=DEV) if case["out"] != "bf16" else None
        st["scale"] = torch.zeros(rows, -(-cols // 128), device=DEV) if case["out"] != "bf16" else None
        return st
    st["ws"] = torch.zeros(128 << 20, dtype=torch.uint8, device=DEV)
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        st["a"] = normal(m, k)
        st["w"] = normal(n, k, std=k ** -0.5)
        st["b"] = normal(n, std=0.5) if case["bias"] else None
        ld = -(-n // 8) * 8
        st["r"] = normal(m, ld) if case["res"] else None
        st["out"] = torch.zeros(m, ld, dtype=torch.float32 if case["f32"] else torch.bfloat16, device=DEV)
        return st
    hk, d, page, seqs = case["hk"], case["d"], case["page"], case["seqs"]
    kl, ql = _lengths(case), _news(case)
    need = [-(-n // page) for n in kl]
    pages, most = sum(need) + 3, max(need) + 1
    # the sequences' pages lie anywhere in the pool; entries behind a sequence's last page are not set
    order = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    held = torch.arange(most, device=DEV) < torch.tensor(need, device=DEV)[:, None]
    st["table"] = torch.full((seqs, most), -1, dtype=torch.int32, device=DEV)
    st["table"][held] = order[:sum(need)]
    # what earlier calls have left in the pool; keys have channels of their own size and mean
    size = torch.rand(hk, 1, d, generator=g, device=DEV) + 0.5
    mean = torch.randn(hk, 1, d, generator=g, device=DEV)
    cache = torch.zeros(pages, hk, _slab(case), dtype=torch.uint8, device=DEV)
    step = max(1, (64 << 20) // (hk * page * d))
    for at in range(0, pages, step):
        n = min(step, pages - at)
        parts = _parts(cache[at:at + n], page, d)
        for key in (True, False):
            x = torch.randn(n, hk, page, d, generator=g, device=DEV)
            code, scale = _quantise((x * size + mean if key else x).to(torch.bfloat16))
            parts[0 if key else 2].copy_(_pack(code, key))
            parts[1 if key else 3].copy_(scale)
    st["cache"] = cache
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    q0 = [0]
    for n in ql:
        q0.append(q0[-1] + n)
    st["qs"], st["ql"], st["kl"] = i32(q0), i32(ql), i32(kl)
    st["max_q"], st["max_k"] = max(ql), max(kl)
    if op == "cache":
        k0 = [0]
        for n in kl:
            k0.append(k0[-1] + n)
        st["ks"] = i32(k0)
        kv = normal(q0[-1], 2 * hk * d)  # keys and values as one projection writes them
        st["k"], st["v"] = kv[:, :hk * d], kv[:, hk * d:]
        st["k_out"] = torch.zeros(k0[-1], hk * d, dtype=torch.bfloat16, device=DEV)
        st["v_out"] = torch.zeros(k0[-1], hk * d, dtype=torch.bfloat16, device=DEV)
    else:
        st["q"] = normal(q0[-1], case["hq"] * d)
        st["out"] = torch.zeros(q0[-1], case["hq"] * d, dtype=torch.bfloat16, device=DEV)
    return st


# --------------------------------------------------------------------------- the plain forms
def _plain_norm(st):
    c = st["case"]
    s = st["x"].float()
    if c["res"]:
        s = s + st["r"].float()
    out = {"sum": s.to(torch.bfloat16)} if c["res"] else {}
    y = s * torch.rsqrt((s * s).mean(-1, keepdim=True) + EPS) * (st["w"].float() + c["offset"])
    if c["out"] != "e4m3":
        out["y"] = y.to(torch.bfloat16)
    if c["out"] != "bf16":
        rows, cols, nb = c["rows"], c["cols"], -(-c["cols"] // 128)
        t = torch.zeros(rows, nb * 128, device=DEV)
        t[:, :cols] = y
        t = t.view(rows, nb, 128)
        top = t.abs().amax(-1).clamp(min=448.0 * 2.0 ** -118)
        v = (t * (448.0 / top)[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        out["q"], out["scale"] = v.view(rows, nb * 128)[:, :cols].contiguous(), top / 448.0
    return out


def _plain_linear(st):
    c = st["case"]
    n = c["n"]
    y = torch.matmul(st["a"].float(), st["w"].float().t())
    if c["bias"]:
        y = y + st["b"].float()
    if c["act"] == "relu":
        y = y.clamp(min=0)
    elif c["act"] == "gelu":
        y = 0.5 * y * (1 + torch.erf(y * math.sqrt(0.5)))
    elif c["act"] == "gelu_tanh":
        y = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    elif c["act"] == "silu":
        y = y / (1 + torch.exp(-y))
    if c["res"]:
        y = y + st["r"][:, :n].float()
    return y if c["f32"] else y.to(torch.bfloat16)


def _places(st, lens, first):
    """Sequence, page and token within the page of `lens` tokens of each sequence from `first` on, packed."""
    c = st["case"]
    seq = torch.repeat_interleave(torch.arange(c["seqs"], device=DEV), lens)
    start = torch.cumsum(lens, 0) - lens
    pos = torch.arange(seq.shape[0], device=DEV) - start[seq] + first[seq]
    return st["table"][seq, pos // c["page"]].long(), pos % c["page"]


def _plain_cache(st):
    c = st["case"]
    hk, d = c["hk"], c["d"]
    kl, ql = st["kl"].long(), st["ql"].long()
    kc, ks, vc, vs = _parts(st["cache"], c["page"], d)
    page, slot = _places(st, ql, kl - ql)
    for x, code, scale, key in ((st["k"], kc, ks, True), (st["v"], vc, vs, False)):
        n, s = _quantise(x.reshape(-1, hk, d))
        code[page, :, slot] = _pack(n, key)
        scale[page, :, slot] = s
    page, slot = _places(st, kl, torch.zeros_like(kl))
    out = {}
    for name, code, scale, key in (("k", kc, ks, True), ("v", vc, vs, False)):
        n = _unpack(code[page, :, slot], key).float() - 8
        out[name] = (n * scale[page, :, slot].float()[..., None]).to(torch.bfloat16).flatten(1)
    return out


def _plain_attn4(st):
    c = st["case"]
    hk, d, g = c["hk"], c["d"], c["hq"] // c["hk"]
    kl, ql = st["kl"].long(), st["ql"].long()
    S, Lq, Lk = c["seqs"], st["max_q"], st["max_k"]
    i, j = torch.arange(Lq, device=DEV), torch.arange(Lk, device=DEV)
    at = torch.minimum(j, kl[:, None] - 1)  # the last key again past the end
    page, slot = st["table"].gather(1, at // c["page"]).long(), at % c["page"]
    kc, ks, vc, vs = _parts(st["cache"], c["page"], d)
    k = ((_unpack(kc[page, :, slot], True).float() - 8) * ks[page, :, slot].float()[..., None]).flatten(-2)  # [S, Lk, hk, d]
    qi = st["qs"][:-1, None].long() + torch.minimum(i, ql[:, None] - 1)
    q = st["q"][qi].float().view(S, Lq, hk, g, d).permute(0, 2, 3, 1, 4).reshape(S, hk, g * Lq, d)
    s = torch.matmul(q, k.permute(0, 2, 3, 1)).view(S, hk, g, Lq, Lk)
    del k
    s.mul_(1 / math.sqrt(d))
    seen = j <= (i + (kl - ql)[:, None])[:, :, None]  # the last query sees the last key
    s.masked_fill_(~seen[:, None, None], -math.inf)
    p = s.sub_(s.amax(-1, keepdim=True)).exp_()
    v = ((_unpack(vc[page, :, slot], False).float() - 8) * vs[page, :, slot].float()[..., None]).flatten(-2)
    o = torch.matmul(p.view(S, hk, g * Lq, Lk), v.permute(0, 2, 1, 3)) / p.sum(-1).view(S, hk, g * Lq, 1)
    o = o.view(S, hk, g, Lq, d).permute(0, 3, 1, 2, 4).reshape(S, Lq, hk * g * d).to(torch.bfloat16)
    return o[i < ql[:, None]]


# ------------------------------------------------------------------------------------- a pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": _own_norm, "linear": _own_linear, "cache": _own_cache, "attn4": _own_attn4}[op](state)
    return {"norm": _plain_norm, "linear": _plain_linear, "cache": _plain_cache, "attn4": _plain_attn4}[op](state)


def _own_norm(st):
    from diffusion_transformer_step_gb300 import dit
    c = st["case"]
    n = c["cols"]
    dit.dit_add_rms_norm(c["rows"], n, st["x"], n, st["r"], n, st["w"], c["offset"], EPS, st["sum"], n, st["y"], n, st["q"],
                         st["scale"])
    out = {"sum": st["sum"]} if c["res"] else {}
    if c["out"] != "e4m3":
        out["y"] = st["y"]
    if c["out"] != "bf16":
        out["q"], out["scale"] = st["q"].view(torch.float8_e4m3fn), st["scale"]
    return out


def _own_linear(st):
    from diffusion_transformer_step_gb300 import dit
    c = st["case"]
    m, n, k, out, r, ws = c["m"], c["n"], c["k"], st["out"], st["r"], st["ws"]
    ld = out.stride(0)
    dit.dit_linear_act(m, n, k, st["a"], k, st["w"], k, st["b"], ACTS.index(c["act"]), r, ld if c["res"] else 0, out, ld, c["f32"],
                       ws, ws.numel())
    return out[:, :n]


def _own_cache(st):
    from diffusion_transformer_step_gb300 import dit
    c = st["case"]
    k, v, ko, vo, ws = st["k"], st["v"], st["k_out"], st["v_out"], st["ws"]
    cache = dit.make_text_cache4(c["hk"], c["d"], st["cache"].shape[0], c["page"], st["table"].shape[1])
    dit.dit_text_cache4_append(cache, c["seqs"], k.shape[0], st["max_q"], st["qs"], st["ql"], st["kl"], st["table"], k, k.stride(0),
                               v, v.stride(0), st["cache"], ws, ws.numel())
    dit.dit_text_cache4_read(cache, c["seqs"], ko.shape[0], st["max_k"], st["ks"], st["kl"], st["table"], st["cache"], ko,
                             ko.stride(0), vo, vo.stride(0), ws, ws.numel())
    return {"k": ko, "v": vo}


def _own_attn4(st):
    from diffusion_transformer_step_gb300 import dit
    c = st["case"]
    q, out, ws = st["q"], st["out"], st["ws"]
    cache = dit.make_text_cache4(c["hk"], c["d"], st["cache"].shape[0], c["page"], st["table"].shape[1])
    a = dit.make_text_attn(c["seqs"], c["hq"], c["hk"], c["d"], q.shape[0], 0, st["max_q"], st["max_k"])
    dit.dit_text_cache4_attention(cache, a, st["qs"], st["ql"], st["kl"], st["table"], q, q.stride(0), st["cache"], out,
                                  out.stride(0), ws, ws.numel())
    return out


# ------------------------------------------------------------------------------ what it takes
def work(case):
    op = case["op"]
    if op == "norm":
        v, out = case["rows"] * case["cols"], {"bf16": 2.0, "e4m3": 1 + 4 / 128, "both": 3 + 4 / 128}[case["out"]]
        return {"bytes": int(v * (2 + (4 if case["res"] else 0) + out) + 2 * case["cols"]), "flops": 8 * v}
    if op == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": 2 * (m * k + n * k) + m * n * ((4 if case["f32"] else 2) + (2 if case["res"] else 0)) +
                (2 * n if case["bias"] else 0), "flops": 2 * m * n * k}
    kl, ql = _lengths(case), _news(case)
    row = 2 * case["hk"] * case["d"]  # values of a token, keys and values
    if op == "cache":  # new rows in and their codes out; the codes before them in, all rows out
        return {"bytes": int(sum(ql) * row * (2 + 0.5625) + (sum(kl) - sum(ql)) * row * 0.5625 + sum(kl) * row * 2),
                "flops": 4 * row * sum(ql) + 2 * row * sum(kl)}
    seen = sum(sum(i + 1 + b - a for i in range(a)) for a, b in zip(ql, kl))
    return {"bytes": int(sum(kl) * row * 0.5625 + 4 * case["hq"] * case["d"] * sum(ql)), "flops": 4 * case["d"] * case["hq"] * seen}


# ----------------------------------------------------------------------- the definition, 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        s = st["x"].double()
        if case["res"]:
            s = s + st["r"].double()
        y = s / torch.sqrt(s.pow(2).sum(-1, keepdim=True) / case["cols"] + EPS) * (st["w"].double() + case["offset"])
        out = {"sum": s} if case["res"] else {}
        if case["out"] != "e4m3":
            out["y"] = y
        if case["out"] != "bf16":
            scale = torch.stack([b.abs().amax(-1) for b in y.split(128, -1)], -1) / 448
            v = y / scale.repeat_interleave(128, 1)[:, :case["cols"]]
            # e4m3: three bits behind the point of a binade, no binade below 2^-6
            step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
            out["q"], out["scale"] = torch.round(v / step) * step, scale
        return out
    if op == "linear":
        n = case["n"]
        y = st["a"].double() @ st["w"].double().t()
        if case["bias"]:
            y += st["b"].double()
        if case["act"] == "relu":
            y = torch.where(y > 0, y, torch.zeros_like(y))
        elif case["act"] == "gelu":
            y = y * torch.special.erfc(-y / math.sqrt(2)) / 2
        elif case["act"] == "gelu_tanh":
            y = y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))
        elif case["act"] == "silu":
            y = y * torch.sigmoid(y)
        return y + st["r"][:, :n].double() if case["res"] else y
    hk, d, page = case["hk"], case["d"], case["page"]
    kl, ql = _lengths(case), _news(case)
    table = st["table"].tolist()
    # where value i of a row is: byte of the row, and how far its code is shifted
    i = torch.arange(d, device=DEV)
    j, u, groups = i // 32, i % 32, d // 32
    word = {True: (u // 8) * groups + j, False: (u // 4) * groups + j}
    byte = {True: word[True] * 4 + (u % 8) // 2, False: word[False] * 2 + (u % 4) // 2}

    def rows(s, key):
        """The values [tokens, heads, d] that a sequence's pages hold."""
        slab = st["cache"][torch.tensor(table[s][:-(-kl[s] // page)], device=DEV)]
        at = 0 if key else page * d * 9 // 16
        code = slab[..., at:at + page * d // 2].reshape(-1, hk, page, d // 2)[..., byte[key]].int()
        code = (code >> ((i % 2) * 4).int()) & 15
        sc = slab[..., at + page * d // 2:at + page * d * 9 // 16].contiguous().view(torch.bfloat16).reshape(-1, hk, page, groups)
        v = (code.double() - 8) * sc.double()[..., j]
        return v.transpose(1, 2).reshape(-1, hk, d)[:kl[s]]

    def rounded(x):
        """Rows as the cache holds them: a bf16 scale per 32, decided on numbers of 32 bits by definition."""
        x = x.reshape(-1, hk, d // 32, 32)
        s = (x.float().abs().amax(-1).clamp(min=7.0 * 2.0 ** -118) / 7).bfloat16()
        return (torch.round(x.float() * (1 / s.float())[..., None]).double() * s.double()[..., None]).reshape(-1, hk, d)

    if op == "cache":
        out = {}
        for name, key in (("k", True), ("v", False)):
            new, got, a = rounded(st[name]), [], 0
            for s in range(case["seqs"]):
                got += [rows(s, key)[:kl[s] - ql[s]], new[a:a + ql[s]]]
                a += ql[s]
            out[name] = torch.cat(got).flatten(1)
        return out
    got, a = [], 0
    for s in range(case["seqs"]):
        k, v, q = rows(s, True), rows(s, False), st["q"][a:a + ql[s]].double().view(ql[s], hk, -1, d)
        z = torch.einsum("qhgd,khd->hgqk", q, k) / math.sqrt(d)
        z = z + torch.full((ql[s], kl[s]), -math.inf, dtype=torch.float64, device=DEV).triu(kl[s] - ql[s] + 1)
        got.append(torch.einsum("hgqk,khd->qhgd", torch.softmax(z, -1), v).reshape(ql[s], -1))
        a += ql[s]
    return torch.cat(got)
