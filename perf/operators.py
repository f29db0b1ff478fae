"""The text-side operators: what one pass through each computes, at the sizes that a text encoder
in front of the diffusion step (or a decoder that rewrites its prompts) runs them with.

  rope    table of rotary positions, plain or scaled for long contexts
  qk      per-head RMSNorm of queries and keys with the rotation in the same pass
  attn    attention with grouped heads over packed or padded sequences, causal or not, from whole
          prompts to single new tokens over a cache
  linear  activations quantised to e4m3 with a scale per 128 values of a row, times e4m3 weights
          with a scale per block of 128 x 128
"""
import math
import random

import torch

own = False

SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3}
DEV = "cuda"


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the table of one padded 512-row prompt, whole heads of 128
        {"name": "rope_512", "op": "rope", "n": 512, "rot": 128, "theta": 1e6, "scaling": "none", "start": 0},
        # the table of a long-context server: 128 Ki positions, a rotation stretched eight times
        {"name": "rope_128k_by_parts", "op": "rope", "n": 131072, "rot": 128, "theta": 5e5, "scaling": "by_parts",
         "start": 0},
        # one decoding step of a batch of seven: the smallest call, latency counts
        {"name": "qk_7_rows", "op": "qk", "rows": 7, "hq": 32, "hk": 8, "d": 128, "rot": 128, "layout": "half",
         "norm": True, "packed": True},
        # a batch of prompts, 10007 rows in all, a quarter of each 64-wide head left unrotated
        {"name": "qk_10007_rows_partial", "op": "qk", "rows": 10007, "hq": 32, "hk": 8, "d": 64, "rot": 48,
         "layout": "interleaved", "norm": True, "packed": True},
        # one 512-token prompt (the text rows of one image)
        {"name": "attn_prompt_512", "op": "attn", "kind": "prompt", "seqs": 1, "lo": 512, "hi": 512, "hq": 32, "hk": 8,
         "d": 128, "causal": True, "padded": False, "lens": 0},
        # eleven prompts of 17 to 1500 tokens packed into one buffer
        {"name": "attn_packed_11", "op": "attn", "kind": "prompt", "seqs": 11, "lo": 17, "hi": 1500, "hq": 32, "hk": 8,
         "d": 128, "causal": True, "padded": False, "lens": 3},
        # a bidirectional encoder with 64-wide heads over a padded batch
        {"name": "attn_encoder_64", "op": "attn", "kind": "prompt", "seqs": 16, "lo": 100, "hi": 512, "hq": 16, "hk": 16,
         "d": 64, "causal": False, "padded": True, "lens": 5},
        # one long document
        {"name": "attn_8192", "op": "attn", "kind": "prompt", "seqs": 1, "lo": 8192, "hi": 8192, "hq": 32, "hk": 8,
         "d": 128, "causal": True, "padded": False, "lens": 0},
        # one new token for each of 48 sequences over caches of 100 to 8192 tokens
        {"name": "attn_decode_48", "op": "attn", "kind": "decode", "seqs": 48, "lo": 100, "hi": 8192, "hq": 32, "hk": 8,
         "d": 128, "causal": True, "padded": True, "lens": 7},
        # a projection of one new token
        {"name": "linear_1", "op": "linear", "m": 1, "n": 4096, "k": 2560},
        # a ragged product: rows, columns and depth all off the tile sizes
        {"name": "linear_1777_ragged", "op": "linear", "m": 1777, "n": 2568, "k": 2064},
        # the widest projection over a batch of prompts
        {"name": "linear_8192", "op": "linear", "m": 8192, "n": 12288, "k": 4096},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "qk", "attn", "attn", "attn", "linear", "linear"])
    if op == "rope":
        return {"op": op, "n": _log_int(rng, 1, 131072), "rot": 2 * rng.randint(2, 64), "theta": rng.choice([1e4, 5e5, 1e6]),
                "scaling": rng.choice(list(SCALINGS)), "start": rng.choice([0, 0, rng.randint(1, 1000000)])}
    if op == "qk":
        d = rng.choice([64, 128])
        hk = rng.randint(1, 8)
        return {"op": op, "rows": _log_int(rng, 1, 10000), "hq": hk * rng.choice([1, 2, 3, 4]), "hk": hk, "d": d,
                "rot": rng.choice([d, d, 8 * rng.randint(1, d // 8)]), "layout": rng.choice(["half", "interleaved"]),
                "norm": rng.random() < 0.75, "packed": rng.random() < 0.75}
    if op == "linear":
        while True:
            c = {"op": op, "m": _log_int(rng, 1, 8192), "n": 8 * _log_int(rng, 16, 1536), "k": 16 * _log_int(rng, 8, 640)}
            if c["m"] * c["n"] * c["k"] <= 8192 * 12288 * 4096:
                return c
    while True:
        hk = rng.randint(1, 8)
        g = rng.choice([1, 2, 3, 4, 5, 8])
        kind = rng.choice(["prompt", "prompt", "decode", "tail"])
        hi = _log_int(rng, 1, 8192)
        c = {"op": op, "kind": kind, "seqs": _log_int(rng, 1, 64), "lo": rng.randint(max(1, hi // 20), hi), "hi": hi,
             "hq": hk * g, "hk": hk, "d": rng.choice([64, 128]), "causal": kind != "prompt" or rng.random() < 0.75,
             "padded": rng.random() < 0.5, "lens": rng.randint(0, 10**6)}
        ql, kl = _lengths(c)
        if c["seqs"] * c["hq"] * max(ql) * max(kl) <= 32 * 8192 * 8192 and c["seqs"] * max(kl) * c["hk"] * c["d"] <= 48 * 8192 * 8 * 128:
            return c


def _lengths(c):
    """Query and key lengths of the sequences: a whole prompt, one new token over a cache, or the
    last part of a prompt whose beginning is in the cache already."""
    r = random.Random(c["lens"])
    kl = [r.randint(c["lo"], c["hi"]) for _ in range(c["seqs"])]
    kl[r.randrange(len(kl))] = c["hi"]
    if c["kind"] == "prompt":
        return list(kl), kl
    if c["kind"] == "decode":
        return [1] * len(kl), kl
    return [r.randint(1, max(1, min(n, 300))) for n in kl], kl


def _spans(lens, padded):
    """Start row of each sequence and the rows of the whole buffer."""
    if padded:
        return [i * max(lens) for i in range(len(lens))], len(lens) * max(lens)
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at[:-1], at[-1]


# ------------------------------------------------------------------------------------ inputs
def _positions(n, packed, device):
    """Positions of `n` packed rows: sequences of 1, 2, 4, ... 512, 512, ... tokens, or one."""
    i = torch.arange(n, device=device)
    if not packed:
        return i.to(torch.int32)
    p = i + 1
    k = torch.floor(torch.log2(p.double())).long().clamp(max=9)
    return torch.where(p < 512, p - (1 << k), (p - 512) % 512).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=g, device=DEV).mul_(std).to(dtype)

    op = case["op"]
    st = {"case": case, "ws": torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)}
    if op == "rope":
        base = int(torch.randint(0, 1000, (1,), generator=g, device=DEV))
        st["pos"] = (torch.arange(case["n"], device=DEV) + case["start"] + base).to(torch.int32)
        st["table"] = torch.zeros(case["n"], case["rot"] // 2, 2, device=DEV)
    elif op == "qk":
        rows, hq, hk, d = case["rows"], case["hq"], case["hk"], case["d"]
        # queries, keys and values as one projection writes them
        st["qkv"] = normal(rows, (hq + 2 * hk) * d)
        st["wq"] = normal(d, std=0.1).add_(1) if case["norm"] else None
        st["wk"] = normal(d, std=0.1).add_(1) if case["norm"] else None
        st["pos"] = _positions(rows, case["packed"], DEV)
        n = int(st["pos"].max()) + 1
        ang = torch.arange(n, device=DEV).double()[:, None] * torch.pow(
            1e6, -torch.arange(case["rot"] // 2, device=DEV).double() * 2 / case["rot"])
        st["table"] = torch.stack([ang.cos(), ang.sin()], -1).float()
        st["q_out"] = torch.zeros(rows, hq * d, dtype=torch.bfloat16, device=DEV)
        st["k_out"] = torch.zeros(rows, hk * d, dtype=torch.bfloat16, device=DEV)
    elif op == "attn":
        hq, hk, d = case["hq"], case["hk"], case["d"]
        ql, kl = _lengths(case)
        qs, rq = _spans(ql, case["padded"])
        ks, rk = _spans(kl, case["padded"])
        if case["kind"] == "prompt":  # one fused buffer of queries, keys and values
            qkv = normal(rq, (hq + 2 * hk) * d)
            st["q"], st["k"], st["v"] = qkv[:, :hq * d], qkv[:, hq * d:(hq + hk) * d], qkv[:, (hq + hk) * d:]
        else:  # queries of their own, a cache of keys and one of values
            st["q"], st["k"], st["v"] = normal(rq, hq * d), normal(rk, hk * d), normal(rk, hk * d)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
        st["ql"], st["kl"], st["qs"], st["ks"] = i32(ql), i32(kl), i32(qs + [rq]), i32(ks + [rk])
        st["max_q"], st["max_k"] = max(ql), max(kl)
        st["out"] = torch.zeros(rq, hq * d, dtype=torch.bfloat16, device=DEV)
    else:
        m, n, k = case["m"], case["n"], case["k"]
        st["x"] = normal(m, k)
        nb, kb = -(-n // 128), -(-k // 128)
        w = normal(n, k, std=60.0, dtype=torch.float32).clamp_(-448, 448)
        st["wq"] = w.to(torch.float8_e4m3fn)
        # a weight of standard deviation near 0.02, with blocks of different sizes
        st["ws_"] = torch.rand(nb, kb, generator=g, device=DEV).mul_(0.5e-3).add_(1e-4)
        st["aq"] = torch.zeros(m, k, dtype=torch.uint8, device=DEV)
        st["as"] = torch.zeros(m, kb, device=DEV)
        st["out"] = torch.zeros(m, n, dtype=torch.bfloat16, device=DEV)
    return st


# --------------------------------------------------------------------------- the plain forms
def _frequencies(case):
    """Radians per position of each pair, in 64 bits."""
    rot, theta, f = case["rot"], case["theta"], _FACTOR
    j = torch.arange(rot // 2, device=DEV).double()
    if case["scaling"] == "ntk":
        theta = theta * f ** (rot / (rot - 2))
    w = torch.pow(theta, -2 * j / rot)
    if case["scaling"] == "linear":
        w = w / f
    if case["scaling"] == "by_parts":
        turns = w * _ORIGINAL / (2 * math.pi)
        keep = ((turns - _LOW) / (_HIGH - _LOW)).clamp(0, 1)
        w = w * keep + w / f * (1 - keep)
    return w


_FACTOR, _LOW, _HIGH, _ORIGINAL, _MAGNITUDE = 8.0, 1.0, 4.0, 16384, 1.2079441541679836


def _plain_rope(st):
    c = st["case"]
    a = st["pos"].double()[:, None] * _frequencies(c)
    m = _MAGNITUDE if c["scaling"] == "by_parts" else 1.0
    return torch.stack([a.cos() * m, a.sin() * m], -1).float()


def _plain_heads(x, w, cs, rot, layout):
    """RMSNorm over the last dimension (where there is a weight), then the rotation of its first
    `rot` values: pairs (2j, 2j + 1), or (j, j + rot/2)."""
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()
    r, rest = x[..., :rot], x[..., rot:]
    a, b = (r[..., 0::2], r[..., 1::2]) if layout == "interleaved" else (r[..., :rot // 2], r[..., rot // 2:])
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    u, v = a * c - b * s, b * c + a * s
    r = torch.stack([u, v], -1).flatten(-2) if layout == "interleaved" else torch.cat([u, v], -1)
    return torch.cat([r, rest], -1).to(torch.bfloat16).flatten(1)


def _plain_qk(st):
    c = st["case"]
    hq, hk, d = c["hq"], c["hk"], c["d"]
    x = st["qkv"].view(-1, hq + 2 * hk, d)
    cs = st["table"][st["pos"].long()]
    return {"q": _plain_heads(x[:, :hq], st["wq"], cs, c["rot"], c["layout"]),
            "k": _plain_heads(x[:, hq:hq + hk], st["wk"], cs, c["rot"], c["layout"])}


def _plain_attn(st):
    c = st["case"]
    hk, d, g = c["hk"], c["d"], c["hq"] // c["hk"]
    ql, kl = st["ql"].long(), st["kl"].long()
    i, j = torch.arange(st["max_q"], device=DEV), torch.arange(st["max_k"], device=DEV)
    qi = st["qs"][:-1, None].long() + torch.minimum(i, ql[:, None] - 1)  # [S, Lq], the last row again past the end
    ki = st["ks"][:-1, None].long() + torch.minimum(j, kl[:, None] - 1)
    S, Lq, Lk = len(ql), len(i), len(j)
    q = st["q"][qi].float().view(S, Lq, hk, g, d).permute(0, 2, 3, 1, 4).reshape(S, hk, g * Lq, d)
    k = st["k"][ki].float().view(S, Lk, hk, d).permute(0, 2, 3, 1)
    v = st["v"][ki].float().view(S, Lk, hk, d).permute(0, 2, 1, 3)
    s = torch.matmul(q, k).view(S, hk, g, Lq, Lk)
    s.mul_(1 / math.sqrt(d))
    seen = (j < kl[:, None])[:, None, :]
    if c["causal"]:  # the last query sees the last key
        seen = seen & (j <= (i + (kl - ql)[:, None])[:, :, None])
    s.masked_fill_(~seen[:, None, None], -math.inf)
    p = s.sub_(s.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(p.view(S, hk, g * Lq, Lk), v) / p.sum(-1).view(S, hk, g * Lq, 1)
    o = o.view(S, hk, g, Lq, d).permute(0, 3, 1, 2, 4).reshape(S, Lq, hk * g * d).to(torch.bfloat16)
    out = torch.zeros_like(st["out"])
    ok = i < ql[:, None]
    out[qi[ok]] = o[ok]
    return out


def _plain_linear(st):
    c = st["case"]
    m, n, k = c["m"], c["n"], c["k"]
    nb, kb = st["ws_"].shape
    x = torch.zeros(m, kb * 128, device=DEV)
    x[:, :k] = st["x"].float()
    x = x.view(m, kb, 128)
    top = x.abs().amax(-1)
    inv = torch.where(top > 0, torch.full_like(top, 448.0) / top, torch.zeros_like(top))
    code = (x * inv[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    a = (code.float() * (top / 448.0)[..., None]).view(m, kb * 128)[:, :k]
    scale = st["ws_"].repeat_interleave(128, 0)[:n].repeat_interleave(128, 1)[:, :k]
    w = st["wq"].float() * scale
    return torch.matmul(a, w.t()).to(torch.bfloat16)


# ------------------------------------------------------------------------------------- a pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "qk": _own_qk, "attn": _own_attn, "linear": _own_linear}[op](state)
    return {"rope": _plain_rope, "qk": _plain_qk, "attn": _plain_attn, "linear": _plain_linear}[op](state)


def _own_rope(st):
    from diffusion_transformer_step_gb300 import dit
    c = st["case"]
    parts = c["scaling"] == "by_parts"
    r = dit.make_text_rope(c["rot"], c["theta"], SCALINGS[c["scaling"]], factor=_FACTOR, low=_LOW, high=_HIGH,
                           original_len=_ORIGINAL, magnitude=_MAGNITUDE if parts else 1.0)
    dit.dit_text_rope_table(r, st["pos"], c["n"], st["table"])
    return st["table"]


def _own_qk(st):
    from diffusion_transformer_step_gb300 import dit
    c = st["case"]
    hq, hk, d = c["hq"], c["hk"], c["d"]
    x, ws = st["qkv"], st["ws"]
    dit.dit_qk_norm_rope(c["rows"], hq, hk, d, c["rot"], dit.DIT_ROPE_HALF if c["layout"] == "half" else dit.DIT_ROPE_INTERLEAVED,
                         x, x.stride(0), x[:, hq * d:], x.stride(0), st["wq"], st["wk"], 1e-6, st["table"],
                         st["table"].shape[0], st["pos"], st["q_out"], hq * d, st["k_out"], hk * d, ws, ws.numel())
    return {"q": st["q_out"], "k": st["k_out"]}


def _own_attn(st):
    from diffusion_transformer_step_gb300 import dit
    c = st["case"]
    q, k, v, out, ws = st["q"], st["k"], st["v"], st["out"], st["ws"]
    a = dit.make_text_attn(c["seqs"], c["hq"], c["hk"], c["d"], q.shape[0], k.shape[0], st["max_q"], st["max_k"],
                           causal=c["causal"], scale=1 / math.sqrt(c["d"]))
    dit.dit_text_attention(a, st["qs"], st["ql"], st["ks"], st["kl"], q, q.stride(0), k, k.stride(0), v, v.stride(0),
                           out, out.stride(0), ws, ws.numel())
    return out


def _own_linear(st):
    from diffusion_transformer_step_gb300 import dit
    c = st["case"]
    m, n, k, ws = c["m"], c["n"], c["k"], st["ws"]
    dit.dit_quantize_blocks_fp8(st["x"], k, m, k, 1, st["aq"], st["as"])
    dit.dit_linear_fp8_blocks(m, n, k, st["aq"], st["as"], st["wq"], st["ws_"], st["out"], n, ws, ws.numel())
    return st["out"]


# ------------------------------------------------------------------------------ what it takes
def work(case):
    op = case["op"]
    if op == "rope":  # positions in, cosine and sine out; about 40 operations for such a pair
        pairs = case["n"] * (case["rot"] // 2)
        return {"bytes": 4 * case["n"] + 8 * pairs, "flops": 40 * pairs}
    if op == "qk":
        v = case["rows"] * (case["hq"] + case["hk"]) * case["d"]
        top = min(case["rows"], 512 if case["packed"] else case["rows"])
        return {"bytes": 4 * v + 4 * case["rows"] + 4 * top * case["rot"], "flops": 8 * v}
    if op == "attn":
        ql, kl = _lengths(case)
        seen = sum(sum(max(0, i + 1 + b - a) for i in range(a)) if case["causal"] else a * b for a, b in zip(ql, kl))
        return {"bytes": 2 * case["d"] * (2 * case["hq"] * sum(ql) + 2 * case["hk"] * sum(kl)) + 8 * len(ql),
                "flops": 4 * case["d"] * case["hq"] * seen}
    m, n, k = case["m"], case["n"], case["k"]
    return {"bytes": 2 * m * k + n * k + 4 * (-(-n // 128)) * (-(-k // 128)) + 2 * m * n, "flops": 2 * m * n * k}


# ----------------------------------------------------------------------- the definition, 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        half = case["rot"] // 2
        rows = []
        for j in range(half):
            f = math.exp(-math.log(case["theta"]) * j / half)
            if case["scaling"] == "ntk":
                f = math.exp(-(math.log(case["theta"]) + math.log(_FACTOR) * half / (half - 1)) * j / half)
            elif case["scaling"] == "linear":
                f /= _FACTOR
            elif case["scaling"] == "by_parts":
                t = min(1.0, max(0.0, (f * _ORIGINAL / math.tau - _LOW) / (_HIGH - _LOW)))
                f = t * f + (1 - t) * f / _FACTOR
            rows.append(f)
        size = _MAGNITUDE if case["scaling"] == "by_parts" else 1.0
        z = torch.outer(st["pos"].double(), torch.tensor(rows, dtype=torch.float64, device=DEV))
        z = torch.polar(torch.full_like(z, size), z)
        return torch.view_as_real(z).contiguous()
    if op == "qk":
        hq, hk, d, rot = case["hq"], case["hk"], case["d"], case["rot"]
        x = st["qkv"].double().view(case["rows"], hq + 2 * hk, d)[:, :hq + hk]
        if case["norm"]:
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / d + 1e-6)
            x = x * torch.cat([st["wq"].double().expand(hq, d), st["wk"].double().expand(hk, d)])
        turn = torch.view_as_complex(st["table"].double()[st["pos"].long()])[:, None]
        j = torch.arange(rot // 2, device=DEV)
        lo, hi = (2 * j, 2 * j + 1) if case["layout"] == "interleaved" else (j, j + rot // 2)
        z = torch.complex(x[..., lo], x[..., hi]) * turn
        y = x.clone()
        y[..., lo], y[..., hi] = z.real, z.imag
        return {"q": y[:, :hq].reshape(case["rows"], -1), "k": y[:, hq:].reshape(case["rows"], -1)}
    if op == "attn":
        hq, hk, d = case["hq"], case["hk"], case["d"]
        ql, kl = _lengths(case)
        q0, rq = _spans(ql, case["padded"])
        k0, _ = _spans(kl, case["padded"])
        out = torch.zeros(rq, hq, d, dtype=torch.float64, device=DEV)
        for a, b, na, nb in zip(q0, k0, ql, kl):
            for h in range(hk):
                k = st["k"][b:b + nb, h * d:(h + 1) * d].double()
                v = st["v"][b:b + nb, h * d:(h + 1) * d].double()
                for r in range(0, na, 2048):  # the rows [r, e) of the sequence
                    e = min(na, r + 2048)
                    heads = slice(h * hq // hk * d, (h + 1) * hq // hk * d)
                    q = st["q"][a + r:a + e, heads].double().view(e - r, hq // hk, d).transpose(0, 1)
                    s = q @ k.t() / math.sqrt(d)
                    if case["causal"]:
                        s = s + torch.full((e - r, nb), -math.inf, dtype=torch.float64, device=DEV).triu(nb - na + r + 1)
                    out[a + r:a + e, h * hq // hk:(h + 1) * hq // hk] = (torch.softmax(s, -1) @ v).transpose(0, 1)
        return out.view(rq, hq * d)
    m, n, k = case["m"], case["n"], case["k"]
    a = torch.zeros(m, k, dtype=torch.float64, device=DEV)
    out = torch.zeros(m, n, dtype=torch.float64, device=DEV)
    w = torch.zeros(n, k, dtype=torch.float64, device=DEV)
    for b in range(0, k, 128):
        x = st["x"][:, b:b + 128].double()
        scale = x.abs().amax(1, keepdim=True) / 448
        # the codes are of x times 448 / max, factor and product numbers of 32 bits by definition:
        # they decide the ties
        v = (x * (1 / torch.where(scale > 0, scale, torch.ones_like(scale))).float().double()).float().double()
        # e4m3: three bits behind the point of a binade, no binade below 2^-6
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        a[:, b:b + 128] = torch.round(v / step) * step * scale
        w[:, b:b + 128] = st["wq"][:, b:b + 128].double() * st["ws_"][:, b // 128].double().repeat_interleave(128)[:n, None]
    torch.matmul(a, w.t(), out=out)
    return out
