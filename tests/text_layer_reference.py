"""The operations of a text layer besides rotation and attention, in 64 bits, and the 4-bit cache bit for
bit, from their formulas (CPU tensors)."""
from __future__ import annotations

import math

import numpy as np
import torch


def add_rms_norm(x, res, w, offset, eps):
    """(s, y) in float64 of bf16 matrices."""
    s = x.double() + (res.double() if res is not None else 0.0)
    y = s / torch.sqrt(s.pow(2).mean(-1, keepdim=True) + eps)
    return s, y * (offset + (w.double() if w is not None else 1.0))


def e4m3_steps(v):
    """Distance of neighbouring e4m3 numbers around v (float64): three bits, no binade below 2^-6."""
    return torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)


ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def activation(z, act):
    if act == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if act == "gelu":
        return z * torch.special.erfc(-z * math.sqrt(0.5)) / 2
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def linear_act(a, w, bias, act, res):
    """(out, size) in float64: size is the sum of the magnitudes that z is made of."""
    z = a.double() @ w.double().t()
    size = a.double().abs() @ w.double().abs().t()
    if bias is not None:
        z, size = z + bias.double(), size + bias.double().abs()
    y = activation(z, act)
    return (y if res is None else y + res.double()), size, z


def linear_act_tolerance(out, size, z, k, res, f32):
    """z is a sum of k + 1 products in fp32, each step off by at most 2^-23 of `size` (truncation); no activation is
    steeper than 1.13.  The activation itself: exponential, reciprocal and erf are each within 2^-20 of 1, its argument
    off by 2^-22 relative, which an exponential of up to 88 turns into 2^-15 of what is then at most
    |z| exp(-|z|)-small: 2^-20 |z| covers both.  Then one addition and one rounding."""
    tol = 1.13 * (k + 2) * 2.0 ** -23 * size + 2.0 ** -20 * z.abs() + 2.0 ** -23 * (out.abs() + (res.double().abs() if res is not None else 0.0))
    return tol + (0.0 if f32 else 2.0 ** -8 * out.abs()) + 1e-30


# ------------------------------------------------------------------------------- the 4-bit cache
def quantise(x):
    """(n int8 [..., d], scale bf16 [..., d / 32]) of bf16 values; n 0 and scale NaN where a value is not finite."""
    g = x.float().reshape(*x.shape[:-1], -1, 32)
    bad = ~g.isfinite().all(-1)
    m = torch.nan_to_num(g, nan=0.0, posinf=0.0, neginf=0.0).abs().amax(-1).clamp(min=7.0 * 2.0 ** -118)
    scale = (m / 7.0).to(torch.bfloat16)
    inv = 1.0 / scale.float()
    n = torch.round(torch.nan_to_num(g, nan=0.0, posinf=0.0, neginf=0.0) * inv[..., None]).clamp(-7, 7)
    n[bad] = 0
    scale[bad] = math.nan
    return n.to(torch.int8).reshape(x.shape), scale


def code_places(d, key):
    """Byte of its row and shift of each of the d values' codes."""
    out = []
    for i in range(d):
        j, u = divmod(i, 32)
        if key:
            out.append((((u // 8) * (d // 32) + j) * 4 + (u % 8) // 2, 4 * (u % 2)))
        else:
            out.append((((u // 4) * (d // 32) + j) * 2 + (u % 4) // 2, 4 * (u % 2)))
    return out


class Cache:
    """The cache's buffer as numpy bytes, written and read value by value."""

    def __init__(self, heads, d, pages, page_size, fill=0):
        self.heads, self.d, self.pages, self.page = heads, d, pages, page_size
        self.half = page_size * d * 9 // 16
        self.raw = np.full((pages, heads, 2 * self.half), fill, np.uint8)

    def put(self, page, slot, k, v):
        """Keys and values [heads, d] (bf16) of one token."""
        for key, x in ((True, k), (False, v)):
            n, scale = quantise(x)
            at = 0 if key else self.half
            row = np.zeros((self.heads, self.d // 2), np.uint8)
            for i, (byte, shift) in enumerate(code_places(self.d, key)):
                row[:, byte] |= ((n[:, i].numpy() + 8).astype(np.uint8) << shift).astype(np.uint8)
            g = self.d // 32
            bits = scale.view(torch.int16).numpy().astype(np.uint16)
            bits[scale.isnan().numpy()] = 0x7fff
            s = at + self.page * self.d // 2 + slot * g * 2
            self.raw[page, :, at + slot * self.d // 2:at + (slot + 1) * self.d // 2] = row
            self.raw[page, :, s:s + 2 * g] = bits.view(np.uint8).reshape(self.heads, 2 * g)

    def codes(self, pages, key):
        """(n int8 [len(pages) * page, heads, d], scale float64 [.., heads, d / 32])."""
        at, d, p = 0 if key else self.half, self.d, self.page
        raw = self.raw[np.asarray(pages, np.int64)]
        c = raw[..., at:at + p * d // 2].reshape(-1, self.heads, p, d // 2).transpose(0, 2, 1, 3).reshape(-1, self.heads, d // 2)
        places = code_places(d, key)
        n = np.stack([(c[..., b] >> s) & 15 for b, s in places], -1).astype(np.int8) - 8
        s = np.ascontiguousarray(raw[..., at + p * d // 2:at + self.half]).view(np.int16)
        s = s.reshape(-1, self.heads, p, d // 32).transpose(0, 2, 1, 3).reshape(-1, self.heads, d // 32)
        return torch.from_numpy(n), torch.from_numpy(np.ascontiguousarray(s)).view(torch.bfloat16).double()

    def values(self, pages, key):
        n, s = self.codes(pages, key)
        return n.double() * s.repeat_interleave(32, -1)


def cache_attention(q, spans, causal, scale, cache, table, left_out=()):
    """(out, tolerance, bad, owned) of q [rows, Hq, d] (bf16) over the cache, spans [(q0, nq, nk)], nothing that a row
    does not see taking part; `bad` where a visible value of V is not finite, or a visible key's scale.  Positions in
    `left_out` (sequence, position) take no part.  The tolerance is each value's own; with size = sum p |v|:

    - the probability times the value's scale is rounded to fp16 (2^-11 size), the output to bf16 (2^-8 |out|);
    - what of such a weight is subnormal in fp16 is off by 2^-25 where the largest of its row is 2^5 or more (2^6 when the
      reference is set, to the accuracy of a logarithm): n visible values of at most 7 steps, n 7 2^-30 of the row's largest
      weight W = max p s / l;
    - a group's 32 products q c (c up to 15) are summed in fp32 in at most 34 steps, each off by 2^-23 of sum |q| 15
      (truncation), and added, times the scale, to -8 sum(q) s, at most 8 steps at 23 sum |q| s: with B = scale * max over the
      visible keys of sum_g s_g sum |q_i|, and A the same of sum |q k|, and the exponent's two roundings at up to 2 A
      in units of log2: e = ((34 * 15 + 8 * 23) B + 12 A) 2^-23.  A query value below 2^-28 of its row's largest, Q, is off by
      2^-34 Q at most: B's share of that is d Q 2^-34 scale max s 15.  Scores off by e move p / l by at most exp(2 e) - 1;
    - codes are subnormal fp16 operands, whose products are lined up as if they were 2^-14: of each of a step's sixteen products
      2^-14 of the step's largest other operand may be cut off.  Scores: d / 16 steps of 16 * 2^-14 Q scale max s, into e.
      Output: 16 * 2^-14 of each step's largest weight, at most 2^-10 U;
    - sums over n visible keys of c f and of 8 f, up to 23 U with U = sum p s, and the exponential (2^-22) and rescales:
      (n + 128) 2^-23 of 23 U.

    The relative part is asserted to be under 5 %, so that no input makes the comparison empty."""
    Hq, d = q.shape[1], q.shape[2]
    Hk = cache.heads
    out = torch.zeros(q.shape, dtype=torch.float64)
    tol, bad, owned = torch.zeros_like(out), torch.zeros(q.shape, dtype=torch.bool), torch.zeros(q.shape[0], dtype=torch.bool)
    for si, (q0, nq, nk) in enumerate(spans):
        owned[q0:q0 + nq] = True
        if nq == 0 or nk == 0:
            continue
        pages = [p if 0 <= p < cache.pages else 0 for p in table[si][:-(-nk // cache.page)]]
        kn, ks = (t[:nk] for t in cache.codes(pages, True))
        vn, vs_all = (t[:nk] for t in cache.codes(pages, False))
        vv_all = vn.double() * vs_all.repeat_interleave(32, -1)
        i, j = torch.arange(nq)[:, None], torch.arange(nk)[None]
        seen = j <= i + (nk - nq) if causal else torch.ones(nq, nk, dtype=torch.bool)
        seen = seen.clone()
        for s, p in left_out:
            if s == si:
                seen[:, p] = False
        for h in range(Hk):
            heads = slice(h * Hq // Hk, (h + 1) * Hq // Hk)
            kbad = ~ks[:, h].isfinite().all(-1)
            sk = torch.nan_to_num(ks[:, h], nan=0.0, posinf=0.0, neginf=0.0)
            kk, vv = kn[:, h].double() * sk.repeat_interleave(32, -1), vv_all[:, h]
            vbad = ~vv.isfinite()
            vv = torch.where(vbad, torch.zeros_like(vv), vv)
            qq = q[q0:q0 + nq, heads].double().transpose(0, 1)
            s = (qq @ kk.t() * scale).masked_fill(~seen, -math.inf)
            A = (qq.abs() @ kk.abs().t() * scale).masked_fill(~seen, 0.0).amax(-1, keepdim=True)
            B = (qq.abs() @ sk.repeat_interleave(32, -1).t() * scale).masked_fill(~seen, 0.0).amax(-1, keepdim=True)
            m = s.amax(-1, keepdim=True)
            p = torch.where(seen, torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m)), torch.zeros_like(s))
            l = p.sum(-1, keepdim=True)
            p = torch.where(l > 0, p / l, torch.zeros_like(p))
            o, size = p @ vv, p @ vv.abs()
            sv = torch.nan_to_num(vs_all[:, h], nan=0.0, posinf=0.0, neginf=0.0)
            U, W = p @ sv.repeat_interleave(32, -1), (p * sv.amax(-1)).amax(-1, keepdim=True)
            e = ((34 * 15 + 8 * 23) * B + 12 * A) * 2.0 ** -23
            e = e + d * qq.abs().amax(-1, keepdim=True) * 2.0 ** -34 * scale * sk.max() * 15
            e = e + d / 16 * 2.0 ** -10 * qq.abs().amax(-1, keepdim=True) * scale * sk.max()
            n = seen.sum(-1)[None, :, None]
            rel = 2.0 ** -11 + torch.expm1(2 * e)
            assert float(rel.max()) < 0.05, float(rel.max())
            off = ((n + 128) * 2.0 ** -23 * 23 + 2.0 ** -10) * U + n * 7 * 2.0 ** -30 * W
            b = (seen.double() @ (vbad | kbad[:, None]).double() > 0)[None].expand_as(o)
            put = lambda x: x.transpose(0, 1)  # noqa: E731
            out[q0:q0 + nq, heads] = put(torch.where(b, torch.zeros_like(o), o))
            tol[q0:q0 + nq, heads] = put(torch.where(b, torch.zeros_like(o), rel * size + off + 2.0 ** -8 * o.abs() + 1e-30))
            bad[q0:q0 + nq, heads] = put(b)
    return out, tol, bad, owned
