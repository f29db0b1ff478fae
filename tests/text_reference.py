"""The text-side operations in 64 bits, from their formulas, for the tests (CPU tensors in,
float64 out)."""
from __future__ import annotations

import math

import numpy as np
import torch


def rope_frequencies(rot, theta, scaling="none", factor=1.0, low=1.0, high=4.0, original_len=1):
    j = np.arange(rot // 2, dtype=np.float64)
    if scaling == "ntk":
        theta = theta * factor ** (rot / (rot - 2))
    w = np.asarray(theta, np.float64) ** (-2 * j / rot)
    if scaling == "linear":
        w = w / factor
    if scaling == "by_parts":
        t = w * original_len / (2 * math.pi)
        g = np.clip((t - low) / (high - low), 0, 1)
        w = g * w + (1 - g) * w / factor
    return w


def rope_table(pos, magnitude=1.0, **kw):
    a = np.asarray(pos, np.float64)[:, None] * rope_frequencies(**kw)
    return np.stack([np.cos(a), np.sin(a)], -1) * magnitude


def qk_norm_rope(x, w, eps, table, rot, layout):
    """x [rows, heads, d] -> (y, |a| + |b| of each value's pair) in float64; table [rows, rot/2, 2]."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt(x.pow(2).mean(-1, keepdim=True) + eps) * w.double()
    y, size = x.clone(), x.abs()
    j = torch.arange(rot // 2)
    lo, hi = (2 * j, 2 * j + 1) if layout == "interleaved" else (j, j + rot // 2)
    if rot:
        c, s = table[:, None, :, 0].double(), table[:, None, :, 1].double()
        a, b = x[..., lo], x[..., hi]
        y[..., lo], y[..., hi] = a * c - b * s, b * c + a * s
        size = size.clone()
        size[..., lo] = (a * c).abs() + (b * s).abs()
        size[..., hi] = (b * c).abs() + (a * s).abs()
    return y, size


def attention(q, k, v, spans, causal, scale):
    """q [rows_q, Hq, d], k and v [rows_k, Hk, d] (any dtype), spans [(q0, nq, k0, nk)].
    Returns (out, sum of p |v|, largest score error bound): float64 of q's shape, zero where no
    sequence is or no key is visible, and a mask of the rows that belong to sequences.  Only
    visible keys and values are ever touched."""
    Hq, Hk, d = q.shape[1], k.shape[1], q.shape[2]
    g = Hq // Hk
    out = torch.zeros(q.shape, dtype=torch.float64)
    size = torch.zeros_like(out)
    owned = torch.zeros(q.shape[0], dtype=torch.bool)
    for q0, nq, k0, nk in spans:
        owned[q0:q0 + nq] = True
        if nq == 0 or nk == 0:
            continue
        qq = q[q0:q0 + nq].double().transpose(0, 1)                     # [Hq, nq, d]
        kk = k[k0:k0 + nk].double().transpose(0, 1).repeat_interleave(g, 0)
        vv = v[k0:k0 + nk].double().transpose(0, 1).repeat_interleave(g, 0)
        s = (qq @ kk.transpose(1, 2)) * scale
        seen = torch.ones(nq, nk, dtype=torch.bool)
        if causal:
            seen = torch.arange(nk)[None] <= torch.arange(nq)[:, None] + (nk - nq)
        s = s.masked_fill(~seen, -math.inf)
        m = s.amax(-1, keepdim=True)
        p = torch.where(seen, torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m)), torch.zeros_like(s))
        l = p.sum(-1, keepdim=True)
        p = torch.where(l > 0, p / l, torch.zeros_like(p))
        out[q0:q0 + nq] = (p @ vv).transpose(0, 1)
        size[q0:q0 + nq] = (p @ vv.abs()).transpose(0, 1)
    return out, size, owned


def attention_tolerance(out, size, q, k, scale):
    """How far a bf16 output may be.  The probabilities are rounded to bf16 (2^-8 of sum p |v|),
    the output once more (2^-8 |o|); a score is a sum of d products in fp32, off by at most
    d 2^-24 sum |q_i k_i| scale <= d 2^-24 |q| |k| scale =: e, twice (score and statistics),
    which moves a probability by 2 e relative, the exponential and the sums of thousands of
    fp32 terms add under 2^-12 of sum p |v| together."""
    qn = q.double().norm(dim=-1).max()
    kn = k.double().norm(dim=-1).max() if k.numel() else torch.zeros(())
    e = float(q.shape[-1] * 2.0 ** -24 * qn * kn * scale)
    return 2.0 ** -8 * (size + out.abs()) + (2 * e + 2.0 ** -12) * size + 1e-30


def quantize_blocks(x, block_rows):
    """(codes uint8, scales fp32) of a bf16 matrix: the definition in fp32, bit for bit."""
    x = x.float()
    rows, cols = x.shape
    rb, cb = -(-rows // block_rows), -(-cols // 128)
    pad = torch.zeros(rb * block_rows, cb * 128)
    pad[:rows, :cols] = x
    t = pad.view(rb, block_rows, cb, 128)
    m = torch.nan_to_num(t, nan=0.0, posinf=math.inf, neginf=-math.inf).abs().amax((1, 3))
    m = m.clamp(min=448.0 * 2.0 ** -118)
    inv = torch.full_like(m, 448.0) / m
    v = (t * inv[:, None, :, None]).reshape(rb * block_rows, cb * 128)[:rows, :cols]
    codes = v.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, m / torch.full_like(m, 448.0)


def dequantize(codes, scale, block_rows):
    rows, cols = codes.shape
    s = scale.double().repeat_interleave(block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
    return codes.view(torch.float8_e4m3fn).double() * s


def linear_blocks(a_q, a_scale, w_q, w_scale):
    """(out, sum of |a| |w|) in float64."""
    a, w = dequantize(a_q, a_scale, 1), dequantize(w_q, w_scale, 128)
    return a @ w.t(), a.abs() @ w.abs().t()


def attention_bound(q, k, v, spans, causal, scale, exact_scores=False):
    """As `attention`, but nothing that a row does not see takes part, in the values or in the tolerance,
    whatever it holds: (out, tolerance, bad, owned) with `bad` where a visible value of V is infinite or NaN
    (out and tolerance 0 there).  The tolerance is each value's own.  With size = sum p |v|:

    - the probabilities and the output are rounded to bf16: 2^-8 size, 2^-8 |out|;
    - a score is a sum of d exact products in fp32, each step off by at most 2^-23 (truncation) of
      A = scale * max over the visible keys of sum |q_i k_i|, and its exponent is rounded twice at up to 2 A
      in units of log2: e = (d + 4) 2^-23 A.  Scores off by e move p / l by at most exp(2 e) - 1.  With
      `exact_scores` (integers whose sums fp32 holds, which the caller sees to) only the exponent's roundings
      are left: a score times scale log2(e), half a step of 2^-24 relative, and the running maximum's share,
      e = 2 * 2^-24 A;
    - sums over n visible keys, the exponential (2^-22) and the running rescales: (n + 128) 2^-23 size.

    The relative part of the tolerance is asserted to be under 5 %, so that no input makes the comparison empty."""
    Hq, Hk, d = q.shape[1], k.shape[1], q.shape[2]
    out = torch.zeros(q.shape, dtype=torch.float64)
    tol, bad, owned = torch.zeros_like(out), torch.zeros(q.shape, dtype=torch.bool), torch.zeros(q.shape[0], dtype=torch.bool)
    for q0, nq, k0, nk in spans:
        owned[q0:q0 + nq] = True
        if nq == 0 or nk == 0:
            continue
        i, j = torch.arange(nq)[:, None], torch.arange(nk)[None]
        seen = j <= i + (nk - nq) if causal else torch.ones(nq, nk, dtype=torch.bool)
        used = seen.any(0)  # keys that some row sees
        for h in range(Hk):
            heads = slice(h * Hq // Hk, (h + 1) * Hq // Hk)
            kk, vv = k[k0:k0 + nk, h].double(), v[k0:k0 + nk, h].double()
            kk = torch.where(used[:, None], kk, torch.zeros_like(kk))
            vbad = ~vv.isfinite()
            vv = torch.where(vbad | ~used[:, None], torch.zeros_like(vv), vv)
            qq = q[q0:q0 + nq, heads].double().transpose(0, 1)  # [g, nq, d]
            s = (qq @ kk.t() * scale).masked_fill(~seen, -math.inf)
            a = (qq.abs() @ kk.abs().t() * abs(scale)).masked_fill(~seen, 0.0).amax(-1, keepdim=True)
            m = s.amax(-1, keepdim=True)
            p = torch.where(seen, torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m)), torch.zeros_like(s))
            l = p.sum(-1, keepdim=True)
            p = torch.where(l > 0, p / l, torch.zeros_like(p))
            o, size = p @ vv, p @ vv.abs()
            e = 2 * 2.0 ** -24 * a if exact_scores else (d + 4) * 2.0 ** -23 * a
            rel = 2.0 ** -8 + torch.expm1(2 * e) + (seen.sum(-1)[None, :, None] + 128) * 2.0 ** -23
            assert float(rel.max()) < 0.05, float(rel.max())
            b = (seen.double() @ vbad.double() > 0)[None].expand_as(o)
            put = lambda x: x.transpose(0, 1)  # noqa: E731
            out[q0:q0 + nq, heads] = put(torch.where(b, torch.zeros_like(o), o))
            tol[q0:q0 + nq, heads] = put(torch.where(b, torch.zeros_like(o), rel * size + 2.0 ** -8 * o.abs() + 1e-30))
            bad[q0:q0 + nq, heads] = put(b)
    return out, tol, bad, owned
