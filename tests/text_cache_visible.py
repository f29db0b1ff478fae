"""Long calls of the attention over the 4-bit cache with inputs that show every block of keys, and what they must give.

With random values an output over n keys shrinks as 1 / sqrt(n) while a sum's bound grows with n: from some 9000 keys on a block
of 128 that is lost, or added twice, moves outputs by less than the bound. Two kinds of inputs do not have that:

- queries of zeros, so that all keys weigh the same, and values of 1 to 7 in one dimension and 0 in the others, a stretch of n / d
  tokens for each dimension: an output is its value times the weight of its stretch, of which sixteen tokens more or fewer are
  3 % at least up to 33000 keys;
- a needle, one key that the query meets with +7 where all others have -7: the output is that token's values."""
import numpy as np
import torch

def dims_of(n, d, head):
    """The dimension that each of n tokens' values have their number in, and the number."""
    stretch = np.arange(n) * d // max(n, 1)
    return (stretch + 5 * head) % d, 1 + (stretch + 3 * head) % 7


def uniform(n, d, head, weight=None):
    """The mean of n such values; `weight` says how often each token counts (a mask, or a slip)."""
    w = np.ones(n) if weight is None else weight
    dim, value = dims_of(n, d, head)
    return torch.from_numpy(np.bincount(dim, weights=value * w, minlength=d) / w.sum())


def uniform_tolerance(want):
    """All weights are equal, 2^6 to the accuracy of a logarithm and an exponential, which are the same for all keys: products with
    codes and their sums are exact in fp32. The sum of the weights is off by 2^-24 of it for each of the at most 2^12 additions
    that follow one another in a run and its join (a run has 4096 keys at most and 32 lanes share it; parts: fewer than
    400), the division and the join's factors by 2^-21, the fp16 weight by 2^-11, the output by half a step of bf16."""
    return (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -12 + 2.0 ** -20) * want.abs()


def write_uniform(st):
    """The values of a test's cache (reference bytes; upload them yourself)."""
    from text_layer_reference import code_places
    r = st.ref
    places = code_places(r.d, False)
    byte, shift = (np.array([p[i] for p in places]) for i in (0, 1))
    r.raw[:, :, r.half:r.half + r.page * r.d // 2] = 0x88
    st.scales(False)[:] = 0x3f80
    for s, n in enumerate(st.lens):
        pos = np.arange(n)
        page = np.array(st.table[s], np.int64)[pos // r.page] if n else pos
        for h in range(r.heads):
            dim, value = dims_of(n, r.d, h)
            r.raw[page, h, r.half + pos % r.page * (r.d // 2) + byte[dim]] = np.where(shift[dim] == 0, 0x88 + value, 0x88 + 16 * value)


def uniform_rows(lens, q_lens, d, heads, group, causal=True):
    """(want, tolerance) of the queries of all sequences, one after another, [rows, heads * group, d] in float64."""
    out = []
    for n, q in zip(lens, q_lens):
        for i in range(q):
            seen = n - q + 1 + i if causal else n
            w = (np.arange(n) < seen).astype(np.float64)
            rows = [uniform(n, d, h, w) if seen > 0 else torch.zeros(d, dtype=torch.float64) for h in range(heads)]
            out.append(torch.stack(rows).repeat_interleave(group, 0))
    want = torch.stack(out)
    return want, uniform_tolerance(want)
