"""Long calls of the attention over the 4-bit cache with inputs that show every block of keys: runs cut by bounds and joined by a
second kernel or in a cluster, even shares, eight and sixteen rows per CTA, several tokens."""
import numpy as np
import pytest
import torch

import text_cache_visible as V
import text_layer_reference as R
from test_text_layer_gpu import DEV, Setup, _check_attention, _i32, _ok, _within, dit, ws  # noqa: F401

pytestmark = pytest.mark.gpu


def _wide(st, keys):
    """A table with room for `keys` tokens of each sequence: the bound of the call."""
    st.max_pages = max(st.max_pages, keys // st.ref.page)
    st.c = st.dit.make_text_cache4(st.ref.heads, st.ref.d, st.ref.pages, st.ref.page, st.max_pages)
    return st


def _run(dit, ws, st, hq, q_lens, q, max_k, causal=True, scale=None):
    d, rows = st.ref.d, sum(q_lens)
    out = torch.full((rows, hq * d), 9.0, dtype=torch.bfloat16, device=DEV)
    a = dit.make_text_attn(len(st.lens), hq, st.ref.heads, d, rows, 0, max(q_lens), max_k, causal=causal, scale=scale)
    assert dit.dit_text_cache4_attention_workspace(st.c, a) <= ws.numel()
    dit.dit_text_cache4_attention(st.c, a, _i32([0] + np.cumsum(q_lens).tolist()), None, _i32(st.lens), st.table_dev(), q, hq * d, st.dev, out,
                                  hq * d, ws, ws.numel())
    _ok(dit, ws)
    return out.view(rows, hq, d)


CASES = [
    # heads of queries and keys, page, new tokens, lengths, bound (0: the longest sequence)
    (4, 1, 64, [1, 1, 2], [20000, 40, 6666], 0),           # runs and a second kernel
    (4, 1, 16, [1, 1, 2], [9999, 40, 3333], 0),
    (4, 1, 256, [1, 1, 2], [33000, 40, 11000], 0),
    (2, 1, 64, [1], [4000], 0),                            # a cluster
    (12, 1, 64, [1], [3900], 0),
    (3, 1, 32, [17, 1], [5000, 100], 0),                   # several tiles of rows
    (4, 1, 64, [1], [30000], 1 << 19),                     # even shares of one sequence
    (12, 1, 64, [1, 1, 1], [9000, 127, 5000], 1 << 19),    # of sixteen rows
    (8, 4, 16, [1] * 5, [30000, 1, 129, 128, 9000], 1 << 17),
    (24, 8, 64, [5, 2], [5001, 4097], 1 << 16),
    (1, 1, 128, [3], [33000], 1 << 19)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk,page,q_lens,lens,bound", CASES)
def test_every_key_counts_once(dit, ws, d, hq, hk, page, q_lens, lens, bound):
    """All keys weigh the same: outputs are the weights of the dimensions' stretches of keys."""
    st = Setup(dit, hk, d, page, lens, seed=page)
    st.fill_random(page)
    V.write_uniform(st)
    st.upload()
    _wide(st, bound)
    q = torch.zeros(sum(q_lens), hq * d, dtype=torch.bfloat16, device=DEV)
    for causal in (True, False):
        want, tol = V.uniform_rows(lens, q_lens, d, hk, hq // hk, causal)
        _within(_run(dit, ws, st, hq, q_lens, q, max(bound, max(lens)), causal), want, tol)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group,page,lens,bound", [(1, 64, [20000, 9000, 700], 0), (3, 16, [9999, 3900, 33], 0), (12, 64, [9000, 5000, 129], 0),
                                                   (2, 64, [30000, 2500, 1], 1 << 17), (9, 256, [9000, 12000, 4097], 1 << 17)])
def test_a_needle_in_every_block(dit, ws, d, group, page, lens, bound):
    """A key that scores 14 d s q above all others, s = 1/4 and q = 1: d = 64 and a scale of 1/8 leave the others exp(-28), at
    most 2^-25 of the weight together. Then the output is that token's values: the weight, one, times the value's scale is rounded to fp16
    (2^-11), the output to bf16 (2^-8); a product of codes loses at most 2^-10 of the scale."""
    heads, hq = 4, 4 * group
    st = Setup(dit, heads, d, page, lens, seed=group)
    st.fill_random(page + d)
    r = st.ref
    r.raw[:, :, :page * d // 2] = 0x11  # keys of -7
    st.scales(True)[:] = 0x3e80         # 0.25
    st.upload()
    _wide(st, bound)
    dev = st.dev.view(r.pages, heads, 2 * r.half)
    q = torch.ones(len(lens), hq * d, dtype=torch.bfloat16, device=DEV)
    rng = np.random.default_rng(d + group)
    # a needle per block of 128 of the longest sequence, places within it drawn; first and last keys, and those at page borders
    places = [np.minimum(np.arange(0, n, 128) + rng.integers(0, 128, -(-n // 128)), n - 1) for n in lens]
    places = [np.concatenate([p, [0, n - 1, n - 1 - (n - 1) % page, max(n - 1 - n % 128, 0)]]) for p, n in zip(places, lens)]
    for turn in range(-(-max(map(len, places)) // heads)):
        spots, want, tol = [], [], []
        for s, n in enumerate(lens):
            for h in range(heads):
                p = int(places[s][(turn * heads + h) % len(places[s])])
                page_no, slot = st.table[s][p // page], p % page
                spots.append((page_no, h, slot))
                codes, scale = r.codes([page_no], False)
                scale = scale[slot, h].repeat_interleave(32)
                v = codes[slot, h].double() * scale
                want.append(v.expand(group, d))
                tol.append(((2.0 ** -8 + 2.0 ** -11 + 2.0 ** -20) * v.abs() + 2.0 ** -10 * scale + 2.0 ** -25 * 8).expand(group, d))
        for page_no, h, slot in spots:
            dev[page_no, h, slot * d // 2:(slot + 1) * d // 2] = 0xff  # +7
        out = _run(dit, ws, st, hq, [1] * len(lens), q, max(bound, max(lens)), scale=0.125)
        for page_no, h, slot in spots:
            dev[page_no, h, slot * d // 2:(slot + 1) * d // 2] = 0x11
        _within(out.view(len(lens), hq, d), torch.stack(want).view(len(lens), hq, d), torch.stack(tol).view(len(lens), hq, d))


def test_a_sequence_without_a_single_page_is_zeros(dit, ws):
    """Its query rows are written, as zeros, and the rows between sequences are not."""
    lens = [100, 40, 33]
    st = Setup(dit, 2, 64, 16, lens, seed=4)
    st.fill_random(12)
    table = st.table_dev()
    table[2, :] = -1
    out = _check_attention(dit, ws, st, 4, [2, 1, 1], left_out=[(2, p) for p in range(33)], table=table, status=0x802)
    assert (out[6] == 0).all() and (out[[1, 2, 4]] != 0).any(1).all() and (out[[0, 3, 5, 7]] == 9.0).all()
