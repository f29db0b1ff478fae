"""Attention over the 4-bit cache where all keys of a call are shared out evenly over the GPU: a CTA has pieces of
several sequences and heads, and a long one is joined from several CTAs.

The bound `max_k` chooses this, so the calls here state one of up to a million keys and a table that has room for
them; tolerances are those of the other tests of this attention."""
import numpy as np
import pytest
import torch

import text_layer_reference as R
from test_text_layer_gpu import DEV, Setup, _bits, _check_attention, _i32, _ok, _randn, _within, dit, ws  # noqa: F401

pytestmark = pytest.mark.gpu


def _setup(dit, heads, d, page, lens, seed, keys=1 << 19):
    """Tables of `keys` tokens, whatever the sequences have; heads * sequences * keys is enough for even shares."""
    assert heads * len(lens) * keys >= 512 * 456
    st = Setup(dit, heads, d, page, lens, seed=seed)
    st.max_pages = keys // page
    st.c = dit.make_text_cache4(heads, d, st.ref.pages, page, st.max_pages)
    st.fill_random(seed)
    st.keys = keys
    return st


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk,page,q_lens,lens,causal", [
    (4, 1, 64, [1], [30000], True),                                                    # one item over all CTAs
    (8, 2, 16, [1] * 5, [3000, 1, 0, 128, 129], True),                                  # whole pieces and cut ones
    (12, 1, 64, [1, 1, 1], [9000, 127, 5000], True),                                    # sixteen rows
    (6, 2, 32, [5, 0, 2, 1], [700, 300, 2500, 64], True),                               # several tokens, one without
    (3, 3, 128, [2, 1], [2049, 1300], False),
    (2, 1, 256, [1] * 40, [37 * i % 900 for i in range(40)], True),                     # sequences shorter than a share
    (2, 2, 16, [1] * 150, [i % 35 for i in range(150)], True),                          # more than are looked up at once
    (4, 4, 64, [1] * 3, [0, 0, 0], True)])
def test_even_shares(dit, ws, d, hq, hk, page, q_lens, lens, causal):
    st = _setup(dit, hk, d, page, lens, seed=hq)
    one = _check_attention(dit, ws, st, hq, q_lens, causal, pad=8, seed=page, max_k=st.keys)
    assert torch.equal(_bits(one), _bits(_check_attention(dit, ws, st, hq, q_lens, causal, pad=8, seed=page, max_k=st.keys)))


def test_even_shares_of_equal_sequences(dit, ws):
    """Shares that end with a sequence's head, one block before it or behind it, or inside what a piece costs."""
    for n in (128 * 6, 128 * 7, 128 * 9 + 1, 128 * 30):
        st = _setup(dit, 2, 128, 64, [n] * 20, seed=n, keys=1 << 14)
        _check_attention(dit, ws, st, 4, [1] * 20, seed=3, max_k=st.keys)


def test_even_shares_more_sequences_than_ctas(dit, ws):
    lens = [1 + (i * 7919) % 300 for i in range(700)]
    st = _setup(dit, 1, 64, 16, lens, seed=2, keys=1 << 13)
    _check_attention(dit, ws, st, 2, [1] * 700, gap=0, seed=3, max_k=st.keys)


def test_even_shares_bad_entries(dit, ws):
    """Sequences with lengths out of range are skipped, pages out of range left out, both are reported; the others have
    their results."""
    lens = [2000, 400, 33, 900]
    st = _setup(dit, 2, 64, 16, lens, seed=4)
    for bad in (-1, st.c.pages):
        table = st.table_dev()
        table[0, 20] = bad
        table[3, 0] = bad
        _check_attention(dit, ws, st, 4, [2, 1, 1, 1], left_out=[(0, p) for p in range(320, 336)] + [(3, p) for p in range(16)], table=table,
                         status=0x802, max_k=st.keys)
    q = _randn(5, 4 * 64, seed=1)
    qd = q.to(DEV)
    want, tol, _, _ = R.cache_attention(q.view(5, 4, 64), [(0, 2, 2000), (2, 1, 400), (3, 1, 33), (4, 1, 900)], True, 64 ** -0.5, st.ref,
                                        st.table)
    a = dit.make_text_attn(4, 4, 2, 64, 5, 0, 2, st.keys)
    rows = ([0, 1], [2], [3], [4])
    for q_off, q_len, k_len, skipped in (([0, 2, 3, 4], [3, 1, 1, 1], lens, 0), ([0, 2, 3, 4], [2, 1, 1, 1], [2000, -1, 33, 900], 1),
                                         ([0, 2, 3, 4], [2, 1, 1, 1], [2000, 400, 33, st.keys + 1], 3),
                                         ([0, -1, 3, 4], [2, 1, 1, 1], lens, 1), ([0, 2, 5, 4], [2, 1, 1, 1], lens, 2)):
        out = torch.full((5, 256), 9.0, dtype=torch.bfloat16, device=DEV)
        dit.dit_text_cache4_attention(st.c, a, _i32(q_off + [5]), _i32(q_len), _i32(k_len), st.table_dev(), qd, 256, st.dev, out, 256, ws,
                                      ws.numel())
        _ok(dit, ws, 0x801)
        for s in range(4):
            if s == skipped:
                assert (out[rows[s]] == 9.0).all()
            else:
                _within(out[rows[s]].view(-1, 4, 64), want[rows[s]], tol[rows[s]])
    # all of them
    out = torch.full((5, 256), 9.0, dtype=torch.bfloat16, device=DEV)
    dit.dit_text_cache4_attention(st.c, a, _i32([0, 2, 3, 4, 5]), _i32([-1] * 4), _i32(lens), st.table_dev(), qd, 256, st.dev, out, 256, ws,
                                  ws.numel())
    _ok(dit, ws, 0x801)
    assert (out == 9.0).all()


@pytest.mark.parametrize("d", [64, 128])
def test_even_shares_bad_values(dit, ws, d):
    """NaN scales behind the keys everywhere, and on single keys: a value reaches the rows that see it, no others."""
    lens = [1500, 200]
    for key in (True, False):
        for pos in (1499, 700, 0):
            st = _setup(dit, 2, d, 32, lens, seed=4)
            s = st.scales(key)
            s[st.table[0][pos // 32], 1, pos % 32, -1] = 0x7fff
            for which in (True, False):
                sc = st.scales(which)
                sc[st.table[0][1499 // 32], :, 1499 % 32 + 1:] = 0x7fff
                sc[st.table[1][199 // 32], :, 199 % 32 + 1:] = 0x7f80
            st.upload()
            _check_attention(dit, ws, st, 4, [3, 1], seed=pos, max_k=st.keys)


def test_even_shares_captured_and_replayed_over_other_lengths(dit, ws):
    """The shares follow the lengths on the device: a graph replayed over shorter, longer, empty and bad ones, beside a second
    graph on the same workspace."""
    full = [3000, 1000, 5000]
    st = _setup(dit, 2, 128, 64, full, seed=5)
    q = _randn(3, 8 * 128, seed=1)
    qd, out = q.to(DEV), torch.zeros(3, 8 * 128, dtype=torch.bfloat16, device=DEV)
    a, qo, kl, table = dit.make_text_attn(3, 8, 2, 128, 3, 0, 1, st.keys), _i32([0, 1, 2, 3]), _i32(full), st.table_dev()
    other = torch.zeros_like(out)
    run = lambda o: dit.dit_text_cache4_attention(st.c, a, qo, None, kl, table, qd, 1024, st.dev, o, 1024, ws, ws.numel(),  # noqa: E731
                                                  torch.cuda.current_stream())
    run(out)
    torch.cuda.synchronize()
    graphs = []
    for o in (out, other):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(o)
        graphs.append(g)
    for lens in (full, [1, 1000, 4999], [0, 0, 5000], [2999, 0, 128], full):
        kl.copy_(_i32(lens))
        for g in (graphs[0], graphs[1], graphs[0]):
            g.replay()
        _ok(dit, ws)
        want, tol, _, _ = R.cache_attention(q.view(3, 8, 128), [(i, 1, n) for i, n in enumerate(lens)], True, 128 ** -0.5, st.ref, st.table)
        _within(out.view(3, 8, 128), want, tol)
        assert torch.equal(_bits(out), _bits(other))


def test_even_shares_value_scales(dit, ws):
    """Scales of the values that rise and fall over the keys, so that the parts' references lie far apart."""
    for sign in (1, -1):
        st = _setup(dit, 1, 128, 64, [4000], seed=6)
        s = st.scales(False)
        for pos in range(4000):
            s[st.table[0][pos // 64], :, pos % 64] = torch.full((1,), 0.1 * 2.0 ** (sign * (pos / 40 - 50))).bfloat16().view(torch.int16).numpy()
        st.upload()
        _check_attention(dit, ws, st, 4, [1], seed=2, max_k=st.keys)
