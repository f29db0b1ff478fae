"""The norm with residual, the product with its epilogue and the 4-bit cache at the ends of their ranges: magnitudes,
offsets that pass 32 bits, streams other than the default one, graphs that share a workspace, long tables.

Against the same 64-bit forms, with the tolerances derived there."""
import math

import numpy as np
import pytest
import torch

import text_layer_reference as R
from test_text_layer_gpu import DEV, Setup, _bits, _check_attention, _i32, _ok, _randn, _within, _norm_tolerance, dit, ws  # noqa: F401

pytestmark = pytest.mark.gpu


def _set_exponents(st, key, exps):
    """Scales 2^e times what they are (0.05 to 0.4), e by [page, head, place, group]."""
    s = st.scales(key)
    v = torch.from_numpy(s.copy()).view(torch.bfloat16).double() * torch.exp2(torch.from_numpy(np.broadcast_to(exps, s.shape).astype(np.float64)))
    s[:] = v.bfloat16().view(torch.int16).numpy()
    st.upload()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", ["2^-60", "2^95", "mixed", "falling", "rising", "zero"])
def test_cache_attention_value_scales(dit, ws, d, kind):
    """Scales of the values over the range that is documented, the same for all or different for each: weights and
    references that follow the products of probability and scale, a sum of probabilities that does not."""
    lens = [700, 90]
    st = Setup(dit, 2, d, 32, lens, seed=3)
    st.fill_random(21)
    rng = np.random.default_rng(5)
    shape = st.scales(False).shape
    if kind == "2^-60":
        _set_exponents(st, False, -60)
    elif kind == "2^95":
        _set_exponents(st, False, 95)
    elif kind == "mixed":
        _set_exponents(st, False, rng.integers(-60, 90, shape))
    elif kind == "zero":
        st.scales(False)[:] = torch.full((1,), 2.0 ** -118).bfloat16().view(torch.int16).numpy()
        r = st.ref
        r.raw[:, :, r.half:r.half + r.page * d // 2] = 0x88  # codes of zero
        st.upload()
    else:
        exps = np.zeros(shape)
        for s, n in enumerate(lens):
            for pos in range(n):
                exps[st.table[s][pos // 32], :, pos % 32] = (-90 if kind == "falling" else 90) * pos / n + (60 if kind == "falling" else -30)
        _set_exponents(st, False, exps.astype(np.int64))
    out = _check_attention(dit, ws, st, 6, [2, 1], seed=d)
    if kind == "zero":
        rows = out[[1, 2, 4], :6 * d]
        assert (rows == 0).all()


def test_cache_attention_large_scales_that_a_row_does_not_see(dit, ws):
    """The last keys' values are 2^95 times the others': the queries before them keep their results to the bit."""
    for d in (64, 128):
        outs = []
        for e in (0, 95):
            st = Setup(dit, 1, d, 64, [300], seed=3)
            st.fill_random(22)
            exps = np.zeros(st.scales(False).shape, np.int64)
            exps[st.table[0][299 // 64], :, 299 % 64] = e
            exps[st.table[0][298 // 64], :, 298 % 64] = e
            _set_exponents(st, False, exps)
            outs.append(_check_attention(dit, ws, st, 4, [4], seed=1))
        # two queries see neither; their references may differ, their weights are the same to fp16's half step
        a, b = outs[0][1:3].double(), outs[1][1:3].double()
        assert float((a - b).norm() / a.norm()) < 2.0 ** -7


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("up", [60, -60])
def test_cache_attention_query_magnitudes(dit, ws, d, up):
    """Queries, and keys' scales, far from one, undone by the other or by the scale."""
    st = Setup(dit, 2, d, 64, [200, 33], seed=6)
    st.fill_random(23)
    _check_attention(dit, ws, st, 4, [2, 1], std=2.0 ** up, scale=2.0 ** -up * d ** -0.5, seed=2)
    _set_exponents(st, True, up)
    _check_attention(dit, ws, st, 4, [2, 1], std=1.0, scale=2.0 ** -up * d ** -0.5, seed=3)
    _check_attention(dit, ws, st, 4, [2, 1], std=2.0 ** -up, scale=d ** -0.5, seed=4)


def test_cache_attention_rows_of_zeros_and_of_one_value(dit, ws):
    """A query of zeros weighs all keys alike; one of a single value, or of the smallest numbers, has its scores."""
    d, hq = 128, 4
    st = Setup(dit, 1, d, 64, [130], seed=7)
    st.fill_random(24)
    q = torch.zeros(1, hq * d).bfloat16()
    q[0, d + 5] = 3.0
    q[0, 2 * d:3 * d] = _randn(d, seed=3) * 2.0 ** -120
    q[0, 3 * d:] = _randn(d, seed=4)
    q[0, 3 * d + 9] = 60.0
    out = torch.zeros_like(q).to(DEV)
    a = dit.make_text_attn(1, hq, 1, d, 1, 0, 1, 130, scale=0.05)
    dit.dit_text_cache4_attention(st.c, a, _i32([0, 1]), None, _i32([130]), st.table_dev(), q.to(DEV), hq * d, st.dev, out, hq * d, ws,
                                  ws.numel())
    _ok(dit, ws)
    want, tol, _, _ = R.cache_attention(q.view(1, hq, d), [(0, 1, 130)], True, 0.05, st.ref, st.table)
    _within(out.view(1, hq, d), want, tol)


def test_cache_of_more_than_four_gigabytes(dit, ws):
    """Pages whose offsets pass 2^31 and 2^32 bytes: append, attention and read give the bits of the same tokens in a
    small cache."""
    heads, d, page, n, hq = 8, 128, 256, 700, 16
    small = dit.make_text_cache4(heads, d, 3, page, 3)
    page_bytes = dit.dit_text_cache4_bytes(small) // 3
    pages = (1 << 32) // page_bytes + 40
    big = dit.make_text_cache4(heads, d, pages, page, 3)
    kv = _randn(n, 2 * heads * d, seed=1).to(DEV)
    q = _randn(1, hq * d, seed=2).to(DEV)
    got = []
    for c, table in ((small, [2, 0, 1]), (big, [pages - 1, (1 << 31) // page_bytes + 1, pages - 3])):
        cache = torch.empty(dit.dit_text_cache4_bytes(c), dtype=torch.uint8, device=DEV)
        t, kl = _i32([table]), _i32([n])
        dit.dit_text_cache4_append(c, 1, n, n, _i32([0, n]), None, kl, t, kv, kv.stride(0), kv[:, heads * d:], kv.stride(0), cache, ws,
                                   ws.numel())
        out, k, v = torch.zeros_like(q), torch.zeros(n, heads * d, dtype=torch.bfloat16, device=DEV), torch.zeros(
            n, heads * d, dtype=torch.bfloat16, device=DEV)
        a = dit.make_text_attn(1, hq, heads, d, 1, 0, 1, n)
        dit.dit_text_cache4_attention(c, a, _i32([0, 1]), None, kl, t, q, hq * d, cache, out, hq * d, ws, ws.numel())
        dit.dit_text_cache4_read(c, 1, n, n, _i32([0, n]), None, t, cache, k, heads * d, v, heads * d, ws, ws.numel())
        _ok(dit, ws)
        got.append([_bits(x) for x in (out, k, v)])
        del cache
    assert all(torch.equal(x, y) for x, y in zip(*got)) and bool((got[0][0] != 0).any())
    torch.cuda.empty_cache()


def test_rows_behind_two_to_the_31_elements(dit, ws):
    """The last rows of buffers whose offsets pass 32 bits, of the norm and of the product."""
    rows, cols, ld = 140000, 16, 16392
    x = torch.zeros(rows, ld, dtype=torch.bfloat16, device=DEV)
    pick = [0, 1, 131007, 131008, rows - 2, rows - 1]
    vals = _randn(len(pick), cols, seed=1)
    for i, r in enumerate(pick):
        x[r, :cols] = vals[i].to(DEV)
    w = _randn(24, cols, seed=2)
    out = torch.full((rows, ld), 5.0, dtype=torch.bfloat16, device=DEV)
    dit.dit_add_rms_norm(rows, cols, x, ld, None, 0, None, 0.0, 1e-6, None, 0, out, ld, None, None)
    _, want = R.add_rms_norm(vals, None, None, 0.0, float(np.float32(1e-6)))
    _within(out[pick, :cols], want, 2.0 ** -8 * want.abs() + _norm_tolerance(want, cols) * 1.01)
    assert (out[pick, cols:] == 5.0).all()
    out.fill_(5.0)
    dit.dit_linear_act(rows, 24, cols, x, ld, w.to(DEV), cols, None, 0, None, 0, out, ld, False, ws, ws.numel())
    _ok(dit, ws)
    want, size, z = R.linear_act(vals, w, None, "none", None)
    _within(out[pick, :24], want, R.linear_act_tolerance(want, size, z, cols, None, False))
    assert (out[pick, 24:] == 5.0).all()
    del x, out
    torch.cuda.empty_cache()


def test_every_call_runs_on_the_stream_it_is_given(dit, ws):
    """Inputs that a stream is still writing (behind a copy of a gigabyte) when the call is made on it."""
    st = Setup(dit, 2, 64, 16, [50, 20], seed=5)
    st.fill_random(31)
    x, w = _randn(40, 256, seed=1), _randn(128, 256, seed=2, std=0.06)
    q, kv = _randn(2, 4 * 64, seed=3), _randn(2, 4 * 64, seed=4)
    a = dit.make_text_attn(2, 4, 2, 64, 2, 0, 1, 50)
    qo, kl, table, wd = _i32([0, 1, 2]), _i32([50, 20]), st.table_dev(), w.to(DEV)
    busy = torch.zeros(1 << 30, dtype=torch.uint8, device=DEV)
    start = st.dev.clone()
    results = []
    for stream in (None, torch.cuda.Stream()):
        st.dev.copy_(start)
        src = [t.to(DEV) for t in (x, q, kv)]
        xin, qin, kvin = (torch.zeros_like(t) for t in src)
        y, o, lin = torch.zeros_like(xin), torch.zeros_like(qin), torch.zeros(40, 128, dtype=torch.bfloat16, device=DEV)
        kb, vb = (torch.zeros(70, 2 * 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        torch.cuda.synchronize()
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            for _ in range(8):
                busy.add_(1)
            for dst, s in zip((xin, qin, kvin), src):
                dst.copy_(s)
            s = stream if stream is not None else torch.cuda.current_stream()
            dit.dit_add_rms_norm(40, 256, xin, 256, None, 0, None, 0.0, 1e-6, None, 0, y, 256, None, None, s)
            dit.dit_linear_act(40, 128, 256, y, 256, wd, 256, None, dit.DIT_ACT_SILU, None, 0, lin, 128, False, ws, ws.numel(), s)
            dit.dit_text_cache4_append(st.c, 2, 2, 1, qo, None, kl, table, kvin, 256, kvin[:, 128:], 256, st.dev, ws, ws.numel(), s)
            dit.dit_text_cache4_attention(st.c, a, qo, None, kl, table, qin, 256, st.dev, o, 256, ws, ws.numel(), s)
            dit.dit_text_cache4_read(st.c, 2, 70, 50, _i32([0, 50, 70]), None, table, st.dev, kb, 128, vb, 128, ws, ws.numel(), s)
            outs = [t.clone() for t in (y, lin, o, kb, vb)]
        torch.cuda.synchronize()
        _ok(dit, ws)
        results.append([_bits(t) for t in outs])
    assert all(torch.equal(a, b) for a, b in zip(*results)) and all(bool((t != 0).any()) for t in results[0])


def test_graphs_that_share_a_workspace(dit, ws):
    """Three captured calls of different sizes on one workspace (one joins runs through it, one joins them in a cluster, one
    has none), replayed in any order on one stream."""
    sets = []
    for i, (d, lens, news) in enumerate(((128, [9000, 8000, 300] * 8, [1] * 24), (64, [900], [2]), (128, [40, 30], [1, 1]))):
        st = Setup(dit, 2, d, 64, lens, seed=i)
        st.fill_random(40 + i)
        rows = sum(news)
        q = _randn(rows, 8 * d, seed=i).to(DEV)
        out = torch.zeros_like(q)
        a = dit.make_text_attn(len(lens), 8, 2, d, rows, 0, max(news), max(lens))
        assert dit.dit_text_cache4_attention_workspace(st.c, a) <= ws.numel()
        sets.append((st, a, _i32([0] + np.cumsum(news).tolist()), _i32(lens), st.table_dev(), q, out))

    def run(s):
        st, a, qo, kl, table, q, out = s
        dit.dit_text_cache4_attention(st.c, a, qo, None, kl, table, q, q.stride(0), st.dev, out, q.stride(0), ws, ws.numel(),
                                      torch.cuda.current_stream())

    want, graphs = [], []
    for s in sets:
        run(s)
        torch.cuda.synchronize()
        want.append(_bits(s[-1]))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(s)
        graphs.append(g)
    for order in ((0, 1, 2, 0, 1, 2), (2, 1, 0, 0, 2, 1), (1, 0, 1, 0, 2, 2)):
        for s in sets:
            s[-1].zero_()
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for s, w in zip(sets, want):
            assert torch.equal(_bits(s[-1]), w)
    _ok(dit, ws)


@pytest.mark.parametrize("d", [64, 128])
def test_no_keys_at_all(dit, ws, d):
    """Queries of a cache without tokens are zeros, also where the bound says that there are none."""
    for max_k in (0, 1, 700):
        st = Setup(dit, 2, d, 16, [0, 0, 0], seed=1)
        st.max_pages = 64
        st.c = dit.make_text_cache4(2, d, st.ref.pages, 16, 64)
        out = _check_attention(dit, ws, st, 4, [1, 3, 0], seed=2, max_k=max_k)
        assert (out[[1, 3, 4, 5]] == 0).all()


def test_many_short_sequences(dit, ws):
    """As many sequences as a call takes, most without tokens, the last with some."""
    seqs, d, page = 16384, 64, 16
    lens = np.zeros(seqs, np.int64)
    lens[[0, 5000, seqs - 1]] = [20, 7, 33]
    st = Setup(dit, 1, d, page, lens.tolist(), seed=9)
    st.fill_random(50)
    news = (lens > 0).astype(np.int64)
    q = _randn(3, 2 * d, seed=1)
    out = torch.full((4, 2 * d), 9.0, dtype=torch.bfloat16, device=DEV)
    off = np.concatenate([[0], np.cumsum(news)])
    a = dit.make_text_attn(seqs, 2, 1, d, 3, 0, 1, 33)
    dit.dit_text_cache4_attention(st.c, a, _i32(off.tolist()), None, _i32(lens.tolist()), st.table_dev(), q.to(DEV), 2 * d, st.dev, out,
                                  2 * d, ws, ws.numel())
    _ok(dit, ws)
    spans = [(i, 1, n) for i, n in enumerate((20, 7, 33))]
    want, tol, _, _ = R.cache_attention(q.view(3, 2, d), spans, True, d ** -0.5, st.ref, [st.table[i] for i in (0, 5000, seqs - 1)])
    _within(out[:3].view(3, 2, d), want, tol)
    assert (out[3] == 9.0).all()


def test_the_same_token_twice_and_pages_that_are_shared(dit, ws):
    """Two sequences with one page table read the same keys; two new tokens on one place leave every other place alone."""
    d, page = 128, 16
    st = Setup(dit, 2, d, page, [40, 40], seed=10)
    st.fill_random(60)
    st.table[1] = st.table[0]
    out = _check_attention(dit, ws, st, 4, [1, 1], gap=0, seed=2)
    assert not torch.equal(_bits(out[0]), _bits(out[1]))
    before = st.dev.clone()
    kv = _randn(2, 4 * d, seed=3).to(DEV)
    st.append(ws, 2, _i32([0, 1, 2]), None, _i32([40, 40]), kv, kv[:, 2 * d:])
    _ok(dit, ws)
    for s in (0, 1):  # what the place may hold is one of the two, byte by byte
        st.ref.put(st.table[0][2], 7, kv[s].cpu()[:2 * d].view(2, d), kv[s].cpu()[2 * d:].view(2, d))
        same = st.dev.cpu() == torch.from_numpy(st.ref.raw.reshape(-1))
        either = same if s == 0 else either | same
    assert bool(either.all())
    changed = (st.dev != before).view(st.c.pages, -1).any(1).cpu().nonzero().flatten().tolist()
    assert changed == [st.table[0][2]]


@pytest.mark.parametrize("m,n,k,pad", [(300, 1000, 4104, 0), (777, 200, 1032, 0), (257, 136, 8192, 8), (600, 1500, 2056, 0), (900, 130, 1024, 0)])
def test_linear_act_rows_off_their_lines(dit, ws, m, n, k, pad):
    """Depths split over clusters, and rows that start between the lines of 128 bytes, with everything in the epilogue."""
    from test_text_layer_gpu import _check_linear
    for seed in (0, 1):
        _check_linear(dit, ws, m, n, k, ("gelu", "silu")[seed], True, True, bool(seed), pad=pad, seed=seed)


def test_operands_that_start_off_their_lines(dit, ws):
    """Operands 16 bytes into a line give the sums of the same operands at its start, within their roundings."""
    m, n, k = 520, 264, 2048
    a, w = _randn(m, k, seed=1), _randn(n, k, seed=2, std=k ** -0.5)
    want, size, z = R.linear_act(a, w, None, "none", None)
    for shift in (0, 8, 24):
        buf, wb = torch.zeros(m * k + 64, dtype=torch.bfloat16, device=DEV), torch.zeros(n * k + 64, dtype=torch.bfloat16, device=DEV)
        av, wv = buf[shift:shift + m * k].view(m, k), wb[shift:shift + n * k].view(n, k)
        av.copy_(a)
        wv.copy_(w)
        out = torch.zeros(m, n, dtype=torch.bfloat16, device=DEV)
        dit.dit_linear_act(m, n, k, av, k, wv, k, None, 0, None, 0, out, n, False, ws, ws.numel())
        _ok(dit, ws)
        _within(out, want, R.linear_act_tolerance(want, size, z, k, None, False))


@pytest.mark.parametrize("m,n,k", [(1 << 20, 8, 8), (1, 1 << 20, 8), (130, 1 << 18, 16), (8, 8, 1 << 20), (300, 9, 1 << 19)])
def test_linear_act_longest_sides(dit, ws, m, n, k):
    """As many rows, columns and as much depth as a call takes."""
    a, w = _randn(m, k, seed=1), _randn(n, k, seed=2, std=k ** -0.5)
    out = torch.zeros(m, n + -n % 8, device=DEV)
    dit.dit_linear_act(m, n, k, a.to(DEV), k, w.to(DEV), k, None, 0, None, 0, out, out.stride(0), True, ws, ws.numel())
    _ok(dit, ws)
    pick = [0, 1, m // 2, m - 1] if m > 4 else list(range(m))
    want, size, z = R.linear_act(a[pick], w, None, "none", None)
    _within(out[pick, :n], want, R.linear_act_tolerance(want, size, z, k, None, True))


def test_add_rms_norm_many_rows(dit):
    """Four million rows of eight columns: several rows of a CTA at once, each CTA many."""
    rows = 1 << 22
    x = _randn(1024, 8, seed=1).repeat(rows // 1024, 1).to(DEV)
    y = torch.zeros_like(x)
    dit.dit_add_rms_norm(rows, 8, x, 8, None, 0, None, 0.0, 1e-6, None, 0, y, 8, None, None)
    torch.cuda.synchronize()
    _, want = R.add_rms_norm(x[:1024].cpu(), None, None, 0.0, float(np.float32(1e-6)))
    _within(y[:1024], want, 2.0 ** -8 * want.abs() + _norm_tolerance(want, 8) * 1.01)
    assert bool((y.view(-1, 1024, 8) == y[:1024]).all())


@pytest.mark.parametrize("d", [64, 128])
def test_cache_of_as_many_heads_as_there_may_be(dit, ws, d):
    heads, lens = 1024, [3, 17]
    st = Setup(dit, heads, d, 16, lens, seed=d)
    kv = _randn(20, 2 * heads * d, seed=1)
    kvd = kv.to(DEV)
    st.append(ws, 20, _i32([0, 3, 20]), None, _i32(lens), kvd, kvd[:, heads * d:])
    _ok(dit, ws)
    row = 0
    for s, n in enumerate(lens):
        for i in range(n):
            st.ref.put(st.table[s][i // 16], i % 16, kv[row, :heads * d].view(heads, d), kv[row, heads * d:].view(heads, d))
            row += 1
    assert st.same()
    _check_attention(dit, ws, st, heads, [1, 2], seed=3)
    _check_attention(dit, ws, st, heads, [1, 2], seed=3, max_k=1 << 20)
