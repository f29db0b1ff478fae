"""The text-side operations on the GPU against 64-bit forms of their formulas, through the C ABI.

Tolerances are derived where they are used: a rounding to bf16 is off by at most 2^-8 of the
value, one to fp32 by 2^-24."""
import math

import numpy as np
import pytest
import torch

import text_reference as R

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def dit():
    from diffusion_transformer_step_gb300 import build_lib
    build_lib.build()
    from diffusion_transformer_step_gb300 import dit as d
    d.lib()
    return d


@pytest.fixture()
def ws():
    return torch.zeros(32 << 20, dtype=torch.uint8, device=DEV)


def _ok(dit, ws):
    st, where = dit.dit_sync_status(ws)
    assert st == dit.DIT_OK, (st, hex(where))


def _randn(*shape, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16)


def _within(got, want, tol):
    err = (got.double().cpu() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), float((err / tol).max()), bad.nonzero()[:4].tolist())


# ------------------------------------------------------------------------------ rotary table
SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3}


@pytest.mark.parametrize("scaling", list(SCALINGS))
@pytest.mark.parametrize("rot,n,start,theta", [(128, 700, 0, 1e6), (2, 1, 5, 1e4), (4, 33, 0, 1e4), (96, 257, 1 << 23, 5e5),
                                               (256, 5, -3, 1e4), (64, 300, -(1 << 24), 1.5)])
def test_text_rope_table(dit, scaling, rot, n, start, theta):
    if scaling == "ntk" and rot == 2:
        pytest.skip("refused: its exponent divides by rot_dim - 2")
    kw = dict(rot=rot, theta=theta, scaling=scaling, factor=8.0, low=1.0, high=4.0, original_len=4096)
    mag = 1.2 if scaling == "by_parts" else 1.0
    r = dit.make_text_rope(rot, theta, SCALINGS[scaling], factor=8.0, low=1.0, high=4.0, original_len=4096, magnitude=mag)
    table = torch.full((n + 1, rot // 2, 2), 7.0, device=DEV)
    pos = torch.arange(n, dtype=torch.int32) + start
    dit.dit_text_rope_table(r, None if start == 0 else pos.to(DEV), n, table)
    torch.cuda.synchronize()
    want = R.rope_table(pos.numpy(), magnitude=np.float32(mag), **kw)
    # the documented bound; the 64-bit angles of the reference are off by 2^24 * 2^-52 at most
    tol = 4 * 2.0 ** -24 * mag + 2.0 ** -27
    err = np.abs(table[:n].cpu().double().numpy() - want)
    assert err.max() <= tol, err.max() / tol
    assert (table[n:] == 7.0).all()


def test_text_rope_table_any_order_of_positions(dit):
    pos = torch.tensor([5, 0, 5, 16777216, -16777216, 99, 1], dtype=torch.int32)
    table = torch.empty(7, 32, 2, device=DEV)
    dit.dit_text_rope_table(dit.make_text_rope(64, 1e4), pos.to(DEV), 7, table)
    want = R.rope_table(pos.numpy(), rot=64, theta=1e4)
    assert np.abs(table.cpu().double().numpy() - want).max() <= 4 * 2.0 ** -24 + 2.0 ** -27
    assert torch.equal(table[0], table[2])


# ---------------------------------------------------------------------- norm and rotation of heads
@pytest.mark.parametrize("layout", ["interleaved", "half"])
@pytest.mark.parametrize("rows,hq,hk,d,rot,norm", [
    (1, 1, 0, 64, 64, True), (1, 32, 8, 128, 128, True), (7, 3, 1, 64, 48, True), (33, 5, 5, 128, 8, False),
    (300, 8, 2, 128, 128, True), (129, 7, 1, 64, 64, False), (65, 2, 2, 128, 0, True), (1025, 16, 4, 128, 104, True)])
def test_qk_norm_rope(dit, ws, layout, rows, hq, hk, d, rot, norm):
    ld = (hq + 2 * hk) * d + 8
    x = _randn(rows, ld, seed=rows)
    wq, wk = (_randn(d, seed=2, std=0.2) + 1, _randn(d, seed=3, std=0.2) + 1) if norm else (None, None)
    top = rows + 3
    table = torch.from_numpy(R.rope_table(np.arange(top), rot=max(rot, 2), theta=1e4)).float()
    index = torch.randperm(top, generator=torch.Generator().manual_seed(1))[:rows].int()
    xd = x.to(DEV)
    qo = torch.full((rows, hq * d + 16), 3.0, dtype=torch.bfloat16, device=DEV)
    ko = torch.full((rows, hk * d + 8), 3.0, dtype=torch.bfloat16, device=DEV)
    dv = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    wqd, wkd, td, ixd = dv(wq), dv(wk), dv(table) if rot else None, dv(index)
    lay = dit.DIT_ROPE_HALF if layout == "half" else dit.DIT_ROPE_INTERLEAVED
    args = (rows, hq, hk, d, rot, lay)
    dit.dit_qk_norm_rope(*args, xd, ld, xd[:, hq * d:], ld, wqd, wkd, 1e-6, td, top, ixd, qo, hq * d + 16, ko, hk * d + 8,
                         ws, ws.numel())
    _ok(dit, ws)
    for part, out, w, h in ((x[:, :hq * d], qo, wq, hq), (x[:, hq * d:(hq + hk) * d], ko, wk, hk)):
        want, size = R.qk_norm_rope(part.reshape(rows, h, d), w, float(np.float32(1e-6)), table[index.long()], rot, layout)
        # one rounding to bf16, and under 16 fp32 roundings of the pair's two products
        tol = 2.0 ** -8 * want.abs() + 16 * 2.0 ** -24 * size + 1e-30
        _within(out[:, :h * d].reshape(rows, h, d), want, tol)
        assert (out[:, h * d:] == 3.0).all()
    # in place gives the same bits, and leaves the values and the padding alone
    yd = x.to(DEV)
    dit.dit_qk_norm_rope(*args, yd, ld, yd[:, hq * d:], ld, wqd, wkd, 1e-6, td, top, ixd, yd, ld, yd[:, hq * d:], ld, ws,
                         ws.numel())
    _ok(dit, ws)
    assert torch.equal(yd[:, :hq * d], qo[:, :hq * d]) and torch.equal(yd[:, hq * d:(hq + hk) * d], ko[:, :hk * d])
    assert torch.equal(yd[:, (hq + hk) * d:].cpu(), x[:, (hq + hk) * d:])
    if rot:
        # without the index, row r reads table row r
        dit.dit_qk_norm_rope(*args, xd, ld, xd[:, hq * d:], ld, wqd, wkd, 1e-6, td[index.long().to(DEV)].contiguous(), rows,
                             None, yd, ld, yd[:, hq * d:], ld, ws, ws.numel())
        _ok(dit, ws)
        assert torch.equal(yd[:, :hq * d], qo[:, :hq * d])


@pytest.mark.parametrize("layout,rows,hq,hk,d,rot,norm", [
    ("half", 4099, 36, 8, 128, 128, True), ("interleaved", 10003, 33, 0, 64, 48, True), ("half", 4001, 40, 1, 128, 64, False),
    ("interleaved", 5003, 17, 17, 128, 128, True), ("half", 7001, 40, 16, 64, 64, True), ("half", 4999, 33, 0, 128, 0, True)])
def test_qk_norm_rope_many_rows(dit, ws, layout, rows, hq, hk, d, rot, norm):
    """Enough rows to be streamed through shared memory: strided, in place, two rows without a table row."""
    ld, heads = (hq + hk) * d + 24, hq + hk
    x = _randn(rows, ld, seed=rows)
    wq, wk = (_randn(d, seed=2, std=0.2) + 1, _randn(d, seed=3, std=0.2) + 1) if norm else (None, None)
    top = 600
    table = torch.from_numpy(R.rope_table(np.arange(top), rot=max(rot, 2), theta=1e4)).float()
    index = torch.randint(0, top, (rows,), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    bad = [5, rows - 1] if rot else []
    given = index.clone()
    given[bad] = torch.tensor([top, -7][:len(bad)], dtype=torch.int32)
    dv = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    lay = dit.DIT_ROPE_HALF if layout == "half" else dit.DIT_ROPE_INTERLEAVED
    xd, td = x.to(DEV), dv(table) if rot else None
    qo = torch.full((rows, hq * d + 8), 3.0, dtype=torch.bfloat16, device=DEV)
    ko = torch.full((rows, hk * d + 16), 3.0, dtype=torch.bfloat16, device=DEV)
    k = xd[:, hq * d:] if hk else None
    norms = dv(wq), dv(wk) if hk else None
    dit.dit_qk_norm_rope(rows, hq, hk, d, rot, lay, xd, ld, k, ld, *norms, 1e-6, td, top, dv(given), qo, hq * d + 8,
                         ko if hk else None, hk * d + 16, ws, ws.numel())
    st, where = dit.dit_sync_status(ws)
    assert (st, where) == (dit.DIT_ERR_INVALID_ARG, 0x601) if bad else st == dit.DIT_OK
    good = torch.ones(rows, dtype=torch.bool)
    good[bad] = False
    for part, out, w, h in ((x[:, :hq * d], qo, wq, hq), (x[:, hq * d:heads * d], ko, wk, hk)):
        if h == 0:
            continue
        want, size = R.qk_norm_rope(part.reshape(rows, h, d), w, float(np.float32(1e-6)), table[index.long()], rot, layout)
        tol = 2.0 ** -8 * want.abs() + 16 * 2.0 ** -24 * size + 1e-30  # as above
        _within(out[:, :h * d].reshape(rows, h, d)[good.to(DEV)], want[good], tol[good])
        assert (out[:, h * d:] == 3.0).all() and (out[(~good).to(DEV)] == 3.0).all()
    yd = x.to(DEV)
    dit.dit_qk_norm_rope(rows, hq, hk, d, rot, lay, yd, ld, yd[:, hq * d:] if hk else None, ld, *norms, 1e-6, td, top,
                         dv(index), yd, ld, yd[:, hq * d:] if hk else None, ld, ws, ws.numel())
    _ok(dit, ws)
    g = good.to(DEV)
    assert torch.equal(yd[g, :hq * d], qo[g, :hq * d]) and torch.equal(yd[g, hq * d:heads * d], ko[g, :hk * d])
    assert torch.equal(yd[:, heads * d:].cpu(), x[:, heads * d:])
    # a few rows alone, row by row, give the same bits
    n = 9
    few = torch.empty(n, hq * d, dtype=torch.bfloat16, device=DEV)
    dit.dit_qk_norm_rope(n, hq, 0, d, rot, lay, xd, ld, None, 0, norms[0], None, 1e-6, td, top, dv(index), few, hq * d, None, 0,
                         ws, ws.numel())
    _ok(dit, ws)
    assert torch.equal(few, yd[:n, :hq * d])


def test_qk_norm_rope_zero_rows_of_x_and_nan(dit, ws):
    """A head of zeros stays zeros (eps keeps the root finite); a NaN stays in its own head."""
    x = _randn(3, 256, seed=1)
    x[0] = 0
    x[1, 5] = math.nan
    w = torch.ones(128, dtype=torch.bfloat16, device=DEV)
    t = torch.from_numpy(R.rope_table(np.arange(3), rot=128, theta=1e4)).float().to(DEV)
    out = torch.empty(3, 256, dtype=torch.bfloat16, device=DEV)
    dit.dit_qk_norm_rope(3, 2, 0, 128, 128, dit.DIT_ROPE_HALF, x.to(DEV), 256, None, 0, w, None, 1e-6, t, 3, None, out, 256,
                         None, 0, ws, ws.numel())
    _ok(dit, ws)
    assert (out[0] == 0).all() and out[1, :128].isnan().all() and out[1:, 128:].isfinite().all()


def test_qk_norm_rope_bad_index_is_reported_and_its_row_left(dit, ws):
    x = _randn(4, 128, seed=4).to(DEV)
    t = torch.from_numpy(R.rope_table(np.arange(4), rot=128, theta=1e4)).float().to(DEV)
    for bad in (-1, 4, 2 ** 31 - 1, -2 ** 31):
        index = torch.tensor([0, bad, 3, 1], dtype=torch.int32, device=DEV)
        out = torch.full((4, 128), 9.0, dtype=torch.bfloat16, device=DEV)
        dit.dit_qk_norm_rope(4, 1, 0, 128, 128, dit.DIT_ROPE_HALF, x, 128, None, 0, None, None, 1e-6, t, 4, index, out, 128,
                             None, 0, ws, ws.numel())
        st, where = dit.dit_sync_status(ws)
        assert st == dit.DIT_ERR_INVALID_ARG and where == 0x601
        _ok(dit, ws)  # cleared
        assert (out[1] == 9.0).all() and (out[[0, 2, 3]] != 9.0).any(1).all()


# ------------------------------------------------------------------------------------ attention
def _spans(ql, kl, gap_q=0, gap_k=0):
    spans, a, b = [], gap_q, gap_k
    for n, m in zip(ql, kl):
        spans.append((a, n, b, m))
        a, b = a + n + gap_q, b + m + gap_k
    return spans, a, b


def _attend(dit, ws, ql, kl, hq, hk, d, causal, scale=None, gap_q=0, gap_k=0, lens=True, fill=None, qstd=1.0, seed=0,
            edit=None, ld_extra=0):
    spans, rq, rk = _spans(ql, kl, gap_q, gap_k)
    scale = d ** -0.5 if scale is None else scale
    q, k, v = _randn(rq, hq, d, seed=seed, std=qstd), _randn(rk, hk, d, seed=seed + 1), _randn(rk, hk, d, seed=seed + 2)
    if fill is not None:  # rows of k and v that belong to no sequence
        own = torch.zeros(rk, dtype=torch.bool)
        for _, _, b, m in spans:
            own[b:b + m] = True
        k[~own] = fill
        v[~own] = fill
    if edit:
        edit(q, k, v, spans)
    want, size, owned = R.attention(q, k, v, spans, causal, float(np.float32(scale)))
    i32 = lambda t: torch.tensor(t, dtype=torch.int32, device=DEV)  # noqa: E731
    qo, ko = i32([s[0] for s in spans] + [rq]), i32([s[2] for s in spans] + [rk])
    qn, kn = (i32(list(ql)), i32(list(kl))) if lens else (None, None)

    def strided(t):
        b = torch.zeros(t.shape[0], t.shape[1] * d + ld_extra, dtype=torch.bfloat16, device=DEV)
        b[:, :t.shape[1] * d] = t.flatten(1).to(DEV)
        return b

    qd, kd, vd = strided(q), strided(k), strided(v)
    out = torch.full((rq, hq * d + ld_extra), 5.0, dtype=torch.bfloat16, device=DEV)
    a = dit.make_text_attn(len(ql), hq, hk, d, rq, rk, max(ql, default=0), max(kl, default=0), causal, scale)
    need = dit.dit_text_attention_workspace(a)
    assert need <= ws.numel()
    call = lambda: dit.dit_text_attention(a, qo, qn, ko, kn, qd, hq * d + ld_extra, kd, hk * d + ld_extra, vd,  # noqa: E731
                                          hk * d + ld_extra, out, hq * d + ld_extra, ws, need)
    call()
    _ok(dit, ws)
    first = out.clone()
    call()
    _ok(dit, ws)
    assert torch.equal(first, out) or first.isnan().any()  # equal calls, equal bits
    got = first[:, :hq * d].reshape(rq, hq, d).cpu()
    assert (first[:, hq * d:] == 5.0).all() and (got[~owned] == 5.0).all()
    return got[owned], want[owned], size[owned], (q, k, float(np.float32(scale)))


def _check_attention(got, want, size, qks):
    fin = want.isfinite()
    assert torch.equal(got.isfinite(), fin)
    tol = R.attention_tolerance(torch.nan_to_num(want), torch.nan_to_num(size), *[torch.nan_to_num(t) for t in qks[:2]], qks[2])
    _within(torch.where(fin, got.double(), 0.0), torch.where(fin, want, 0.0), tol)


@pytest.mark.parametrize("hq,hk,d", [(4, 1, 128), (2, 2, 64), (6, 2, 128), (5, 1, 64), (8, 8, 128), (14, 2, 64), (64, 1, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_text_attention_lengths(dit, ws, hq, hk, d, causal):
    """Whole prompts from no token to past two key tiles, packed without gaps."""
    ql = [1, 2, 0, 31, 127, 128, 129, 5, 300]
    _check_attention(*_attend(dit, ws, ql, ql, hq, hk, d, causal, lens=False))


@pytest.mark.parametrize("hq,hk,d", [(8, 2, 128), (4, 4, 64), (7, 1, 128)])
@pytest.mark.parametrize("causal", [True, False])
def test_text_attention_tails_and_caches(dit, ws, hq, hk, d, causal):
    """Queries that are the last part of their keys, in padded slots; rows between the slots
    hold NaN and are neither used nor written."""
    ql = [1, 3, 40, 130, 1, 257, 17, 1]
    kl = [1, 200, 40, 131, 1000, 300, 640, 128]
    _check_attention(*_attend(dit, ws, ql, kl, hq, hk, d, causal, gap_q=3, gap_k=5, fill=math.nan))


@pytest.mark.parametrize("fill", [math.inf, -math.inf, 3.3e38])
def test_text_attention_ignores_rows_behind_the_keys(dit, ws, fill):
    _check_attention(*_attend(dit, ws, [64, 65, 1], [64, 65, 130], 4, 2, 128, True, gap_k=7, fill=fill))


@pytest.mark.parametrize("d", [64, 128])
def test_text_attention_rows_without_a_key(dit, ws, d):
    """No keys at all, and causal queries before the first key: zeros."""
    got, want, size, qk = _attend(dit, ws, [5, 200, 1, 140], [0, 60, 0, 3], 4, 1, d, True)
    assert (got[:5] == 0).all() and (got[5:145] == 0).all() and (got[205] == 0).all()
    _check_attention(got, want, size, qk)
    got, want, size, qk = _attend(dit, ws, [5, 1], [0, 0], 4, 1, d, False)
    assert (got == 0).all()


@pytest.mark.parametrize("seqs,nk,hq,hk,d", [(1, 5000, 8, 2, 128), (3, 2049, 4, 1, 64), (2, 4096, 16, 1, 128), (1, 1, 32, 8, 128),
                                             (40, 129, 8, 8, 64), (5, 1000, 12, 1, 128), (1, 3001, 64, 1, 64)])
def test_text_attention_single_tokens(dit, ws, seqs, nk, hq, hk, d):
    kl = [max(1, nk - 37 * i) for i in range(seqs)]
    _check_attention(*_attend(dit, ws, [1] * seqs, kl, hq, hk, d, True, gap_k=2, fill=math.nan))


@pytest.mark.parametrize("nq,nk,hq,hk", [(4, 3000, 4, 1), (16, 2000, 2, 2), (33, 1500, 8, 2), (2, 700, 8, 1)])
def test_text_attention_few_queries_over_long_keys(dit, ws, nq, nk, hq, hk):
    for causal in (True, False):
        _check_attention(*_attend(dit, ws, [nq, 1, nq], [nk, 5, nk - 300], hq, hk, 128, causal))


@pytest.mark.parametrize("nq,nk,hq,hk,d", [(1, 20000, 4, 1, 128), (4, 9001, 8, 2, 64), (20, 17000, 3, 1, 128), (130, 4500, 1, 1, 64)])
def test_text_attention_joins_of_many_parts(dit, ws, nq, nk, hq, hk, d):
    """Few rows over so many keys that a row's parts are more than a warp's lanes, or as many as the
    tiles are cut into; the sequences behind them have keys for some of their parts only."""
    _check_attention(*_attend(dit, ws, [nq, min(nq, 3), nq], [nk, 3, nk // 3], hq, hk, d, True, gap_k=1, fill=math.nan))


@pytest.mark.parametrize("nq,nk", [(40, 3000), (3, 12000)])
def test_text_attention_bad_value_in_one_of_many_parts(dit, ws, nq, nk):
    """A value in the last part is infinite: the queries before it keep their results over all parts."""
    at = nk - nq // 2 - 1
    def edit(q, k, v, spans):
        v[at, 0, 3] = math.inf
    got, want, size, qk = _attend(dit, ws, [nq], [nk], 3, 1, 128, True, edit=edit)
    blind = at - (nk - nq)  # queries that do not see it
    clean = R.attention(qk[0], qk[1], _randn(nk, 1, 128, seed=2), [(0, nq, 0, nk)], True, qk[2])
    _check_attention(got[:blind], clean[0][:blind], clean[1][:blind], qk)
    assert not got[blind:, :, 3].isfinite().any()
    assert got[blind:][..., [c for c in range(128) if c != 3]].isfinite().all()


@pytest.mark.parametrize("seqs", [65, 300, 1500])
@pytest.mark.parametrize("hq,hk,d,causal", [(4, 1, 128, True), (3, 3, 64, False)])
def test_text_attention_many_sequences(dit, ws, seqs, hq, hk, d, causal):
    """More sequences than one warp can search: the tiles are listed first.  Every 7th is empty,
    every 11th longer than a tile."""
    kl = [0 if i % 7 == 3 else 300 + i % 50 if i % 11 == 0 and i < 200 else 1 + (i * 37) % 40 for i in range(seqs)]
    kl[0] = 301
    _check_attention(*_attend(dit, ws, kl, kl, hq, hk, d, causal, lens=False))
    _check_attention(*_attend(dit, ws, [min(n, 17) for n in kl], kl, hq, hk, d, causal, gap_q=1, gap_k=1, fill=math.inf))


@pytest.mark.parametrize("hq,hk", [(3, 1), (5, 1), (12, 4), (16, 2), (32, 1)])
def test_text_attention_group_sizes_over_items(dit, ws, hq, hk):
    """Groups that do and do not divide a warp's rows, more items than SMs in one call."""
    ql = [700, 33, 512, 1, 257, 640, 128, 90]
    _check_attention(*_attend(dit, ws, ql, ql, hq, hk, 64, True))


def test_text_attention_single_tokens_without_keys(dit, ws):
    got, want, size, qk = _attend(dit, ws, [1, 1, 0, 1], [0, 700, 3, 5], 4, 2, 128, True)
    assert (got[0] == 0).all()
    _check_attention(got, want, size, qk)
    got, _, _, _ = _attend(dit, ws, [1], [0], 8, 8, 64, False)
    assert (got == 0).all()
    # causal queries before the first key
    got, want, size, qk = _attend(dit, ws, [4], [2], 4, 1, 128, True)
    assert (got[:2] == 0).all()
    _check_attention(got, want, size, qk)


def test_text_attention_bounds_wider_than_the_lengths(dit, ws):
    """max_q and max_k are upper bounds only: the same bits as with tight ones, on the same kernel."""
    hq, hk, d = 8, 2, 128
    q, k, v = _randn(300, hq, d, seed=1), _randn(300, hk, d, seed=2), _randn(300, hk, d, seed=3)
    i32 = lambda t: torch.tensor(t, dtype=torch.int32, device=DEV)  # noqa: E731
    want, size, _ = R.attention(q, k, v, [(0, 200, 0, 200), (200, 100, 200, 100)], True, d ** -0.5)
    dev = [t.flatten(1).to(DEV) for t in (q, k, v)]
    for mq, mk in ((200, 200), (300, 300), (100000, 1 << 24)):
        out = torch.zeros(300, hq * d, dtype=torch.bfloat16, device=DEV)
        a = dit.make_text_attn(2, hq, hk, d, 300, 300, mq, mk)
        dit.dit_text_attention(a, i32([0, 200, 300]), None, i32([0, 200, 300]), None, dev[0], hq * d, dev[1], hk * d, dev[2],
                               hk * d, out, hq * d, ws, ws.numel())
        _ok(dit, ws)
        _check_attention(out.reshape(300, hq, d).cpu(), want, size, (q, k, d ** -0.5))


@pytest.mark.parametrize("scale,qstd", [(1.0, 4.0), (0.02, 1.0), (3.0, 1.0)])
def test_text_attention_sharp_and_flat_scores(dit, ws, scale, qstd):
    """Scores over hundreds (one key takes everything, the running maximum moves often) and flat ones."""
    _check_attention(*_attend(dit, ws, [300, 1, 1], [300, 900, 130], 4, 2, 128, True, scale=scale, qstd=qstd))


def test_text_attention_growing_scores(dit, ws):
    """Every key scores above all before it, by steps of many powers of two."""
    def edit(q, k, v, spans):
        q[:] = 0
        k[:] = 0
        q[..., 0] = 8
        k[..., 0] = torch.arange(k.shape[0])[:, None].float().to(torch.bfloat16)
    for ql, kl in (([700], [700]), ([1], [700])):
        _check_attention(*_attend(dit, ws, ql, kl, 4, 2, 128, True, edit=edit, scale=0.25))
        _check_attention(*_attend(dit, ws, ql, kl, 4, 2, 128, False, edit=edit, scale=0.25))


def test_text_attention_very_low_scores(dit, ws):
    """All scores near -2^16: the maximum, not zero, is what exponentials are taken against."""
    def edit(q, k, v, spans):
        q[..., 0] = -256
        k[..., 0] = 256
    _check_attention(*_attend(dit, ws, [200, 1], [200, 400], 4, 2, 64, True, edit=edit, scale=1.0))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("ql,kl", [([300], [300]), ([1], [300]), ([40], [700])])
def test_text_attention_bad_value_reaches_only_queries_that_see_it(dit, ws, ql, kl, bad):
    """One infinite or NaN value in V, late in the sequence: queries before it stay finite and
    right, queries that see it get it."""
    at = kl[0] - 20

    def edit(q, k, v, spans):
        v[spans[0][2] + at, 0, 3] = bad
    got, want, size, qk = _attend(dit, ws, ql, kl, 4, 1, 128, True, edit=edit)
    blind = max(0, ql[0] - 20)  # queries before the bad key
    clean = R.attention(*[t for t in (qk[0], qk[1])], torch.nan_to_num(_randn(kl[0], 1, 128, seed=2), 0), [(0, ql[0], 0, kl[0])],
                        True, qk[2])
    _check_attention(got[:blind], clean[0][:blind], clean[1][:blind], qk) if blind else None
    assert not got[blind:, :, 3].isfinite().any()
    keep = [c for c in range(128) if c != 3]
    assert got[blind:][..., keep].isfinite().all()


# Calls of more than 304 tiles of 16 query rows (heads of a group among them) are worked on in tiles
# of 128 rows, smaller ones 16 rows at a time: the next tests hold what the ones above hold on either side.
@pytest.mark.parametrize("hq,hk,d", [(32, 8, 128), (12, 12, 64), (40, 8, 128), (64, 16, 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_text_attention_many_tiles(dit, ws, hq, hk, d, causal):
    """Odd lengths, sequences without queries or keys, more queries than keys, gaps of NaN between."""
    ql = [129, 1, 0, 64, 300, 65, 7, 250]
    kl = [129, 200, 5, 0, 300, 30, 129, 511]
    _check_attention(*_attend(dit, ws, ql, kl, hq, hk, d, causal, gap_q=3, gap_k=2, fill=math.nan))
    _check_attention(*_attend(dit, ws, ql, kl, hq, hk, d, causal, lens=False, ld_extra=8))


@pytest.mark.parametrize("seqs,n,hq,hk,d,causal", [
    (1, 17, 4, 1, 128, True), (1, 100, 32, 32, 64, False), (1, 77, 32, 8, 128, True), (3, 300, 2, 1, 64, True), (2, 40, 8, 2, 128, False),
    (1, 1200, 2, 2, 64, True), (70, 5, 8, 2, 64, True)])
def test_text_attention_small_prompts(dit, ws, seqs, n, hq, hk, d, causal):
    """Prompts of a few tiles of 16 rows, ragged, and their last parts over a cache."""
    kl = [max(1, n - 3 * i) for i in range(seqs)]
    _check_attention(*_attend(dit, ws, kl, kl, hq, hk, d, causal, lens=False))
    _check_attention(*_attend(dit, ws, [max(1, x // 2) for x in kl], kl, hq, hk, d, causal, gap_q=1, gap_k=3, fill=math.inf))
    _check_attention(*_attend(dit, ws, kl, [x // 2 for x in kl], hq, hk, d, causal))  # rows that see nothing


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("nk", [300, 129, 1000])
def test_text_attention_bad_value_in_a_tile(dit, ws, nk, bad):
    """As below and above, with enough heads for tiles of 128 rows: the queries that do not see the bad
    value keep their results, and so do the other heads."""
    at, hq, hk = nk - 40, 32, 8
    def edit(q, k, v, spans):
        v[at, 3, 5] = bad
    got, want, size, qk = _attend(dit, ws, [nk], [nk], hq, hk, 128, True, edit=edit)
    clean = R.attention(qk[0], qk[1], _randn(nk, hk, 128, seed=2), [(0, nk, 0, nk)], True, qk[2])
    mine = [h for h in range(hq) if h // 4 == 3]
    other = [h for h in range(hq) if h // 4 != 3]
    keep = [c for c in range(128) if c != 5]
    _check_attention(got[:at], clean[0][:at], clean[1][:at], qk)
    assert got[:, other].isfinite().all() and got[at:, mine][..., keep].isfinite().all()
    assert not got[at:, mine][..., 5].isfinite().any()


def test_text_attention_bad_key_in_a_tile(dit, ws):
    def edit(q, k, v, spans):
        k[250, 2, 7] = math.nan
    got, want, size, qk = _attend(dit, ws, [300], [300], 32, 8, 128, True, edit=edit)
    mine = [h for h in range(32) if h // 4 == 2]
    assert got[:250].isfinite().all() and got[250:, mine].isnan().all()
    assert got[:, [h for h in range(32) if h not in mine]].isfinite().all()


@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("nk", [4, 300, 1000, 3000])
def test_text_attention_bad_value_between_few_queries(dit, ws, nk, bad):
    """Four last queries, the last but one key's value bad: the first two do not see it."""
    def edit(q, k, v, spans):
        v[nk - 2, 0, 3] = bad
    got, want, size, qk = _attend(dit, ws, [4], [nk], 4, 1, 128, True, edit=edit)
    clean = R.attention(qk[0], qk[1], _randn(nk, 1, 128, seed=2), [(0, 4, 0, nk)], True, qk[2])
    _check_attention(got[:2], clean[0][:2], clean[1][:2], qk)
    assert not got[2:, :, 3].isfinite().any()
    assert got[2:][..., [c for c in range(128) if c != 3]].isfinite().all()


def test_text_attention_bad_key_reaches_only_queries_that_see_it(dit, ws):
    def edit(q, k, v, spans):
        k[250, 0, 7] = math.nan
    got, want, size, qk = _attend(dit, ws, [300], [300], 4, 1, 128, True, edit=edit)
    assert got[:250].isfinite().all() and got[250:].isnan().all()


def test_text_attention_shared_key_rows_and_strides(dit, ws):
    """Two sequences that read the same keys (a shared prompt), row strides wider than the heads."""
    hq, hk, d, nk = 8, 2, 128, 333
    q, k, v = _randn(9, hq, d, seed=1), _randn(nk, hk, d, seed=2), _randn(nk, hk, d, seed=3)
    spans = [(0, 5, 0, nk), (5, 4, 0, nk)]
    want, size, _ = R.attention(q, k, v, spans, False, d ** -0.5)
    kv = torch.cat([k.flatten(1), v.flatten(1), k.flatten(1)], 1).to(DEV).contiguous()
    ldkv = kv.shape[1]
    buf = torch.zeros(9, 2 * hq * d, dtype=torch.bfloat16, device=DEV)  # queries and outputs side by side
    buf[:, :hq * d] = q.flatten(1).to(DEV)
    i32 = lambda t: torch.tensor(t, dtype=torch.int32, device=DEV)  # noqa: E731
    a = dit.make_text_attn(2, hq, hk, d, 9, nk, 5, nk, causal=False)
    dit.dit_text_attention(a, i32([0, 5, 9]), None, i32([0, 0, 0]), i32([nk, nk]), buf, 2 * hq * d, kv, ldkv, kv[:, hk * d:],
                           ldkv, buf[:, hq * d:], 2 * hq * d, ws, ws.numel())
    _ok(dit, ws)
    _check_attention(buf[:, hq * d:].reshape(9, hq, d).cpu(), want, size, (q, k, d ** -0.5))
    assert torch.equal(buf[:, :hq * d].cpu(), q.flatten(1))


def test_text_attention_far_rows(dit, ws):
    """Key rows whose byte offsets pass 2^32 and element offsets pass 2^31."""
    hq, hk, d = 4, 1, 64
    ld, rows = 1 << 12, (1 << 20) + 300  # 8.6 GB each
    k = torch.zeros(rows, ld, dtype=torch.bfloat16, device=DEV)
    nk, nq = 300, 200
    kk, vv, q = _randn(nk, hk, d, seed=1), _randn(nk, hk, d, seed=2), _randn(nq, hq, d, seed=3)
    k[rows - nk:, :d] = kk[:, 0].to(DEV)
    k[rows - nk:, d:2 * d] = vv[:, 0].to(DEV)
    out = torch.zeros(nq, hq * d, dtype=torch.bfloat16, device=DEV)
    i32 = lambda t: torch.tensor(t, dtype=torch.int32, device=DEV)  # noqa: E731
    for n in (nq, 1):
        want, size, _ = R.attention(q[:n], kk, vv, [(0, n, 0, nk)], True, d ** -0.5)
        a = dit.make_text_attn(1, hq, hk, d, n, rows, n, nk, causal=True)
        dit.dit_text_attention(a, i32([0, n]), None, i32([rows - nk, rows]), None, q.flatten(1).to(DEV), hq * d, k, ld,
                               k[:, d:], ld, out, hq * d, ws, ws.numel())
        _ok(dit, ws)
        _check_attention(out[:n].reshape(n, hq, d).cpu(), want, size, (q[:n], kk, d ** -0.5))


def test_text_attention_bad_lengths_are_reported_and_skipped(dit, ws):
    hq, hk, d = 2, 1, 128
    q, k = _randn(40, hq * d).to(DEV), _randn(60, d).to(DEV)
    i32 = lambda t: torch.tensor(t, dtype=torch.int32, device=DEV)  # noqa: E731
    good = ([0, 20, 40], [10, 20], [0, 30, 60], [30, 30])
    for which, entry, value in ((0, 1, -1), (0, 1, 21), (0, 1, 2 ** 31 - 1), (1, 1, -1), (1, 1, 21), (2, 1, 31), (2, 1, -5),
                                (3, 1, 31), (3, 1, -2), (3, 1, 2 ** 31 - 1)):
        arr = [list(x) for x in good]
        arr[which][entry] = value
        out = torch.full((40, hq * d), 5.0, dtype=torch.bfloat16, device=DEV)
        a = dit.make_text_attn(2, hq, hk, d, 40, 60, 20, 30, causal=False)
        qo, ql, ko, kl = map(i32, arr)
        dit.dit_text_attention(a, qo, ql, ko, kl, q, hq * d, k, d, k, d, out, hq * d, ws, ws.numel())
        st, where = dit.dit_sync_status(ws)
        assert st == dit.DIT_ERR_INVALID_ARG and where == 0x501, (which, value, st, hex(where))
        assert (out[10:] == 5.0).all() and (out[:10] != 5.0).any()  # the good sequence is done, nothing else written


def test_text_attention_far_rows_in_tiles(dit, ws):
    """Far key rows as above, with enough heads for tiles of 128 rows."""
    hq, hk, d = 32, 8, 64
    ld, rows = 1 << 12, (1 << 20) + 300
    k = torch.zeros(rows, ld, dtype=torch.bfloat16, device=DEV)
    nk, nq = 300, 200
    kk, vv, q = _randn(nk, hk, d, seed=1), _randn(nk, hk, d, seed=2), _randn(nq, hq, d, seed=3)
    k[rows - nk:, :hk * d] = kk.flatten(1).to(DEV)
    k[rows - nk:, hk * d:2 * hk * d] = vv.flatten(1).to(DEV)
    out = torch.zeros(nq, hq * d, dtype=torch.bfloat16, device=DEV)
    i32 = lambda t: torch.tensor(t, dtype=torch.int32, device=DEV)  # noqa: E731
    want, size, _ = R.attention(q, kk, vv, [(0, nq, 0, nk)], True, d ** -0.5)
    a = dit.make_text_attn(1, hq, hk, d, nq, rows, nq, nk, causal=True)
    dit.dit_text_attention(a, i32([0, nq]), None, i32([rows - nk, rows]), None, q.flatten(1).to(DEV), hq * d, k, ld,
                           k[:, hk * d:], ld, out, hq * d, ws, ws.numel())
    _ok(dit, ws)
    _check_attention(out.reshape(nq, hq, d).cpu(), want, size, (q, kk, d ** -0.5))


@pytest.mark.parametrize("seqs", [2, 66])
def test_text_attention_bad_lengths_in_tiles(dit, ws, seqs):
    """Bad entries as above, with enough heads for tiles of 128 rows, and so many sequences that the
    tiles are listed first."""
    hq, hk, d = 128, 64, 64
    q, k = _randn(20 * seqs, hq * d).to(DEV), _randn(30 * seqs, hk * d).to(DEV)
    i32 = lambda t: torch.tensor(t, dtype=torch.int32, device=DEV)  # noqa: E731
    good = ([20 * i for i in range(seqs + 1)], [10] + [20] * (seqs - 1), [30 * i for i in range(seqs + 1)], [30] * seqs)
    for which, value in ((0, -1), (0, 20 * seqs), (1, -1), (1, 21), (2, 30 * seqs - 29), (3, 31), (3, -2)):
        arr = [list(x) for x in good]
        arr[which][seqs - 1] = value
        out = torch.full((20 * seqs, hq * d), 5.0, dtype=torch.bfloat16, device=DEV)
        a = dit.make_text_attn(seqs, hq, hk, d, 20 * seqs, 30 * seqs, 20, 30, causal=False)
        need = dit.dit_text_attention_workspace(a)
        qo, ql, ko, kl = map(i32, arr)
        dit.dit_text_attention(a, qo, ql, ko, kl, q, hq * d, k, hk * d, k, hk * d, out, hq * d, ws, need)
        st, where = dit.dit_sync_status(ws)
        assert st == dit.DIT_ERR_INVALID_ARG and where == 0x501, (which, value, st, hex(where))
        last = 20 * (seqs - 1)
        assert (out[last:] == 5.0).all() and (out[:10] != 5.0).any()  # the bad sequence is left, the others done
        assert (out[10:20] == 5.0).all() and (seqs == 2 or (out[20:last] != 5.0).any(1).all())


# ------------------------------------------------------------------------------ block-scaled e4m3
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols", [(1, 16), (5, 128), (127, 144), (129, 400), (300, 4096), (128, 2560), (1000, 1008)])
def test_quantize_blocks_bit_exact(dit, block_rows, rows, cols):
    x = _randn(rows, cols, seed=rows + cols)
    x[0] *= 1e-30
    if rows > 4:
        x[1] = 0
        x[2] *= 1e30
        x[3, :16] = 1.1e-38
        x[4, 3] = math.nan
    ld = cols + 24
    xd = torch.full((rows, ld), 1e38, dtype=torch.bfloat16, device=DEV)
    xd[:, :cols] = x.to(DEV)
    rb, cb = -(-rows // block_rows), -(-cols // 128)
    q = torch.full((rows * cols + 64,), 77, dtype=torch.uint8, device=DEV)
    sc = torch.full((rb * cb + 16,), 7.0, device=DEV)
    dit.dit_quantize_blocks_fp8(xd, ld, rows, cols, block_rows, q, sc)
    torch.cuda.synchronize()
    codes, scale = R.quantize_blocks(x, block_rows)
    assert torch.equal(sc[:rb * cb].cpu().view(rb, cb), scale)
    got = q[:rows * cols].view(rows, cols).cpu()
    nan = x.isnan()
    assert torch.equal(got[~nan], codes[~nan]) and ((got[nan] & 127) == 127).all()
    assert (q[rows * cols:] == 77).all() and (sc[rb * cb:] == 7.0).all()


@pytest.mark.parametrize("m,n,k", [(1, 8, 16), (1, 4096, 2560), (2, 136, 272), (16, 1000, 1008), (17, 264, 144), (64, 128, 128),
                                   (65, 512, 640), (127, 2568, 400), (128, 256, 256), (129, 520, 384), (300, 256, 4096),
                                   (257, 1288, 1296), (1777, 2568, 2064), (3, 8, 20000), (513, 128, 16), (40, 3000, 512), (489, 1168, 9616), (65, 8, 2048), (1567, 408, 5120)])
def test_linear_fp8_blocks(dit, ws, m, n, k):
    x, w = _randn(m, k, seed=1), _randn(n, k, seed=2, std=0.05)
    x[:, :min(k, 40)] *= 30  # blocks of unlike scales
    w[:, -min(k, 100):] *= 8
    aq, asc = R.quantize_blocks(x, 1)
    wq, wsc = R.quantize_blocks(w, 128)
    ld = n + 16
    out = torch.full((m + 1, ld), 5.0, dtype=torch.bfloat16, device=DEV)
    need = dit.dit_linear_fp8_blocks_workspace(m, n, k)
    assert need <= ws.numel()
    args = [t.to(DEV) for t in (aq, asc, wq, wsc)]
    dit.dit_linear_fp8_blocks(m, n, k, *args, out, ld, ws, need)
    _ok(dit, ws)
    first = out.clone()
    dit.dit_linear_fp8_blocks(m, n, k, *args, out, ld, ws, need)
    _ok(dit, ws)
    assert torch.equal(first, out)
    if m * n * k < 1e9:
        want, size = R.linear_blocks(aq, asc, wq, wsc)
    else:
        a, b = (R.dequantize(q, s, r).to(DEV) for q, s, r in ((aq, asc, 1), (wq, wsc, 128)))
        want, size = (a @ b.t()).cpu(), (a.abs() @ b.abs().t()).cpu()
    # products of e4m3 values are exact in fp32; a block sums 128 of them and the blocks add up,
    # each addition and scaling off by at most 2^-23 (truncation) of the sum of magnitudes
    tol = 2.0 ** -8 * want.abs() + (128 + 2 + -(-k // 128)) * 2.0 ** -23 * size + 1e-30
    _within(out[:m, :n], want, tol)
    assert (out[:m, n:] == 5.0).all() and (out[m:] == 5.0).all()


def test_linear_fp8_blocks_nan_stays_in_its_row(dit, ws):
    m, n, k = 130, 128, 256
    x, w = _randn(m, k, seed=1), _randn(n, k, seed=2)
    x[5, 9] = math.nan
    xd = x.to(DEV)
    aq, asc = torch.empty(m, k, dtype=torch.uint8, device=DEV), torch.empty(m, 2, device=DEV)
    dit.dit_quantize_blocks_fp8(xd, k, m, k, 1, aq, asc)
    wq, wsc = (t.to(DEV) for t in R.quantize_blocks(w, 128))
    out = torch.empty(m, n, dtype=torch.bfloat16, device=DEV)
    dit.dit_linear_fp8_blocks(m, n, k, aq, asc, wq, wsc, out, n, ws, ws.numel())
    _ok(dit, ws)
    assert out[5].isnan().all() and out[[i for i in range(m) if i != 5]].isfinite().all()


# --------------------------------------------------------------------------- a run of them together
class Layer:
    """The attention half of one encoder layer on packed prompts: e4m3 projection to queries,
    keys and values, their norms and rotation in place, attention, e4m3 projection back."""

    def __init__(self, dit, lens, hidden=512, hq=8, hk=2, d=128, seed=0):
        self.dit, self.lens, self.hidden, self.hq, self.hk, self.d = dit, lens, hidden, hq, hk, d
        self.rows = sum(lens)
        self.wide = (hq + 2 * hk) * d
        self.w_in, self.w_out = _randn(self.wide, hidden, seed=seed + 1, std=0.05), _randn(hidden, hq * d, seed=seed + 2, std=0.05)
        self.nq, self.nk = _randn(d, seed=seed + 3, std=0.1) + 1, _randn(d, seed=seed + 4, std=0.1) + 1
        self.q_in, self.q_out = (self._weight(w) for w in (self.w_in, self.w_out))
        self.norms = [t.to(DEV) for t in (self.nq, self.nk)]
        self.off = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)
        self.pos = torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]).to(DEV)
        self.table = torch.empty(max(lens), d // 2, 2, device=DEV)
        dit.dit_text_rope_table(dit.make_text_rope(d, 1e6), None, max(lens), self.table)
        self.x = torch.zeros(self.rows, hidden, dtype=torch.bfloat16, device=DEV)
        e = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t, device=DEV)  # noqa: E731
        self.a8, self.a_s = e(self.rows, hidden, t=torch.uint8), e(self.rows, -(-hidden // 128), t=torch.float32)
        self.b8, self.b_s = e(self.rows, hq * d, t=torch.uint8), e(self.rows, -(-hq * d // 128), t=torch.float32)
        self.raw, self.qkv, self.ctx, self.y = e(self.rows, self.wide), e(self.rows, self.wide), e(self.rows, hq * d), e(self.rows, hidden)
        self.attn = dit.make_text_attn(len(lens), hq, hk, d, self.rows, self.rows, max(lens), max(lens))
        need = max(dit.dit_text_attention_workspace(self.attn), dit.dit_linear_fp8_blocks_workspace(self.rows, self.wide, hidden),
                   dit.dit_linear_fp8_blocks_workspace(self.rows, hidden, hq * d))
        self.ws = torch.zeros(need, dtype=torch.uint8, device=DEV)

    def _weight(self, w):
        n, k = w.shape
        q = torch.empty(n, k, dtype=torch.uint8, device=DEV)
        s = torch.empty(-(-n // 128), -(-k // 128), device=DEV)
        self.dit.dit_quantize_blocks_fp8(w.to(DEV), k, n, k, 128, q, s)
        torch.cuda.synchronize()
        return q, s

    def __call__(self):
        dit, d, hq, hk, n = self.dit, self.d, self.hq, self.hk, self.ws.numel()
        dit.dit_quantize_blocks_fp8(self.x, self.hidden, self.rows, self.hidden, 1, self.a8, self.a_s)
        dit.dit_linear_fp8_blocks(self.rows, self.wide, self.hidden, self.a8, self.a_s, *self.q_in, self.qkv, self.wide, self.ws, n)
        self.raw.copy_(self.qkv)
        q, k, v, w = self.qkv, self.qkv[:, hq * d:], self.qkv[:, (hq + hk) * d:], self.wide
        dit.dit_qk_norm_rope(self.rows, hq, hk, d, d, dit.DIT_ROPE_HALF, q, w, k, w, *self.norms, 1e-6, self.table,
                             self.table.shape[0], self.pos, q, w, k, w, self.ws, n)
        dit.dit_text_attention(self.attn, self.off, None, self.off, None, q, w, k, w, v, w, self.ctx, hq * d, self.ws, n)
        dit.dit_quantize_blocks_fp8(self.ctx, hq * d, self.rows, hq * d, 1, self.b8, self.b_s)
        dit.dit_linear_fp8_blocks(self.rows, self.hidden, hq * d, self.b8, self.b_s, *self.q_out, self.y, self.hidden, self.ws, n)

    def check(self):
        """Each stage against the 64-bit form of its formula on what the stage before it wrote."""
        _ok(self.dit, self.ws)
        d, hq, hk, rows = self.d, self.hq, self.hk, self.rows
        c = lambda t: t.cpu()  # noqa: E731
        lin_tol = lambda want, size, k: 2.0 ** -8 * want.abs() + (130 + -(-k // 128)) * 2.0 ** -23 * size  # noqa: E731
        for x, a8, a_s, (wq, wsc), w, y in ((self.x, self.a8, self.a_s, self.q_in, self.w_in, self.raw),
                                            (self.ctx, self.b8, self.b_s, self.q_out, self.w_out, self.y)):
            codes, scale = R.quantize_blocks(c(x), 1)
            assert torch.equal(codes, c(a8)) and torch.equal(scale, c(a_s))
            wc, wscale = R.quantize_blocks(w, 128)
            assert torch.equal(wc, c(wq)) and torch.equal(wscale, c(wsc))
            want, size = R.linear_blocks(codes, scale, wc, wscale)
            _within(y, want, lin_tol(want, size, w.shape[1]))
        raw, qkv = c(self.raw), c(self.qkv)
        table = c(self.table)[c(self.pos).long()]
        for a, h, w in ((0, hq, self.nq), (hq * d, hk, self.nk)):
            want, size = R.qk_norm_rope(raw[:, a:a + h * d].reshape(rows, h, d), w, float(np.float32(1e-6)), table, d, "half")
            _within(qkv[:, a:a + h * d].reshape(rows, h, d), want, 2.0 ** -8 * want.abs() + 16 * 2.0 ** -24 * size)
        assert torch.equal(qkv[:, (hq + hk) * d:], raw[:, (hq + hk) * d:])
        o = c(self.off).tolist()
        spans = [(o[i], n, o[i], n) for i, n in enumerate(self.lens)]
        q, k, v = qkv[:, :hq * d].reshape(rows, hq, d), qkv[:, hq * d:(hq + hk) * d].reshape(rows, hk, d), qkv[:, (hq + hk) * d:].reshape(rows, hk, d)
        want, size, _ = R.attention(q, k, v, spans, True, float(np.float32(d ** -0.5)))
        _check_attention(c(self.ctx).reshape(rows, hq, d), want, size, (q, k, d ** -0.5))


@pytest.mark.parametrize("lens", [[1], [77, 1, 300, 40]])
def test_encoder_layer(dit, lens):
    layer = Layer(dit, lens)
    layer.x.copy_(_randn(layer.rows, layer.hidden, seed=9))
    layer()
    layer.check()


def test_encoder_layer_captured_and_replayed(dit):
    """One graph of the whole run, replayed on new inputs, other lengths and another stream;
    a second graph of another layer, with a workspace of its own, replayed at the same time."""
    layers = [Layer(dit, [77, 1, 300, 40]), Layer(dit, [200, 150], seed=50)]
    graphs = []
    side = torch.cuda.Stream()
    for layer in layers:
        layer.x.copy_(_randn(layer.rows, layer.hidden, seed=9))
        with torch.cuda.stream(side):
            layer()
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            layer()
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for lens in ([77, 1, 300, 40], [1, 290, 120, 7]):
        a = layers[0]
        a.lens = lens
        a.off.copy_(torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32))
        a.pos[:sum(lens)].copy_(torch.cat([torch.arange(n, dtype=torch.int32) for n in lens]))
        for layer in layers:
            layer.x.copy_(_randn(layer.rows, layer.hidden, seed=sum(lens)))
            layer.y.zero_()
        torch.cuda.synchronize()
        for _ in range(3):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for layer in layers:
            layer.check()


def test_encoder_layer_two_host_threads(dit):
    """Two layers on two streams from two threads at once give the bits of one at a time."""
    import threading
    layers = [Layer(dit, [200, 90]), Layer(dit, [1, 130, 60], seed=30)]
    want = []
    for layer in layers:
        layer.x.copy_(_randn(layer.rows, layer.hidden, seed=5))
        layer()
        torch.cuda.synchronize()
        want.append(layer.y.clone())

    def work(layer):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(10):
                layer()
            torch.cuda.current_stream().synchronize()
    threads = [threading.Thread(target=work, args=(layer,)) for layer in layers]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    for layer, w in zip(layers, want):
        assert torch.equal(layer.y, w)
        layer.check()
