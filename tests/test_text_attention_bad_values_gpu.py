"""Infinite and NaN values of V that some rows of a tile see and others do not: the rows that do not see them
keep their results, on every path of dit_text_attention and at every length."""
import math

import pytest
import torch

import text_reference as R
from attention_calls import DEV, attend, check, i32, split_tiles_bytes
from test_text_ops_gpu import _randn, dit  # noqa: F401

pytestmark = pytest.mark.gpu


def _qkv(nq, nk, hq, hk, d, seed=0):
    return _randn(nq, hq, d, seed=seed), _randn(nk, hk, d, seed=seed + 1), _randn(nk, hk, d, seed=seed + 2)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("back", [2, 20, 150, 299])
def test_split_tiles(dit, bad, d, back):  # noqa: F811
    """The last 300 of 3366 tokens of three heads on one: tiles of 128 rows, their keys in six parts.  The parts
    of the rows that do not see the value are worked out again, the joined rows with them."""
    q, k, v = _qkv(300, 3366, 3, 1, d)
    v[3366 - back, 0, 3] = bad
    got, ws = attend(dit, q, k, v, [(0, 300, 0, 3366)])
    assert ws == split_tiles_bytes(1, 3, 1, d, 300, 300, 3366)  # the path that this test is for
    check(got, R.attention_bound(q, k, v, [(0, 300, 0, 3366)], True, d ** -0.5))


@pytest.mark.parametrize("hq,hk,d,nq,nk", [
    (32, 8, 128, 300, 300), (32, 8, 128, 1000, 1000), (12, 12, 64, 700, 700), (64, 8, 64, 500, 1111),  # tiles
    (3, 1, 128, 300, 3366),                                                                             # split tiles
    (4, 1, 128, 300, 300), (3, 1, 64, 20, 200), (3, 1, 128, 20, 4000), (5, 1, 128, 40, 7000)])          # rows in sixteens
def test_rows_that_see_some_bad_values_and_not_others(dit, hq, hk, d, nq, nk):  # noqa: F811
    """Bad values close together in different dimensions of one head: a row may see the first and not the
    second, so that it is worked out again and still gets what it sees."""
    q, k, v = _qkv(nq, nk, hq, hk, d, seed=5)
    h = hk - 1
    for i, (back, value) in enumerate(((nq + 3, -math.inf), (nq - 3, math.nan), (nq // 2 + 2, math.inf), (nq // 2, math.nan),
                                       (nq // 2 - 7, -math.inf), (9, math.nan), (2, math.inf), (1, math.nan))):
        v[max(0, nk - back), h, 3 + 5 * i] = value
    spans = [(0, nq, 0, nk)]
    check(attend(dit, q, k, v, spans)[0], R.attention_bound(q, k, v, spans, True, d ** -0.5))


@pytest.mark.parametrize("hq,hk,d", [(32, 8, 128), (6, 6, 64)])
def test_a_bad_value_in_every_tile(dit, hq, hk, d):  # noqa: F811
    q, k, v = _qkv(1500, 1500, hq, hk, d, seed=3)
    for t, j in enumerate(range(40, 1500, 61)):
        v[j, :, t % d] = math.nan
    spans = [(0, 700, 0, 700), (700, 800, 700, 800)]
    check(attend(dit, q, k, v, spans)[0], R.attention_bound(q, k, v, spans, True, d ** -0.5))


def test_values_that_are_all_nan(dit):  # noqa: F811
    """Every row sees a NaN in every dimension; the other key heads do not notice."""
    for n in (40, 900):
        q, k, v = _qkv(n, n, 32, 8, 128, seed=7)
        v[:, 2] = math.nan
        check(attend(dit, q, k, v, [(0, n, 0, n)])[0], R.attention_bound(q, k, v, [(0, n, 0, n)], True, 128 ** -0.5))


@pytest.mark.parametrize("seqs", [1, 64, 72])
def test_more_bad_rows_than_a_block_notes_down(dit, seqs):  # noqa: F811
    """4096 work items or more with a bad value each, 27 to a CTA, more than it takes before it repairs rows
    and goes on: of one sequence, of as many as one warp searches, and of more, whose tiles are listed first.
    Against the same call on values that are all finite, and the size of the sums from |v|."""
    n, h, d = 16384 if seqs == 1 else 256 * seqs, 64, 64
    g = torch.Generator(device=DEV).manual_seed(1)
    q, k, v = (torch.randn(n, h * d, generator=g, device=DEV).to(torch.bfloat16) for _ in range(3))
    dirty = v.clone().view(n, h, d)
    t = torch.arange(n // 256, device=DEV)
    dirty[256 * t + 200, :, t % d] = math.nan
    a = dit.make_text_attn(seqs, h, h, d, n, n, n // seqs, n // seqs)
    ws = torch.zeros(dit.dit_text_attention_workspace(a), dtype=torch.uint8, device=DEV)
    off = i32([i * (n // seqs) for i in range(seqs + 1)])

    def run(values):
        out = torch.full_like(q, 5.0)
        dit.dit_text_attention(a, off, None, off, None, q, h * d, k, h * d, values, h * d, out, h * d, ws, ws.numel())
        assert dit.dit_sync_status(ws)[0] == dit.DIT_OK
        return out.view(n, h, d)
    got, want, size = run(dirty.view(n, h * d)), run(v), run(v.abs())
    sees = torch.zeros(n, 1, d, dtype=torch.bool, device=DEV)
    for i in t.tolist():  # the value of tokens 256 i + 200, dimension i mod d, and the rows of its sequence behind it
        sees[256 * i + 200:(256 * i // (n // seqs) + 1) * (n // seqs), 0, i % d] = True
    assert torch.equal(got.isnan(), sees.expand(n, h, d))
    # both sides: probabilities and outputs rounded to bf16, sums of up to 16384 terms and the error of a
    # score (64 products, |q| |k| scale <= 20) in fp32; `size` itself within 2 %
    tol = 2 * ((2.0 ** -8 + 2 * 68 * 2.0 ** -23 * 20 + n * 2.0 ** -23) * 1.02 * size.float() + 2.0 ** -8 * want.float().abs())
    err = (torch.where(sees, torch.zeros_like(got), got).float() - torch.where(sees, torch.zeros_like(want), want).float()).abs()
    assert (err <= tol).all(), float((err / tol).max())


def test_a_bad_value_at_the_end_of_a_long_sequence(dit):  # noqa: F811
    """262144 tokens, one NaN twenty before the end: the rows before it are worked out again over all their
    keys, which takes longer than the kernel's roles may wait for one another if they did meanwhile."""
    n, d = 1 << 18, 64
    q, k, v = _qkv(n, n, 1, 1, d, seed=11)
    v[n - 20, 0, 7] = math.nan
    got, _ = attend(dit, q, k, v, [(0, n, 0, n)])
    assert got[:n - 20].isfinite().all() and got[n - 20:, 0, 7].isnan().all()
    for first in (n - 256, n - 48):
        m = 32
        rows = [(0, m, 0, first + m)]
        check(got[first:first + m], R.attention_bound(q[first:first + m], k[:first + m], v[:first + m], rows, True, d ** -0.5))


@pytest.mark.parametrize("hq,hk,d,n", [(32, 8, 128, 700), (4, 1, 64, 60), (3, 1, 128, 300)])
def test_every_row_sees_every_value_without_a_mask(dit, hq, hk, d, n):  # noqa: F811
    nk = 3366 if hq == 3 else n
    q, k, v = _qkv(n, nk, hq, hk, d, seed=9)
    v[5, hk - 1, 3], v[nk - 1, 0, 7], v[nk // 2] = math.nan, -math.inf, math.nan if hq == 3 else 1.0
    spans = [(0, n, 0, nk)]
    check(attend(dit, q, k, v, spans, causal=False)[0], R.attention_bound(q, k, v, spans, False, d ** -0.5))


@pytest.mark.parametrize("hq,hk,d,nq,nk", [(32, 8, 128, 700, 700), (4, 1, 64, 60, 60), (3, 1, 128, 300, 3366), (8, 8, 128, 1, 9000)])
@pytest.mark.parametrize("causal", [True, False])
def test_large_values_do_not_overflow_the_sums(dit, causal, hq, hk, d, nq, nk):  # noqa: F811
    """Up to 2^98, as documented: the sums of probabilities times values are divided at the end."""
    q, k, v = _qkv(nq, nk, hq, hk, d, seed=13)
    v = (v.float().clamp(-4, 4) * 2.0 ** 96).to(torch.bfloat16)
    spans = [(0, nq, 0, nk)]
    check(attend(dit, q, k, v, spans, causal)[0], R.attention_bound(q, k, v, spans, causal, d ** -0.5))
