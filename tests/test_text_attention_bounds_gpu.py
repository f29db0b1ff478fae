"""dit_text_attention against 64 bits with a tolerance of its own for every value, from what that value's row
sees: rows behind the keys, sequences listed first, short and split calls, very low scores, wide bounds."""
import math

import pytest
import torch

import text_reference as R
from attention_calls import attend, check, split_tiles_bytes
from test_text_ops_gpu import _randn, dit  # noqa: F401

pytestmark = pytest.mark.gpu
FILLS = [math.nan, math.inf, -math.inf, 3.3e38]


def _inputs(ql, kl, hq, hk, d, gap_q=0, gap_k=0, fill=None, seed=0):
    """Sequences with rows between, before and behind them, which hold `fill` in k and v and NaN in q."""
    spans, a, b = [], gap_q, gap_k
    for n, m in zip(ql, kl):
        spans.append((a, n, b, m))
        a, b = a + n + gap_q, b + m + gap_k
    q, k, v = _randn(a, hq, d, seed=seed), _randn(b, hk, d, seed=seed + 1), _randn(b, hk, d, seed=seed + 2)
    if fill is not None:
        own_q, own_k = torch.zeros(a, dtype=torch.bool), torch.zeros(b, dtype=torch.bool)
        for q0, n, k0, m in spans:
            own_q[q0:q0 + n] = True
            own_k[k0:k0 + m] = True
        q[~own_q] = math.nan
        k[~own_k] = fill
        v[~own_k] = fill
    return q, k, v, spans


def _held(dit, q, k, v, spans, causal=True, scale=None, exact=False):  # noqa: F811
    scale = q.shape[2] ** -0.5 if scale is None else scale
    got, ws = attend(dit, q, k, v, spans, causal, scale)
    check(got, R.attention_bound(q, k, v, spans, causal, scale, exact))
    return ws


@pytest.mark.parametrize("fill", FILLS)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("ql,kl,hq,hk,d", [
    ([64, 65, 1], [64, 65, 130], 4, 2, 128), ([1, 1, 1], [130, 1, 700], 8, 2, 64),           # sixteen rows at a time
    ([129, 64, 300, 1], [129, 200, 300, 77], 32, 8, 128), ([100, 257], [100, 300], 16, 16, 64)])  # tiles
def test_rows_behind_the_keys(dit, fill, causal, ql, kl, hq, hk, d):  # noqa: F811
    _held(dit, *_inputs(ql, kl, hq, hk, d, 3, 7, fill), causal)


@pytest.mark.parametrize("fill", FILLS)
@pytest.mark.parametrize("d", [64, 128])
def test_rows_behind_the_keys_of_split_tiles(dit, fill, d):  # noqa: F811
    ql, kl = [300, 2], [3366, 1500]
    q, k, v, spans = _inputs(ql, kl, 3, 1, d, 3, 7, fill)
    assert _held(dit, q, k, v, spans) == split_tiles_bytes(2, 3, 1, d, q.shape[0], 300, 3366)


@pytest.mark.parametrize("fill", FILLS)
@pytest.mark.parametrize("seqs", [65, 300])
@pytest.mark.parametrize("hq,hk,d,causal", [(4, 1, 128, True), (3, 3, 64, False), (32, 8, 64, True)])
def test_many_sequences_over_caches(dit, fill, seqs, hq, hk, d, causal):  # noqa: F811
    """More sequences than one warp can search, with fewer queries than keys and rows between them."""
    kl = [0 if i % 7 == 3 else 300 + i % 50 if i % 11 == 0 and i < 200 else 1 + (i * 37) % 40 for i in range(seqs)]
    _held(dit, *_inputs([min(n, 17) for n in kl], kl, hq, hk, d, 1, 1, fill), causal)


@pytest.mark.parametrize("fill", FILLS)
@pytest.mark.parametrize("seqs,n,hq,hk,d,causal", [
    (1, 17, 4, 1, 128, True), (1, 100, 32, 32, 64, False), (1, 77, 32, 8, 128, True), (3, 300, 2, 1, 64, True),
    (2, 40, 8, 2, 128, False), (1, 1200, 2, 2, 64, True), (70, 5, 8, 2, 64, True)])
def test_small_prompts_over_caches(dit, fill, seqs, n, hq, hk, d, causal):  # noqa: F811
    kl = [max(1, n - 3 * i) for i in range(seqs)]
    _held(dit, *_inputs([max(1, x // 2) for x in kl], kl, hq, hk, d, 1, 3, fill), causal)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("ql,kl,hq,hk,d", [
    ([200, 1], [200, 400], 4, 2, 64), ([300, 40], [300, 700], 32, 8, 64), ([300], [3366], 3, 1, 128)])
def test_very_low_scores(dit, ql, kl, hq, hk, d, causal):  # noqa: F811
    """All scores at -2^16 and a little: the maximum, not zero, is what exponentials are taken against.  The
    values are small integers, so that every sum on the way to a score is one that fp32 holds."""
    q, k, v, spans = _inputs(ql, kl, hq, hk, d)
    g = torch.Generator().manual_seed(4)
    q = torch.zeros(q.shape).to(torch.bfloat16)
    k = torch.zeros(k.shape).to(torch.bfloat16)
    q[..., 1:9] = torch.randint(0, 2, (*q.shape[:2], 8), generator=g).to(torch.bfloat16)
    k[..., 1:9] = torch.randint(-1, 2, (*k.shape[:2], 8), generator=g).to(torch.bfloat16)
    q[..., 0], k[..., 0] = -256, 256
    _held(dit, q, k, v, spans, causal, 1.0, exact=True)


@pytest.mark.parametrize("hq,hk,d", [(32, 8, 128), (12, 12, 64)])
@pytest.mark.parametrize("causal", [True, False])
def test_lengths_in_tiles(dit, hq, hk, d, causal):  # noqa: F811
    ql = [129, 1, 0, 64, 300, 65, 7, 250, 31]
    kl = [129, 200, 5, 0, 300, 30, 129, 511, 31]
    _held(dit, *_inputs(ql, kl, hq, hk, d, 2, 2, math.nan), causal)


@pytest.mark.parametrize("hq,hk", [(8, 2), (32, 8)])
def test_bounds_wider_than_the_lengths_change_no_bits(dit, hq, hk):  # noqa: F811
    """max_q and max_k choose how the work is split and nothing else: where the choice is the same, so are
    the bits."""
    d = 128
    q, k, v, spans = _inputs([200, 100], [200, 100], hq, hk, d)
    # eight heads on two: sixteen rows at a time up to 250 tokens; 32 on 8: tiles, at any of these
    bounds = [(200, 200), (240, 250)] if hq == 8 else [(200, 200), (300, 300), (100000, 1 << 24)]
    outs = [attend(dit, q, k, v, spans, max_q=a, max_k=b)[0] for a, b in bounds]
    for o in outs[1:]:
        assert torch.equal(o, outs[0])
    check(outs[0], R.attention_bound(q, k, v, spans, True, d ** -0.5))
