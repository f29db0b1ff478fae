"""The tolerance that the attention tests on the GPU use (text_reference.attention_bound) against the kernels'
arithmetic restated on the CPU: it lets that pass and slips of one key fail, and nothing that a row does not
see widens it."""
import math

import pytest
import torch

import text_reference as R

SPANS = [(1, 64, 2, 64), (66, 65, 70, 65), (132, 1, 140, 130)]
ROWS_Q, ROWS_K = 134, 275


def _inputs(fill=None, seed=0, d=128):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn(n, h, d, generator=g).to(torch.bfloat16) for n, h in ((ROWS_Q, 4), (ROWS_K, 2), (ROWS_K, 2)))
    if fill is not None:
        own = torch.zeros(ROWS_K, dtype=torch.bool)
        for _, _, b, n in SPANS:
            own[b:b + n] = True
        k[~own] = fill
        v[~own] = fill
    return q, k, v


def _restated(q, k, v, causal, scale, slip=None):
    """fp32 scores and statistics, probabilities rounded to bf16, one rounding of the output."""
    out = torch.full(q.shape, 5.0, dtype=torch.bfloat16)
    for q0, nq, k0, nk in SPANS:
        for i in range(nq):
            n = min(nk, i + nk - nq + 1) if causal else nk
            n += {"one key more": 1, "one key less": -1}.get(slip, 0)
            for h in range(q.shape[1]):
                kk, vv = k[k0:k0 + n, h // 2].float(), v[k0:k0 + n, h // 2].float()
                x = (kk @ q[q0 + i, h].float()) * scale
                if slip == "first key twice" and n > 1:
                    x[1], vv = x[0], torch.cat([vv[:1], vv[:1], vv[2:]])
                if n <= 0:
                    out[q0 + i, h] = 0
                    continue
                p = torch.exp(x - x.max())
                out[q0 + i, h] = ((p.to(torch.bfloat16).float() @ vv) / p.sum()).to(torch.bfloat16)
    return out


def _fits(got, bound):
    want, tol, bad, owned = bound
    fin = got.isfinite()
    if not torch.equal(fin[owned], ~bad[owned]):
        return False
    err = (torch.where(bad, torch.zeros_like(got), got).double() - want).abs()
    return bool((err <= tol)[owned].all())


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("fill", [None, math.nan, math.inf, -math.inf, 3.3e38])
def test_the_bar_holds_the_kernels_arithmetic_and_no_slip(causal, fill):
    q, k, v = _inputs(fill)
    scale = 128 ** -0.5
    bound = R.attention_bound(q, k, v, SPANS, causal, scale)
    assert (bound[1][bound[3]] < 0.05).all()  # sums of values of size 1: what lies behind the keys widens nothing
    assert _fits(_restated(q, k, v, causal, scale), bound)
    for slip in ("one key more", "one key less", "first key twice"):
        assert not _fits(_restated(q, k, v, causal, scale, slip), bound), slip


def test_the_bar_does_not_depend_on_what_is_not_seen():
    want = R.attention_bound(*_inputs(0.0), SPANS, True, 0.1)
    for fill in (math.nan, math.inf, 3.3e38):
        got = R.attention_bound(*_inputs(fill), SPANS, True, 0.1)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_bad_values_are_expected_where_they_are_seen():
    q, k, v = _inputs()
    v[2 + 40, 1, 9] = math.inf
    want, tol, bad, owned = R.attention_bound(q, k, v, SPANS, True, 0.1)
    rows = torch.zeros(ROWS_Q, dtype=torch.bool)
    rows[1 + 40:1 + 64] = True
    assert torch.equal(bad[:, 2, 9], rows) and torch.equal(bad[:, 3, 9], rows) and int(bad.sum()) == 2 * 24
