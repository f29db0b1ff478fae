"""Attention over the 4-bit cache where the values that a row sees lie as far apart as scales may, with scores alike: keys whose
values all but vanish keep their part of the sum of probabilities."""
import numpy as np
import pytest

from test_text_layer_gpu import Setup, _check_attention, dit, ws  # noqa: F401
from test_text_layer_limits_gpu import _set_exponents

pytestmark = pytest.mark.gpu


def _exponents(kind, n):
    """One exponent per key: small ones before large ones, behind them, in turns by the 32 keys of a warp, one large key alone."""
    pos = np.arange(n)
    large = {"rise": pos >= n // 2, "fall": pos < n // 2, "warps": pos // 32 % 4 == 2, "last": pos == n - 1, "first": pos == 0,
             "blocks": pos // 128 % 2 == 1}[kind]
    return np.where(large, 95, -60)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", ["rise", "fall", "warps", "blocks", "last", "first"])
@pytest.mark.parametrize("hq,page,lens,bound", [
    (4, 32, [300], 0),               # one CTA
    (4, 64, [2000], 0),              # a cluster
    (12, 16, [1500], 0),
    (4, 64, [6000, 700], 0),         # runs and a second kernel
    (4, 64, [5000, 700], 1 << 20),   # even shares
    (12, 32, [3000, 130], 1 << 20)])
def test_scales_far_apart(dit, ws, d, kind, hq, page, lens, bound):
    st = Setup(dit, 1, d, page, lens, seed=3)
    st.fill_random(21)
    exps = np.zeros(st.scales(False).shape, np.int64)
    for s, n in enumerate(lens):
        e = _exponents(kind, n)
        for pos in range(n):
            exps[st.table[s][pos // page], :, pos % page] = e[pos]
    _set_exponents(st, False, exps)
    st.max_pages = max(st.max_pages, bound // page)
    st.c = dit.make_text_cache4(1, d, st.ref.pages, page, st.max_pages)
    _check_attention(dit, ws, st, hq, [1] * len(lens), seed=d, max_k=max(bound, max(lens)))
    # all keys alike: the large ones' values, divided by the number of all keys
    _check_attention(dit, ws, st, hq, [1] * len(lens), seed=d, std=0.0, max_k=max(bound, max(lens)))
