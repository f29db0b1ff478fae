"""Attention over the 4-bit cache where queries and scale are so small that the factor of their scores is below any fp32 number."""
import pytest

from test_text_layer_gpu import Setup, _check_attention, dit, ws  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("std,scale", [(2.0 ** -120, 2.0 ** -60), (2.0 ** -118, 1e-30), (2.0 ** -112, 2.0 ** -49), (1.0, 2.0 ** -60),
                                       (2.0 ** -120, 2.0 ** -10)])
def test_scores_that_all_but_vanish(dit, ws, d, std, scale):
    """The smallest queries times the smallest scales, down to factors below any fp32 number: all visible keys weigh the
    same, and what a row does not see stays out of it."""
    st = Setup(dit, 2, d, 16, [100, 33, 8], seed=7)
    st.fill_random(24)
    _check_attention(dit, ws, st, 6, [3, 1, 8], seed=1, std=std, scale=scale)
    _check_attention(dit, ws, st, 6, [3, 1, 8], seed=1, std=std, scale=scale, causal=False)
    st.max_pages = (1 << 19) // 16  # even shares
    st.c = dit.make_text_cache4(2, d, st.ref.pages, 16, st.max_pages)
    _check_attention(dit, ws, st, 4, [2, 1, 1], seed=2, std=std, scale=scale, max_k=1 << 19)
