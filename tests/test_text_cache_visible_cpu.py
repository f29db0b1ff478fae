"""The inputs that make every block of a long cache visible, against slips planted in what they give, and against the 64-bit
softmax over the same bytes."""
import numpy as np
import pytest
import torch

import text_cache_visible as V
import text_layer_reference as R

SIZES = [(64, 9000), (64, 9999), (64, 33000), (128, 4000), (128, 20000), (128, 30000), (128, 33000)]


@pytest.mark.parametrize("d,n", SIZES)
def test_a_missing_or_doubled_block_passes_the_bar(d, n):
    """Every block of 128 keys, every warp's 32 of one and every sixteen, lost, or counted twice."""
    want = V.uniform(n, d, 1)
    tol = V.uniform_tolerance(want)
    for size in (128, 32, 16):
        for at in range(0, n, size * max(1, n // size // 300)):
            for times in (0.0, 2.0):
                w = np.ones(n)
                w[at:at + size] = times
                if at + size <= n:
                    assert ((V.uniform(n, d, 1, w) - want).abs() > 3 * tol).any(), (size, at, times)


@pytest.mark.parametrize("d,n", SIZES)
def test_slips_of_whole_pieces_pass_the_bar(d, n):
    """Two parts joined with weights that stand a tenth of a power of two apart, a head's values under its neighbour."""
    want = V.uniform(n, d, 1)
    tol = V.uniform_tolerance(want)
    for cut in (1000, n // 2, n - 200):
        w = np.ones(n)
        w[:cut] = 2.0 ** 0.1
        assert ((V.uniform(n, d, 1, w) - want).abs() > tol).any()
    assert ((V.uniform(n, d, 2) - want).abs() > 3 * tol).any()


class _Setup:
    def __init__(self, heads, d, page, lens):
        self.lens = lens
        need = [-(-n // page) for n in lens]
        order = np.random.default_rng(0).permutation(sum(need) + 1).tolist()
        self.table = []
        for n in need:
            self.table.append(order[:n])
            order = order[n:]
        self.ref = R.Cache(heads, d, sum(need) + 1, page)

    def scales(self, key):
        r = self.ref
        at = (0 if key else r.half) + r.page * r.d // 2
        return r.raw[:, :, at:at + r.page * r.d // 16].view(np.int16).reshape(r.pages, r.heads, r.page, r.d // 32)


@pytest.mark.parametrize("d,page", [(64, 16), (128, 64)])
def test_the_written_values_are_those(d, page):
    """The bytes read by the value-by-value reader, and the softmax over them."""
    st = _Setup(2, d, page, [200, 37])
    st.ref.raw[:] = 0x39  # keys: any finite codes and scales
    V.write_uniform(st)
    for s, n in enumerate(st.lens):
        v = st.ref.values(st.table[s], False)[:n]
        for h in range(2):
            want = torch.zeros(n, d, dtype=torch.float64)
            dim, value = (torch.from_numpy(x) for x in V.dims_of(n, d, h))
            want[torch.arange(n), dim] = value.double()
            assert torch.equal(v[:, h], want)
    q = torch.zeros(4, 4, d).bfloat16()
    out, _, bad, owned = R.cache_attention(q, [(0, 3, 200), (3, 1, 37)], True, 0.1, st.ref, st.table)
    want, _ = V.uniform_rows(st.lens, [3, 1], d, 2, 2)
    assert not bad.any() and owned.all()
    torch.testing.assert_close(out, want, rtol=1e-12, atol=1e-12)
