"""The product with bias, activation and residual on small whole numbers, where every sum is exact in fp32 whatever its order:
outputs equal the 64-bit ones bit for bit, and every 64-deep block of depth shows in them.

With random operands the bound of an fp32 sum passes the outputs themselves from some ten thousand columns of depth on; here a block
that is lost, read twice or read from its neighbour changes an output by whole numbers."""
import math

import pytest
import torch

import text_layer_reference as R
from test_text_layer_gpu import DEV, _ok, dit, ws  # noqa: F401

pytestmark = pytest.mark.gpu


def _whole(rows, cols, most, g):
    return torch.randint(-most, most + 1, (rows, cols), generator=g, device=DEV, dtype=torch.int32).to(torch.bfloat16)


def _operands(m, n, k, pad, seed):
    """a and w of -3 .. 3 (a's first row to 4), NaN behind their rows. Partial sums stay within 12 k <= 12 * 2^20 < 2^24. In the
    first column of each 64-deep block w is 1, so that a's first row can be moved where a block adds nothing to out[0, 0]."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    a, w = (torch.full((r, k + p), math.nan, dtype=torch.bfloat16, device=DEV) for r, p in ((m, pad), (n, 2 * pad)))
    a[:, :k], w[:, :k] = _whole(m, k, 3, g), _whole(n, k, 3, g)
    w[:, :k:64] = 1
    first = torch.nn.functional.pad(a[0, :k].double() * w[0, :k].double(), (0, -k % 64)).view(-1, 64).sum(-1)
    a[0, :k:64] += (first == 0).to(torch.bfloat16)
    first = torch.nn.functional.pad(a[0, :k].double() * w[0, :k].double(), (0, -k % 64)).view(-1, 64).sum(-1)
    assert bool((first != 0).all()) and float(a[:, :k].abs().max()) <= 4 and 12 * k + 64 < 1 << 24
    return a, w, g


def _check(dit, ws, m, n, k, pad=0, bias=True, res=True, act="none", seed=0):
    a, w, g = _operands(m, n, k, pad, seed)
    ld = n + -n % 8 + pad
    b = _whole(1, n, 9, g)[0].contiguous() if bias else None
    r = _whole(m, ld, 9, g) if res else None
    z = a[:, :k].double() @ w[:, :k].double().t() + (b.double() if bias else 0.0)
    want = (z.clamp(min=0.0) if act == "relu" else z) + (r[:, :n].double() if res else 0.0)
    for f32 in (True, False):
        out = torch.full((m + 1, ld), 0.5, dtype=torch.float32 if f32 else torch.bfloat16, device=DEV)
        dit.dit_linear_act(m, n, k, a, k + pad, w, k + 2 * pad, b, R.ACTS.index(act), r, ld if res else 0, out, ld, f32, ws, ws.numel())
        _ok(dit, ws)
        # fp32 holds the sums; bf16 is their one rounding
        exact = want.float() if f32 else want.float().to(torch.bfloat16)
        wrong = out[:m, :n] != exact
        assert not bool(wrong.any()), (f32, int(wrong.sum()), wrong.nonzero()[:4].tolist())
        assert bool((out[m] == 0.5).all()) and bool((out[:m, n:] == 0.5).all())


@pytest.mark.parametrize("m,n,k", [(8, 8, 1 << 20), (300, 9, 1 << 19), (1, 1, 100000), (1, 1, 1 << 20), (40, 130, 1 << 18), (100, 9, 1 << 19),
                                   (130, 257, 1 << 17), (200, 100, 100000), (255, 9, 20008), (520, 260, 65544)])
def test_deep_products(dit, ws, m, n, k):
    """Rings that wrap around thousands of times, splits of the depth whose parts are joined, a last block of eight columns."""
    _check(dit, ws, m, n, k, seed=m)
    if k % 64:
        _check(dit, ws, m, n, k, pad=8, seed=n)


@pytest.mark.parametrize("m", [1, 16, 17, 32, 33, 64, 65, 128, 129, 256, 300, 777])
@pytest.mark.parametrize("n,k,pad", [(130, 8192, 0), (2560, 4096, 0), (1000, 2568, 8), (4095, 1032, 0), (12288, 520, 8)])
def test_every_split(dit, ws, m, n, k, pad):
    """Both kernels with one to eight splits, tiles of 128, 192 and 256 columns, rows on their lines and off them."""
    _check(dit, ws, m, n, k, pad, seed=m + n)


@pytest.mark.parametrize("m,n,k", [(2000, 3001, 264), (4100, 1160, 520), (1 << 20, 8, 8), (1, 1 << 20, 8), (130, 1 << 18, 16)])
def test_many_tiles_and_longest_sides(dit, ws, m, n, k):
    for bias, res, act in ((True, True, "relu"), (False, False, "none"), (True, False, "none"), (False, True, "relu")):
        _check(dit, ws, m, n, k, 0, bias, res, act, seed=k)


@pytest.mark.parametrize("m", [3, 100, 130, 600])
def test_extreme_values_in_every_row_and_column(dit, ws, m):
    """Pre-activations far out on both sides, infinite and NaN, seventeen times over the columns, so that whole pieces of 32 and
    the last single columns both have them: the limits of the activations, the same bits in every row."""
    k, times = 64, 17
    z = torch.tensor([0.0, -0.0, 90.0, -90.0, 1e4, -1e4, 3e38, -3e38, math.inf, -math.inf, math.nan, 12.0, -12.0, 0.5, -0.5, 1e-30])
    b = z.bfloat16().repeat(times)
    n = len(b)
    a, w, bd = torch.zeros(m, k, dtype=torch.bfloat16, device=DEV), torch.zeros(n, k, dtype=torch.bfloat16, device=DEV), b.to(DEV)
    x = b.double()
    fin = x.isfinite()
    for act in R.ACTS:
        want = R.activation(x, act)
        for f32 in (True, False):
            out = torch.full((m, n), 5.0, dtype=torch.float32 if f32 else torch.bfloat16, device=DEV)
            dit.dit_linear_act(m, n, k, a, k, w, k, bd, R.ACTS.index(act), None, 0, out, n, f32, ws, ws.numel())
            _ok(dit, ws)
            bits = out.view(torch.int32 if f32 else torch.int16)
            assert bool((bits == bits[:1]).all()), (act, f32)
            got = out[0].double().cpu()
            # exponential, reciprocal and polynomial within 2^-18; the tail of a probability within 1e-6; a rounding
            tol = (2.0 ** -18 + (0.0 if f32 else 2.0 ** -8)) * want.abs() + 1e-6
            assert bool(((got - want).abs()[fin] <= tol[fin]).all()), (act, f32)
            inf, ninf, nan = (torch.arange(times) * 16 + i for i in (8, 9, 10))
            assert bool((got[inf] == math.inf).all()) and bool(got[nan].isnan().all())
            if act in ("none", "relu"):
                assert bool((got[ninf] == (-math.inf if act == "none" else 0.0)).all())
