"""The norm with residual, the product with bias, activation and residual, and the 4-bit cache on the GPU, against
64-bit forms of their formulas, through the C ABI.

Tolerances are derived where they are used: a rounding to bf16 is off by at most 2^-8 of the value, one to
fp32 by 2^-24, one to e4m3 by half a step of three bits."""
import math
import threading

import numpy as np
import pytest
import torch

import text_layer_reference as R

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
    return torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)


def _ok(dit, ws, want=None):
    st, where = dit.dit_sync_status(ws)
    if want is None:
        assert st == dit.DIT_OK, (st, hex(where))
    else:
        assert (st, where) == (dit.DIT_ERR_INVALID_ARG, want), (st, hex(where))


def _randn(*shape, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16)


def _within(got, want, tol):
    err = (got.double().cpu() - want).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (int(bad.sum()), float((err / tol).max()), bad.nonzero()[:4].tolist())


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _bits(t):
    return t.cpu().contiguous().view(torch.int16)


# ---------------------------------------------------------------------------------- norm with residual
def _norm_tolerance(y, cols):
    """Relative error of y before its rounding: the squares' sum has cols / 1024 + 32 + 10 additions in a row at most
    and each square a rounding (halved by the root), rsqrt is within 2 units, four roundings follow."""
    return ((cols / 1024 + 43) / 2 + 2 * 2 + 4) * 2.0 ** -24 * y.abs()


def _check_norm(dit, rows, cols, res, w, offset, kind, pad=0, in_place=None, seed=0, x=None):
    x = _randn(rows, cols + pad, seed=seed) if x is None else x
    r = _randn(rows, cols + 2 * pad, seed=seed + 1, std=3.0) if res else None
    wt = (_randn(cols, seed=seed + 2, std=0.3) + (1 - offset)).bfloat16() if w else None
    xd, rd, wd = x.to(DEV), r.to(DEV) if res else None, wt.to(DEV) if w else None
    sd = torch.full((rows, cols + 3 * pad), 7.0, dtype=torch.bfloat16, device=DEV)
    yd = torch.full((rows, cols + pad), 7.0, dtype=torch.bfloat16, device=DEV) if kind != "e4m3" else None
    if in_place == "res":
        sd = rd
    elif in_place == "x":
        sd = xd
    elif in_place == "swap":  # the sum over the residual, the norm over x
        sd, yd = rd, xd if yd is not None else None
    qd = torch.full((rows + 1, cols), 0x55, dtype=torch.uint8, device=DEV) if kind != "bf16" else None
    nb = -(-cols // 128)
    cd = torch.full((rows + 1, nb), 7.0, device=DEV) if kind != "bf16" else None
    ld = lambda t: 0 if t is None else t.stride(0)  # noqa: E731
    dit.dit_add_rms_norm(rows, cols, xd, ld(xd), rd, ld(rd), wd, offset, 1e-6, sd, ld(sd), yd, ld(yd), qd, cd)
    torch.cuda.synchronize()
    xs, rs = x[:, :cols], r[:, :cols] if res else None
    s, y = R.add_rms_norm(xs, rs, wt, offset, float(np.float32(1e-6)))
    # the sum is one fp32 addition, rounded
    want = (xs.float() + (rs.float() if res else 0.0)).bfloat16()
    assert torch.equal(_bits(sd[:, :cols]), _bits(want))
    tol = _norm_tolerance(y, cols)
    if yd is not None:
        _within(yd[:, :cols], y, 2.0 ** -8 * y.abs() + tol * 1.01 + 1e-30)
        if pad and in_place is None:
            assert (yd[:, cols:] == 7.0).all() and (sd[:, cols:] == 7.0).all()
        if in_place == "swap" and pad:
            assert torch.equal(_bits(xd[:, cols:]), _bits(x[:, cols:])) and torch.equal(_bits(rd[:, cols:]), _bits(r[:, cols:]))
    if qd is not None:
        pd = torch.zeros(rows, nb * 128, dtype=torch.float64)
        pd[:, :cols] = y.abs()
        top = pd.view(rows, nb, 128).amax(-1).clamp(min=448 * 2.0 ** -118)
        # maximum, one division
        _within(cd[:rows], top / 448, (top / 448) * ((cols / 1024 + 43) / 2 + 12) * 2.0 ** -24)
        codes = qd[:rows].cpu().view(torch.float8_e4m3fn).double()
        scale = (top / 448).repeat_interleave(128, 1)[:, :cols]
        v = y / scale
        # half a step of three bits, and what the roundings before it move the value by (across a step: half of
        # the larger one)
        slack = ((cols / 1024 + 43) / 2 + 20) * 2.0 ** -24 * v.abs()
        _within(codes, v, R.e4m3_steps(v.abs() + slack) / 2 * (1 + 1e-9) + slack)
        assert (qd[rows] == 0x55).all() and (cd[rows] == 7.0).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "both"])
@pytest.mark.parametrize("rows,cols,res,w,offset,pad", [
    (1, 16, True, True, 0.0, 0), (1, 4096, True, True, 0.0, 0), (7, 2560, True, True, 1.0, 8), (33, 144, False, True, 0.0, 16),
    (5, 32768, True, True, 0.0, 8), (3, 8208, True, False, 0.0, 0), (300, 1040, False, False, 2.0, 24), (19, 16400, True, True, 1.0, 0),
    (2049, 128, True, True, 0.0, 0), (4500, 272, True, True, 0.0, 8)])
def test_add_rms_norm(dit, kind, rows, cols, res, w, offset, pad):
    _check_norm(dit, rows, cols, res, w, offset, kind, pad, seed=rows + cols)


@pytest.mark.parametrize("cols", [8, 24, 1000, 2568, 8200, 32760])
def test_add_rms_norm_columns_of_eights(dit, cols):
    _check_norm(dit, 11, cols, True, True, 0.0, "bf16", 8, seed=cols)


@pytest.mark.parametrize("in_place", ["res", "x", "swap"])
@pytest.mark.parametrize("rows,cols", [(3, 4096), (700, 1032), (1, 20000)])
def test_add_rms_norm_in_place(dit, in_place, rows, cols):
    _check_norm(dit, rows, cols, True, True, 0.0, "bf16", 8, in_place)


def test_add_rms_norm_small_and_large_rows(dit):
    """A row of zeros, one of the smallest numbers, one near the documented bound, NaN and infinity in one row each."""
    x = _randn(6, 512, seed=3)
    x[0] = 0.0
    x[1] *= 2.0 ** -60
    x[2] *= 2.0 ** 53
    x[4, 100], x[5, 7] = math.nan, math.inf
    xd, w = x.to(DEV), torch.ones(512, dtype=torch.bfloat16, device=DEV)
    y, q, sc = torch.empty_like(xd), torch.empty(6, 512, dtype=torch.uint8, device=DEV), torch.empty(6, 4, device=DEV)
    dit.dit_add_rms_norm(6, 512, xd, 512, None, 0, w, 0.0, 1e-6, None, 0, y, 512, q, sc)
    torch.cuda.synchronize()
    _, want = R.add_rms_norm(x, None, None, 0.0, float(np.float32(1e-6)))
    ok = [0, 1, 2, 3]
    _within(y[ok], want[ok], 2.0 ** -8 * want[ok].abs() + _norm_tolerance(want[ok], 512) * 1.01 + 1e-30)
    assert y[4].isnan().all() and y[5, 7].isnan()
    assert (q[0] == 0).all() and (q[4].view(torch.float8_e4m3fn).float().isnan()).all()
    # the scale of a block of zeros is the quantiser's floor, and finite
    assert float(sc[0, 0]) == 2.0 ** -118


def test_add_rms_norm_feeds_the_block_product(dit, ws):
    """Its codes and scales are those of the quantiser on the same values (a power of two as gain and a norm of one
    make y a bf16 number), and the block-scaled product takes them."""
    rows, cols, n = 70, 640, 256
    x = torch.where(_randn(rows, cols, seed=4) > 0, 1.0, -1.0).bfloat16()
    w = torch.ones(cols, dtype=torch.bfloat16, device=DEV) * 2
    xd = x.to(DEV)
    q, sc, y = torch.empty(rows, cols, dtype=torch.uint8, device=DEV), torch.empty(rows, 5, device=DEV), torch.empty_like(xd)
    dit.dit_add_rms_norm(rows, cols, xd, cols, None, 0, w, 0.0, 0.0, None, 0, y, cols, q, sc)
    q2, sc2 = torch.empty_like(q), torch.empty_like(sc)
    dit.dit_quantize_blocks_fp8(y, cols, rows, cols, 1, q2, sc2)
    torch.cuda.synchronize()
    assert torch.equal(q, q2) and torch.equal(sc, sc2)
    wq, wsc = torch.empty(n, cols, dtype=torch.uint8, device=DEV), torch.empty(2, 5, device=DEV)
    wt = _randn(n, cols, seed=5, std=0.05)
    dit.dit_quantize_blocks_fp8(wt.to(DEV), cols, n, cols, 128, wq, wsc)
    out = torch.empty(rows, n, dtype=torch.bfloat16, device=DEV)
    dit.dit_linear_fp8_blocks(rows, n, cols, q, sc, wq, wsc, out, n, ws, ws.numel())
    _ok(dit, ws)
    a = q.cpu().view(torch.float8_e4m3fn).double() * sc.cpu().double().repeat_interleave(128, 1)
    b = wq.cpu().view(torch.float8_e4m3fn).double() * wsc.cpu().double().repeat_interleave(128, 0).repeat_interleave(128, 1)
    want = a @ b.t()
    _within(out, want, 2.0 ** -8 * want.abs() + (cols + 8) * 2.0 ** -23 * (a.abs() @ b.abs().t()))


# -------------------------------------------------------------------- bias, activation, residual
def _check_linear(dit, ws, m, n, k, act, bias, res, f32, in_place=False, pad=0, seed=0):
    a, w = _randn(m, k + pad, seed=seed), _randn(n, k + 2 * pad, seed=seed + 1, std=k ** -0.5)
    b = _randn(n, seed=seed + 2) if bias else None
    ld = n + -n % 8 + pad
    r = _randn(m, ld, seed=seed + 3, std=2.0) if res else None
    dt = torch.float32 if f32 else torch.bfloat16
    od = torch.full((m + 1, ld), 5.0, dtype=dt, device=DEV)
    rd = r.to(DEV) if res else None
    if in_place:
        od[:m] = rd
        rd = od
    ad, wd, bd = a.to(DEV), w.to(DEV), b.to(DEV) if bias else None
    dit.dit_linear_act(m, n, k, ad, k + pad, wd, k + 2 * pad, bd, R.ACTS.index(act), rd, ld if res else 0, od, ld, f32, ws, ws.numel())
    _ok(dit, ws)
    rr = r[:, :n] if res else None
    want, size, z = R.linear_act(a[:, :k], w[:, :k], b, act, rr)
    _within(od[:m, :n], want, R.linear_act_tolerance(want, size, z, k, rr, f32))
    assert (od[m] == 5.0).all()
    if in_place:
        assert torch.equal(_bits(od[:m, n:]), _bits(r[:, n:]))
    else:
        assert (od[:m, n:] == 5.0).all()
    return od


@pytest.mark.parametrize("act", R.ACTS)
@pytest.mark.parametrize("m,n,k,f32", [(1, 1, 8, False), (3, 137, 72, True), (20, 64, 512, False), (70, 300, 264, True), (300, 520, 136, False)])
def test_linear_act_activations(dit, ws, act, m, n, k, f32):
    _check_linear(dit, ws, m, n, k, act, True, True, f32, seed=m)


@pytest.mark.parametrize("bias,res", [(False, False), (True, False), (False, True)])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("m,n,k,pad", [
    (1, 2560, 4096, 0), (1, 1, 100000, 0), (2, 5, 8, 8), (16, 129, 1032, 8), (17, 1000, 2568, 0), (32, 33, 64, 8), (33, 4095, 136, 0),
    (64, 256, 5160, 8), (65, 257, 72, 8), (100, 1, 64, 8), (255, 9, 20008, 0), (256, 256, 128, 0), (257, 513, 520, 8), (777, 130, 2056, 0)])
def test_linear_act_sizes(dit, ws, bias, res, f32, m, n, k, pad):
    _check_linear(dit, ws, m, n, k, "none", bias, res, f32, pad=pad, seed=m + n)


@pytest.mark.parametrize("m,n,k", [(1, 700, 2048), (50, 333, 264), (130, 257, 4096), (1000, 776, 520)])
def test_linear_act_residual_in_place(dit, ws, m, n, k):
    _check_linear(dit, ws, m, n, k, "gelu", True, True, False, in_place=True, pad=8)


@pytest.mark.parametrize("m,n,k,act", [(2000, 3001, 256, "silu"), (4097, 1160, 264, "gelu_tanh"), (8192, 640, 72, "relu")])
def test_linear_act_many_tiles(dit, ws, m, n, k, act):
    """More tiles than the GPU runs at once."""
    _check_linear(dit, ws, m, n, k, act, True, True, False, seed=n)


@pytest.mark.parametrize("m,n,k", [(1, 512, 4096), (40, 1000, 2048), (200, 300, 8192), (1500, 2000, 512)])
def test_linear_act_equal_calls_give_equal_bits(dit, ws, m, n, k):
    one = _check_linear(dit, ws, m, n, k, "silu", True, True, False, seed=9)
    for _ in range(3):
        assert torch.equal(_bits(_check_linear(dit, ws, m, n, k, "silu", True, True, False, seed=9)), _bits(one))


@pytest.mark.parametrize("m", [3, 100, 600])
def test_linear_act_extreme_values(dit, ws, m):
    """Pre-activations far out on both sides, infinite, and NaN: the activations' limits; rows do not mix."""
    k = 64
    z = torch.tensor([0.0, -0.0, 90.0, -90.0, 1e4, -1e4, 3e38, -3e38, math.inf, -math.inf, math.nan, 12.0, -12.0, 0.5, -0.5, 1e-30])
    n = len(z)
    a, w, b = torch.zeros(m, k).bfloat16(), torch.zeros(n, k).bfloat16(), z.bfloat16()
    for act in R.ACTS:
        out = torch.full((m, n), 5.0, device=DEV)
        dit.dit_linear_act(m, n, k, a.to(DEV), k, w.to(DEV), k, b.to(DEV), R.ACTS.index(act), None, 0, out, n, True, ws, ws.numel())
        _ok(dit, ws)
        got, x = out.double().cpu(), b.double()
        want = R.activation(x, act)
        fin = x.isfinite()
        assert torch.equal(got, got[:1].expand_as(got)) or act in R.ACTS and bool((got.isnan() == got[:1].isnan()).all())
        # the underflow of a tail: anything from -1e-6 to 0
        assert ((got[0] - want).abs()[fin] <= 2.0 ** -18 * want.abs()[fin] + 1e-6).all(), (act, got[0], want)
        assert got[0, 10].isnan() and got[0, 8] == math.inf
        assert got[0, 9] == (0.0 if act == "relu" else -math.inf) or act in ("gelu", "gelu_tanh", "silu")
    # an infinite row of a leaves the others finite
    a[1] = math.inf
    w[:] = 1.0
    out = torch.full((m, n), 5.0, device=DEV)
    dit.dit_linear_act(m, n, k, a.to(DEV), k, w.to(DEV), k, None, 0, None, 0, out, n, True, ws, ws.numel())
    _ok(dit, ws)
    assert (out[1] == math.inf).all() and (out[[0, 2]] == 0).all()


# ------------------------------------------------------------------------------------ the 4-bit cache
class Setup:
    """Sequences over a cache with shuffled pages on both sides: the reference's bytes and the GPU's."""

    def __init__(self, dit, heads, d, page, lens, seed=0, spare=2, fill=0xa5):
        self.dit, self.lens = dit, list(lens)
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // page) for n in lens]
        self.max_pages = max(need + [1]) + 1
        pages = sum(need) + spare
        order = torch.randperm(pages, generator=g).tolist()
        self.table = []
        for n in need:
            self.table.append(order[:n])
            order = order[n:]
        self.ref = R.Cache(heads, d, pages, page, fill)
        self.c = dit.make_text_cache4(heads, d, pages, page, self.max_pages)
        assert dit.dit_text_cache4_bytes(self.c) == self.ref.raw.size
        self.dev = torch.full((self.ref.raw.size,), fill, dtype=torch.uint8, device=DEV)

    def table_dev(self, fill=-1):
        return _i32([t + [fill] * (self.max_pages - len(t)) for t in self.table])

    def fill_random(self, seed=0):
        """Every place random codes (1 to 15) and scales, without the append."""
        rng = np.random.default_rng(seed)
        r = self.ref
        codes = rng.integers(1, 16, (2,) + r.raw.shape[:2] + (r.page * r.d,), dtype=np.uint8)
        scales = torch.from_numpy(rng.uniform(0.05, 0.4, (2,) + r.raw.shape[:2] + (r.page * r.d // 32,))).bfloat16()
        for h in range(2):
            at = h * r.half
            r.raw[:, :, at:at + r.page * r.d // 2] = codes[h, ..., 0::2] | (codes[h, ..., 1::2] << 4)
            r.raw[:, :, at + r.page * r.d // 2:at + r.half] = scales[h].view(torch.int16).numpy().view(np.uint8)
        self.upload()

    def upload(self):
        self.dev.copy_(torch.from_numpy(self.ref.raw.reshape(-1)))

    def scales(self, key):
        """A writable view [pages, heads, page, d / 32] of the scales' bits."""
        r = self.ref
        at = (0 if key else r.half) + r.page * r.d // 2
        return r.raw[:, :, at:at + r.page * r.d // 16].view(np.int16).reshape(r.pages, r.heads, r.page, r.d // 32)

    def append(self, ws, rows, q_off, q_len, k_len, k, v, max_q=None, table=None):
        self.dit.dit_text_cache4_append(self.c, len(self.lens), rows, rows if max_q is None else max_q, q_off, q_len, k_len,
                                        self.table_dev() if table is None else table, k, k.stride(0), v, v.stride(0), self.dev, ws,
                                        ws.numel())

    def same(self):
        return torch.equal(self.dev.cpu(), torch.from_numpy(self.ref.raw.reshape(-1)))


@pytest.mark.parametrize("heads,d,page,lens,news", [
    (1, 64, 16, [1], [1]), (2, 128, 16, [1, 16, 17, 40], [1, 16, 1, 23]), (3, 64, 64, [0, 65, 130, 5], [0, 1, 130, 0]),
    (8, 128, 64, [700, 3], [129, 3]), (5, 128, 256, [300, 256, 257], [45, 256, 1]), (1, 64, 128, [129] * 40, [2] * 40)])
def test_cache_append_bit_for_bit(dit, ws, heads, d, page, lens, news):
    """New rows of a fused buffer land in their places as the formula says, and nothing else changes; two calls, the
    second for the tokens after the first's."""
    st = Setup(dit, heads, d, page, lens, seed=page)
    start = [n - a for n, a in zip(lens, news)]
    for part in (0, 1):  # the first half of each sequence's new tokens, then the rest
        count = [a // 2 if part == 0 else a - a // 2 for a in news]
        off = np.concatenate([[3], 3 + np.cumsum(count)])
        rows = int(off[-1]) + 2
        kv = _randn(rows, 2 * heads * d + 8, seed=part, std=2.0)
        kv[rows // 2] *= 2.0 ** -50
        kvd = kv.to(DEV)
        end = [s + (news[i] // 2 if part == 0 else news[i]) for i, s in enumerate(start)]
        by_len = part == 1
        st.append(ws, rows, _i32(off.tolist()), _i32(count) if by_len else None, _i32(end), kvd, kvd[:, heads * d:])
        _ok(dit, ws)
        for s in range(len(lens)):
            for i in range(count[s]):
                pos, row = end[s] - count[s] + i, int(off[s]) + i
                st.ref.put(st.table[s][pos // page], pos % page, kv[row, :heads * d].view(heads, d),
                           kv[row, heads * d:2 * heads * d].view(heads, d))
        assert st.same()


def test_cache_append_rounding(dit, ws):
    """Values spread evenly up to the largest of their group, of groups whose scale rounds either way, zeros,
    subnormals and the largest numbers: bit for bit."""
    d, n = 64, 64
    x = torch.zeros(n, 1, d)
    for i in range(n):
        top = [7.0, 1.0, 3.0, 0.4375, 2.0 ** -126, 2.0 ** 127, 1e-30, 0.0][i % 8] * (1 + (i // 8) / 16)
        x[i, 0] = torch.linspace(-1, 1, d) * top
        x[i, 0, 31] = top
    x = x.clamp(-3.3e38, 3.3e38).bfloat16()
    st = Setup(dit, 1, d, 16, [n], spare=0)
    xd = x.view(n, d).to(DEV)
    st.append(ws, n, _i32([0, n]), None, _i32([n]), xd, xd)
    _ok(dit, ws)
    for i in range(n):
        st.ref.put(st.table[0][i // 16], i % 16, x[i], x[i])
    assert st.same()


def test_cache_append_marks_what_is_not_finite(dit, ws):
    heads, d = 2, 128
    st = Setup(dit, heads, d, 32, [40], seed=1)
    k, v = _randn(40, heads * d, seed=1), _randn(40, heads * d, seed=2)
    k[3, 5], k[39, 255], v[0, 0], v[17, 100] = math.nan, math.inf, -math.inf, math.nan
    st.append(ws, 40, _i32([0, 40]), None, _i32([40]), k.to(DEV), v.to(DEV))
    _ok(dit, ws)
    for i in range(40):
        st.ref.put(st.table[0][i // 32], i % 32, k[i].view(heads, d), v[i].view(heads, d))
    assert st.same()
    # read back: the 32 values of each marked group are NaN, the others finite
    ko, vo = (torch.zeros(40, heads * d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    dit.dit_text_cache4_read(st.c, 1, 40, 40, _i32([0, 40]), None, st.table_dev(), st.dev, ko, heads * d, vo, heads * d, ws, ws.numel())
    _ok(dit, ws)
    for out, where in ((ko, [(3, 0), (39, 7)]), (vo, [(0, 0), (17, 3)])):
        nan = out.cpu().isnan().view(40, -1, 32)
        assert nan.sum() == 32 * len(where) and all(nan[i, j].all() for i, j in where)


def test_cache_append_bad_entries(dit, ws):
    """Lengths and pages out of range: those tokens are not written, the others are, and the call is reported."""
    heads, d, page = 1, 64, 16
    k = _randn(40, d, seed=5).to(DEV)

    def run(q_off, q_len, k_len, table, max_q=40):
        st = Setup(dit, heads, d, page, [20, 20], seed=2)
        t = table(st)
        st.append(ws, 40, _i32(q_off), _i32(q_len), _i32(k_len), k, k, max_q, t)
        return st

    def expect(st, tokens):
        for s, pos, row in tokens:
            st.ref.put(st.table[s][pos // page], pos % page, k[row].cpu().view(1, d), k[row].cpu().view(1, d))
        assert st.same()

    plain = lambda st: st.table_dev()  # noqa: E731
    second = [(1, i, 20 + i) for i in range(20)]
    for q_off, q_len, k_len, max_q in (([-1, 20, 40], [20, 20], [20, 20], 40), ([0, 20, 40], [-1, 20], [20, 20], 40),
                                       ([0, 20, 40], [20, 20], [19, 20], 40), ([0, 20, 40], [20, 20], [-5, 20], 40),
                                       ([21, 20, 40], [20, 20], [20, 20], 40), ([0, 20, 40], [20, 20], [1 << 30, 20], 40),
                                       ([0, 20, 40], [33, 20], [33, 20], 32), ([1 << 30, 20, 40], [20, 20], [20, 20], 40),
                                       ([0, 20, 40], [20, 20], [16 * 3 + 1, 20], 40)):
        st = run(q_off, q_len, k_len, plain, max_q)
        _ok(dit, ws, 0x801)
        expect(st, second)
    for bad in (-1, 1 << 30):
        def table(st, bad=bad):
            t = st.table_dev()
            t[0, 1] = bad
            return t
        st = run([0, 20, 40], [20, 20], [20, 20], table)
        _ok(dit, ws, 0x802)
        expect(st, [(0, i, i) for i in range(16)] + second)
    _ok(dit, ws)


@pytest.mark.parametrize("heads,d,page,lens", [(1, 64, 16, [1]), (2, 128, 16, [5, 0, 16, 33]), (8, 128, 64, [129, 64, 1]),
                                               (3, 64, 256, [255, 257]), (2, 64, 32, [9] * 50)])
def test_cache_read(dit, ws, heads, d, page, lens):
    """Exactly n * scale rounded to bf16, in its rows; the rows between and the columns behind stay."""
    st = Setup(dit, heads, d, page, lens, seed=7)
    st.fill_random(3)
    off, at = [], 2
    for n in lens:
        off.append(at)
        at += n + 3
    wide = heads * d
    buf = torch.full((at, 2 * wide + 16), 9.0, dtype=torch.bfloat16, device=DEV)
    dit.dit_text_cache4_read(st.c, len(lens), at, max(lens), _i32(off + [at]), _i32(lens), st.table_dev(), st.dev, buf, buf.stride(0),
                             buf[:, wide + 8:], buf.stride(0), ws, ws.numel())
    _ok(dit, ws)
    want = torch.full((at, 2 * wide + 16), 9.0, dtype=torch.bfloat16)
    for s, n in enumerate(lens):
        if n:
            want[off[s]:off[s] + n, :wide] = st.ref.values(st.table[s], True)[:n].flatten(1).bfloat16()
            want[off[s]:off[s] + n, wide + 8:2 * wide + 8] = st.ref.values(st.table[s], False)[:n].flatten(1).bfloat16()
    assert torch.equal(_bits(buf), _bits(want))
    # packed, without lengths, over a table with a bad page and one sequence too long for the buffer
    if len(lens) > 2:
        off = np.concatenate([[0], np.cumsum(lens)]).tolist()
        table = st.table_dev()
        table[0, 0] = st.c.pages
        off[-1] += 1
        buf = torch.full((off[-2], wide), 9.0, dtype=torch.bfloat16, device=DEV)
        other = buf.clone()
        dit.dit_text_cache4_read(st.c, len(lens), off[-2], max(lens) + 1, _i32(off), None, table, st.dev, buf, wide, other, wide, ws,
                                 ws.numel())
        stt, where = dit.dit_sync_status(ws)
        assert stt == dit.DIT_ERR_INVALID_ARG and where in (0x801, 0x802)
        want = torch.full((off[-2], wide), 9.0, dtype=torch.bfloat16)
        for s, n in enumerate(lens[:-1]):
            if n:
                want[off[s]:off[s] + n] = st.ref.values(st.table[s], True)[:n].flatten(1).bfloat16()
        want[:min(page, lens[0])] = 9.0
        want[off[-3] + lens[-2]:] = 9.0
        assert torch.equal(_bits(buf), _bits(want))


# --------------------------------------------------------------------- attention over the 4-bit cache
def _check_attention(dit, ws, st, hq, q_lens, causal=True, scale=None, pad=0, gap=1, left_out=(), table=None, status=None, seed=0,
                     std=1.0, max_q=None, max_k=None, stream=None):
    """Queries in a strided buffer with `gap` rows between sequences that must stay as they are."""
    d, lens = st.ref.d, st.lens
    off, at = [], gap
    for n in q_lens:
        off.append(at)
        at += n + gap
    q = _randn(at, hq * d + pad, seed=seed, std=std)
    qd = q.to(DEV)
    out = torch.full((at, hq * d + 2 * pad), 9.0, dtype=torch.bfloat16, device=DEV)
    a = dit.make_text_attn(len(lens), hq, st.ref.heads, d, at, 0, max(q_lens) if max_q is None else max_q,
                           max(lens) if max_k is None else max_k, causal=causal, scale=scale)
    assert dit.dit_text_cache4_attention_workspace(st.c, a) <= ws.numel()
    dit.dit_text_cache4_attention(st.c, a, _i32(off + [at]), _i32(q_lens), _i32(lens), st.table_dev() if table is None else table, qd,
                                  qd.stride(0), st.dev, out, out.stride(0), ws, ws.numel(), stream)
    _ok(dit, ws, status)
    spans = list(zip(off, q_lens, lens))
    want, tol, bad, owned = R.cache_attention(q[:, :hq * d].reshape(at, hq, d), spans, causal, d ** -0.5 if scale is None else scale,
                                              st.ref, st.table, left_out)
    got = out[:, :hq * d].reshape(at, hq, d).cpu()
    assert (got[bad].isnan() | got[bad].isinf()).all()
    _within(torch.where(bad, torch.zeros_like(got), got)[owned], want[owned], tol[owned])
    assert (out.cpu()[~owned] == 9.0).all() and (out[:, hq * d:] == 9.0).all()
    return out


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk,page,q_lens,lens,causal", [
    (1, 1, 16, [1], [1], True), (4, 1, 16, [1, 1, 1], [1, 15, 16], True), (8, 2, 64, [1] * 5, [17, 63, 64, 65, 700], True),
    (6, 2, 32, [3, 1, 2], [3, 100, 33], True), (16, 1, 64, [1, 1], [257, 1000], True), (24, 1, 128, [1, 2], [129, 300], True),
    (64, 1, 64, [1], [200], True), (2, 2, 256, [5, 0, 7], [300, 40, 0], False), (8, 8, 16, [9, 4], [9, 2], True),
    (4, 2, 64, [70, 1], [130, 5], True), (12, 4, 32, [1] * 20, list(range(0, 400, 20)), False), (5, 1, 64, [8], [2000], True),
    (3, 3, 128, [17], [17], True)])
def test_cache_attention(dit, ws, d, hq, hk, page, q_lens, lens, causal):
    st = Setup(dit, hk, d, page, lens, seed=hq)
    st.fill_random(hq + d)
    _check_attention(dit, ws, st, hq, q_lens, causal, pad=8, seed=page)


@pytest.mark.parametrize("d,page,n", [(128, 64, 20000), (64, 16, 9999), (128, 256, 33000)])
def test_cache_attention_long(dit, ws, d, page, n):
    """Keys split over the GPU and joined; a short sequence beside the long one."""
    st = Setup(dit, 1, d, page, [n, 40, n // 3], seed=1)
    st.fill_random(5)
    _check_attention(dit, ws, st, 4, [1, 1, 2], seed=3)


def test_cache_attention_peaked_scores(dit, ws):
    """Scores that rise along the keys, so that the running maximum moves in every block, and a large scale."""
    for d in (64, 128):
        st = Setup(dit, 2, d, 64, [900, 333], seed=2)
        st.fill_random(9)
        s = st.scales(True)
        for t, n in ((0, 900), (1, 333)):
            for pos in range(n):
                s[st.table[t][pos // 64], :, pos % 64] = torch.full((1,), 0.02 + 0.4 * pos / n).bfloat16().view(torch.int16).numpy()
        st.upload()
        _check_attention(dit, ws, st, 4, [2, 1], seed=1, scale=0.25)
        _check_attention(dit, ws, st, 4, [2, 1], seed=2, scale=1e-3, causal=False)


@pytest.mark.parametrize("d", [64, 128])
def test_cache_attention_bad_values(dit, ws, d):
    """NaN scales behind the keys, and on visible and invisible keys: a value reaches the rows that see it, no others."""
    page, lens = 32, [100, 40]
    for key in (True, False):
        for pos in (99, 98, 60, 0):
            st = Setup(dit, 2, d, page, lens, seed=4)
            st.fill_random(11)
            s = st.scales(key)
            s[st.table[0][pos // page], 1, pos % page, -1] = 0x7fff
            for which in (True, False):  # everything behind the last token of both sequences
                sc = st.scales(which)
                sc[st.table[0][3], :, 4:] = 0x7fff
                sc[st.table[1][1], :, 8:] = 0x7f80
            st.upload()
            _check_attention(dit, ws, st, 4, [3, 1], seed=pos)


def test_cache_attention_bad_entries(dit, ws):
    """A page out of range is left out of the sums, a sequence with lengths out of range is skipped; both are reported."""
    page, lens = 16, [100, 40, 33]
    st = Setup(dit, 2, 64, page, lens, seed=4)
    st.fill_random(12)
    for bad in (-1, st.c.pages, 1 << 30):
        table = st.table_dev()
        table[0, 2] = bad
        _check_attention(dit, ws, st, 4, [2, 1, 1], left_out=[(0, p) for p in range(32, 48)], table=table, status=0x802)
    table = st.table_dev()
    table[2, :] = -1  # a sequence without a single page: zeros
    out = _check_attention(dit, ws, st, 4, [2, 1, 1], left_out=[(2, p) for p in range(33)], table=table, status=0x802)
    assert (out[7] == 0).all() or (out == 0).any()
    q = _randn(4, 4 * 64).to(DEV)
    out = torch.full((4, 4 * 64), 9.0, dtype=torch.bfloat16, device=DEV)
    good = dit.make_text_attn(3, 4, 2, 64, 4, 0, 2, 100)
    for q_off, q_len, k_len in (([0, 2, 3], [3, 1, 1], lens), ([-1, 2, 3], [2, 1, 1], lens), ([0, 2, 3], [2, 1, 1], [101, 40, 33]),
                                ([0, 2, 3], [2, 1, 1], [-1, 40, 33]), ([3, 2, 3], [2, 1, 1], lens), ([0, 2, 3], [-1, 1, 1], lens)):
        out.fill_(9.0)
        dit.dit_text_cache4_attention(st.c, good, _i32(q_off + [4]), _i32(q_len), _i32(k_len), st.table_dev(), q, 256, st.dev, out, 256, ws,
                                      ws.numel())
        _ok(dit, ws, 0x801)
        assert (out[:2] == 9.0).all() and (out[2:] != 9.0).any(1).all()


def test_cache_attention_bounds_above_the_lengths(dit, ws):
    """max_q and max_k well above what the sequences need choose other splits, not other results."""
    st = Setup(dit, 2, 128, 64, [300, 70], seed=6)
    st.fill_random(13)
    for max_q, max_k in ((1, 300), (1, 20000), (50, 1 << 24), (1, 1 << 24)):
        _check_attention(dit, ws, st, 8, [1, 1], max_q=max_q, max_k=max_k)


def test_cache_attention_equal_calls_give_equal_bits(dit, ws):
    st = Setup(dit, 2, 128, 64, [3000, 700, 90], seed=8)
    st.fill_random(14)
    one = _check_attention(dit, ws, st, 8, [1, 2, 1])
    for _ in range(3):
        assert torch.equal(_bits(_check_attention(dit, ws, st, 8, [1, 2, 1])), _bits(one))


def test_cache_attention_agrees_with_attention_on_what_is_read_back(dit, ws):
    """A chunk of a long prompt: appended, read back, and attended to either way."""
    heads, hq, d, page, lens, news = 2, 8, 128, 64, [500, 130], [150, 130]
    st = Setup(dit, heads, d, page, lens, seed=9)
    st.fill_random(15)
    rows = sum(news)
    kv = _randn(rows, 2 * heads * d, seed=3).to(DEV)
    q = _randn(rows, hq * d, seed=4).to(DEV)
    qo, kl = _i32([0, 150, 280]), _i32(lens)
    st.append(ws, rows, qo, None, kl, kv, kv[:, heads * d:])
    ko = torch.zeros(630, heads * d, dtype=torch.bfloat16, device=DEV)
    vo = torch.zeros_like(ko)
    k_off = _i32([0, 500, 630])
    dit.dit_text_cache4_read(st.c, 2, 630, 500, k_off, kl, st.table_dev(), st.dev, ko, heads * d, vo, heads * d, ws, ws.numel())
    out, out4 = torch.zeros_like(q), torch.zeros_like(q)
    a = dit.make_text_attn(2, hq, heads, d, rows, 630, 150, 500)
    dit.dit_text_attention(a, qo, None, k_off, None, q, hq * d, ko, heads * d, vo, heads * d, out, hq * d, ws, ws.numel())
    dit.dit_text_cache4_attention(st.c, a, qo, None, kl, st.table_dev(), q, hq * d, st.dev, out4, hq * d, ws, ws.numel())
    _ok(dit, ws)
    # the rounding of n * scale to bf16 (2^-8 of keys and values) is all that differs, besides both sides' own
    err = (out.float() - out4.float()).norm() / out.float().norm()
    assert float(err) < 2.0 ** -6, float(err)


# ----------------------------------------------------------------------------- a layer of a decoder
class Layer:
    """One decoder layer for new tokens over the 4-bit cache, every operation the library's: norm -> product with bias ->
    per-head norm and rotation -> append -> attention -> output product + residual -> norm to e4m3 -> block-scaled product
    -> product with activation and residual.  `check` compares each stage with the 64-bit form on what the stage
    before it wrote."""

    def __init__(self, dit, lens, news, seed=0, d=64, hq=4, hk=2, hidden=256, mlp=384, page=16):
        self.dit, self.d, self.hq, self.hk, self.hidden, self.mlp = dit, d, hq, hk, hidden, mlp
        self.st = Setup(dit, hk, d, page, lens, seed=seed)
        self.st.fill_random(seed)
        self.news, self.rows = news, sum(news)
        wide = (hq + 2 * hk) * d
        h = lambda *s, i, std: _randn(*s, seed=100 * seed + i, std=std)  # noqa: E731
        self.cpu = dict(x=h(self.rows, hidden, i=0, std=1.0), n1=h(hidden, i=1, std=0.1) + 1, wqkv=h(wide, hidden, i=2, std=0.06),
                        bqkv=h(wide, i=3, std=0.3), qn=h(d, i=4, std=0.1) + 1, kn=h(d, i=5, std=0.1) + 1,
                        wo=h(hidden, hq * d, i=6, std=0.06), n2=h(hidden, i=7, std=0.1) + 1, wu=h(mlp, hidden, i=8, std=0.06),
                        wd=h(hidden, mlp, i=9, std=0.05), bd=h(hidden, i=10, std=0.1))
        self.p = {n: t.to(DEV) for n, t in self.cpu.items()}
        z = lambda *s, dt=torch.bfloat16: torch.zeros(*s, dtype=dt, device=DEV)  # noqa: E731
        r = self.rows
        self.y1, self.qkv, self.att, self.x2 = z(r, hidden), z(r, wide), z(r, hq * d), z(r, hidden)
        self.s2, self.q8, self.s8 = z(r, hidden), z(r, hidden, dt=torch.uint8), z(r, -(-hidden // 128), dt=torch.float32)
        self.wq, self.wsc = z(mlp, hidden, dt=torch.uint8), z(-(-mlp // 128), -(-hidden // 128), dt=torch.float32)
        self.up, self.out = z(r, mlp), z(r, hidden)
        dit.dit_quantize_blocks_fp8(self.p["wu"], hidden, mlp, hidden, 128, self.wq, self.wsc)
        self.table = z(max(lens) + 1, d // 2, 2, dt=torch.float32)
        dit.dit_text_rope_table(dit.make_text_rope(d, 1e4), None, max(lens) + 1, self.table)
        self.pages, self.q_off, self.kl = self.st.table_dev(), _i32([0] + np.cumsum(news).tolist()), _i32(lens)
        self.pos = _i32([n - a + i for n, a in zip(lens, news) for i in range(a)])
        self.ws = torch.zeros(32 << 20, dtype=torch.uint8, device=DEV)
        self.a = dit.make_text_attn(len(lens), hq, hk, d, r, 0, max(news), max(lens))
        torch.cuda.synchronize()

    def run(self, stream=None):
        t, p, d, hq, hk, r, hidden, mlp, ws = self.dit, self.p, self.d, self.hq, self.hk, self.rows, self.hidden, self.mlp, self.ws
        n, wide = ws.numel(), self.qkv.stride(0)
        t.dit_add_rms_norm(r, hidden, p["x"], hidden, None, 0, p["n1"], 0.0, 1e-6, None, 0, self.y1, hidden, None, None, stream)
        t.dit_linear_act(r, wide, hidden, self.y1, hidden, p["wqkv"], hidden, p["bqkv"], t.DIT_ACT_NONE, None, 0, self.qkv, wide, False, ws, n,
                         stream)
        q, k, v = self.qkv, self.qkv[:, hq * d:], self.qkv[:, (hq + hk) * d:]
        t.dit_qk_norm_rope(r, hq, hk, d, d, t.DIT_ROPE_HALF, q, wide, k, wide, p["qn"], p["kn"], 1e-6, self.table, self.table.shape[0],
                           self.pos, q, wide, k, wide, ws, n, stream)
        t.dit_text_cache4_append(self.st.c, len(self.news), r, max(self.news), self.q_off, None, self.kl, self.pages, k, wide, v, wide,
                                 self.st.dev, ws, n, stream)
        t.dit_text_cache4_attention(self.st.c, self.a, self.q_off, None, self.kl, self.pages, q, wide, self.st.dev, self.att, hq * d, ws, n,
                                    stream)
        t.dit_linear_act(r, hidden, hq * d, self.att, hq * d, p["wo"], hq * d, None, t.DIT_ACT_NONE, p["x"], hidden, self.x2, hidden, False,
                         ws, n, stream)
        t.dit_add_rms_norm(r, hidden, self.x2, hidden, None, 0, p["n2"], 0.0, 1e-6, None, 0, None, 0, self.q8, self.s8, stream)
        t.dit_linear_fp8_blocks(r, mlp, hidden, self.q8, self.s8, self.wq, self.wsc, self.up, mlp, ws, n, stream)
        t.dit_linear_act(r, hidden, mlp, self.up, mlp, p["wd"], mlp, p["bd"], t.DIT_ACT_SILU, self.x2, hidden, self.out, hidden, False, ws, n,
                         stream)

    def outputs(self):
        return [t.clone() for t in (self.qkv, self.st.dev, self.att, self.x2, self.q8, self.s8, self.up, self.out)]

    def check(self):
        _ok(self.dit, self.ws)
        c, d, hq, hk, lens = self.cpu, self.d, self.hq, self.hk, self.st.lens
        eps = float(np.float32(1e-6))
        _, y = R.add_rms_norm(c["x"], None, c["n1"], 0.0, eps)
        _within(self.y1, y, 2.0 ** -8 * y.abs() + _norm_tolerance(y, self.hidden) * 1.01)
        qkv = self.qkv.cpu()
        # the values are neither normed nor turned: the product itself
        vs = slice((hq + hk) * d, None)
        want, size, z = R.linear_act(self.y1.cpu(), c["wqkv"][vs], c["bqkv"][vs], "none", None)
        _within(qkv[:, vs], want, R.linear_act_tolerance(want, size, z, self.hidden, None, False))
        # the cache holds the keys and values of the buffer
        ref, at = self.st.ref, 0
        for s, a in enumerate(self.news):
            for i in range(a):
                pos = lens[s] - a + i
                ref.put(self.st.table[s][pos // ref.page], pos % ref.page, qkv[at, hq * d:(hq + hk) * d].view(hk, d),
                        qkv[at, (hq + hk) * d:].view(hk, d))
                at += 1
        assert self.st.same()
        off = np.cumsum([0] + list(self.news))
        want, tol, _, _ = R.cache_attention(qkv[:, :hq * d].reshape(-1, hq, d), [(int(off[s]), a, lens[s]) for s, a in enumerate(self.news)],
                                            True, d ** -0.5, ref, self.st.table)
        _within(self.att.view(-1, hq, d), want, tol)
        want, size, z = R.linear_act(self.att.cpu(), c["wo"], None, "none", c["x"])
        _within(self.x2, want, R.linear_act_tolerance(want, size, z, hq * d, c["x"], False))
        s8 = self.s8.cpu().double().repeat_interleave(128, 1)[:, :self.hidden]
        a8 = self.q8.cpu().view(torch.float8_e4m3fn).double() * s8
        _, y = R.add_rms_norm(self.x2.cpu(), None, c["n2"], 0.0, eps)
        v = y / s8
        _within(a8, y, (R.e4m3_steps(v.abs() * 1.001) / 2 + v.abs() * 64 * 2.0 ** -24) * s8)
        w8 = self.wq.cpu().view(torch.float8_e4m3fn).double() * self.wsc.cpu().double().repeat_interleave(128, 0)[:self.mlp].repeat_interleave(128, 1)[:, :self.hidden]
        want = a8 @ w8.t()
        _within(self.up, want, 2.0 ** -8 * want.abs() + (self.hidden + 8) * 2.0 ** -23 * (a8.abs() @ w8.abs().t()))
        want, size, z = R.linear_act(self.up.cpu(), c["wd"], c["bd"], "silu", self.x2.cpu())
        _within(self.out, want, R.linear_act_tolerance(want, size, z, self.mlp, self.x2.cpu(), False))


@pytest.mark.parametrize("lens,news,kw", [([37, 1, 100], [1, 1, 1], {}), ([37, 20, 100, 64], [5, 20, 1, 33], {}),
                                          ([300, 70], [1, 3], dict(d=128, hq=8, hk=2, hidden=384, mlp=512, page=64))])
def test_decoder_layer(dit, lens, news, kw):
    layer = Layer(dit, lens, news, seed=1, **kw)
    layer.run()
    layer.check()


def test_decoder_layer_captured_and_replayed(dit):
    """Two layers captured on workspaces of their own, replayed at once on two streams, then again over other lengths,
    pages and inputs: the bits of the eager calls."""
    layers = [Layer(dit, [37, 30, 100], [1, 1, 1], seed=s) for s in (2, 3)]
    graphs = []
    for l in layers:
        l.run()  # one-time set-up outside the capture
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            l.run()
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in layers]

    def replay():
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()

    replay()
    for l in layers:
        l.check()
    for l in layers:
        lens = [n - 5 for n in l.st.lens]
        l.kl.copy_(_i32(lens))
        l.pos.copy_(_i32([n - 1 for n in lens]))
        x = _randn(l.rows, l.hidden, seed=77)
        l.p["x"].copy_(x)
        l.cpu["x"], l.st.lens = x, lens
    replay()
    for l in layers:
        l.check()
        got = l.outputs()
        l.run()
        torch.cuda.synchronize()
        for x, y in zip(got, l.outputs()):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_decoder_layer_from_two_threads(dit):
    """Two host threads on streams and workspaces of their own, twenty calls each: the one-thread bits."""
    layers = [Layer(dit, [64, 7, 250], [2, 1, 1], seed=s) for s in (4, 5)]
    want = []
    for l in layers:
        l.run()
        torch.cuda.synchronize()
        want.append(l.outputs())
    errors = []

    def work(l):
        try:
            s = torch.cuda.Stream()
            for _ in range(20):
                l.run(s)
            s.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=(l,)) for l in layers]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for l, w in zip(layers, want):
        _ok(dit, l.ws)
        for x, y in zip(w, l.outputs()):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
