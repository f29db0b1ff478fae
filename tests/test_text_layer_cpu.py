"""Refusals of the norm with residual, the product with bias, activation and residual, and the 4-bit cache, without
a GPU: each call fails its checks before any launch; and the 64-bit forms hold what they state."""
import math

import numpy as np
import pytest
import torch

import text_layer_reference as R

FAKE = 0x10000  # 16-byte aligned, never dereferenced
B1, B2, B3, B4, B5, B6, B7 = (FAKE + (i << 32) for i in range(1, 8))


@pytest.fixture(scope="module")
def dit():
    from diffusion_transformer_step_gb300 import build_lib
    build_lib.build()
    from diffusion_transformer_step_gb300 import dit as d
    d.lib()
    return d


def _refused(dit, call, want=None):
    before = dit.dit_launch_count()
    with pytest.raises(dit.DitError) as e:
        call()
    assert e.value.status == (dit.DIT_ERR_INVALID_ARG if want is None else want)
    assert dit.dit_launch_count() == before


NORM = dict(rows=4, cols=256, x=B1, ldx=256, res=B2, ld_res=264, w=B3, offset=0.0, eps=1e-6, sum_out=B4, ld_sum=256, y=B5,
            ldy=256, q=B6, scale=B7)


@pytest.mark.parametrize("change,st", [
    ({"cols": 0}, 2), ({"cols": 260}, 2), ({"cols": 32776}, 2), ({"cols": 248}, 2), ({"rows": -1}, 1), ({"rows": (1 << 26) + 1}, 1),
    ({"eps": -1e-6}, 1), ({"eps": math.nan}, 1), ({"eps": math.inf}, 1), ({"offset": math.nan}, 1), ({"offset": math.inf}, 1),
    ({"y": None, "q": None, "scale": None}, 1), ({"scale": None}, 1), ({"q": None}, 1), ({"ldx": 248}, 1), ({"ldx": 260}, 1),
    ({"ld_res": 255}, 1), ({"ld_sum": (1 << 24) + 8}, 1), ({"ldy": 0}, 1), ({"x": None}, 1), ({"x": B1 + 8}, 1), ({"res": B2 + 2}, 1),
    ({"w": B3 + 4}, 1), ({"sum_out": B4 + 1}, 1), ({"y": B5 + 8}, 1), ({"q": B6 + 8}, 1), ({"scale": B7 + 4}, 1),
    # outputs over the inputs or over one another
    ({"sum_out": B1 + 16}, 1), ({"y": B1 + 16}, 1), ({"sum_out": B2}, 1), ({"y": B2 + 512, "ldy": 264}, 1), ({"y": B4}, 1), ({"y": B3}, 1),
    ({"sum_out": B3 + 496}, 1), ({"q": B1}, 1), ({"q": B2 + 512}, 1), ({"q": B3}, 1), ({"q": B5 + 1024}, 1), ({"scale": B6 + 512}, 1),
    ({"scale": B4}, 1)])
def test_add_rms_norm_refusals(dit, change, st):
    _refused(dit, lambda: dit.dit_add_rms_norm(*{**NORM, **change}.values(), stream=0), st)


def test_nothing_to_do_is_no_launch(dit):
    before = dit.dit_launch_count()
    dit.dit_add_rms_norm(*{**NORM, "rows": 0}.values(), stream=0)
    none = dict.fromkeys(("x", "res", "sum_out", "y", "q", "scale"))  # as the pointers of tensors without elements
    dit.dit_add_rms_norm(*{**NORM, **none, "rows": 0}.values(), stream=0)
    dit.dit_linear_act(*{**LIN, "rows": 0, "a": None}.values(), stream=0)
    dit.dit_linear_act(*{**LIN, "rows": 0, "a": 0, "res": 0, "out": 0}.values(), stream=0)
    c = dit.make_text_cache4(**CACHE)
    for change in ({"seqs": 0}, {"rows": 0}, {"max_q": 0}):
        dit.dit_text_cache4_append(c, *{**APPEND, **change, "q_off": None}.values(), stream=0)
    for change in ({"seqs": 0}, {"rows": 0}, {"max_k": 0}):
        dit.dit_text_cache4_read(c, *{**READ, **change, "k_off": None}.values(), stream=0)
    for change in ({"seqs": 0}, {"rows_q": 0}, {"max_q": 0}):
        a = dit.make_text_attn(**{**AT, **change})
        dit.dit_text_cache4_attention(c, a, *{**ATTN, "q_off": None}.values(), stream=0)
    assert dit.dit_launch_count() == before


LIN = dict(rows=4, n_out=100, k=256, a=B1, lda=256, w=B2, ldw=256, bias=B3, act=2, res=B4, ld_res=104, out=B5, ld_out=104, f32=False,
           ws=B6, ws_bytes=1 << 26)


@pytest.mark.parametrize("change,st", [
    ({"rows": -1}, 1), ({"rows": (1 << 20) + 1}, 1), ({"n_out": 0}, 1), ({"n_out": (1 << 20) + 1}, 1), ({"k": 0}, 1), ({"k": 252}, 1),
    ({"k": 264}, 1), ({"act": -1}, 1), ({"act": 5}, 1), ({"lda": 260}, 1), ({"ldw": 248}, 1), ({"ld_res": 96}, 1), ({"ld_out": 96}, 1),
    ({"ld_out": 100}, 1), ({"a": None}, 1), ({"w": B2 + 8}, 1), ({"bias": B3 + 2}, 1), ({"res": B4 + 8}, 1), ({"out": None}, 1),
    ({"ws": None}, 1), ({"ws_bytes": 255}, 3),
    # the output over an operand; over the residual only exactly, and only where both are bf16
    ({"out": B1}, 1), ({"out": B2 + 16}, 1), ({"out": B3 + 192}, 1), ({"out": B4 + 16}, 1), ({"out": B4, "ld_out": 112}, 1),
    ({"out": B4, "f32": True}, 1), ({"out": B1 - 16, "f32": True}, 1)])
def test_linear_act_refusals(dit, change, st):
    _refused(dit, lambda: dit.dit_linear_act(*{**LIN, **change}.values(), stream=0), st)


def test_linear_act_workspace(dit):
    """Bounded for any sizes, refused when it is a byte short."""
    for m, n, k in ((0, 1, 8), (1, 8, 16), (300, 256, 4096), (65, 128, 1 << 20), (489, 1168, 9616), (8192, 12288, 4096),
                    (1 << 20, 8, 1 << 20), (1 << 20, 1 << 20, 1 << 20), (777, 1544, 5160), (200, 100, 100000)):
        need = dit.dit_linear_act_workspace(m, n, k)
        assert 256 <= need <= 256 + 48 * (1 << 20)
        if m:
            _refused(dit, lambda: dit.dit_linear_act(*{**LIN, "rows": m, "n_out": n, "k": k, "lda": k, "ldw": k, "ld_res": n + -n % 8,
                                                       "ld_out": n + -n % 8, "ws_bytes": need - 1}.values(), stream=0), dit.DIT_ERR_WORKSPACE)
    for args in ((-1, 8, 8), (1, 0, 8), (1, 8, 12)):
        _refused(dit, lambda: dit.dit_linear_act_workspace(*args))


CACHE = dict(heads_k=2, head_dim=128, pages=10, page_size=64, max_pages=4)
SLAB = 64 * 128 * 9 // 8


@pytest.mark.parametrize("change,st", [
    ({"head_dim": 96}, 2), ({"head_dim": 256}, 2), ({"page_size": 8}, 2), ({"page_size": 48}, 2), ({"page_size": 512}, 2), ({"heads_k": 0}, 1),
    ({"heads_k": 1025}, 1), ({"pages": 0}, 1), ({"pages": (1 << 24) + 1}, 1), ({"max_pages": 0}, 1), ({"max_pages": (1 << 18) + 1}, 1)])
def test_cache_refusals(dit, change, st):
    c = dit.make_text_cache4(**{**CACHE, **change})
    _refused(dit, lambda: dit.dit_text_cache4_bytes(c), st)
    _refused(dit, lambda: dit.dit_text_cache4_append(c, *APPEND.values(), stream=0), st)
    _refused(dit, lambda: dit.dit_text_cache4_read(c, *READ.values(), stream=0), st)
    a = dit.make_text_attn(**AT)
    _refused(dit, lambda: dit.dit_text_cache4_attention(c, a, *ATTN.values(), stream=0), st)


def test_cache_bytes(dit):
    assert dit.dit_text_cache4_bytes(dit.make_text_cache4(**CACHE)) == 10 * 2 * SLAB
    assert dit.dit_text_cache4_bytes(dit.make_text_cache4(1024, 128, 1 << 24, 256, 1 << 16)) == (1 << 34) * 256 * 144


APPEND = dict(seqs=2, rows=8, max_q=5, q_off=FAKE, q_len=None, k_len=FAKE, table=FAKE, k=B1, ldk=512, v=B1 + 512, ldv=512, cache=B2,
              ws=FAKE, ws_bytes=256)
READ = dict(seqs=2, rows=300, max_k=200, k_off=FAKE, k_len=None, table=FAKE, cache=B2, k=B3, ldk=512, v=B3 + 512, ldv=512, ws=FAKE,
            ws_bytes=256)
MOVE = [({"seqs": -1}, 1), ({"seqs": 16385}, 1), ({"rows": -1}, 1), ({"rows": (1 << 28) + 1}, 1), ({"ldk": 248}, 1), ({"ldv": 260}, 1),
        ({"ldk": (1 << 24) + 8}, 1), ({"k": None}, 1), ({"v": None}, 1), ({"k": B4 + 8}, 1), ({"table": None}, 1), ({"table": FAKE + 2}, 1),
        ({"cache": None}, 1), ({"cache": B2 + 8}, 1), ({"ws": None}, 1), ({"ws_bytes": 255}, 3), ({"k": B2}, 1), ({"v": B2 + 20 * SLAB - 16}, 1)]


@pytest.mark.parametrize("change,st", MOVE + [({"max_q": -1}, 1), ({"max_q": (1 << 24) + 1}, 1), ({"q_off": None}, 1), ({"q_off": FAKE + 2}, 1),
                                              ({"q_len": FAKE + 2}, 1), ({"k_len": None}, 1), ({"k_len": FAKE + 1}, 1)])
def test_cache_append_refusals(dit, change, st):
    c = dit.make_text_cache4(**CACHE)
    _refused(dit, lambda: dit.dit_text_cache4_append(c, *{**APPEND, **change}.values(), stream=0), st)


@pytest.mark.parametrize("change,st", MOVE + [({"max_k": -1}, 1), ({"k_off": None}, 1), ({"k_off": FAKE + 2}, 1), ({"k_len": FAKE + 2}, 1),
                                              ({"v": B3}, 1), ({"v": B3 + 256}, 1)])
def test_cache_read_refusals(dit, change, st):
    c = dit.make_text_cache4(**CACHE)
    _refused(dit, lambda: dit.dit_text_cache4_read(c, *{**READ, **change}.values(), stream=0), st)


AT = dict(seqs=2, heads_q=8, heads_k=2, head_dim=128, rows_q=64, rows_k=0, max_q=40, max_k=200, causal=True, scale=0.1)
ATTN = dict(q_off=FAKE, q_len=None, k_len=FAKE, table=FAKE, q=B1, ldq=1024, cache=B2, out=B3, ldo=1024, ws=B4, ws_bytes=1 << 26)


@pytest.mark.parametrize("change,st", [
    ({"heads_k": 4}, 1), ({"head_dim": 64}, 1), ({"head_dim": 96}, 2), ({"heads_q": 7}, 1), ({"heads_q": 130}, 1), ({"seqs": -1}, 1),
    ({"seqs": 16385}, 1), ({"rows_q": -1}, 1), ({"max_q": -1}, 1), ({"max_k": (1 << 24) + 1}, 1), ({"scale": 0.0}, 1), ({"scale": math.nan}, 1)])
def test_cache_attention_size_refusals(dit, change, st):
    c, a = dit.make_text_cache4(**CACHE), dit.make_text_attn(**{**AT, **change})
    _refused(dit, lambda: dit.dit_text_cache4_attention(c, a, *ATTN.values(), stream=0), st)
    _refused(dit, lambda: dit.dit_text_cache4_attention_workspace(c, a), st)


@pytest.mark.parametrize("change,st", [
    ({"q_off": None}, 1), ({"q_off": FAKE + 2}, 1), ({"q_len": FAKE + 1}, 1), ({"k_len": None}, 1), ({"k_len": FAKE + 2}, 1),
    ({"table": None}, 1), ({"table": FAKE + 1}, 1), ({"q": None}, 1), ({"q": B1 + 8}, 1), ({"cache": None}, 1), ({"cache": B2 + 8}, 1),
    ({"out": None}, 1), ({"out": B3 + 8}, 1), ({"ldq": 1016}, 1), ({"ldo": 1028}, 1), ({"ws": None}, 1), ({"ws_bytes": 255}, 3),
    ({"out": B1}, 1), ({"out": B2 + 20 * SLAB - 16}, 1), ({"out": B2 - 16}, 1)])
def test_cache_attention_argument_refusals(dit, change, st):
    c, a = dit.make_text_cache4(**CACHE), dit.make_text_attn(**AT)
    _refused(dit, lambda: dit.dit_text_cache4_attention(c, a, *{**ATTN, **change}.values(), stream=0), st)


def test_cache_attention_workspace_over_the_range(dit):
    """Some bytes for any documented sizes, without an overflow or a division by zero; none refused."""
    for seqs in (1, 7, 16384):
        for hq, hk in ((1, 1), (1024, 16), (1024, 1024)):
            for max_q in (1, 17, 1 << 24):
                for max_k in (0, 1, 255, 1 << 24):
                    for page in (16, 256):
                        c = dit.make_text_cache4(hk, 128, 1 << 24, page, (1 << 24) // page)
                        a = dit.make_text_attn(seqs, hq, hk, 128, 1 << 28, 0, max_q, max_k)
                        assert 256 <= dit.dit_text_cache4_attention_workspace(c, a) < 1 << 34


def test_cache_attention_workspace_stays_small(dit):
    """At most 2^17 rows of parts, whichever way the keys are cut: by bounds, into clusters, in even shares."""
    for d in (64, 128):
        for seqs in (1, 9, 48, 456, 1024, 1025, 16384):
            for hq, hk in ((1, 1), (32, 8), (96, 8), (1024, 1024)):
                for max_q in (1, 2, 5, 500):
                    for max_k in (1, 128, 512, 513, 2048, 2049, 5001, 32768, 1 << 20, 1 << 24):
                        c = dit.make_text_cache4(hk, d, 1 << 20, 64, (1 << 24) // 64)
                        a = dit.make_text_attn(seqs, hq, hk, d, 1 << 20, 0, max_q, max_k)
                        need = dit.dit_text_cache4_attention_workspace(c, a)
                        assert 256 <= need <= 1024 + (1 << 17) * (8 + 4 * d) + 456 * 16, (d, seqs, hq, hk, max_q, max_k, need)


def test_kernel_classes_have_names(dit):
    names = [dit.dit_kernel_class_name(i) for i in range(40)]
    for n in ("add_rms_norm", "linear_act", "text_cache4_append", "text_cache4_read", "text_cache4_attention",
              "text_cache4_join"):
        assert names.count(n) == 1


# ------------------------------------------------------------------- the reference forms themselves
@pytest.mark.parametrize("d", [64, 128])
def test_reference_cache_round_trip(d):
    g = torch.Generator().manual_seed(d)
    c = R.Cache(3, d, 4, 16)
    k, v = torch.randn(16, 3, d, generator=g).bfloat16(), torch.randn(16, 3, d, generator=g).bfloat16()
    for i in range(16):
        c.put(2, i, k[i], v[i])
    for key, x in ((True, k), (False, v)):
        got = c.values([2], key)
        step = x.double().reshape(16, 3, -1, 32).abs().amax(-1, keepdim=True) / 7
        # half a step, the scale's own rounding at up to 7.03 steps, the largest value clamped to 7 of them
        err = (got.reshape(16, 3, -1, 32) - x.double().reshape(16, 3, -1, 32)).abs()
        assert (err <= step * (0.5 + 7.03 * 2.0 ** -8)).all()
        for row in (R.code_places(d, key),):
            assert len(set(row)) == d and max(b for b, _ in row) == d // 2 - 1
    assert (c.raw[[0, 1, 3]] == 0).all()


def test_reference_quantiser_marks_what_is_not_finite():
    x = torch.ones(4, 64).bfloat16()
    x[0, 3], x[1, 40], x[2, 0] = math.nan, math.inf, -math.inf
    n, s = R.quantise(x)
    assert s.isnan().tolist() == [[True, False], [False, True], [True, False], [False, False]]
    assert (n[3] == 7).all() and (n[0, :32] == 0).all()


def test_reference_attention_is_the_textbook_softmax():
    g = torch.Generator().manual_seed(0)
    c = R.Cache(2, 64, 3, 16)
    for i in range(20):
        c.put([2, 0][i // 16], i % 16, torch.randn(2, 64, generator=g).bfloat16(), torch.randn(2, 64, generator=g).bfloat16())
    q = torch.randn(3, 4, 64, generator=g).bfloat16()
    out, tol, bad, owned = R.cache_attention(q, [(0, 3, 20)], True, 0.125, c, [[2, 0]])
    k, v = c.values([2, 0], True)[:20], c.values([2, 0], False)[:20]
    for i in range(3):
        for h in range(4):
            s = (k[:18 + i, h // 2] @ q[i, h].double()) * 0.125
            torch.testing.assert_close(out[i, h], torch.softmax(s, 0) @ v[:18 + i, h // 2])
    assert owned.all() and not bad.any() and (tol < 0.05).all()


def test_bars_reject_planted_slips():
    """The attention's tolerance against slips planted in its inputs: one key left out, two tokens' values swapped,
    the scales of neighbouring groups exchanged, the mask one token off."""
    g = torch.Generator().manual_seed(1)
    n = 40
    k, v = torch.randn(n, 2, 64, generator=g).bfloat16(), torch.randn(n, 2, 64, generator=g).bfloat16()
    q = torch.randn(2, 4, 64, generator=g).bfloat16()

    def cache(kk, vv, scales=False):
        c = R.Cache(2, 64, 3, 16)
        for i in range(n):
            c.put(i // 16, i % 16, kk[i], vv[i])
        if scales:
            s = c.raw[:, :, 512:576].reshape(3, 2, 16, 2, 2)
            s[:] = s[:, :, :, ::-1].copy()
        return c

    run = lambda c, causal=True, out=(): R.cache_attention(q, [(0, 2, n)], causal, 0.125, c, [[0, 1, 2]], out)  # noqa: E731
    want, tol, _, _ = run(cache(k, v))
    swapped = v.clone()
    swapped[[3, 4]] = v[[4, 3]]
    for other in (run(cache(k, v), out=[(0, 7)]), run(cache(k, swapped)), run(cache(k, v, True)), run(cache(k, v), causal=False)):
        assert ((other[0] - want).abs() > tol).any()
    assert np.isfinite(tol.numpy()).all()
