"""Refusals of the text-side operations, without a GPU: each call fails its checks before any
launch; and the 64-bit forms that the GPU tests compare with hold what they state."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

import text_reference as R

FAKE = 0x10000  # 16-byte aligned, never dereferenced


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


def test_text_rope_refusals(dit):
    ok = dict(rot_dim=64, theta=1e4, scaling=3, factor=4.0, low=1.0, high=4.0, original_len=128, magnitude=1.0)
    inf, nan = math.inf, math.nan
    for change, st in (({"rot_dim": 63}, 2), ({"rot_dim": 0}, 2), ({"rot_dim": 258}, 2), ({"theta": 1.0}, 1), ({"theta": nan}, 1),
                       ({"theta": inf}, 1), ({"scaling": 4}, 1), ({"scaling": -1}, 1), ({"factor": 0.5}, 1), ({"factor": nan}, 1),
                       ({"low": 4.0}, 1), ({"low": -1.0}, 1), ({"high": nan}, 1), ({"original_len": 0}, 1), ({"magnitude": 0.0}, 1),
                       ({"magnitude": inf}, 1), ({"rot_dim": 2, "scaling": 2}, 2), ({"scaling": 2, "factor": 0.0}, 1)):
        r = dit.make_text_rope(**{**ok, **change})
        _refused(dit, lambda: dit.dit_text_rope_table(r, None, 4, FAKE, stream=0), st)
    r = dit.make_text_rope(**ok)
    for args in ((None, -1, FAKE), (None, (1 << 24) + 1, FAKE), (FAKE + 2, 4, FAKE), (None, 4, FAKE + 4), (None, 4, None)):
        _refused(dit, lambda: dit.dit_text_rope_table(r, *args, stream=0))
    dit.dit_text_rope_table(r, None, 0, None, stream=0)  # nothing to do


QK = dict(rows=4, heads_q=8, heads_k=2, head_dim=128, rot_dim=128, layout=1, q_dev=FAKE, ldq=1536, k_dev=FAKE + 2048, ldk=1536,
          q_norm=FAKE, k_norm=FAKE, eps=1e-6, table_dev=FAKE, table_rows=4, table_row_dev=None, q_out_dev=FAKE + (1 << 20),
          ldq_out=1024, k_out_dev=FAKE + (1 << 21), ldk_out=256, ws=FAKE, ws_bytes=256, stream=0)


@pytest.mark.parametrize("change,st", [
    ({"head_dim": 96}, 2), ({"rot_dim": 12}, 2), ({"rot_dim": 136}, 2), ({"rot_dim": -8}, 2), ({"rows": -1}, 1),
    ({"rows": (1 << 26) + 1}, 1), ({"heads_q": 0}, 1), ({"heads_k": -1}, 1), ({"layout": 2}, 1), ({"eps": -1.0}, 1),
    ({"eps": math.nan}, 1), ({"eps": math.inf}, 1), ({"q_norm": None}, 1), ({"k_norm": None}, 1), ({"ldq": 1020}, 1), ({"ldq": 1016}, 1),
    ({"ldk": 255}, 1), ({"ldq_out": 1016}, 1), ({"ldk_out": 248}, 1), ({"rows": 5}, 1), ({"table_dev": None}, 1),
    ({"q_dev": FAKE + 2}, 1), ({"q_dev": None}, 1), ({"k_out_dev": None}, 1), ({"ws": None}, 1), ({"ws_bytes": 255}, 3),
    ({"table_row_dev": FAKE + 2}, 1), ({"table_rows": -1, "table_row_dev": FAKE}, 1),
    # outputs that lie half over the inputs, or over each other
    ({"q_out_dev": FAKE + 16, "ldq_out": 1536}, 1), ({"q_out_dev": FAKE}, 1), ({"k_out_dev": FAKE, "ldk_out": 1536}, 1),
    ({"k_out_dev": FAKE + (1 << 20) + 16}, 1), ({"q_out_dev": FAKE + 1024, "ldq_out": 1536}, 1)])
def test_qk_norm_rope_refusals(dit, change, st):
    _refused(dit, lambda: dit.dit_qk_norm_rope(**{**QK, **change}), st)


def test_nothing_to_do_is_no_launch(dit):
    before = dit.dit_launch_count()
    dit.dit_qk_norm_rope(**{**QK, "rows": 0, "q_dev": None})
    for change in ({"seqs": 0}, {"rows_q": 0}, {"max_q": 0}):
        a = dit.make_text_attn(**{**AT, **change})
        dit.dit_text_attention(a, *AT_ARGS.values(), stream=0)
    assert dit.dit_launch_count() == before


AT = dict(seqs=2, heads_q=8, heads_k=2, head_dim=128, rows_q=64, rows_k=64, max_q=40, max_k=40, causal=True, scale=0.1)
AT_ARGS = dict(q_off=FAKE, q_len=None, k_off=FAKE, k_len=None, q_dev=FAKE, ldq=1536, k_dev=FAKE + 2048, ldk=1536,
               v_dev=FAKE + 2560, ldv=1536, out_dev=FAKE + (1 << 20), ldo=1024, ws=FAKE, ws_bytes=1 << 24)


@pytest.mark.parametrize("change,st", [
    ({"head_dim": 96}, 2), ({"heads_q": 7}, 1), ({"heads_q": 0}, 1), ({"heads_k": 0}, 1), ({"heads_q": 130}, 1), ({"seqs": -1}, 1),
    ({"seqs": 16385}, 1), ({"rows_q": -1}, 1), ({"rows_k": (1 << 28) + 1}, 1), ({"max_q": -1}, 1), ({"max_k": (1 << 24) + 1}, 1),
    ({"scale": 0.0}, 1), ({"scale": -1.0}, 1), ({"scale": math.nan}, 1), ({"scale": math.inf}, 1), ({"scale": 2e30}, 1)])
def test_text_attention_size_refusals(dit, change, st):
    a = dit.make_text_attn(**{**AT, **change})
    _refused(dit, lambda: dit.dit_text_attention(a, *AT_ARGS.values(), stream=0), st)
    _refused(dit, lambda: dit.dit_text_attention_workspace(a), st)


@pytest.mark.parametrize("change,st", [
    ({"q_off": None}, 1), ({"k_off": None}, 1), ({"q_off": FAKE + 2}, 1), ({"q_len": FAKE + 1}, 1), ({"q_dev": None}, 1),
    ({"k_dev": None}, 1), ({"v_dev": FAKE + 8}, 1), ({"out_dev": None}, 1), ({"ldq": 1016}, 1), ({"ldq": 1028}, 1), ({"ldk": 248}, 1),
    ({"ldv": (1 << 24) + 8}, 1), ({"ldo": 1020}, 1), ({"ws": None}, 1), ({"ws_bytes": 255}, 3),
    # the output over the queries, the keys or the values
    ({"out_dev": FAKE}, 1), ({"out_dev": FAKE + 2048, "ldo": 1536}, 1), ({"out_dev": FAKE + 2560, "ldo": 1536}, 1)])
def test_text_attention_argument_refusals(dit, change, st):
    a = dit.make_text_attn(**AT)
    _refused(dit, lambda: dit.dit_text_attention(a, *{**AT_ARGS, **change}.values(), stream=0), st)


def test_text_attention_workspace_is_bounded(dit):
    """At least the status word, no more than a few bytes a value of the output, for any sizes."""
    for seqs, nq, nk in ((1, 1, 1 << 20), (64, 1, 8192), (16384, 1, 128), (1, 8192, 8192), (3, 17, 70000)):
        a = dit.make_text_attn(seqs, 32, 8, 128, seqs * nq, seqs * nk, nq, nk)
        n = dit.dit_text_attention_workspace(a)
        assert 256 <= n <= 256 + max(64 << 20, 0)


@pytest.mark.parametrize("args", [
    (FAKE, 128, 0, 128, 1, FAKE, FAKE), (FAKE, 128, 4, 120, 1, FAKE, FAKE), (FAKE, 120, 4, 128, 1, FAKE, FAKE),
    (FAKE, 132, 4, 128, 1, FAKE, FAKE), (FAKE, 128, 4, 128, 64, FAKE, FAKE), (FAKE, 128, 4, 128, 0, FAKE, FAKE),
    (None, 128, 4, 128, 1, FAKE, FAKE), (FAKE, 128, 4, 128, 1, FAKE + 8, FAKE), (FAKE, 128, 4, 128, 1, FAKE, None),
    (FAKE, 128, (1 << 20) + 1, 128, 1, FAKE, FAKE),
    # buffers over one another
    (FAKE, 128, 4, 128, 1, FAKE + 1008, FAKE + 4096), (FAKE, 128, 4, 128, 1, FAKE + 4096, FAKE + 4096 + 496),
    (FAKE, 128, 4, 128, 1, FAKE + 4096, FAKE + 1008)])
def test_quantize_blocks_refusals(dit, args):
    _refused(dit, lambda: dit.dit_quantize_blocks_fp8(*args, stream=0))


B1, B2, B3, B4 = (FAKE + (i << 24) for i in (1, 2, 3, 4))
LIN = dict(rows=4, n_out=128, k=256, a=B1, a_s=B2, w=B3, w_s=B4, out=FAKE, ld=128, ws=FAKE, ws_bytes=1 << 24)


@pytest.mark.parametrize("change,st", [
    ({"rows": 0}, 1), ({"rows": (1 << 20) + 1}, 1), ({"n_out": 0}, 1), ({"n_out": 132}, 1), ({"k": 0}, 1), ({"k": 264}, 1),
    ({"ld": 120}, 1), ({"ld": 132}, 1), ({"a": None}, 1), ({"a_s": FAKE + 4}, 1), ({"w": FAKE + 8}, 1), ({"w_s": None}, 1),
    ({"out": FAKE + 2}, 1), ({"ws": None}, 1), ({"ws_bytes": 255}, 3),
    # the output over an operand or its scales
    ({"out": B1 + 1008}, 1), ({"out": B2 - 16}, 1), ({"out": B3 + 16}, 1), ({"out": B4}, 1)])
def test_linear_fp8_blocks_refusals(dit, change, st):
    _refused(dit, lambda: dit.dit_linear_fp8_blocks(*{**LIN, **change}.values(), stream=0), st)


def test_linear_fp8_blocks_workspace(dit):
    """Bounded for any sizes, and refused when it is a byte short."""
    for m, n, k in ((1, 8, 16), (300, 256, 4096), (65, 128, 1 << 20), (489, 1168, 9616), (8192, 12288, 4096), (1 << 20, 8, 1 << 20)):
        assert 256 <= dit.dit_linear_fp8_blocks_workspace(m, n, k) <= 256 + 10 * (1 << 20)
    need = dit.dit_linear_fp8_blocks_workspace(300, 256, 4096)
    assert need > 256
    _refused(dit, lambda: dit.dit_linear_fp8_blocks(*{**LIN, "rows": 300, "n_out": 256, "k": 4096, "ld": 256,
                                                      "ws_bytes": need - 1}.values(), stream=0), dit.DIT_ERR_WORKSPACE)


def test_kernel_classes_have_names(dit):
    names = [dit.dit_kernel_class_name(i) for i in range(32)]
    for n in ("text_rope_table", "qk_norm_rope", "text_attention", "text_attention_join", "quantize_blocks_fp8",
              "linear_fp8_blocks", "linear_fp8_join"):
        assert names.count(n) == 1


# ------------------------------------------------------------------- the 64-bit forms themselves
def test_reference_attention_is_the_textbook_softmax():
    g = torch.Generator().manual_seed(0)
    q, k, v = (torch.randn(5, h, 64, generator=g) for h in (4, 2, 2))
    out, size, _ = R.attention(q, k, v, [(0, 5, 0, 5)], True, 0.125)
    for i in range(5):
        for h in range(4):
            s = (k[:i + 1, h // 2].double() @ q[i, h].double()) * 0.125
            torch.testing.assert_close(out[i, h], torch.softmax(s, 0) @ v[:i + 1, h // 2].double())
    assert (size >= out.abs() - 1e-12).all()


def test_reference_by_parts_keeps_fast_pairs_and_stretches_slow_ones():
    w0 = R.rope_frequencies(128, 1e6)
    w = R.rope_frequencies(128, 1e6, "by_parts", 8.0, 1.0, 4.0, 16384)
    assert w[0] == w0[0] and np.isclose(w[-1], w0[-1] / 8) and (w <= w0).all() and (w >= w0 / 8 - 1e-18).all()


def test_reference_quantiser_round_trip():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(130, 200, generator=g).to(torch.bfloat16)
    for r in (1, 128):
        q, s = R.quantize_blocks(x, r)
        err = (R.dequantize(q, s, r) - x.double()).abs()
        # half a step of three bits, or half the smallest step
        assert (err <= 2.0 ** -4 * x.double().abs() * 1.001 + 2.0 ** -10 * 448 * float(s.max()) / 448 * 1.001).all()
