"""The even shares of the attention over the 4-bit cache are as many as CTAs run at once: what the workspace has room for says how
many the plan cuts."""
import pytest

SMS = 152


@pytest.fixture(scope="module")
def dit():
    from diffusion_transformer_step_gb300 import build_lib
    build_lib.build()
    from diffusion_transformer_step_gb300 import dit as d
    d.lib()
    return d


def _shares(dit, d, hq, hk, new, seqs=32, max_k=1 << 15):
    """Shares of a long call of few rows: two rows of parts for each query row of each (8 bytes and a row of fp32, the first
    array rounded up to 256 bytes), and 16 bytes for where it cuts."""
    rows = new * hq // hk
    c = dit.make_text_cache4(hk, d, 1 << 16, 64, 1 << 10)
    need = dit.dit_text_cache4_attention_workspace(c, dit.make_text_attn(seqs, hq, hk, d, seqs * new, 0, new, max_k)) - 256
    fits = [s for s in range(1, 8 * SMS) if -(-2 * s * rows * 8 // 256) * 256 + 2 * s * rows * d * 4 + 16 * s == need]
    assert len(fits) == 1, (need, fits)
    return fits[0]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk,new,per_sm", [(8, 8, 1, 3), (32, 8, 1, 3), (64, 8, 1, 3), (8, 1, 1, 3), (72, 8, 1, 2), (96, 8, 1, 2), (24, 8, 5, 2),
                                              (16, 1, 1, 2), (8, 8, 16, 2)])
def test_shares_are_the_ctas_that_run_at_once(dit, d, hq, hk, new, per_sm):
    """Three CTAs of eight rows per SM. A CTA of sixteen has five warps of 168 registers (64-wide heads; a scheduler's 16384 hold
    three of those warps) or four of 255 (two): two per SM."""
    assert 16384 // (168 * 32) * 4 // 5 == 2 and 16384 // (255 * 32) * 4 // 4 == 2 and 16384 // (128 * 32) * 4 // 5 == 3
    assert _shares(dit, d, hq, hk, new) == per_sm * SMS
