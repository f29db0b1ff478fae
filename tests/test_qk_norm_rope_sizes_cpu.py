"""Rows x heads of dit_qk_norm_rope beyond what one launch covers: refused as an argument, before any launch."""
import pytest

FAKE = 1 << 16  # 16-byte aligned, never dereferenced


@pytest.mark.parametrize("rows,heads_q,heads_k", [(1 << 26, 1024, 1024), (1 << 26, 512, 1), (1 << 26, 1, 512), (34000000, 1024, 8)])
def test_too_many_heads_are_refused(rows, heads_q, heads_k):
    from diffusion_transformer_step_gb300 import build_lib
    build_lib.build()
    from diffusion_transformer_step_gb300 import dit
    before = dit.dit_launch_count()
    for d in (64, 128):
        far = [FAKE + (i << 52) for i in range(4)]  # buffers of terabytes, apart from one another
        ld = 1024 * d
        with pytest.raises(dit.DitError) as e:
            dit.dit_qk_norm_rope(rows, heads_q, heads_k, d, 0, dit.DIT_ROPE_HALF, far[0], ld, far[1], ld, None, None, 1e-6, None, 0,
                                 None, far[2], ld, far[3], ld, FAKE, 256, stream=0)
        assert e.value.status == dit.DIT_ERR_INVALID_ARG
    assert dit.dit_launch_count() == before
