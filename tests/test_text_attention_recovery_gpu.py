"""What a workspace is left with, and how dit_sync_status makes it usable again."""
import pytest
import torch

import text_reference as R
from test_text_ops_gpu import DEV, _check_attention, _ok, _randn, dit  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("left", [(0, 0, 5, 0), (0, 0, 0, 3), (0, 0, 0xffffffff, 0xffffffff), (0, 0x501, 7, 1)])
def test_sync_status_zeroes_the_work_counters(dit, left):  # noqa: F811
    """Counters that a call did not leave at zero (a workspace never zeroed, two calls at once on it)
    would make the next call skip items; after dit_sync_status the next call is right."""
    hq, hk, d, n = 32, 8, 128, 400
    q, k, v = _randn(n, hq, d, seed=1), _randn(n, hk, d, seed=2), _randn(n, hk, d, seed=3)
    a = dit.make_text_attn(1, hq, hk, d, n, n, n, n)
    ws = torch.zeros(dit.dit_text_attention_workspace(a), dtype=torch.uint8, device=DEV)
    words = ws[:16].view(torch.int32)
    words.copy_(torch.tensor([x - (1 << 32) if x >= 1 << 31 else x for x in left], dtype=torch.int32))
    assert dit.dit_sync_status(ws)[0] == dit.DIT_OK
    assert (words == 0).all()
    off = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    out = torch.zeros(n, hq * d, dtype=torch.bfloat16, device=DEV)
    dev = [t.flatten(1).to(DEV) for t in (q, k, v)]
    dit.dit_text_attention(a, off, None, off, None, dev[0], hq * d, dev[1], hk * d, dev[2], hk * d, out, hq * d, ws, ws.numel())
    _ok(dit, ws)
    assert (words == 0).all()
    want, size, _ = R.attention(q, k, v, [(0, n, 0, n)], True, d ** -0.5)
    _check_attention(out.reshape(n, hq, d).cpu(), want, size, (q, k, d ** -0.5))


def test_sync_status_reports_once_and_clears(dit):  # noqa: F811
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    for word, want in ((1, dit.DIT_ERR_TIMEOUT), (4, dit.DIT_ERR_INVALID_ARG), (5, dit.DIT_ERR_TIMEOUT)):
        ws[:16].view(torch.int32).copy_(torch.tensor([word, 0x501, 2, 1], dtype=torch.int32))
        assert dit.dit_sync_status(ws) == (want, 0x501)
        assert (ws == 0).all()
        assert dit.dit_sync_status(ws) == (dit.DIT_OK, 0)


@pytest.mark.parametrize("byte", [0xff, 0x7f, 0x00])
@pytest.mark.parametrize("seqs", [2, 70])
def test_split_tiles_whatever_the_workspace_held(dit, byte, seqs):  # noqa: F811
    """Tiles whose keys are split: only the status block has to be zero.  The last sequence's length is
    out of range, so its tiles have no rows to join; it is left, the others are right."""
    hq, hk, d = 3, 1, 128
    nq, nk = (300, 3366) if seqs == 2 else (4, 3366)
    ql = [nq] + [1] * (seqs - 2) + [2]
    q, k, v = _randn(sum(ql), hq, d, seed=1), _randn(nk, hk, d, seed=2), _randn(nk, hk, d, seed=3)
    qo = [sum(ql[:i]) for i in range(seqs + 1)]
    a = dit.make_text_attn(seqs, hq, hk, d, sum(ql), nk, 300, nk)
    ws = torch.full((dit.dit_text_attention_workspace(a),), byte, dtype=torch.uint8, device=DEV)
    assert ws.numel() > 256 * 1024  # parts
    ws[:256] = 0
    i32 = lambda t: torch.tensor(t, dtype=torch.int32, device=DEV)  # noqa: E731
    out = torch.full((sum(ql), hq * d), 5.0, dtype=torch.bfloat16, device=DEV)
    dev = [t.flatten(1).to(DEV) for t in (q, k, v)]
    dit.dit_text_attention(a, i32(qo), None, i32([0] * seqs), i32([nk] * (seqs - 1) + [nk + 1]), dev[0], hq * d, dev[1], hk * d,
                           dev[2], hk * d, out, hq * d, ws, ws.numel())
    assert dit.dit_sync_status(ws) == (dit.DIT_ERR_INVALID_ARG, 0x501)
    n = sum(ql) - 2
    assert (out[n:] == 5.0).all()
    want, size, _ = R.attention(q[:n], k, v, [(qo[i], ql[i], 0, nk) for i in range(seqs - 1)], True, d ** -0.5)
    _check_attention(out[:n].reshape(n, hq, d).cpu(), want, size, (q[:n], k, d ** -0.5))
