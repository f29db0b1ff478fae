"""One dit_text_attention call on CPU tensors, for the GPU tests: laid out, run twice, its rows returned."""
import torch

DEV = "cuda"


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def attend(dit, q, k, v, spans, causal=True, scale=None, max_q=None, max_k=None):
    """q [rows_q, Hq, d], k and v [rows_k, Hk, d] bf16, spans [(q0, nq, k0, nk)].  Rows of the output that no
    sequence owns hold 5.  The workspace is exactly as large as it has to be, and behind its status block
    full of NaN.  Returns the output and the workspace's size."""
    (rows_q, hq, d), (rows_k, hk, _) = q.shape, k.shape
    a = dit.make_text_attn(len(spans), hq, hk, d, rows_q, rows_k, max(s[1] for s in spans) if max_q is None else max_q,
                           max(s[3] for s in spans) if max_k is None else max_k, causal, scale)
    ws = torch.full((dit.dit_text_attention_workspace(a),), 0xff, dtype=torch.uint8, device=DEV)
    ws[:256] = 0
    dq, dk, dv = (t.flatten(1).to(DEV) for t in (q, k, v))
    out = torch.full_like(dq, 5.0)
    lens = [i32([s[e] for s in spans] + [0]) for e in range(4)]
    bits = []
    for _ in range(2):
        dit.dit_text_attention(a, *lens, dq, hq * d, dk, hk * d, dv, hk * d, out, hq * d, ws, ws.numel())
        st, where = dit.dit_sync_status(ws)
        assert st == dit.DIT_OK, (st, hex(where))
        bits.append(out.view(torch.int16).clone())
    assert torch.equal(*bits)  # equal calls, equal bits
    return out.reshape(rows_q, hq, d).cpu(), ws.numel()


def check(got, bound):
    """Against text_reference.attention_bound."""
    want, tol, bad, owned = bound
    assert (got[~owned] == 5.0).all()
    fin = got.isfinite()
    assert torch.equal(fin[owned], ~bad[owned]), ((~fin & ~bad)[owned].sum(), (fin & bad)[owned].sum())
    err = (torch.where(bad, torch.zeros_like(got), got).double() - want).abs()
    err[~owned] = 0
    over = err > tol
    assert not over.any(), (int(over.sum()), float((err / tol.clamp(min=1e-300))[over].max()), over.nonzero()[:4].tolist())


def split_tiles_bytes(seqs, hq, hk, d, rows_q, max_q, max_k):
    """The workspace of a call (of up to 64 sequences) whose keys are split over tiles of 128 rows: two rows
    of parts per pair of tiles, key head and split."""
    up = lambda x: -(-x // 256) * 256  # noqa: E731
    pair = 2 * (128 // (hq // hk))
    tiles = min(rows_q // pair + seqs, seqs * -(-max_q // pair))
    splits = min(152 // (tiles * hk), -(-max_k // 128) // 4, 32)
    assert splits > 1
    n = tiles * hk * splits * 256
    return 256 + up(tiles * 8) + up(n * 8) + up(n * d * 4)
