"""Prompts padded to a fixed number of rows whose padding rows are queries too, as the step reads its text
features: row i of a prompt of n tokens sees the keys j <= i that are tokens.  That is two calls of
dit_text_attention on one output: the tokens, causal, and the padding rows over all tokens, without a mask."""
import pytest
import torch

import text_reference as R
from attention_calls import DEV, check, i32
from test_text_ops_gpu import _randn, dit  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hk,d,rows,lens", [(32, 8, 128, 512, [77, 512, 1, 300]), (32, 8, 128, 512, [9]), (8, 8, 64, 96, [0, 95, 96, 31])])
def test_padding_rows_are_queries(dit, hq, hk, d, rows, lens):  # noqa: F811
    n, b = rows * len(lens), len(lens)
    q, k, v = _randn(n, hq, d, seed=1), _randn(n, hk, d, seed=2), _randn(n, hk, d, seed=3)
    qkv = torch.cat([t.flatten(1) for t in (q, k, v)], 1).to(DEV)
    ld = qkv.shape[1]
    out = torch.full((n, hq * d), 5.0, dtype=torch.bfloat16, device=DEV)
    # the lengths stay on the device, so a captured pair of calls replays with others
    start, tokens = i32([rows * i for i in range(b)] + [n]), i32(lens)
    rest_start, rest = start[:-1] + tokens, rows - tokens
    calls = [(dit.make_text_attn(b, hq, hk, d, n, n, rows, rows, causal=True), start, tokens),
             (dit.make_text_attn(b, hq, hk, d, n, n, rows, rows, causal=False), rest_start, rest)]
    ws = torch.zeros(max(dit.dit_text_attention_workspace(c[0]) for c in calls), dtype=torch.uint8, device=DEV)

    def run():
        for a, q_off, q_len in calls:
            dit.dit_text_attention(a, q_off, q_len, start, tokens, qkv, ld, qkv[:, hq * d:], ld, qkv[:, (hq + hk) * d:], ld, out,
                                   hq * d, ws, ws.numel())
    run()
    assert dit.dit_sync_status(ws)[0] == dit.DIT_OK
    spans = [[(rows * i, m, rows * i, m) for i, m in enumerate(lens)],
             [(rows * i + m, rows - m, rows * i, m) for i, m in enumerate(lens)]]
    got = out.reshape(n, hq, d).cpu()
    for s, causal in zip(spans, (True, False)):
        want, tol, bad, owned = R.attention_bound(q, k, v, s, causal, d ** -0.5)
        part = torch.where(owned[:, None, None], got, torch.full_like(got, 5.0))
        check(part, (want, tol, bad, owned))
    first = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        run()
    out.fill_(5.0)
    graph.replay()
    assert dit.dit_sync_status(ws)[0] == dit.DIT_OK and torch.equal(first, out)
