"""Small fixed cases for profiler captures: one dual-stream or single-stream block at the
1024x1024 shape (512 text + 4096 image tokens, hidden 3072), or the per-step modulation at
klein width (batch 1), run `--reps` times through the C ABI.  About 1 GB on the device for
a block (its GEMMs read more than the 129 MB L2); 341 MB of modulation weights for the
modulation.

    python -m diffusion_transformer_step_gb300.profile_case --block single --reps 2
    python -m diffusion_transformer_step_gb300.profile_case --block modulation --reps 3
    python -m diffusion_transformer_step_gb300.profile_case --block single --fp8 --reps 2

The text-side operations at one size each: attention of a 4096-token causal prompt (32 query heads
on 8 of 128), of 16 new tokens over 8192 keys, the block-scaled e4m3 product 4096 x 4864 x 4096, norm
and rotation of 40000 rows of 40 heads of 128.

    python -m diffusion_transformer_step_gb300.profile_case --text attention --reps 2
    python -m diffusion_transformer_step_gb300.profile_case --text decode --reps 2
    python -m diffusion_transformer_step_gb300.profile_case --text linear --reps 2
    python -m diffusion_transformer_step_gb300.profile_case --text qk --reps 2

The norm of 16384 rows of 4096 with residual and both outputs, the product 4096 x 4096 x 4096 with bias, SiLU
and residual, 512 new tokens into the 4-bit cache of each of 16 sequences of 8192 and all of them read back, 16 new tokens
over that cache (one each).

    python -m diffusion_transformer_step_gb300.profile_case --text norm --reps 2
    python -m diffusion_transformer_step_gb300.profile_case --text linear_act --reps 2
    python -m diffusion_transformer_step_gb300.profile_case --text cache4 --reps 2
    python -m diffusion_transformer_step_gb300.profile_case --text decode4 --reps 2

`--fp8` runs the block with every projection in e4m3 (per-row activation and per-output-channel
weight scales, the library's low-precision variant).
"""
import argparse

import torch

from diffusion_transformer_step_gb300 import build_lib, dit, synth


def text_case(kind, reps):
    dev, hq, hk, d = "cuda", 32, 8, 128
    g = synth.generator(0, dev)
    ws = torch.zeros(64 << 20, dtype=torch.uint8, device=dev)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    if kind in ("attention", "decode"):
        seqs, nq, nk = (1, 4096, 4096) if kind == "attention" else (16, 1, 8192)
        q = synth.normal((seqs * nq, hq * d), 1.0, g, dev)
        kv = synth.normal((seqs * nk, 2 * hk * d), 1.0, g, dev)
        out = torch.empty_like(q)
        a = dit.make_text_attn(seqs, hq, hk, d, seqs * nq, seqs * nk, nq, nk)
        qo, ko = i32([i * nq for i in range(seqs + 1)]), i32([i * nk for i in range(seqs + 1)])
        run = lambda: dit.dit_text_attention(a, qo, None, ko, None, q, hq * d, kv, 2 * hk * d, kv[:, hk * d:],  # noqa: E731
                                             2 * hk * d, out, hq * d, ws, ws.numel())
    elif kind == "linear":
        m, n, k = 4096, 4864, 4096
        x, w = synth.normal((m, k), 1.0, g, dev), synth.normal((n, k), 0.02, g, dev)
        aq, wq = (torch.empty((r, k), dtype=torch.uint8, device=dev) for r in (m, n))
        a_s, w_s = torch.empty((m, k // 128), device=dev), torch.empty((n // 128, k // 128), device=dev)
        dit.dit_quantize_blocks_fp8(w, k, n, k, 128, wq, w_s)
        out = torch.empty((m, n), dtype=torch.bfloat16, device=dev)

        def run():
            dit.dit_quantize_blocks_fp8(x, k, m, k, 1, aq, a_s)
            dit.dit_linear_fp8_blocks(m, n, k, aq, a_s, wq, w_s, out, n, ws, ws.numel())
    elif kind == "norm":
        rows, cols = 16384, 4096
        x, res = (synth.normal((rows, cols), 1.0, g, dev) for _ in range(2))
        w = torch.ones(cols, dtype=torch.bfloat16, device=dev)
        s, y = torch.empty_like(x), torch.empty_like(x)
        q, sc = torch.empty((rows, cols), dtype=torch.uint8, device=dev), torch.empty((rows, cols // 128), device=dev)
        run = lambda: dit.dit_add_rms_norm(rows, cols, x, cols, res, cols, w, 0.0, 1e-6, s, cols, y, cols, q, sc)  # noqa: E731
    elif kind == "linear_act":
        m = n = k = 4096
        x, w, res = synth.normal((m, k), 1.0, g, dev), synth.normal((n, k), 0.02, g, dev), synth.normal((m, n), 1.0, g, dev)
        b, out = synth.normal((n,), 1.0, g, dev), torch.empty((m, n), dtype=torch.bfloat16, device=dev)
        run = lambda: dit.dit_linear_act(m, n, k, x, k, w, k, b, dit.DIT_ACT_SILU, res, n, out, n, False, ws, ws.numel())  # noqa: E731
    elif kind in ("cache4", "decode4"):
        seqs, nk, page, nq = 16, 8192, 64, 512 if kind == "cache4" else 1
        c = dit.make_text_cache4(hk, d, seqs * nk // page, page, nk // page)
        cache = torch.empty(dit.dit_text_cache4_bytes(c), dtype=torch.uint8, device=dev)
        pages = torch.randperm(c.pages, generator=g, device=dev).to(torch.int32)
        kv = synth.normal((seqs * nk, 2 * hk * d), 1.0, g, dev)
        v, wide = kv[:, hk * d:], 2 * hk * d
        full, kl, qo = i32([i * nk for i in range(seqs + 1)]), i32([nk] * seqs), i32([i * nq for i in range(seqs + 1)])
        dit.dit_text_cache4_append(c, seqs, seqs * nk, nk, full, None, kl, pages, kv, wide, v, wide, cache, ws, ws.numel())
        if kind == "cache4":
            out = torch.empty_like(kv)

            def run():
                dit.dit_text_cache4_append(c, seqs, seqs * nq, nq, qo, None, kl, pages, kv, wide, v, wide, cache, ws, ws.numel())
                dit.dit_text_cache4_read(c, seqs, seqs * nk, nk, full, None, pages, cache, out, wide, out[:, hk * d:], wide, ws,
                                         ws.numel())
        else:
            q = synth.normal((seqs, hq * d), 1.0, g, dev)
            out = torch.empty_like(q)
            a = dit.make_text_attn(seqs, hq, hk, d, seqs, 0, 1, nk)
            run = lambda: dit.dit_text_cache4_attention(c, a, qo, None, kl, pages, q, hq * d, cache, out, hq * d, ws,  # noqa: E731
                                                        ws.numel())
    else:
        rows, wide = 40000, (hq + hk) * d
        x = synth.normal((rows, wide), 1.0, g, dev)
        w = torch.ones(d, dtype=torch.bfloat16, device=dev)
        table = torch.empty((rows, d // 2, 2), device=dev)
        dit.dit_text_rope_table(dit.make_text_rope(d, 1e6), None, rows, table)
        out = torch.empty_like(x)
        run = lambda: dit.dit_qk_norm_rope(rows, hq, hk, d, d, dit.DIT_ROPE_HALF, x, wide, x[:, hq * d:], wide, w, w,  # noqa: E731
                                           1e-6, table, rows, None, out, wide, out[:, hq * d:], wide, ws, ws.numel())
    for _ in range(reps):
        run()
    st, where = dit.dit_sync_status(ws)
    assert st == dit.DIT_OK, f"status {st} at site {where:#x}"
    print(f"profile_case text {kind} x{reps}: ok")


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--block", choices=["single", "dual", "modulation"], default="single")
    ap.add_argument("--reps", type=int, default=2)
    ap.add_argument("--fp8", action="store_true", help="every block projection in e4m3")
    ap.add_argument("--text", choices=["attention", "decode", "linear", "qk", "norm", "linear_act", "cache4", "decode4"])
    args = ap.parse_args()
    build_lib.build()
    if args.text:
        text_case(args.text, args.reps)
        return
    dev = "cuda"
    wl = synth.WORKLOADS["single_block_1024"]
    wd = wl.widths
    g = synth.generator(0, dev)
    if args.block == "modulation":
        W = dit.DeviceWeights(wd, {"mod": synth.mod_weights(wd, g, dev), "dual": [], "single": []}, device=dev)
        sigma = torch.full((1,), 0.75, dtype=torch.float32, device=dev)
        mod = torch.empty((1, 17 * wd.hidden), dtype=torch.bfloat16, device=dev)
        ws = torch.zeros(1 << 20, dtype=torch.uint8, device=dev)
        for _ in range(args.reps):
            dit.dit_modulation(W.w, sigma, 1, mod, ws, ws.numel())
        st, where = dit.dit_sync_status(ws)
        assert st == dit.DIT_OK, f"device wait gave up at site {where:#x}"
        print(f"profile_case modulation x{args.reps}: ok")
        return
    if args.block == "dual":
        logical = {"dual": [(synth.stream_weights(wd, g, dev), synth.stream_weights(wd, g, dev))], "single": []}
    else:
        logical = {"dual": [], "single": [synth.single_weights(wd, g, dev)]}
    W = dit.DeviceWeights(wd, logical, device=dev, fp8="all" if args.fp8 else False)
    bi = synth.block_inputs(wl, 0, dev)
    shape = dit.make_shape(wl.batch, wl.n_txt, wl.n_img, wl.n_ref)
    ids = dit.dit_token_ids(shape, *wl.grid)
    N = wl.n_tokens
    rope = torch.empty((N, 64, 2), dtype=torch.float32, device=dev)
    dit.dit_rope_table(W.cfg, ids.to(dev), N, rope)
    nbytes = dit.dit_workspace_size(W.cfg, shape)
    ws = torch.zeros(nbytes, dtype=torch.uint8, device=dev)
    fwd = dit.dit_dual_block_fwd if args.block == "dual" else dit.dit_single_block_fwd
    for _ in range(args.reps):
        fwd(W.w, 0, shape, bi["x"], bi["mod"], rope, ws, nbytes)
    st, where = dit.dit_sync_status(ws)
    assert st == dit.DIT_OK, f"device wait gave up at site {where:#x}"
    print(f"profile_case {args.block}{' e4m3' if args.fp8 else ''} x{args.reps}: ok")


if __name__ == "__main__":
    main()
