"""Runs one call of the library on a seeded synthetic layer, for profiling
(ncu) and quick timing.

    python -m post_weight_quantization_awq_b200.run_case --op search --tokens 16384 \
        --in 4096 --out 4096 [--alphas 20] [--clips 20] [--bits 4] [--repeat 3] [--form gram|cached_y|fused]

--op is one of: stats, search, clip, pack, layer (all four calls), w4a16 (the
GEMM on the packed output, Y = X Wd^T with Wd = RN16((q - z) scale); with
--w4a16-form fused the weights are dequantised tile by tile inside the GEMM), and
the serving calls: lora (the packed projection with --adapters adapters of --rank
over the tokens), moe (--experts packed experts of in -> out -> in, --top-k of
them a token, up to 64 tokens), norm (rows of --in channels: residual, norm of
the block's output and the next block's norm).  Inputs follow the heavy-tailed
recipe of the synthetic module (1% outlier channels x U[20, 50], W ~ N(0,
0.02)).  Prints the CUDA-event time of the last repeat.
"""

from __future__ import annotations

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def serving(a) -> int:
    """The calls on a packed layer: lora, moe, norm."""
    import torch

    import post_weight_quantization_awq_b200 as awq
    from synthetic import OutlierSpec, gaussian_weight, heavy_tailed_activations

    T, cfg = a.tokens, awq.AwqConfig.make(w_bit=a.bits)
    X = heavy_tailed_activations(T, a.inn, OutlierSpec(0.01, 20.0, 50.0), a.seed).cuda()
    gen = torch.Generator().manual_seed(a.seed)

    def normal(*shape, std=1.0):
        return (torch.randn(shape, generator=gen) * std).half().cuda()

    def packed(out, inn, seed):
        t = (torch.empty((inn, out // 8), dtype=torch.int32, device="cuda"),
             torch.empty((inn // 128, out // 8), dtype=torch.int32, device="cuda"),
             torch.empty((inn // 128, out), dtype=torch.float16, device="cuda"))
        one = torch.ones(inn, dtype=torch.float32, device="cuda")
        awq.awq_quant_pack(gaussian_weight(out, inn, seed).cuda(), one, None, cfg, *t)
        return t

    ws = None
    if a.op == "lora":
        w = packed(a.out, a.inn, a.seed)
        A, B = normal(a.adapters, a.rank, a.inn, std=a.inn ** -0.5), normal(a.adapters, a.out, a.rank, std=0.02)
        c = torch.full((a.adapters,), 0.5, device="cuda")
        ids = torch.randint(-1, a.adapters, (T,), generator=gen, dtype=torch.int32).cuda()
        if T > 64:  # prompts: a request's tokens stand together
            ids = ids.sort().values
        Y = torch.empty((T, a.out), dtype=torch.float16, device="cuda")
        ws = torch.empty(awq.awq_w4a16_lora_workspace_size(T, a.inn, a.out, a.rank, cfg), dtype=torch.uint8,
                         device="cuda")

        def once():
            awq.awq_w4a16_lora_gemm(X, *w, cfg, A, B, c, ids, Y, ws)
    elif a.op == "moe":
        router = normal(a.experts, a.inn, std=a.inn ** -0.5)
        gu = [torch.stack(t) for t in zip(*(packed(2 * a.out, a.inn, a.seed + 2 * e) for e in range(a.experts)))]
        dn = [torch.stack(t) for t in zip(*(packed(a.inn, a.out, a.seed + 2 * e + 1) for e in range(a.experts)))]
        Y = torch.empty_like(X)
        ids = torch.empty((T, a.top_k), dtype=torch.int32, device="cuda")
        weights = torch.empty((T, a.top_k), dtype=torch.float32, device="cuda")
        ws = torch.empty(awq.awq_w4a16_moe_workspace_size(T, a.inn, a.out, a.experts, a.top_k, cfg),
                         dtype=torch.uint8, device="cuda")

        def once():
            awq.awq_w4a16_moe(X, router, gu, dn, cfg, True, None, Y, ids, weights, ws)
    else:
        R, post, pre = normal(T, a.inn), normal(a.inn), normal(a.inn)
        r, n = torch.empty_like(R), torch.empty_like(R)

        def once():
            awq.awq_block_norm(R, X, post, None, 1.0, pre, 1e-6, r, n)

    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(a.repeat):
        e0.record()
        once()
        e1.record()
    torch.cuda.synchronize()
    if ws is not None:
        awq.awq_device_status(ws)
    print(f"{a.op}: T={T} in={a.inn} out={a.out} last call {e0.elapsed_time(e1):.3f} ms")
    return 0


def main(argv=None) -> int:
    import torch

    import post_weight_quantization_awq_b200 as awq
    from synthetic import OutlierSpec, gaussian_weight, heavy_tailed_activations

    ap = argparse.ArgumentParser()
    ap.add_argument("--op", choices=("stats", "search", "clip", "pack", "layer", "w4a16", "lora", "moe", "norm"),
                    required=True)
    ap.add_argument("--tokens", type=int, default=16384)
    ap.add_argument("--in", dest="inn", type=int, default=4096)
    ap.add_argument("--out", type=int, default=4096)
    ap.add_argument("--alphas", type=int, default=20)
    ap.add_argument("--clips", type=int, default=20)
    ap.add_argument("--bits", type=int, default=4)
    ap.add_argument("--repeat", type=int, default=3)
    ap.add_argument("--seed", type=int, default=1)
    ap.add_argument("--form", choices=("direct", "gram", "cached_y", "fused"), default="direct",
                    help="alpha-search scoring form")
    ap.add_argument("--w4a16-form", choices=("auto", "fused"), default="auto",
                    help="auto: the workspace awq_w4a16_workspace_size asks for (dequantise once "
                         "for many tokens, split-K for few); fused: 256 bytes (dequantise per tile)")
    ap.add_argument("--rank", type=int, default=16, help="lora: the adapters' rank")
    ap.add_argument("--adapters", type=int, default=8, help="lora: their number")
    ap.add_argument("--experts", type=int, default=8, help="moe: the number of experts")
    ap.add_argument("--top-k", type=int, default=2, help="moe: experts of a token")
    a = ap.parse_args(argv)
    if a.op in ("lora", "moe", "norm"):
        return serving(a)

    X = heavy_tailed_activations(a.tokens, a.inn, OutlierSpec(0.01, 20.0, 50.0), a.seed).cuda()
    W = gaussian_weight(a.out, a.inn, a.seed).cuda()
    cfg = awq.AwqConfig.make(w_bit=a.bits, n_alpha=a.alphas, n_clip=a.clips,
                             search_form={"direct": awq.abi.SEARCH_DIRECT, "gram": awq.abi.SEARCH_GRAM,
                                          "cached_y": awq.abi.SEARCH_CACHED_Y,
                                          "fused": awq.abi.SEARCH_FUSED}[a.form])
    ws = awq.alloc_workspace(a.tokens, a.inn, a.out, cfg)
    abar = torch.empty(a.inn, dtype=torch.float64, device="cuda")
    mse = torch.empty(a.alphas, dtype=torch.float64, device="cuda")
    best = torch.empty(1, dtype=torch.int32, device="cuda")
    s_best = torch.ones(a.inn, dtype=torch.float32, device="cuda")
    clip_idx = torch.zeros((a.out, a.inn // 128), dtype=torch.uint8, device="cuda")
    g = 128
    qw = torch.empty((a.inn, a.out // 8), dtype=torch.int32, device="cuda")
    qz = torch.empty((a.inn // g, a.out // 8), dtype=torch.int32, device="cuda")
    sc = torch.empty((a.inn // g, a.out), dtype=torch.float16, device="cuda")
    awq.awq_act_stats(X, abar)
    if a.op == "w4a16":
        awq.awq_quant_pack(W, s_best, None, cfg, qw, qz, sc)
        Y = torch.empty((a.tokens, a.out), dtype=torch.float16, device="cuda")
        nws = 256 if a.w4a16_form == "fused" else awq.awq_w4a16_workspace_size(a.tokens, a.inn, a.out, cfg)
        ws16 = torch.empty(nws, dtype=torch.uint8, device="cuda")

    def once():
        if a.op == "stats":
            awq.awq_act_stats(X, abar)
        elif a.op == "search":
            awq.awq_search_scale(X, W, abar, cfg, ws, s_best, mse, best)
        elif a.op == "clip":
            awq.awq_search_clip(X, W, s_best, cfg, ws, clip_idx)
        elif a.op == "pack":
            awq.awq_quant_pack(W, s_best, clip_idx if a.clips else None, cfg, qw, qz, sc)
        elif a.op == "w4a16":
            awq.awq_w4a16_gemm(X, qw, qz, sc, cfg, Y, ws16)
        else:
            awq.quantize_layer(X, W, cfg, ws=ws)

    e0, e1 = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for _ in range(a.repeat):
        e0.record()
        once()
        e1.record()
    torch.cuda.synchronize()
    awq.awq_device_status(ws)
    ms = e0.elapsed_time(e1)
    extra = ""
    if a.op == "w4a16":
        extra = f", {2.0 * a.tokens * a.inn * a.out / (ms * 1e-3) / 1e12:.1f} TFLOP/s"
    print(f"{a.op}: T={a.tokens} in={a.inn} out={a.out} last call {ms:.3f} ms{extra}")
    return 0


if __name__ == "__main__":
    sys.exit(main())
