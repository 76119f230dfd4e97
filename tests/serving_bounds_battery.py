"""Runs every serving call on ragged shapes and saves the results (imported by
test_gpu_serving_bounds.py, which runs it once with the debug library, AWQ_LIB=debug,
and once with the release library in child processes).  Usage:
python tests/serving_bounds_battery.py OUT.pt"""

import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import post_weight_quantization_awq_b200 as awq  # noqa: E402


def _randn(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g) * std).half().cuda()


def _packed(g, lead, inn, out, group):
    words = lambda *s: torch.randint(-2 ** 31, 2 ** 31 - 1, s, generator=g, dtype=torch.int64).to(torch.int32).cuda()  # noqa: E731
    return (words(*lead, inn, out // 8), words(*lead, inn // group, out // 8),
            (torch.rand((*lead, inn // group, out), generator=g) * 0.01 + 0.001).half().cuda())


def run(out_path: str) -> None:
    res = {}
    # adapters: each tile of tokens, whole and in groups of 16, both forms past 64 tokens
    # (a request per token and in runs), ranks of several passes, odd values
    for T, inn, out, rank, n, group, odd in [
            (1, 192, 96, 8, 1, 64, False), (5, 1024, 288, 24, 3, 128, True), (13, 320, 544, 40, 4, 32, False),
            (20, 512, 8224, 16, 3, 64, False), (45, 256, 800, 72, 5, 64, True), (64, 128, 32768, 8, 4, 64, False),
            (65, 64, 32, 256, 9, 64, False), (130, 192, 288, 24, 3, 32, True), (300, 512, 544, 136, 40, 128, False),
            (700, 256, 8224, 16, 3, 128, True)]:
        g = torch.Generator().manual_seed(T + out)
        X, (q, z, s) = _randn(g, T, inn), _packed(g, (), inn, out, group)
        A, B = _randn(g, n, rank, inn, std=inn ** -0.5), _randn(g, n, out, rank, std=0.1)
        c = (torch.rand(n, generator=g) + 0.5).cuda()
        ids = torch.randint(-1, n, (T,), generator=g, dtype=torch.int32)
        if T % 2 == 0:
            ids = ids.sort().values
        if odd:
            B[0, out - 1, rank - 1] = float("inf")
            c[n - 1] = 3e5
        cfg = awq.AwqConfig.make(group_size=group)
        Y = torch.empty((T, out), dtype=torch.float16, device="cuda")
        ws = torch.empty(awq.awq_w4a16_lora_workspace_size(T, inn, out, rank, cfg), dtype=torch.uint8, device="cuda")
        awq.awq_w4a16_lora_gemm(X, q, z, s, cfg, A, B, c, ids.cuda(), Y, ws)
        awq.awq_device_status(ws)
        res[f"lora{T}"] = Y.cpu()
    # experts: logits alone and together, H by each block and between barriers, entries of
    # more than 24 tokens, padding
    for T, hidden, inter, E, k, group, masked in [
            (1, 512, 320, 4, 2, 64, False), (3, 192, 704, 33, 7, 32, True), (8, 576, 2112, 16, 4, 64, False),
            (9, 1088, 64, 5, 3, 64, True), (37, 256, 1408, 16, 4, 32, True), (64, 640, 896, 3, 2, 128, False),
            (64, 128, 128, 256, 16, 64, False)]:
        g = torch.Generator().manual_seed(T + inter)
        X, router = _randn(g, T, hidden), _randn(g, E, hidden, std=0.05)
        gu, dn = _packed(g, (E,), hidden, 2 * inter, group), _packed(g, (E,), inter, hidden, group)
        mask = (torch.arange(T) % 3 != 1).to(torch.uint8).cuda() if masked else None
        cfg = awq.AwqConfig.make(group_size=group)
        Y = torch.empty_like(X)
        ids = torch.empty((T, k), dtype=torch.int32, device="cuda")
        wt = torch.empty((T, k), dtype=torch.float32, device="cuda")
        ws = torch.empty(awq.awq_w4a16_moe_workspace_size(T, hidden, inter, E, k, cfg), dtype=torch.uint8,
                         device="cuda")
        awq.awq_w4a16_moe(X, router, gu, dn, cfg, True, mask, Y, ids, wt, ws)
        awq.awq_device_status(ws)
        res[f"moe{T}_{E}"] = {"Y": Y.cpu(), "ids": ids.cpu(), "wt": wt.cpu()}
    # norms: each team of threads
    for T, d in [(3, 8), (7, 264), (5, 520), (4, 1032), (9, 2056), (3, 4104), (2, 8200), (3, 16392), (2, 32768)]:
        g = torch.Generator().manual_seed(d)
        R, V, gate, post, pre = (_randn(g, *s) for s in ((T, d), (T, d), (T, d), (d,), (d,)))
        r, n = torch.empty_like(R), torch.empty_like(R)
        awq.awq_block_norm(R, V, post, gate, 0.5, pre, 1e-6, r, n)
        res[f"norm{d}"] = {"r": r.cpu(), "n": n.cpu()}
    torch.cuda.synchronize()
    ok, message = True, ""
    try:
        awq.awq_bounds_status()
    except awq.AwqError as e:
        ok, message = False, str(e)
    res["bounds"] = {"enabled": awq.awq_bounds_checks_enabled(), "ok": ok, "message": message}
    torch.save(res, out_path)


if __name__ == "__main__":
    run(sys.argv[1])
