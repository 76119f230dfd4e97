"""The serving calls as a decoder block runs them, on a projection that the
library quantised itself: norm, packed projection with adapters, residual and
norm, mixture-of-experts layer on packed experts, residual and norm.  Every
stage is checked against its fp64 form on the inputs that it got, and the whole
chain captured into a graph and replayed gives the bits of the eager calls."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import post_weight_quantization_awq_b200 as awq
from gpu_helpers import need_cuda
from serving_oracle import block_norm, lora, lora_tolerance, moe, random_packed, ulp16
from synthetic import OutlierSpec, gaussian_weight, heavy_tailed_activations

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    need_cuda()


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class Block:
    """d -> d projection with adapters, and E experts of d -> inter -> d."""

    def __init__(self, T, d=512, inter=320, E=6, k=2, rank=16, adapters=3, seed=1):
        rng = np.random.default_rng(seed)
        self.T, self.d, self.k, self.rank = T, d, k, rank
        X = heavy_tailed_activations(max(T, 64), d, OutlierSpec(0.01, 20.0, 50.0), seed).cuda()
        q = awq.quantize_layer(X, gaussian_weight(d, d, seed).cuda(), awq.AwqConfig.make())
        self.packed = [q.qweight, q.qzeros, q.scales]
        # the projection's input is divided by s: folded into the norm before it
        self.pre1 = _dev((1 + 0.1 * rng.standard_normal(d)).astype(np.float16))
        awq.awq_fold_inv_scale(self.pre1, q.s_best)
        self.cfg, self.cfg64 = awq.AwqConfig.make(), awq.AwqConfig.make(group_size=64)
        f = lambda *s: rng.standard_normal(s).astype(np.float16)  # noqa: E731
        self.A, self.B = f(adapters, rank, d) * np.float16(d ** -0.5), f(adapters, d, rank) * np.float16(0.1)
        self.c = rng.uniform(0.5, 2, adapters).astype(np.float32)
        self.ids = rng.integers(-1, adapters, T).astype(np.int32)
        self.router = (f(E, d) * np.float16(0.05))
        self.gu = [random_packed(d, 2 * inter, 64, rng) for _ in range(E)]
        self.dn = [random_packed(inter, d, 64, rng) for _ in range(E)]
        self.post, self.pre2, self.pre3 = f(d), f(d), f(d)
        self.mask = (np.arange(T) % 7 != 3).astype(np.uint8)
        self.r0 = f(T, d) * np.float16(2)
        h = lambda *s: torch.full(s, 3.0, dtype=torch.float16, device="cuda")  # noqa: E731
        self.t = dict(r0=_dev(self.r0), n1=h(T, d), p=h(T, d), r1=h(T, d), n2=h(T, d), y=h(T, d), r2=h(T, d),
                      n3=h(T, d), eids=torch.empty((T, k), dtype=torch.int32, device="cuda"),
                      wt=torch.empty((T, k), dtype=torch.float32, device="cuda"))
        self.w = dict(A=_dev(self.A), B=_dev(self.B), c=_dev(self.c), ids=_dev(self.ids), router=_dev(self.router),
                      gu=[_dev(np.stack([p[i] for p in self.gu])) for i in range(3)],
                      dn=[_dev(np.stack([p[i] for p in self.dn])) for i in range(3)],
                      post=_dev(self.post), pre2=_dev(self.pre2), pre3=_dev(self.pre3), mask=_dev(self.mask))
        b = lambda n: torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda")  # noqa: E731
        self.ws1 = b(awq.awq_w4a16_lora_workspace_size(T, d, d, rank, self.cfg))
        self.ws2 = b(awq.awq_w4a16_moe_workspace_size(T, d, inter, E, k, self.cfg64))

    def step(self):
        t, w = self.t, self.w
        awq.awq_block_norm(t["r0"], None, None, None, 1.0, self.pre1, 1e-6, None, t["n1"])
        awq.awq_w4a16_lora_gemm(t["n1"], *self.packed, self.cfg, w["A"], w["B"], w["c"], w["ids"], t["p"], self.ws1)
        awq.awq_block_norm(t["r0"], t["p"], None, None, 1.0, w["pre2"], 1e-6, t["r1"], t["n2"])
        awq.awq_w4a16_moe(t["n2"], w["router"], w["gu"], w["dn"], self.cfg64, True, w["mask"], t["y"], t["eids"],
                          t["wt"], self.ws2)
        awq.awq_block_norm(t["r1"], t["y"], w["post"], None, 0.5, w["pre3"], 1e-6, t["r2"], t["n3"])

    def status(self):
        awq.awq_device_status(self.ws1)
        awq.awq_device_status(self.ws2)

    def host(self, name):
        return self.t[name].cpu().numpy()


def _norm_close(got, want, part, d):
    """test_gpu_block_norm's bound, for both outputs."""
    rel = (8 + d / 64 + 8 + 2) * 2.0 ** -24
    r, n = want
    if got[0] is not None:
        assert np.all(np.abs(got[0] - r) <= rel * part + 0.5 * ulp16(np.abs(r) + rel * part))
    tol = rel * (part * np.where(r == 0, 0, np.abs(n) / np.maximum(np.abs(r), 1e-30)) + 2 * np.abs(n))
    assert np.all(np.abs(got[1] - n) <= tol + 0.5 * ulp16(np.abs(n) + tol))


@pytest.mark.parametrize("T", [1, 7, 20, 64])
def test_block_stage_by_stage_and_replayed(T):
    b = Block(T)
    b.step()
    b.status()
    h = {k: b.host(k) for k in b.t}
    f = {k: v.astype(np.float64) for k, v in h.items()}
    pre1 = b.pre1.cpu().numpy()
    _norm_close((None, f["n1"]), block_norm(b.r0, None, None, None, 1.0, pre1, 1e-6), np.abs(f["r0"]), b.d)
    packed = [p.cpu().numpy() for p in b.packed]
    Y, mags = lora(h["n1"], packed, 128, b.A, b.B, b.c, b.ids)
    assert np.all(np.abs(f["p"] - Y) <= lora_tolerance(Y, mags, b.d, b.rank, rounded=False))
    want = block_norm(b.r0, h["p"], None, None, 1.0, b.pre2, 1e-6)
    _norm_close((f["r1"], f["n2"]), want, np.abs(f["r0"]) + np.abs(want[0] - f["r0"]), b.d)
    Y, ids, wt, tol = moe(h["n2"], b.router, b.gu, b.dn, 64, b.k, True, b.mask)
    assert np.array_equal(h["eids"], ids) and np.all(np.abs(h["wt"] - wt) <= 2.0 ** -19 * wt + 2.0 ** -140)
    assert np.all(np.abs(f["y"] - Y) <= tol) and not f["y"][b.mask == 0].any()
    want = block_norm(h["r1"], h["y"], b.post, None, 0.5, b.pre3, 1e-6)
    _norm_close((f["r2"], f["n3"]), want, np.abs(f["r1"]) + np.abs(want[0] - f["r1"]), b.d)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        b.step()
    for k in b.t:
        if k != "r0":
            b.t[k].zero_()
    for _ in range(3):
        g.replay()
    b.status()
    for k in b.t:
        assert np.array_equal(b.host(k).view(np.uint8), h[k].view(np.uint8)), k
    del g


CAPTURE_FIRST = """
import torch
from test_gpu_serving_chain import Block
b = Block({T})
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    b.step()
g.replay()
b.status()
got = {{k: v.clone() for k, v in b.t.items()}}
b.step()
b.status()
assert all(torch.equal(v, got[k]) for k, v in b.t.items())
print("same")
"""


@pytest.mark.parametrize("T", [5, 33])
def test_block_captured_by_its_first_call(T):
    """In a process whose first serving calls are the captured ones."""
    here = os.path.dirname(os.path.abspath(__file__))
    env = dict(os.environ, PYTHONPATH=os.pathsep.join([os.path.dirname(here), here]))
    r = subprocess.run([sys.executable, "-c", CAPTURE_FIRST.format(T=T)], env=env, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("args", [
    "--op lora --tokens 3 --in 512 --out 256 --adapters 2", "--op lora --tokens 100 --in 512 --out 288 --rank 24",
    "--op moe --tokens 5 --in 256 --out 384 --experts 4 --top-k 3", "--op norm --tokens 70 --in 4096"])
def test_run_case_serving_ops(args, capsys):
    from post_weight_quantization_awq_b200 import run_case
    assert run_case.main(args.split() + ["--repeat", "2"]) == 0
    assert args.split()[1] + ": T=" in capsys.readouterr().out


@pytest.mark.parametrize("T", [3, 40])
def test_calls_behind_two_streams_that_join(T):
    """Each call's inputs come from two streams that meet before it (X from one, the
    residual from another), captured and eager: the call waits for both."""
    b = Block(T)
    b.step()
    b.status()
    want = {k: v.clone() for k, v in b.t.items()}
    src = {k: want[k].clone() for k in ("n1", "r0", "p", "n2", "r1", "y")}
    big = torch.zeros((64 << 20,), device="cuda")
    side = torch.cuda.Stream()

    def calls():
        t, w = b.t, b.w
        main = torch.cuda.current_stream()
        for first, second, call in (
                ("n1", "r0", lambda: awq.awq_w4a16_lora_gemm(t["n1"], *b.packed, b.cfg, w["A"], w["B"], w["c"],
                                                             w["ids"], t["p"], b.ws1)),
                ("r0", "p", lambda: awq.awq_block_norm(t["r0"], t["p"], None, None, 1.0, w["pre2"], 1e-6, t["r1"],
                                                       t["n2"])),
                ("n2", "r1", lambda: awq.awq_w4a16_moe(t["n2"], w["router"], w["gu"], w["dn"], b.cfg64, True, w["mask"],
                                                       t["y"], t["eids"], t["wt"], b.ws2)),
                ("r1", "y", lambda: awq.awq_block_norm(t["r1"], t["y"], w["post"], None, 0.5, w["pre3"], 1e-6, t["r2"],
                                                       t["n3"]))):
            t[first].zero_()
            t[second].zero_()
            side.wait_stream(main)
            with torch.cuda.stream(side):
                big.add_(1.0)  # late
                t[first].copy_(src[first])
            t[second].copy_(src[second])
            main.wait_stream(side)
            call()

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    for run in (g.replay, calls):
        for k in ("p", "n2", "y", "eids", "wt", "r2", "n3"):
            b.t[k].zero_()
        torch.cuda.synchronize()
        run()
        b.status()
        torch.cuda.synchronize()
        for k in ("p", "n2", "y", "eids", "wt", "r2", "n3"):
            assert torch.equal(b.t[k], want[k]), k
    del g
