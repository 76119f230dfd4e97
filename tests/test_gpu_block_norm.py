"""GPU parity of the norms around a block (awq_block_norm) against fp64.

Tolerance per value, before the first run: r' = R + c gate v' carries at most
8 fp32 roundings and the norm factor's own (a sum of d squares: d / 32 + 16
roundings at most in a thread and its butterfly, halved by the square root, and
two ulps of rsqrt), each 2^-24 relative, applied to |R| + |c gate v'|; n
carries as much again for its own factor.  Then half an fp16 ulp."""

import numpy as np
import pytest
import torch

import post_weight_quantization_awq_b200 as awq
from gpu_helpers import need_cuda
from serving_oracle import block_norm, ulp16

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    need_cuda()


def _inputs(T, d, post, gate, seed):
    rng = np.random.default_rng(seed)
    f = lambda *s: rng.standard_normal(s).astype(np.float16)  # noqa: E731
    R, V = f(T, d) * np.float16(2), f(T, d) * np.float16(3)
    V[:, rng.random(d) < 0.02] *= np.float16(30)
    return (R, V, f(d) if post else None, {"none": None, "channel": f(d), "token": f(T, d)}[gate], f(d))


def _dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _check(got, R, V, post, gate, c, pre, eps, d):
    r, n = block_norm(R, V, post, gate, c, pre, eps)
    rel = (8 + d / 64 + 8 + 2) * 2.0 ** -24
    part = np.abs(R.astype(np.float64)) + np.abs(r - R.astype(np.float64))
    if got[0] is not None:
        e = np.abs(got[0].astype(np.float64) - r)
        tol = rel * part
        assert np.all(e <= tol + 0.5 * ulp16(np.abs(r) + tol)), e.max()
    if got[1] is not None:
        scale = np.abs(n) / np.maximum(np.abs(r), 1e-30)
        tol = rel * (part * np.where(r == 0, 0, scale) + np.abs(n)) + rel * np.abs(n)
        e = np.abs(got[1].astype(np.float64) - n)
        assert np.all(e <= tol + 0.5 * ulp16(np.abs(n) + tol)), e.max()


@pytest.mark.parametrize("T,d", [(1, 8), (3, 64), (5, 248), (1, 256), (9, 264), (4, 512), (7, 1016), (2, 1032),
                                 (33, 2048), (3, 2056), (1, 4096), (17, 4104), (5, 8192), (2, 8200), (3, 16384),
                                 (2, 16392), (1, 32768), (300, 128), (1000, 5120)])
@pytest.mark.parametrize("post,gate", [(False, "none"), (True, "none"), (True, "channel"), (False, "token"),
                                       (True, "token")])
def test_norm_parity(T, d, post, gate):
    R, V, p, g, pre = _inputs(T, d, post, gate, T + d)
    ro, no = (torch.empty((T, d), dtype=torch.float16, device="cuda") for _ in range(2))
    awq.awq_block_norm(_dev(R), _dev(V), _dev(p), _dev(g), 0.7, _dev(pre), 1e-5, ro, no)
    _check((ro.cpu().numpy(), no.cpu().numpy()), R, V, p, g, 0.7, pre, 1e-5, d)


@pytest.mark.parametrize("T,d", [(3, 64), (20, 1024), (2, 9000)])
def test_norm_optional_parts(T, d):
    """Without V (the first norm of a model), without pre, and with one output."""
    R, V, p, g, pre = _inputs(T, d, True, "token", d)
    no = torch.empty((T, d), dtype=torch.float16, device="cuda")
    ro = torch.empty_like(no)
    awq.awq_block_norm(_dev(R), None, None, None, 5.0, _dev(pre), 1e-6, None, no)
    _check((None, no.cpu().numpy()), R, None, None, None, 5.0, pre, 1e-6, d)
    awq.awq_block_norm(_dev(R), _dev(V), _dev(p), _dev(g), -1.5, None, 1e-6, ro, no)
    _check((ro.cpu().numpy(), no.cpu().numpy()), R, V, p, g, -1.5, None, 1e-6, d)
    ro.zero_()
    awq.awq_block_norm(_dev(R), _dev(V), None, None, 1.0, None, 0.0, ro, None)
    _check((ro.cpu().numpy(), None), R, V, None, None, 1.0, None, 0.0, d)
    awq.awq_block_norm(_dev(R), None, None, None, 1.0, None, 0.0, ro, None)
    assert np.array_equal(ro.cpu().numpy().view(np.uint16), R.view(np.uint16))


@pytest.mark.parametrize("T,d", [(5, 72), (65, 4096), (3, 20000)])
def test_norm_in_place_and_strided(T, d):
    """R_out over R and N_out over V, rows of a wider buffer: the bits of the
    separate outputs, and nothing beside the rows is written."""
    R, V, p, g, pre = _inputs(T, d, True, "channel", d)
    ro, no = (torch.empty((T, d), dtype=torch.float16, device="cuda") for _ in range(2))
    awq.awq_block_norm(_dev(R), _dev(V), _dev(p), _dev(g), 0.5, _dev(pre), 1e-6, ro, no)
    wide = [torch.full((T + 1, d + 24), 9.0, dtype=torch.float16, device="cuda") for _ in range(2)]
    r, v = wide[0][:T, :d], wide[1][:T, :d]
    r.copy_(_dev(R))
    v.copy_(_dev(V))
    awq.awq_block_norm(r, v, _dev(p), _dev(g), 0.5, _dev(pre), 1e-6, r, v)
    assert torch.equal(r, ro) and torch.equal(v, no)
    for w in wide:
        assert bool((w[:, d:] == 9.0).all()) and bool((w[T:] == 9.0).all())


def test_norm_non_finite_rows_stay_apart_and_zero_rows_are_zero():
    T, d = 6, 1024
    R, V, p, g, pre = _inputs(T, d, True, "none", 3)
    R[4], V[4] = 0, 0
    outs = []
    for bad in (False, True):
        if bad:
            V[1, 7], R[2, 9], V[3, 0] = np.inf, np.nan, -np.inf
        ro, no = (torch.empty((T, d), dtype=torch.float16, device="cuda") for _ in range(2))
        awq.awq_block_norm(_dev(R), _dev(V), _dev(p), None, 1.0, _dev(pre), 1e-6, ro, no)
        outs.append((ro.cpu().numpy(), no.cpu().numpy()))
    keep = [0, 4, 5]
    for a, b in zip(*outs):
        assert np.array_equal(a[keep].view(np.uint16), b[keep].view(np.uint16))
        assert np.all(a[4] == 0) and all(np.isnan(b[i]).any() for i in (1, 2, 3))


def test_norm_large_values_do_not_overflow_the_statistics():
    """Rows at fp16's largest value: squares sum to 2^32 d in fp32."""
    T, d = 2, 8192
    R = np.full((T, d), 60000.0, np.float16)
    no = torch.empty((T, d), dtype=torch.float16, device="cuda")
    awq.awq_block_norm(_dev(R), None, None, None, 1.0, None, 1e-6, None, no)
    assert np.all(np.abs(no.cpu().numpy().astype(np.float64) - 1.0) <= 2.0 ** -11)


def test_norm_captured_and_on_another_stream():
    T, d = 40, 4096
    R, V, p, g, pre = _inputs(T, d, True, "token", 1)
    ro, no = (torch.empty((T, d), dtype=torch.float16, device="cuda") for _ in range(2))
    args = [_dev(p), _dev(g), 0.5, _dev(pre), 1e-6]
    r, v = _dev(R), _dev(V)
    awq.awq_block_norm(r, v, *args, ro, no)
    want = no.clone()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        awq.awq_block_norm(r, v, *args, ro, no)
    no.zero_()
    gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(no, want)
    s = torch.cuda.Stream()
    no.zero_()
    torch.cuda.synchronize()
    awq.awq_block_norm(r, v, *args, ro, no, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(no, want)


def test_norm_tensors_the_call_cannot_read_are_refused():
    T, d = 3, 64
    h = lambda *s: torch.zeros(s, dtype=torch.float16, device="cuda")  # noqa: E731
    ok = dict(R=h(T, d), V=h(T, d), post=h(d), gate=h(d), pre=h(d), ro=h(T, d), no=h(T, d))
    for name, bad in (("R", ok["R"].float()), ("R", ok["R"].cpu()), ("V", h(d, T).T), ("V", h(T, 128)),
                      ("post", h(d + 8)), ("post", h(2 * d)[::2]), ("gate", h(T + 1, d)), ("gate", h(8)),
                      ("pre", h(d).bfloat16()), ("ro", h(T + 1, d)), ("no", h(T, d).cpu())):
        a = dict(ok, **{name: bad})
        with pytest.raises(awq.AwqError) as e:
            awq.awq_block_norm(a["R"], a["V"], a["post"], a["gate"], 1.0, a["pre"], 1e-6, a["ro"], a["no"])
        assert e.value.status_name == "AWQ_ERR_INVALID_ARG", name


def test_norm_rows_past_two_to_the_31():
    """Rows whose values begin past 2^31 values of R and of the outputs."""
    d = 32768
    T = (1 << 31) // d + 3
    R = torch.zeros((T, d), dtype=torch.float16, device="cuda")
    rng = np.random.default_rng(2)
    rows = [0, 65535, 65536, T - 1]
    Rn = rng.standard_normal((len(rows), d)).astype(np.float16)
    for r, v in zip(rows, Rn):
        R[r] = _dev(v)
    pre = rng.standard_normal(d).astype(np.float16)
    no = torch.full((T, d), 3.0, dtype=torch.float16, device="cuda")
    awq.awq_block_norm(R, None, None, None, 1.0, _dev(pre), 1e-6, None, no)
    got = np.stack([no[r].cpu().numpy() for r in rows])
    _check((None, got), Rn, None, None, None, 1.0, pre, 1e-6, d)
    assert not bool(no[1].any())
