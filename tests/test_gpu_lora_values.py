"""awq_w4a16_lora_gemm on values that a request may bring or a wait may leave:
what one adapter or token row holds stays with its own rows, and a wait that
runs out is never lost."""

import numpy as np
import pytest

import post_weight_quantization_awq_b200 as awq
from gpu_helpers import need_cuda
from serving_oracle import lora, lora_tolerance
from test_gpu_lora import _case, _run

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    need_cuda()


@pytest.mark.parametrize("T,rank", [(1, 8), (6, 64), (40, 16)])
def test_lora_wait_that_runs_out_is_never_lost(monkeypatch, T, rank):
    """Waits that give up after one poll, many calls: a call whose status is clean
    has the bits of the undisturbed one."""
    X, packed, A, B, c, ids = _case(T, 4096, 1056, rank, 4, 128, T)
    want = _run(X, packed, 128, A, B, c, ids).view(np.uint16)
    monkeypatch.setenv("AWQ_FAULT", "timeout")
    for _ in range(40):
        try:
            assert np.array_equal(_run(X, packed, 128, A, B, c, ids).view(np.uint16), want)
        except awq.AwqError as e:
            assert e.status_name == "AWQ_ERR_TIMEOUT"
    monkeypatch.delenv("AWQ_FAULT")
    assert np.array_equal(_run(X, packed, 128, A, B, c, ids).view(np.uint16), want)


def _kind(v):
    """0 finite, 1 +inf, 2 -inf, 3 NaN."""
    return np.where(np.isnan(v), 3, np.where(np.isposinf(v), 1, np.where(np.isneginf(v), 2, 0)))


def _same_or_close(got, want, tol):
    """Infinities and NaN where the definition has them, the rest within tol."""
    got = got.astype(np.float64)
    assert np.array_equal(_kind(got), _kind(want)), np.argwhere(_kind(got) != _kind(want))[:5]
    ok = np.isfinite(want)
    assert np.all(np.abs(got[ok] - want[ok]) <= tol[ok]), np.abs(got[ok] - want[ok]).max()


@pytest.mark.parametrize("T,inn,out,rank,n,group,order", [
    (6, 256, 96, 16, 3, 64, "mixed"), (13, 256, 96, 8, 3, 64, "mixed"), (40, 256, 288, 72, 5, 64, "mixed"),
    (64, 256, 1056, 24, 4, 128, "runs"), (66, 256, 96, 16, 3, 64, "mixed"),
    (90, 256, 544, 8, 4, 32, "mixed"), (300, 512, 288, 72, 5, 128, "mixed"), (300, 256, 1056, 40, 9, 64, "runs"),
    (600, 256, 8224, 16, 3, 128, "mixed")])
def test_lora_non_finite_b_stays_with_its_rows(T, inn, out, rank, n, group, order):
    """Infinities and NaN in B of some adapters: the rows of the others, and those
    without one, keep their bits; an adapter's own rows are the definition's."""
    X, packed, A, B, c, ids = _case(T, inn, out, rank, n, group, T + out, order)
    clean = _run(X, packed, group, A, B, c, ids)
    rng = np.random.default_rng(T)
    bad = B.copy()
    for a, v in ((0, np.inf), (2, np.nan), (2, -np.inf)):
        for o, r in ((0, 0), (out - 1, rank - 1), (int(rng.integers(out)), int(rng.integers(rank)))):
            bad[a, o, r] = v
    got = _run(X, packed, group, A, bad, c, ids)
    other = (ids != 0) & (ids != 2)
    assert np.array_equal(got[other].view(np.uint16), clean[other].view(np.uint16))
    with np.errstate(invalid="ignore"):
        Yo, _ = lora(X, packed, group, A, bad, c, ids)
    _, mags = lora(X, packed, group, A, B, c, ids)
    tol = lora_tolerance(np.where(np.isfinite(Yo), Yo, 0), mags, inn, rank, rounded=T > 64)
    _same_or_close(got, Yo, tol)


@pytest.mark.parametrize("T", [6, 13, 40, 90])
def test_lora_infinite_rank_row_beside_large_ones(T):
    """One infinite value of U beside others past fp16's range: the infinity decides."""
    X, packed, A, B, c, ids = _case(T, 256, 96, 16, 2, 64, T)
    ids[:] = np.arange(T) % 3 - 1
    c[1] = 1e6
    B[1] = (B[1].astype(np.float64) * 1e-3).astype(np.float16)
    B[1][:, 3] = np.where(np.arange(96) % 2 == 0, 0.5, -0.5)
    A[1, 3, 7] = np.inf
    with np.errstate(invalid="ignore"):
        Yo, _ = lora(X, packed, 64, A, B, c, ids)
    fin = A.copy()
    fin[1, 3, 7] = 0
    _, mags = lora(X, packed, 64, fin, B, c, ids)
    assert (_kind(Yo[ids == 1]) != 3).all() and not np.isfinite(Yo[ids == 1]).any()
    _same_or_close(_run(X, packed, 64, A, B, c, ids), Yo,
                   lora_tolerance(np.where(np.isfinite(Yo), Yo, 0), mags, 256, 16, T > 64))


@pytest.mark.parametrize("T,rank", [(5, 16), (40, 64), (65, 16), (90, 8), (300, 136), (300, 64), (700, 16)])
@pytest.mark.parametrize("c2,b2", [(3e5, 2e-5), (2e-7, 1e5)])
def test_lora_scaled_products_past_fp16(T, rank, c2, b2):
    """c_a U past fp16's largest value, or below its smallest normal one, with B_a
    scaled the other way: Y is an ordinary value, and as near as ever.  The codes
    are the zero points, so that the low-rank part stands alone."""
    X, packed, A, B, c, ids = _case(T, 512, 288, rank, 3, 128, T + rank)
    packed = (np.repeat(packed[1], 128, axis=0), packed[1], packed[2])
    ids[0] = 1
    c[1] = c2
    B[1] = (B[1].astype(np.float64) * b2).astype(np.float16)
    Yo, mags = lora(X, packed, 128, A, B, c, ids)
    got = _run(X, packed, 128, A, B, c, ids)
    _same_or_close(got, Yo, lora_tolerance(Yo, mags, 512, rank, rounded=T > 64))


@pytest.mark.parametrize("T", [1, 2, 5, 8, 9, 16, 30, 64, 65, 130])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_lora_infinite_inputs(T, group):
    """An infinite input gives an infinity of its weight's sign in every output (NaN
    where the code is the zero point), its row alone."""
    X, packed, A, B, c, ids = _case(T, 512, 288, 16, 3, group, T + group)
    ids[::2] = -1
    X[0, 300], X[T // 2, 5], X[T - 1, 511] = np.inf, -np.inf, np.inf
    with np.errstate(invalid="ignore"):
        Yo, _ = lora(X, packed, group, A, B, c, ids)
    _, mags = lora(np.where(np.isfinite(X), X, 0), packed, group, A, B, c, ids)
    tol = lora_tolerance(np.where(np.isfinite(Yo), Yo, 0), mags, 512, 16, rounded=T > 64)
    got = _run(X, packed, group, A, B, c, ids)
    _same_or_close(got, Yo, tol)
