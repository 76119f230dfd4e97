"""GPU parity of the packed projection with per-token low-rank adapters
(awq_w4a16_lora_gemm) against its fp64 form."""

import numpy as np
import pytest
import torch

import post_weight_quantization_awq_b200 as awq
from gpu_helpers import need_cuda
from serving_oracle import lora, lora_tolerance, random_packed

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    need_cuda()


def _case(T, inn, out, rank, n, group, seed, order="mixed", integer=False):
    rng = np.random.default_rng(seed)
    packed = random_packed(inn, out, group, rng, pow2=integer)
    if integer:  # every sum an integer multiple of 2^-4 below 2^20: exact in fp32
        X = rng.integers(-3, 4, size=(T, inn)).astype(np.float16)
        A = rng.integers(-1, 2, size=(n, rank, inn)).astype(np.float16)
        A[:, :, 16:] = 0  # |u| <= 48: exact in fp16 too
        B = rng.integers(-2, 3, size=(n, out, rank)).astype(np.float16)
        c = np.exp2(rng.integers(-1, 2, size=n)).astype(np.float32)
    else:
        boost = np.where(rng.random(inn) < 0.02, 30.0, 1.0)
        X = (rng.standard_normal((T, inn)) * boost).astype(np.float16)
        A = (rng.standard_normal((n, rank, inn)) / np.sqrt(inn)).astype(np.float16)
        B = (rng.standard_normal((n, out, rank)) * 0.1).astype(np.float16)
        c = rng.uniform(0.25, 2.0, size=n).astype(np.float32)
    ids = rng.integers(-1, n, size=T).astype(np.int32)
    if order == "runs":
        ids = np.sort(ids)
    return X, packed, A, B, c, ids


def _run(X, packed, group, A, B, c, ids, stream=None, Y=None):
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    cfg = awq.AwqConfig.make(group_size=group)
    T, inn, out = X.shape[0], X.shape[1], packed[2].shape[1]
    Y = torch.empty((T, out), dtype=torch.float16, device="cuda") if Y is None else Y
    ws = torch.empty(awq.awq_w4a16_lora_workspace_size(T, inn, out, A.shape[1], cfg), dtype=torch.uint8, device="cuda")
    ws.fill_(0xA5)  # nothing of it may be relied on
    awq.awq_w4a16_lora_gemm(d(X) if isinstance(X, np.ndarray) else X, *map(d, packed), cfg, d(A), d(B), d(c), d(ids),
                            Y, ws, stream)
    awq.awq_device_status(ws, stream)
    return Y.cpu().numpy()


SHAPES = [
    (1, 512, 256, 8, 1, 128), (2, 64, 32, 8, 3, 64), (3, 192, 96, 16, 2, 64), (7, 1024, 544, 24, 5, 32),
    (8, 4096, 288, 16, 4, 128), (9, 640, 256, 32, 3, 128), (16, 2048, 1056, 64, 16, 128), (17, 320, 512, 8, 4, 64),
    (31, 96 * 4, 800, 40, 7, 32), (33, 1024, 256, 128, 2, 128), (45, 832, 352, 256, 3, 64), (48, 256, 64, 16, 9, 32),
    (64, 1152, 480, 16, 6, 128), (65, 512, 256, 16, 4, 128), (130, 192, 288, 24, 3, 64), (300, 1024, 544, 64, 40, 32),
    (777, 640, 768, 72, 5, 128), (1100, 256, 96, 8, 2, 32)]


@pytest.mark.parametrize("T,inn,out,rank,n,group", SHAPES)
@pytest.mark.parametrize("order", ["mixed", "runs"])
def test_lora_parity(T, inn, out, rank, n, group, order):
    X, packed, A, B, c, ids = _case(T, inn, out, rank, n, group, T + inn + out, order)
    Yg = _run(X, packed, group, A, B, c, ids)
    Yo, mags = lora(X, packed, group, A, B, c, ids)
    tol = lora_tolerance(Yo, mags, inn, rank, rounded=T > 64)
    err = np.abs(Yg.astype(np.float64) - Yo)
    assert np.all(err <= tol), (err.max(), np.unravel_index(np.argmax(err - tol), err.shape))


@pytest.mark.parametrize("T,inn,out,rank,n,group", SHAPES)
def test_lora_exact_sums(T, inn, out, rank, n, group):
    """Integer inputs, steps and adapter scales that are powers of two: every
    weight, product and partial sum is exact (fp32, and fp16 for U and the
    weights), so Y is the rounded exact sum bit for bit."""
    X, packed, A, B, c, ids = _case(T, inn, out, rank, n, group, 7 * T + inn, integer=True)
    Yo, _ = lora(X, packed, group, A, B, c, ids)
    assert np.abs(Yo).max() < 2 ** 15
    Yg = _run(X, packed, group, A, B, c, ids)
    assert np.array_equal(Yg.view(np.uint16), Yo.astype(np.float16).view(np.uint16))


@pytest.mark.parametrize("T", [5, 40, 150])
def test_lora_without_adapters_and_twice(T):
    """All ids -1: the projection alone, whatever the adapters hold (NaN here);
    and the same call twice gives the same bits."""
    X, packed, A, B, c, ids = _case(T, 512, 288, 16, 3, 128, T)
    Yo, mags = lora(X, packed, 128, A, B, c, np.full(T, -1))
    Yg = _run(X, packed, 128, A * np.nan, B * np.nan, c * np.nan, np.full(T, -1, np.int32))
    assert np.all(np.abs(Yg - Yo) <= lora_tolerance(Yo, mags, 512, 16, T > 64))
    a, b = (_run(X, packed, 128, A, B, c, ids) for _ in range(2))
    assert np.array_equal(a.view(np.uint16), b.view(np.uint16))


@pytest.mark.parametrize("T", [6, 90])
def test_lora_nan_adapter_stays_with_its_rows(T):
    """A non-finite adapter or token row touches its own rows of Y alone."""
    X, packed, A, B, c, ids = _case(T, 256, 96, 16, 3, 64, T)
    ids[:] = np.arange(T) % 3
    clean = _run(X, packed, 64, A, B, c, ids)
    A2 = A.copy()
    A2[1] = np.nan
    X2 = X.copy()
    X2[3, 5] = np.inf
    got = _run(X2, packed, 64, A2, B, c, ids)
    other = (ids != 1) & (np.arange(T) != 3)
    assert np.array_equal(got[other].view(np.uint16), clean[other].view(np.uint16))
    assert np.isnan(got[ids == 1]).all() and not np.isfinite(got[3]).all()


@pytest.mark.parametrize("T", [4, 33, 200])
def test_lora_strided_rows_and_stream(T):
    """X and Y rows wider than the product, on a stream of its own; nothing is
    written past out or below the last row."""
    X, packed, A, B, c, ids = _case(T, 192, 96, 8, 2, 64, T)
    s = torch.cuda.Stream()
    Xb = torch.full((T, 192 + 40), float("nan"), dtype=torch.float16, device="cuda")
    Xb[:, :192] = torch.from_numpy(X).cuda()
    Yb = torch.full((T + 3, 96 + 8), 7.0, dtype=torch.float16, device="cuda")
    torch.cuda.synchronize()
    want = _run(X, packed, 64, A, B, c, ids)
    with torch.cuda.stream(s):
        _run(Xb[:, :192], packed, 64, A, B, c, ids, Y=Yb[:T, :96])
    got = Yb.cpu().numpy()
    assert np.array_equal(got[:T, :96].view(np.uint16), want.view(np.uint16))
    assert np.all(got[:, 96:] == 7.0) and np.all(got[T:] == 7.0)


@pytest.mark.parametrize("T", [5, 70])
@pytest.mark.parametrize("bad", [3, -2, 2 ** 31 - 1, -2 ** 31])
def test_lora_bad_adapter_id_is_reported(T, bad):
    """An id outside [-1, n): the row gets the projection alone, the others
    are as ever, and the status names it; the next call is clean."""
    X, packed, A, B, c, ids = _case(T, 256, 96, 16, 3, 64, T)
    want = _run(X, packed, 64, A, B, c, np.where(np.arange(T) == 2, -1, ids).astype(np.int32))
    Y = torch.empty((T, 96), dtype=torch.float16, device="cuda")
    ids2 = ids.copy()
    ids2[2] = bad
    with pytest.raises(awq.AwqError) as e:
        _run(X, packed, 64, A, B, c, ids2, Y=Y)
    assert e.value.status_name == "AWQ_ERR_INVALID_ARG" and "adapter" in str(e.value)
    assert np.array_equal(Y.cpu().numpy().view(np.uint16), want.view(np.uint16))
    _run(X, packed, 64, A, B, c, ids)


def test_lora_captured_and_replayed_with_new_inputs():
    """One captured call, replayed after X and the ids changed in place."""
    for T in (3, 100):
        X, packed, A, B, c, ids = _case(T, 512, 256, 16, 4, 128, T)
        X2, _, _, _, _, ids2 = _case(T, 512, 256, 16, 4, 128, T + 1)
        cfg = awq.AwqConfig.make()
        d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        x, i = d(X), d(ids)
        w, ad = [d(p) for p in packed], [d(A), d(B), d(c)]
        Y = torch.empty((T, 256), dtype=torch.float16, device="cuda")
        ws = torch.empty(awq.awq_w4a16_lora_workspace_size(T, 512, 256, 16, cfg), dtype=torch.uint8, device="cuda")
        awq.awq_w4a16_lora_gemm(x, *w, cfg, *ad, i, Y, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            awq.awq_w4a16_lora_gemm(x, *w, cfg, *ad, i, Y, ws)
        for XX, ii in ((X2, ids2), (X, ids)):
            x.copy_(d(XX))
            i.copy_(d(ii))
            g.replay()
            got = Y.cpu().numpy()
            assert np.array_equal(got.view(np.uint16), _run(XX, packed, 128, A, B, c, ii).view(np.uint16))
        del g


@pytest.mark.parametrize("T", [5, 100])
def test_lora_two_at_once_with_a_workspace_each(T):
    """The same weights and adapters, two batches, two streams, interleaved."""
    X, packed, A, B, c, ids = _case(T, 1024, 544, 16, 4, 128, T)
    X2, _, _, _, _, ids2 = _case(T, 1024, 544, 16, 4, 128, T + 1)
    cfg = awq.AwqConfig.make()
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    w, ad = [d(p) for p in packed], [d(A), d(B), d(c)]
    calls, want = [], [_run(XX, packed, 128, A, B, c, ii) for XX, ii in ((X, ids), (X2, ids2))]
    for XX, ii in ((X, ids), (X2, ids2)):
        n = awq.awq_w4a16_lora_workspace_size(T, 1024, 544, 16, cfg)
        calls.append((d(XX), d(ii), torch.zeros((T, 544), dtype=torch.float16, device="cuda"),
                      torch.empty(n, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for x, i, Y, ws, s in calls:
            awq.awq_w4a16_lora_gemm(x, *w, cfg, *ad, i, Y, ws, s.cuda_stream)
    for (x, i, Y, ws, s), y in zip(calls, want):
        awq.awq_device_status(ws, s.cuda_stream)
        assert np.array_equal(Y.cpu().numpy().view(np.uint16), y.view(np.uint16))


@pytest.mark.parametrize("T,rank", [(5, 8), (6, 64), (12, 16), (40, 64), (100, 16)])
def test_lora_wait_that_runs_out_is_reported(monkeypatch, T, rank):
    """Every bounded wait gives up after one poll; whether one does depends on how
    soon the copies land, so the call either names the timeout or is right, and
    the next call is right."""
    X, packed, A, B, c, ids = _case(T, 4096, 1056, rank, 4, 128, T)
    want = _run(X, packed, 128, A, B, c, ids)
    monkeypatch.setenv("AWQ_FAULT", "timeout")
    try:
        got = _run(X, packed, 128, A, B, c, ids)
        assert np.array_equal(got.view(np.uint16), want.view(np.uint16))
    except awq.AwqError as e:
        assert e.status_name == "AWQ_ERR_TIMEOUT"
    monkeypatch.delenv("AWQ_FAULT")
    assert np.array_equal(_run(X, packed, 128, A, B, c, ids).view(np.uint16), want.view(np.uint16))


@pytest.mark.parametrize("T", [1, 40, 300])
def test_lora_adapters_past_two_to_the_31(T):
    """An adapter's rows that begin past 2^31 bytes, and past 2^31 values."""
    n, rank, inn, out = 2100, 256, 4096, 64
    rng = np.random.default_rng(T)
    packed = random_packed(inn, out, 128, rng)
    X = rng.standard_normal((T, inn)).astype(np.float16)
    ids = np.array([0, 1, n // 2, n - 1, -1])[rng.integers(0, 5, T)].astype(np.int32)
    ids[0] = n - 1
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    A = torch.zeros((n, rank, inn), dtype=torch.float16, device="cuda")
    B, c = np.zeros((n, out, rank), np.float16), np.ones(n, np.float32)
    few = sorted(set(ids) - {-1})
    An = {a: (rng.standard_normal((rank, inn)) / 64).astype(np.float16) for a in few}
    for a in few:
        A[a] = d(An[a])
        B[a] = rng.standard_normal((out, rank)) * 0.1
    cfg = awq.AwqConfig.make()
    Y = torch.empty((T, out), dtype=torch.float16, device="cuda")
    ws = torch.empty(awq.awq_w4a16_lora_workspace_size(T, inn, out, rank, cfg), dtype=torch.uint8, device="cuda")
    awq.awq_w4a16_lora_gemm(d(X), *map(d, packed), cfg, A, d(B), d(c), d(ids), Y, ws)
    awq.awq_device_status(ws)
    short = np.array([few.index(a) if a >= 0 else -1 for a in ids])
    Yo, mags = lora(X, packed, 128, np.stack([An[a] for a in few]), np.stack([B[a] for a in few]),
                    np.ones(len(few)), short)
    err = np.abs(Y.cpu().numpy().astype(np.float64) - Yo)
    assert np.all(err <= lora_tolerance(Yo, mags, inn, rank, T > 64)), err.max()


def test_lora_tensors_the_call_cannot_read_are_refused():
    X, packed, A, B, c, ids = _case(4, 256, 96, 16, 3, 64, 1)
    cfg = awq.AwqConfig.make(group_size=64)
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    ok = dict(X=d(X), q=d(packed[0]), z=d(packed[1]), s=d(packed[2]), A=d(A), B=d(B), c=d(c), ids=d(ids),
              Y=torch.full((4, 96), 7.0, dtype=torch.float16, device="cuda"),
              ws=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))
    for name, bad in (("X", ok["X"].double()), ("X", ok["X"].cpu()), ("X", d(X.T).T), ("q", ok["q"].T),
                      ("q", ok["q"][:128]), ("s", ok["s"].float()), ("A", ok["A"].transpose(1, 2)),
                      ("B", ok["B"][:2]), ("c", ok["c"].half()), ("ids", ok["ids"].long()), ("ids", ok["ids"][:3]),
                      ("Y", ok["Y"][:3]), ("Y", ok["Y"].bfloat16()), ("ws", ok["ws"].cpu())):
        a = dict(ok, **{name: bad})
        with pytest.raises(awq.AwqError) as e:
            awq.awq_w4a16_lora_gemm(a["X"], a["q"], a["z"], a["s"], cfg, a["A"], a["B"], a["c"], a["ids"], a["Y"],
                                    a["ws"])
        assert e.value.status_name == "AWQ_ERR_INVALID_ARG", name
    assert bool((ok["Y"] == 7.0).all())


@pytest.mark.parametrize("T,inn,out,rank,n,group", [
    # as many tiles as make groups of 16 tokens fill the SMs, and more, where all tokens stay in one block
    (20, 256, 12288, 24, 3, 128), (45, 128, 12288, 8, 5, 64), (64, 192, 12288, 16, 2, 32),
    (20, 128, 39936, 8, 3, 128), (45, 128, 32768, 40, 7, 128), (64, 128, 32768, 8, 4, 64), (45, 64, 39936, 8, 2, 32),
    # past 64 tokens: few rows and many tiles, one row of tiles that is not full, ranks of several passes
    (70, 64, 39936, 8, 3, 64), (129, 192, 8224, 120, 9, 32), (257, 128, 4096, 56, 48, 128), (90, 64, 32, 256, 30, 64)])
def test_lora_many_tiles_and_passes(T, inn, out, rank, n, group):
    X, packed, A, B, c, ids = _case(T, inn, out, rank, n, group, T + out)
    Yg = _run(X, packed, group, A, B, c, ids)
    Yo, mags = lora(X, packed, group, A, B, c, ids)
    err = np.abs(Yg.astype(np.float64) - Yo)
    assert np.all(err <= lora_tolerance(Yo, mags, inn, rank, rounded=T > 64)), err.max()


@pytest.mark.parametrize("T", [2, 12, 40, 150])
def test_lora_two_graphs_share_a_workspace(T):
    """Two captured calls of different inputs on one workspace, replayed in turn."""
    cfg = awq.AwqConfig.make()
    d = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
    ws = torch.empty(awq.awq_w4a16_lora_workspace_size(T, 512, 544, 16, cfg), dtype=torch.uint8, device="cuda")
    graphs = []
    for seed in (T, T + 1):
        X, packed, A, B, c, ids = _case(T, 512, 544, 16, 4, 128, seed)
        Y = torch.zeros((T, 544), dtype=torch.float16, device="cuda")
        t = [d(X), *map(d, packed)], [d(A), d(B), d(c), d(ids), Y]
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            awq.awq_w4a16_lora_gemm(*t[0], cfg, *t[1], ws)
        graphs.append((g, t, _run(X, packed, 128, A, B, c, ids)))
    for g, t, want in graphs * 3:
        t[1][-1].zero_()
        g.replay()
        assert np.array_equal(t[1][-1].cpu().numpy().view(np.uint16), want.view(np.uint16))
    awq.awq_device_status(ws)
    del g, graphs
