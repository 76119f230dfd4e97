"""GPU parity of the mixture-of-experts layer on packed experts
(awq_w4a16_moe) against its fp64 form."""

import numpy as np
import pytest
import torch

import post_weight_quantization_awq_b200 as awq
from gpu_helpers import need_cuda
from serving_oracle import moe, random_packed

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    need_cuda()


def _case(T, hidden, inter, E, group, seed):
    rng = np.random.default_rng(seed)
    boost = np.where(rng.random(hidden) < 0.02, 20.0, 1.0)
    X = (rng.standard_normal((T, hidden)) * boost).astype(np.float16)
    router = (rng.standard_normal((E, hidden)) * 0.05).astype(np.float16)
    gu = [random_packed(hidden, 2 * inter, group, rng, std=0.02) for _ in range(E)]
    dn = [random_packed(inter, hidden, group, rng, std=0.02) for _ in range(E)]
    return X, router, gu, dn


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


class _Layer:
    def __init__(self, X, router, gu, dn, group, k, ren, mask=None):
        self.x, self.router = (_dev(X) if isinstance(X, np.ndarray) else X), _dev(router)
        self.gu = [_dev(np.stack([p[i] for p in gu])) for i in range(3)]
        self.dn = [_dev(np.stack([p[i] for p in dn])) for i in range(3)]
        self.cfg, self.ren = awq.AwqConfig.make(group_size=group), ren
        self.mask = None if mask is None else _dev(np.asarray(mask, np.uint8))
        T, hidden = X.shape
        n = awq.awq_w4a16_moe_workspace_size(T, hidden, self.dn[0].shape[1], router.shape[0], k, self.cfg)
        self.ws = torch.full((n,), 0xA5, dtype=torch.uint8, device="cuda")
        self.Y = torch.full((T, hidden), 7.0, dtype=torch.float16, device="cuda")
        self.ids = torch.full((T, k), 99, dtype=torch.int32, device="cuda")
        self.wt = torch.full((T, k), 99.0, dtype=torch.float32, device="cuda")

    def call(self, stream=None):
        awq.awq_w4a16_moe(self.x, self.router, self.gu, self.dn, self.cfg, self.ren, self.mask, self.Y, self.ids,
                          self.wt, self.ws, stream)

    def run(self, stream=None):
        self.call(stream)
        awq.awq_device_status(self.ws, stream)
        return self.Y.cpu().numpy(), self.ids.cpu().numpy(), self.wt.cpu().numpy()


def _check(got, X, router, gu, dn, group, k, ren, mask=None):
    Y, ids, wt, tol = moe(X, router, gu, dn, group, k, ren, mask)
    assert np.array_equal(got[1], ids)
    # relative 2^-19 (exponent, exp, division); below fp32's smallest normal
    # value 2^-126 the output's step is 2^-149 whatever the value, and exp and
    # the division are off by a few such steps: less than 2^-140
    assert np.all(np.abs(got[2] - wt) <= 2.0 ** -19 * np.abs(wt) + 2.0 ** -140)
    err = np.abs(got[0].astype(np.float64) - Y)
    assert np.all(err <= tol), (err.max(), np.unravel_index(np.argmax(err - tol), err.shape))


@pytest.mark.parametrize("T,hidden,inter,E,k,group,ren", [
    (1, 64, 64, 1, 1, 64, True), (1, 512, 256, 8, 2, 128, True), (2, 320, 192, 5, 5, 64, False),
    (3, 128, 64, 33, 7, 32, True), (5, 2048, 384, 64, 8, 128, False), (8, 1024, 640, 4, 1, 128, True),
    (9, 256, 512, 6, 3, 64, True), (16, 576, 320, 3, 2, 32, False), (17, 512, 128, 16, 16, 128, True),
    (33, 384, 704, 2, 1, 64, True), (37, 1024, 256, 40, 4, 128, False), (64, 512, 384, 8, 2, 128, True),
    (64, 192, 64, 256, 8, 64, False), (64, 128, 128, 20, 16, 32, True), (7, 8192, 64, 4, 2, 64, True),
    (4, 64, 8192, 4, 2, 64, True),
    # so many pairs, channels and tiles of hidden that every value of H is made once for all blocks
    (8, 64, 16448, 16, 16, 64, True), (64, 576, 1088, 20, 16, 64, False), (64, 1088, 704, 18, 16, 32, True)])
def test_moe_parity(T, hidden, inter, E, k, group, ren):
    X, router, gu, dn = _case(T, hidden, inter, E, group, T + hidden + E)
    got = _Layer(X, router, gu, dn, group, k, ren).run()
    _check(got, X, router, gu, dn, group, k, ren)


@pytest.mark.parametrize("T", [1, 6, 50])
def test_moe_masked_rows(T):
    """Masked rows (NaN in them) meet no expert: ids -1, weights 0, Y 0, the
    other rows' bits do not change with what the masked rows hold; with every
    row masked the layer writes zeros."""
    X, router, gu, dn = _case(T, 256, 192, 6, 64, T)
    mask = np.arange(T) % 3 != 1
    outs = []
    for fill in (0.0, np.nan):
        Z = X.copy()
        Z[~mask] = fill
        outs.append(_Layer(Z, router, gu, dn, 64, 2, True, mask).run())
        _check(outs[-1], np.where(mask[:, None], X, 0).astype(np.float16), router, gu, dn, 64, 2, True, mask)
    for a, b in zip(*outs):
        assert np.array_equal(a, b)
    Y, ids, wt = _Layer(X, router, gu, dn, 64, 2, True, np.zeros(T)).run()
    assert not Y.any() and not wt.any() and np.all(ids == -1)


@pytest.mark.parametrize("T,E,k", [(3, 8, 4), (20, 48, 5), (11, 200, 16)])
def test_moe_ties_go_to_the_lowest_expert(T, E, k):
    """Equal router rows give equal logits: the lowest experts are chosen, in
    order (all equal; pairs of equals; zeros of both signs)."""
    X, router, gu, dn = _case(T, 128, 64, E, 64, E)
    for kind in ("all", "pairs", "zero"):
        r = router.copy()
        if kind == "all":
            r[:] = r[0]
        elif kind == "pairs":
            r[1::2] = r[0:E - E % 2:2]
        else:
            r[:] = 0.0
            r[::2] = -0.0
        got = _Layer(X, r, gu, dn, 64, k, False).run()
        _check(got, X, r, gu, dn, 64, k, False)
        if kind != "pairs":
            assert np.all(got[1] == np.arange(k))


@pytest.mark.parametrize("T", [8, 31, 33, 64])
def test_moe_all_tokens_meet_one_expert(T):
    X, router, gu, dn = _case(T, 512, 320, 8, 64, T)
    X[:, 0], router[:, 0] = 4.0, 0.0
    router[5, 0], router[2, 0] = 60.0, 30.0
    got = _Layer(X, router, gu, dn, 64, 2, True).run()
    assert np.all(got[1] == [5, 2])
    _check(got, X, router, gu, dn, 64, 2, True)


def test_moe_non_finite_row_stays_apart():
    """A row with a NaN or an infinity gets valid, distinct experts and a
    non-finite result; the rows that share experts with it are within bounds."""
    T = 12
    X, router, gu, dn = _case(T, 256, 128, 5, 64, 3)
    Z = X.copy()
    Z[4, 7], Z[9, 0] = np.nan, np.inf
    Y, ids, wt = _Layer(Z, router, gu, dn, 64, 3, True).run()
    want = moe(X, router, gu, dn, 64, 3, True)
    keep = [t for t in range(T) if t not in (4, 9)]
    assert np.array_equal(ids[keep], want[1][keep])
    assert np.all(np.abs(Y[keep] - want[0][keep]) <= want[3][keep])
    for t in (4, 9):
        assert sorted(set(ids[t])) == sorted(ids[t]) and ids[t].min() >= 0 and ids[t].max() < 5
        assert not np.isfinite(Y[t]).all()


@pytest.mark.parametrize("T", [2, 40])
def test_moe_strided_rows_and_repeat(T):
    X, router, gu, dn = _case(T, 192, 128, 4, 64, T)
    a = _Layer(X, router, gu, dn, 64, 2, True)
    want = a.run()
    again = a.run()
    for p, q in zip(want, again):
        assert np.array_equal(p, q)
    xb = torch.full((T, 192 + 24), float("nan"), dtype=torch.float16, device="cuda")
    xb[:, :192] = _dev(X)
    b = _Layer(X, router, gu, dn, 64, 2, True)
    b.x = xb[:, :192]
    yb = torch.full((T + 2, 192 + 8), 5.0, dtype=torch.float16, device="cuda")
    b.Y = yb[:T, :192]
    got = b.run()
    for p, q in zip(want, got):
        assert np.array_equal(p, q)
    assert bool((yb[:, 192:] == 5.0).all()) and bool((yb[T:] == 5.0).all())


@pytest.mark.parametrize("T", [3, 30])
def test_moe_captured_replayed_and_on_two_streams(T):
    """A captured call replayed after X changed; then two layers at once on two
    streams, each with its workspace."""
    X, router, gu, dn = _case(T, 512, 256, 8, 128, T)
    X2 = _case(T, 512, 256, 8, 128, T + 100)[0]
    a, b = _Layer(X, router, gu, dn, 128, 2, True), _Layer(X2, router, gu, dn, 128, 2, True)
    want, want2 = a.run(), b.run()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.call()
    a.x.copy_(_dev(X2))
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(a.Y.cpu().numpy(), want2[0]) and np.array_equal(a.ids.cpu().numpy(), want2[1])
    a.x.copy_(_dev(X))
    s, r = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        a.call(s.cuda_stream)
        b.call(r.cuda_stream)
    awq.awq_device_status(a.ws, s.cuda_stream)
    awq.awq_device_status(b.ws, r.cuda_stream)
    assert np.array_equal(a.Y.cpu().numpy(), want[0]) and np.array_equal(b.Y.cpu().numpy(), want2[0])
    del g


def test_moe_barrier_that_runs_out_is_reported(monkeypatch):
    """Every bounded wait gives up after one poll: the status says so, and the
    next call is right."""
    X, router, gu, dn = _case(4, 512, 256, 8, 128, 1)
    a = _Layer(X, router, gu, dn, 128, 2, True)
    want = a.run()
    monkeypatch.setenv("AWQ_FAULT", "timeout")
    with pytest.raises(awq.AwqError) as e:
        a.run()
    assert e.value.status_name == "AWQ_ERR_TIMEOUT"
    monkeypatch.delenv("AWQ_FAULT")
    for p, q in zip(want, a.run()):
        assert np.array_equal(p, q)


@pytest.mark.parametrize("T,hidden,inter,E,k", [(8, 64, 16448, 16, 16), (64, 576, 1088, 20, 16)])
def test_moe_shared_h_timeout_is_reported(monkeypatch, T, hidden, inter, E, k):
    """The same where H is made between two barriers."""
    X, router, gu, dn = _case(T, hidden, inter, E, 64, 5)
    a = _Layer(X, router, gu, dn, 64, k, True)
    want = a.run()
    monkeypatch.setenv("AWQ_FAULT", "timeout")
    with pytest.raises(awq.AwqError) as e:
        a.run()
    assert e.value.status_name == "AWQ_ERR_TIMEOUT"
    monkeypatch.delenv("AWQ_FAULT")
    for p, q in zip(want, a.run()):
        assert np.array_equal(p, q)


def test_moe_tensors_the_call_cannot_read_are_refused():
    X, router, gu, dn = _case(3, 128, 64, 4, 64, 9)
    for change in (dict(x=_dev(X).float()), dict(x=_dev(X).T), dict(router=_dev(router).cpu()),
                   dict(Y=torch.empty((3, 64), dtype=torch.float16, device="cuda")),
                   dict(ids=torch.empty((3, 2), dtype=torch.int64, device="cuda")),
                   dict(wt=torch.empty((2, 2), dtype=torch.float32, device="cuda")),
                   dict(mask=torch.ones(3, dtype=torch.bool, device="cuda")),
                   dict(ws=torch.empty(1 << 20, dtype=torch.uint8))):
        a = _Layer(X, router, gu, dn, 64, 2, True)
        for k, v in change.items():
            setattr(a, k, v)
        with pytest.raises(awq.AwqError) as e:
            a.call()
        assert e.value.status_name == "AWQ_ERR_INVALID_ARG", change
        assert bool((a.Y == 7.0).all()) or "Y" in change


@pytest.mark.parametrize("T", [1, 6, 30])
def test_moe_two_graphs_share_a_workspace(T):
    """Two captured layers of different inputs on one workspace, replayed in turn."""
    layers = []
    for seed in (T, T + 50):
        X, router, gu, dn = _case(T, 256, 192, 6, 64, seed)
        a = _Layer(X, router, gu, dn, 64, 2, True)
        want = a.run()
        if layers:
            a.ws = layers[0][0].ws
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            a.call()
        layers.append((a, g, want))
    for a, g, want in layers * 3:
        a.Y.zero_()
        g.replay()
        assert np.array_equal(a.Y.cpu().numpy(), want[0]) and np.array_equal(a.ids.cpu().numpy(), want[1])
    awq.awq_device_status(layers[0][0].ws)
    del g, layers


def test_moe_choices_that_are_not_a_power_of_two():
    """3, 6 and 11 experts a token: lanes without a choice in the last sum."""
    for k in (3, 6, 11):
        X, router, gu, dn = _case(5, 192, 128, 12, 64, k)
        _check(_Layer(X, router, gu, dn, 64, k, False).run(), X, router, gu, dn, 64, k, False)
