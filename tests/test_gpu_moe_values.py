"""awq_w4a16_moe on values at a border: logits that are equal or nearly so, H past
fp16's range."""

import numpy as np
import pytest

from gpu_helpers import need_cuda
from serving_oracle import weights
from test_gpu_moe import _case, _Layer

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    need_cuda()


def _near_ties(T, hidden, E, seed, near):
    """x on grids of 2^-4 (below 64) and 2^-12 (below 1/4), router rows on one of 2^-9
    (below 2): products are multiples of 2^-21 below 2^7, and sums of 16384 of them exact
    in 64 bits, not in 32.  x repeats its values, and a router row is another one with
    its entries exchanged between equal values of x, so that the exact logits of a token
    are equal; `near` adds one step of the grid to one entry of some rows, where x is
    small."""
    rng = np.random.default_rng(seed)
    base = rng.integers(-1023, 1024, size=hidden // 8) / np.where(rng.random(hidden // 8) < 0.3, 16.0, 4096.0)
    x = np.repeat(base, 8)
    X = np.stack([x * s for s in rng.choice([1.0, -1.0], T)])
    row = rng.integers(-1023, 1024, size=hidden) / 512.0
    rows = []
    for _ in range(E):
        r = row.reshape(-1, 8).copy()
        for g in r:
            rng.shuffle(g)
        rows.append(r.reshape(-1))
    rows = np.stack(rows)
    where = rng.permutation(hidden)
    X, rows = X[:, where], rows[:, where]
    if near:
        j = int(np.flatnonzero((np.abs(X[0]) < 0.25) & (X[0] != 0))[0])
        for e in range(0, E, 3):
            rows[e, j] += (1 if rng.random() < 0.5 else -1) / 512.0
    return X.astype(np.float16), rows.astype(np.float16)


@pytest.mark.parametrize("T,hidden,E,k", [
    (1, 512, 4, 2), (1, 4096, 8, 3), (1, 4096, 9, 4), (3, 2048, 24, 5), (8, 1024, 64, 8), (9, 4096, 16, 4),
    (40, 512, 200, 16), (64, 16384, 8, 2)])
@pytest.mark.parametrize("near", [False, True])
def test_moe_choice_is_the_definitions_at_a_border(T, hidden, E, k, near):
    """Logits that are equal in exact arithmetic, though their products stand in
    another order, go to the lowest expert; logits one step of the products' grid
    apart go by size."""
    X, rows = _near_ties(T, hidden, E, hidden + E, near)
    _, _, gu, dn = _case(T, hidden, 64, 1, 64, E)
    whole = lambda a, unit: np.rint(a.astype(np.float64) * unit).astype(np.int64)  # noqa: E731
    exact = whole(X, 4096) @ whole(rows, 512).T
    want = np.stack([sorted(range(E), key=lambda e: (-exact[t, e], e))[:k] for t in range(T)])
    assert (not near) == all((exact[t] == exact[t, 0]).all() for t in range(T))
    got = _Layer(X, rows, gu * E, dn * E, 64, k, True).run()
    assert np.array_equal(got[1], want)


def _plain(X, router, gu, dn, group, k):
    """Y with H rounded to fp16 (infinite past its range)."""
    Y = []
    x = X.astype(np.float64)
    logits = x @ router.astype(np.float64).T
    for t in range(X.shape[0]):
        order = sorted(range(router.shape[0]), key=lambda e: (-logits[t, e], e))[:k]
        p = np.exp(logits[t, order] - logits[t].max())
        p /= p.sum()
        y = 0
        for e, pe in zip(order, p):
            Wg, Wd = weights(gu[e], group)[0], weights(dn[e], group)[0]
            g, u = np.split(Wg @ x[t], 2)
            with np.errstate(over="ignore", invalid="ignore"):
                h = (g / (1 + np.exp(-g)) * u).astype(np.float16).astype(np.float64)
                y = y + pe * (Wd @ h)
        Y.append(y)
    return np.stack(Y)


def _set(words, o, values):
    """Codes (or zero points) of output o, one a row of words."""
    u = words.view(np.uint32)
    u[:, o // 8] &= np.uint32(~(0xF << (4 * (o % 8))) & 0xFFFFFFFF)
    u[:, o // 8] |= (np.asarray(values, np.uint32) << np.uint32(4 * (o % 8))).astype(np.uint32)


@pytest.mark.parametrize("T,E,k", [(1, 4, 2), (2, 3, 2), (5, 2, 1), (12, 8, 2), (20, 8, 2), (30, 3, 2)])
def test_moe_h_past_fp16(T, E, k):
    """A value of H past fp16's largest is an infinity, however many tokens its expert
    has: every output of its token is an infinity of the down weight's sign, or NaN
    where that weight is 0 or two infinities meet; the other rows stay finite."""
    X, router, gu, dn = _case(T, 128, 64, E, 64, T + E)
    for e in range(E):
        for o in (5, 64 + 5):  # channel 5 of gate and up: 240 x_0
            _set(gu[e][0], o, [15] + [0] * 127)
            _set(gu[e][1], o, [0, 0])
            gu[e][2][:, o] = 16.0
    X[:, 0], router[:, 0] = 0.25, 0.0
    hit = T // 2
    X[hit, 0] = 2.0
    want = _plain(X, router, gu, dn, 64, k)
    assert not np.isfinite(want[hit]).any() and np.isinf(want[hit]).any()
    got = _Layer(X, router, gu, dn, 64, k, True).run()[0]
    assert np.array_equal(np.isnan(got[hit]), np.isnan(want[hit]))
    inf = ~np.isnan(want[hit])
    assert np.array_equal(got[hit][inf], want[hit][inf])
    rest = np.arange(T) != hit
    assert np.isfinite(got[rest]).all() and np.isfinite(want[rest]).all()
