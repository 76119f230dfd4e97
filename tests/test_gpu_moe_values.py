"""awq_w4a16_moe on values at a border: H past fp16's range."""

import numpy as np
import pytest

from gpu_helpers import need_cuda
from serving_oracle import weights
from test_gpu_moe import _case, _Layer

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    need_cuda()


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
