"""What the bounds of the experts' layer's tests can see (CPU, on the oracle): a unit
of 128 rows of one expert left out stands far above them."""

import numpy as np
import pytest

from serving_exact import ROW_BOUND, row_distance
from serving_oracle import random_packed, weights


@pytest.mark.parametrize("hidden,inter,k,group", [(64, 8192, 2, 64), (8192, 64, 2, 64), (4096, 1024, 8, 128),
                                                  (1088, 704, 16, 32)])
def test_a_lost_unit_shows_in_the_row_distance(hidden, inter, k, group):
    rng = np.random.default_rng(hidden + inter)
    x = rng.standard_normal(hidden) * np.where(rng.random(hidden) < 0.02, 20.0, 1.0)
    p = np.full(k, 1.0 / k)
    parts, hs, wgs, wds = [], [], [], []
    for _ in range(k):
        wg = weights(random_packed(hidden, 2 * inter, group, rng), group)[0]
        wd = weights(random_packed(inter, hidden, group, rng), group)[0]
        g, u = np.split(wg @ x, 2)
        hs.append(g / (1 + np.exp(-g)) * u)
        parts.append(wd @ hs[-1])
        wgs.append(wg)
        wds.append(wd)
    Y = sum(a * b for a, b in zip(p, parts))[None]
    # as the calls round: H and Y to fp16
    R = sum(a * (w @ h.astype(np.float16).astype(np.float64)) for a, w, h in zip(p, wds, hs)).astype(np.float16)[None]
    assert row_distance(R, Y)[0] < ROW_BOUND / 1.5
    # the last 128 rows of one expert's down product, and of its gate|up product
    h = hs[0].copy()
    h[-128:] = 0
    lost = Y + p[0] * (wds[0] @ h - parts[0])
    assert row_distance(lost, Y)[0] > 10 * ROW_BOUND
    z = x.copy()
    z[-128:] = 0
    g, u = np.split(wgs[0] @ z, 2)
    lost = Y + p[0] * (wds[0] @ (g / (1 + np.exp(-g)) * u) - parts[0])
    assert row_distance(lost, Y)[0] > 10 * ROW_BOUND
