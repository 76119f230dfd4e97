"""Experts' layers whose every value is exact in the types that hold it, and the
norm-wise distance of the layer's outputs, for tests/test_gpu_moe_exact.py and
tests/test_serving_moe_checks.py."""

import numpy as np

from oracle import awq_oracle as O


def pack(codes):
    """Codes [out, in] (zero points [out, groups]) -> int32 words [in, out / 8]."""
    out, inn = codes.shape
    c = codes.astype(np.uint32).reshape(out // 8, 8, inn)
    words = np.zeros((out // 8, inn), np.uint32)
    for p in range(8):
        words |= c[:, p] << np.uint32(4 * p)
    return np.ascontiguousarray(words.T).view(np.int32)


def packed(w, step, group, rng):
    """A packed layer of the weights w [out, in] (whole numbers of [-1, 1]) times
    `step`, zero points at random."""
    out, inn = w.shape
    z = rng.integers(1, 15, size=(out, inn // group))
    codes = w + np.repeat(z, group, axis=1)
    q = pack(codes)
    assert np.array_equal(O.unpack_nibbles(q), codes)
    return q, pack(z), np.full((inn // group, out), step, np.float16)


def layer(T, hidden, inter, E, k, group, seed, free=False):
    """X, router, gate|up, down and the exact Y of a layer in which gate's sums are
    whole numbers of at least 32, so that silu(g) is g, H is a whole number, the k
    chosen experts of a token weigh exactly 1 / k, and every partial sum is exact in
    fp32.  In one half of the channels gate is constant and up any sum, in the other
    gate any sum and up constant, so that H is exact in fp16 too; `free`: both are any
    sum, and H has up to 15 bits."""
    rng = np.random.default_rng(seed)
    X = rng.integers(-1, 2, size=(T, hidden))
    X[:, 0] = 128
    # experts in sets of k with one router row: a token's logits tie inside a set
    sets = rng.integers(-2, 3, size=(E // k, hidden))
    sets[:, 0] = 0
    router = np.repeat(sets, k, axis=0)
    logits = X @ router.T
    ids = np.stack([sorted(range(E), key=lambda e: (-logits[t, e], e))[:k] for t in range(T)])
    gu, dn, Y = [], [], np.zeros((T, hidden), np.int64)
    half = np.arange(inter) % 2 == 0
    unit = 1 if free else 128  # of which every value of H is a multiple
    for e in range(E):
        wg, wu = rng.integers(-1, 2, size=(2, inter, hidden))
        wg[:, 0], wu[:, 0] = 1, 0
        if not free:
            wg[half, 1:], wu[~half, 1:], wu[~half, 0] = 0, 0, 1
        wd = rng.integers(-1, 2, size=(hidden, inter))
        gu.append(packed(np.concatenate([wg, wu]), 1.0, group, rng))
        dn.append(packed(wd, 2.0 ** -7, group, rng))
        rows = np.flatnonzero((ids == e).any(1))
        g, u = X[rows] @ wg.T, X[rows] @ wu.T
        assert rows.size == 0 or g.min() >= 32
        h = g * u
        if not free:
            assert np.array_equal(h.astype(np.float16).astype(np.int64), h)
        assert not (h % unit).any() and np.abs(h // unit).sum(1, initial=0).max(initial=0) < 2 ** 24
        Y[rows] += h @ wd.T
    Yo = Y.astype(np.float64) / 128 / k
    assert np.abs(Yo).max() < 65504
    return X.astype(np.float16), router.astype(np.float16), gu, dn, Yo.astype(np.float16), ids.astype(np.int32)


# A value of H, and of Y, is off by its rounding to fp16: at most 2^-11 of it, 2^-11 / sqrt(3)
# in the mean square.  The down weights have signs at random, so that H's errors meet in Y
# as H itself does, and Y's two errors together are 2^-11 sqrt(2 / 3) = 4.0e-4 of Y's mean
# square at most; the fp32 sums add less than 1e-5.  Twice that, for the spread of a row's
# mean square over 64 outputs.
ROW_BOUND = 8e-4


def row_distance(got, want):
    """Root mean square error of each row, relative to the row."""
    got = np.asarray(got, np.float64)
    return np.sqrt(((got - want) ** 2).mean(1) / (want ** 2).mean(1))
