"""Plain fp64 forms of the serving operators (adapter product, norms around a
block, mixture-of-experts layer) and random packed layers for their tests."""

import numpy as np

from oracle import awq_oracle as O


def ulp16(v):
    a = np.abs(np.asarray(v, dtype=np.float64))
    return np.exp2(np.floor(np.log2(np.maximum(a, 2.0 ** -14))) - 10)


def random_packed(inn, out, group, rng, pow2=False, std=0.02):
    """qweight, qzeros, scales with random codes and zero points; steps 2^e
    (e in -4..2) or values around std / 4."""
    qw = rng.integers(-2 ** 31, 2 ** 31, size=(inn, out // 8)).astype(np.int32)
    qz = rng.integers(-2 ** 31, 2 ** 31, size=(inn // group, out // 8)).astype(np.int32)
    if pow2:
        sc = np.exp2(rng.integers(-4, 3, size=(inn // group, out)))
    else:
        sc = std / 4 * np.exp(0.3 * rng.standard_normal((inn // group, out)))
    return qw, qz, sc.astype(np.float16)


def weights(packed, group):
    """W [out, in] fp64 = (q - z) scale, and the magnitudes (q + z) scale that
    bound the sums of codes and of zero points apart from each other."""
    qw, qz, sc = packed
    q = O.unpack_nibbles(qw).astype(np.float64)
    z = np.repeat(O.unpack_nibbles(qz).astype(np.float64), group, axis=1)
    s = np.repeat(sc.astype(np.float64).T, group, axis=1)
    return (q - z) * s, (q + z) * s


def lora(X, packed, group, A, B, c, ids):
    """(Y fp64, magnitude sums): Y = X W^T + c_a (X A_a^T) B_a^T.  The second
    value is (sum |x| (q + z) s, sum |x| |W|, |c| |x| |A| |B|, |c u| |B|)."""
    X = X.astype(np.float64)
    W, mag = weights(packed, group)
    Y = X @ W.T
    m_code, m_w = np.abs(X) @ mag.T, np.abs(X) @ np.abs(W).T
    m_low, m_u = np.zeros_like(Y), np.zeros_like(Y)
    for t, a in enumerate(ids):
        if 0 <= a < A.shape[0]:
            Aa, Ba, ca = A[a].astype(np.float64), B[a].astype(np.float64), float(c[a])
            u = ca * (Aa @ X[t])
            Y[t] += Ba @ u
            m_low[t] = abs(ca) * (np.abs(Ba) @ (np.abs(Aa) @ np.abs(X[t])))
            m_u[t] = np.abs(Ba) @ np.abs(u)
    return Y, (m_code, m_w, m_low, m_u)


def lora_tolerance(Y, mags, inn, rank, rounded):
    """Per output: one fp16 rounding of the result, and what the fp32 sums may
    lose.  A sum of n terms on the tensor cores or in FMAs loses at most
    2^-23 of the running magnitude per addition (truncation counted), so at
    most n 2^-23 of the sum of the magnitudes: n = in + 8 for the codes' and
    the zero points' sums with their scaling, in + rank + 8 for the low-rank
    part.  `rounded` (more than 64 tokens): the weights and U are rounded to
    fp16 first, 2^-11 of each product."""
    m_code, m_w, m_low, m_u = mags
    acc = (inn + 8) * 2.0 ** -23 * m_code + (inn + rank + 8) * 2.0 ** -23 * m_low
    if rounded:
        acc = acc + 2.0 ** -11 * (m_w + m_u)
    return acc + 0.5 * ulp16(np.abs(Y) + acc)


def block_norm(R, V, post, gate, c, pre, eps):
    """(r' or None, n) in fp64; the inputs fp16 or None."""
    r = R.astype(np.float64)
    if V is not None:
        v = V.astype(np.float64)
        if post is not None:
            v = v / np.sqrt((v * v).mean(1, keepdims=True) + eps) * post.astype(np.float64)
        if gate is not None:
            v = v * gate.astype(np.float64)
        r = r + float(np.float32(c)) * v
    n = r / np.sqrt((r * r).mean(1, keepdims=True) + eps)
    if pre is not None:
        n = n * pre.astype(np.float64)
    return r, n


def moe(X, router, gate_up, down, group, top_k, renormalize, mask=None):
    """(Y, ids, weights, tolerance) in fp64: gate_up and down are lists of one
    packed layer per expert.  The tolerance per output follows the roundings:
    n-term fp32 sums lose at most n 2^-23 of the sums of magnitudes
    (lora_tolerance), silu(g) u carries g's and u's errors by its derivatives
    (|silu'| < 1.1) and one fp16 rounding, the softmax weights 2^-19 (their
    exponent, exp and division), then one fp16 rounding of the result (and one
    fp32 subnormal step where everything underflows)."""
    T, h = X.shape
    E = router.shape[0]
    x = X.astype(np.float64)
    logits = np.where(np.isfinite(x), x, 0) @ router.astype(np.float64).T
    Y, tol = np.zeros((T, h)), np.zeros((T, h))
    ids = np.full((T, top_k), -1, np.int32)
    wt = np.zeros((T, top_k))
    cache = {}
    for t in range(T):
        if mask is not None and not mask[t]:
            continue
        order = sorted(range(E), key=lambda e: (-logits[t, e], e))[:top_k]
        p = np.exp(logits[t] - logits[t].max())
        p = p[order] / (p[order].sum() if renormalize else p.sum())
        ids[t], wt[t] = order, p
        for e, pe in zip(order, p):
            if e not in cache:
                cache[e] = weights(gate_up[e], group) + weights(down[e], group)
            Wg, Mg, Wd, Md = cache[e]
            inter = Wd.shape[1]
            gu = Wg @ x[t]
            dgu = (h + 8) * 2.0 ** -23 * (Mg @ np.abs(x[t]))
            g, u = gu[:inter], gu[inter:]
            sig = 1 / (1 + np.exp(-g))
            H = g * sig * u
            dH = 1.1 * dgu[:inter] * (np.abs(u) + dgu[inter:]) + np.abs(g * sig) * dgu[inter:]
            dH = dH + 2.0 ** -11 * np.abs(H) + 2.0 ** -21 * np.abs(H) + 2.0 ** -25
            Y[t] += pe * (Wd @ H)
            tol[t] += pe * (np.abs(Wd) @ dH + ((inter + 64) * 2.0 ** -23) * (Md @ np.abs(H)))
            tol[t] += pe * 2.0 ** -19 * np.abs(Wd @ H)
    tol = tol + 0.5 * ulp16(np.abs(Y) + tol)
    return Y, ids, wt, tol
