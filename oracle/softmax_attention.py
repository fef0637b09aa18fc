"""fp64 oracle of the exact softmax attention and its backward, with shared key/value heads,
lengths, causal and windowed masks (numpy; test infrastructure only).

Query i of Lq stands at position i + Lk - Lq and sees key j < Lk iff, when causal,
j <= position and, with a window w > 0, j > position - w.  Rows without keys and rows past
the length give O = 0, lse = -inf and no gradient.

Beside the values, ``forward`` and ``backward`` return how far a kernel may be off that
rounds P, dS and its outputs to bf16 and does everything else in fp32 (`U` = half a bf16
step, relative): each bound is the sum of absolute terms times the relative error of each,
so it holds for any order of summation.
"""
import numpy as np

U = 2.0 ** -8


def host64(x):
    return x.double().cpu().numpy() if hasattr(x, "cpu") else np.asarray(x, dtype=np.float64)


def visible(nq, nk, lq, lk, causal, window):
    i, j = np.arange(nq)[:, None], np.arange(nk)[None]
    m = (i < lq) & (j < lk)
    if causal:
        m &= j <= i + lk - lq
        if window:
            m &= j > i + lk - lq - window
    return m


def _units(Q, K, q_lengths, k_lengths, causal, window):
    b, hq, nq, _ = Q.shape
    hk, nk = K.shape[1], K.shape[2]
    for bi in range(b):
        lq = nq if q_lengths is None else min(max(int(q_lengths[bi]), 0), nq)
        lk = nk if k_lengths is None else min(max(int(k_lengths[bi]), 0), nk)
        m = visible(nq, nk, lq, lk, causal, window)
        for h in range(hq):
            yield bi, h, h // (hq // hk), lq, lk, m


def _probabilities(q, k, m, scale, d):
    """(p, lse, eps): eps is the relative error of p from the fp32 sums of Q.K."""
    s = np.where(m, scale * (q @ k.T), -np.inf)
    top = s.max(1, keepdims=True, initial=-np.inf)
    top = np.where(np.isfinite(top), top, 0.0)
    e = np.exp(s - top)
    total = e.sum(1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (top + np.log(total))[:, 0]
    p = e / np.where(total == 0, 1.0, total)
    # fp32 sums of d products: at most d 2^-23 of their absolute terms, in s and in lse; the
    # exponential's argument is rounded to 2^-24 of its size, the exponential to 2^-22
    terms = scale * (np.abs(q) @ np.abs(k).T)
    size = np.where(m, terms, 0.0).max(initial=0.0)
    return p, lse, 2 * d * 2.0 ** -23 * size + 2.0 ** -22 * size + 2.0 ** -20


def _sums(n):
    """fp32 sums of n terms: the product's accumulator takes 16 terms a step (n / 16 roundings
    of 2^-23), the row sum runs in four strands (n / 4 of 2^-24), joined in a few steps."""
    return n * 2.0 ** -25 + 2.0 ** -20


def _valid_rows(x, n):
    y = np.array(x[:n])
    return np.concatenate([y, np.zeros((x.shape[0] - n, x.shape[1]))])


def forward(Q, K, V, q_lengths=None, k_lengths=None, causal=False, window=0, scale=None):
    """(O, lse, bound of |O error|, bound of |lse error|)."""
    Q, K, V = host64(Q), host64(K), host64(V)
    b, hq, nq, d = Q.shape
    scale = d ** -0.5 if scale is None else scale
    O, lse = np.zeros(Q.shape), np.full((b, hq, nq), -np.inf)
    bO, bl = np.zeros(Q.shape), np.zeros((b, hq, nq))
    for bi, h, kv, lq, lk, m in _units(Q, K, q_lengths, k_lengths, causal, window):
        q, k, v = (_valid_rows(Q[bi, h], lq), _valid_rows(K[bi, kv], lk),
                   _valid_rows(V[bi, kv], lk))
        p, l, eps = _probabilities(q, k, m, scale, d)
        O[bi, h], lse[bi, h] = p @ v, l
        # P rounded once, O rounded once, fp32 sums over the keys and the row sum
        sums = _sums(K.shape[2])
        bO[bi, h] = (U + eps + sums) * (p @ np.abs(v)) + U * np.abs(O[bi, h])
        bl[bi, h] = eps + sums + 2.0 ** -22 * np.abs(np.where(np.isfinite(l), l, 0.0))
    return O, lse, bO, bl


def backward(Q, K, V, dO, q_lengths=None, k_lengths=None, causal=False, window=0, scale=None,
             O=None):
    """((dQ, dK, dV), their bounds, the part of the bounds that comes from delta = dO.O with O
    rounded to bf16: one error for a whole row, which sums over keys do not average out).

    With O, the forward's result as the kernel was given it, delta is taken from that: then its
    rounding is no error, and that part is zero."""
    Q, K, V, dO = host64(Q), host64(K), host64(V), host64(dO)
    O = None if O is None else host64(O)
    d = Q.shape[3]
    scale = d ** -0.5 if scale is None else scale
    out = [np.zeros(Q.shape), np.zeros(K.shape), np.zeros(K.shape)]
    bound = [np.zeros(Q.shape), np.zeros(K.shape), np.zeros(K.shape)]
    rows = [np.zeros(Q.shape), np.zeros(K.shape), np.zeros(K.shape)]
    for bi, h, kv, lq, lk, m in _units(Q, K, q_lengths, k_lengths, causal, window):
        q, g = _valid_rows(Q[bi, h], lq), _valid_rows(dO[bi, h], lq)
        k, v = _valid_rows(K[bi, kv], lk), _valid_rows(V[bi, kv], lk)
        p, _, eps = _probabilities(q, k, m, scale, d)
        dp = g @ v.T
        o = p @ v if O is None else _valid_rows(O[bi, h], lq)
        delta = ((p * dp) if O is None else g * o).sum(1, keepdims=True)
        ds = p * (dp - delta)
        out[0][bi, h] += scale * (ds @ k)
        out[1][bi, kv] += scale * (ds.T @ q)
        out[2][bi, kv] += p.T @ g
        # dK and dV sum over the queries of every head of the group, dQ over the keys
        sums = _sums(max(q.shape[0] * (Q.shape[1] // K.shape[1]), k.shape[0]))
        # delta from the rounded O (none where it is the one given), dP and delta as fp32 sums of
        # d products
        e_delta = (np.abs(g) * np.abs(o)).sum(1, keepdims=True) * ((U if O is None else 0.0) + d * 2.0 ** -23)
        e_dp = d * 2.0 ** -23 * (np.abs(g) @ np.abs(v).T)
        e_ds = (U + eps + sums) * np.abs(ds) + p * (e_delta + e_dp) * (1 + U) + eps * p * np.abs(delta)
        bound[0][bi, h] += scale * (e_ds @ np.abs(k))
        bound[1][bi, kv] += scale * (e_ds.T @ np.abs(q))
        if O is None:
            rows[0][bi, h] += scale * ((p * e_delta) @ np.abs(k))
            rows[1][bi, kv] += scale * ((p * e_delta).T @ np.abs(q))
        bound[2][bi, kv] += (U + eps + sums) * (p.T @ np.abs(g))
    for x, y in zip(bound, out):
        x += U * np.abs(y) * (1 + U)
    return tuple(out), tuple(bound), tuple(rows)
