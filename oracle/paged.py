"""fp64 oracle of the paged key/value cache: rows by table, appended and kept rows, trees of
drafted tokens, attention over the pages (numpy; test infrastructure only).

``forward`` returns bounds as oracle.softmax_attention does, for the same roundings.
"""
import numpy as np

from oracle import rotary
from oracle import softmax_attention as att
from oracle.softmax_attention import U, host64


def rows(cache, table, length):
    """Rows 0 .. length - 1 of one sequence, [hk][length][d]; pages that are not there are zeros."""
    pages, hk, page, d = cache.shape
    out = np.zeros((hk, length, d))
    for j in range(length):
        x = int(table[j // page])
        if 0 <= x < pages:
            out[:, j] = cache[x, :, j % page]
    return out


def place(cache, table, at):
    """(page, row) of row `at` of one sequence, or None."""
    page = cache.shape[2]
    if not 0 <= at < len(table) * page:
        return None
    x = int(table[at // page])
    return (x, at % page) if 0 <= x < cache.shape[0] else None


def append(K, V, k_cache, v_cache, table, starts, counts=None, f=None, positions=None, rot=0,
           interleaved=False, amplitude=1.0, Q=None):
    """(k_cache, v_cache, turned Q or None), the caches as float64 copies."""
    K, V, kc, vc = host64(K), host64(V), host64(k_cache).copy(), host64(v_cache).copy()
    b, _, n, _ = K.shape
    starts = [int(x) for x in starts]
    if f is not None:
        if positions is None:
            positions = np.array([[s + i for i in range(n)] for s in starts])
        K = rotary.rotate(K, f, positions, rot, interleaved, amplitude)
        Q = None if Q is None else rotary.rotate(Q, f, positions, rot, interleaved, amplitude)
    for bi in range(b):
        for i in range(n if counts is None else min(max(int(counts[bi]), 0), n)):
            to = place(kc, table[bi], starts[bi] + i)
            if to:
                kc[to[0], :, to[1]], vc[to[0], :, to[1]] = K[bi, :, i], V[bi, :, i]
    return kc, vc, Q


def keep(k_cache, v_cache, table, starts, path, counts=None):
    old = [host64(k_cache), host64(v_cache)]
    new = [x.copy() for x in old]
    b, m = path.shape
    for bi in range(b):
        for i in range(m if counts is None else min(max(int(counts[bi]), 0), m)):
            node = int(path[bi][i])
            to = place(old[0], table[bi], int(starts[bi]) + i)
            source = place(old[0], table[bi], int(starts[bi]) + node)
            if node >= i and to and source:
                for x, y in zip(new, old):
                    x[to[0], :, to[1]] = y[source[0], :, source[1]]
    return tuple(new)


def ancestors(parents):
    """True where node i sees node j: [b][n][n]."""
    b, n = parents.shape
    out = np.zeros((b, n, n), dtype=bool)
    for bi in range(b):
        for i in range(n):
            j = i
            while j >= 0:
                out[bi, i, j] = True
                up = int(parents[bi][j])
                j = up if -1 <= up < j else -1
    return out


def words(bits):
    """A mask [b][n][n] as int64 words [b][n][ceil(n / 64)]."""
    b, n, _ = bits.shape
    w = np.zeros((b, n, -(-n // 64) * 64), dtype=np.uint8)
    w[:, :, :n] = bits
    return np.packbits(w, axis=2, bitorder="little").view(np.uint64).view(np.int64)


def forward(Q, k_cache, v_cache, table, k_lengths, q_lengths=None, causal=False, window=0,
            scale=None, tree=None):
    """(O, lse, bound of |O error|, bound of |lse error|); tree: a mask [b][nq][nq] in place of
    causal and window."""
    Q, kc, vc = host64(Q), host64(k_cache), host64(v_cache)
    b, hq, nq, d = Q.shape
    hk, page = kc.shape[1], kc.shape[2]
    scale = d ** -0.5 if scale is None else scale
    O, lse = np.zeros(Q.shape), np.full((b, hq, nq), -np.inf)
    bO, bl = np.zeros(Q.shape), np.zeros((b, hq, nq))
    for bi in range(b):
        lk = min(max(int(k_lengths[bi]), 0), len(table[bi]) * page)
        lq = nq if q_lengths is None else min(max(int(q_lengths[bi]), 0), nq)
        K, V = rows(kc, table[bi], lk), rows(vc, table[bi], lk)
        m = att.visible(nq, lk, lq, lk, causal, window)
        if tree is not None:
            for j in range(max(lk - lq, 0), lk):
                m[:, j] &= tree[bi][:, j - (lk - lq)]
        for h in range(hq):
            q, k, v = att._valid_rows(Q[bi, h], lq), K[h // (hq // hk)], V[h // (hq // hk)]
            p, l, eps = att._probabilities(q, k, m, scale, d)
            O[bi, h], lse[bi, h] = p @ v, l
            sums = att._sums(max(lk, 1))
            bO[bi, h] = (U + eps + sums) * (p @ np.abs(v)) + U * np.abs(O[bi, h])
            bl[bi, h] = eps + sums + 2.0 ** -22 * np.abs(np.where(np.isfinite(l), l, 0.0))
    return O, lse, bO, bl
