"""GPU tests of the exact softmax attention (linformer_softmax_attn_fwd / _bwd through the
Python binding) against the fp64 oracle, elementwise within the oracle's derived bounds, and
within 5e-3 in the 2-norm: three independent roundings of relative size at most 2^-8, rms
2^-8 / sqrt(3), give sqrt(3) x 2^-8 / sqrt(3) = 3.9e-3, and the fp32 part is below 1e-3.
The rounding of O that delta = dO.O takes over is one error for a whole row of dS, which sums
over the keys do not average out: its bound is allowed on top."""
import numpy as np
import pytest
import torch

import rank_linear_complexity_gb300.linformer as lf
from oracle import softmax_attention as orc

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF = torch.bfloat16


def tensors(b, hq, hk, nq, nk, d, seed=0, gain=1.5, packed=False):
    """Q, K, V, dO on the device; packed: Q, K and V as slices of one fused buffer."""
    g = torch.Generator().manual_seed(seed)

    def rand(h, n, s):
        return (torch.randn(b, h, n, d, generator=g) * s).to(BF)

    Q, K, V, dO = rand(hq, nq, gain), rand(hk, nk, gain), rand(hk, nk, 1), rand(hq, nq, 1)
    if packed:
        buf = torch.full((b, nq, (hq + 2 * hk) * d), float("nan"), dtype=BF, device=DEV)
        views, at = [], 0
        for x in (Q, K, V):
            h = x.shape[1]
            v = buf[:, :, at:at + h * d].view(b, nq, h, d).transpose(1, 2)
            v.copy_(x)
            views.append(v)
            at += h * d
        wide = torch.empty(b, nq, hq, d, dtype=BF, device=DEV).transpose(1, 2)
        return (*views, wide.copy_(dO))
    return tuple(x.to(DEV) for x in (Q, K, V, dO))


def lengths(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV)


def status():
    torch.cuda.synchronize()
    assert lf.linformer_debug_read_device_status() == 0


def within(got, ref, bound, name, rows=None):
    got, bad = orc.host64(got), np.isinf(ref)
    assert np.array_equal(got[bad], ref[bad]), name
    err = np.abs(np.where(bad, 0, got) - np.where(bad, 0, ref))
    assert np.isfinite(err).all(), f"{name}: not finite"
    over = err > bound
    assert not over.any(), f"{name}: {over.sum()} over, worst {(err - bound).max()} at " \
                           f"{np.unravel_index((err - bound).argmax(), err.shape)}"
    if ref.size >= 4096 and np.linalg.norm(ref[~bad]) > 0:
        rel = np.linalg.norm(err[~bad]) / np.linalg.norm(ref[~bad])
        extra = 0 if rows is None else np.linalg.norm(rows) / np.linalg.norm(ref)
        assert rel <= 5e-3 + extra, f"{name}: 2-norm {rel}"


CASES = {
    # name: b, hq, hk, nq, nk, d, options
    "one": (1, 1, 1, 1, 1, 64, {}),
    "prompt": (2, 4, 2, 77, 77, 64, dict(causal=True, packed=True)),
    "cross": (1, 3, 3, 130, 201, 40, {}),
    "token": (2, 8, 2, 1, 1000, 128, dict(k=[1000, 0])),
    "tokens_causal": (1, 8, 1, 5, 515, 96, dict(causal=True)),
    "window": (2, 2, 2, 300, 300, 128, dict(causal=True, window=100)),
    "ragged_empty_rows": (3, 6, 3, 257, 129, 80, dict(causal=True, q=[257, 30, 129],
                                                      k=[129, 77, 1])),
    "odd_group": (1, 5, 1, 200, 384, 64, {}),
    "token_split": (1, 2, 2, 1, 9000, 64, {}),
    "encoder": (2, 12, 12, 640, 640, 64, dict(q=[640, 161], k=[640, 161])),
    "tokens_window_split": (1, 16, 2, 3, 4000, 128, dict(causal=True, window=700)),
    "many_items": (6, 16, 8, 384, 384, 128, dict(causal=True, packed=True)),
    "many_short": (40, 6, 3, 100, 140, 64, dict(q=list(range(0, 100, 5)) * 2,
                                                k=list(range(7, 127, 3)))),
    "smallest_head": (2, 2, 1, 150, 150, 8, dict(causal=True)),
    "ends_in_tile": (2, 1, 1, 256, 256, 128, dict(q=[128, 129], k=[128, 129])),
}


def options(o):
    kw = dict(causal=o.get("causal", False), window=o.get("window", 0))
    return kw, o.get("q"), o.get("k")


def poison(Q, K, V, dO, q, k):
    """Rows past the lengths hold NaN."""
    for bi in range(Q.shape[0]):
        if q is not None:
            Q[bi, :, q[bi]:] = float("nan")
            dO[bi, :, q[bi]:] = float("nan")
        if k is not None:
            K[bi, :, k[bi]:] = float("nan")
            V[bi, :, k[bi]:] = float("nan")


@pytest.mark.parametrize("name", CASES)
def test_forward(name):
    b, hq, hk, nq, nk, d, o = CASES[name]
    kw, q, k = options(o)
    Q, K, V, dO = tensors(b, hq, hk, nq, nk, d, seed=nq + nk, packed=o.get("packed", False))
    poison(Q, K, V, dO, q, k)
    O, lse = lf.softmax_attention(Q, K, V, lengths(q), lengths(k), **kw)
    status()
    ref, rl, bO, bl = orc.forward(Q, K, V, q, k, **kw)
    within(O, ref, bO, "O")
    within(lse, rl, bl, "lse")


@pytest.mark.parametrize("name", CASES)
def test_backward(name):
    b, hq, hk, nq, nk, d, o = CASES[name]
    kw, q, k = options(o)
    Q, K, V, dO = tensors(b, hq, hk, nq, nk, d, seed=nq + nk + 1, packed=o.get("packed", False))
    poison(Q, K, V, dO, q, k)
    ref, rl, _, _ = orc.forward(Q, K, V, q, k, **kw)
    O = torch.from_numpy(ref).to(DEV, BF)
    lse = torch.from_numpy(rl).to(DEV, torch.float32)
    if q is not None:
        for bi in range(b):
            O[bi, :, q[bi]:] = float("nan")
    got = lf.softmax_attention_backward(Q, K, V, O, dO, lse, lengths(q), lengths(k), **kw)
    status()
    refs, bounds, rows = orc.backward(Q, K, V, dO, q, k, **kw)
    for n, g, r, e, w in zip(("dQ", "dK", "dV"), got, refs, bounds, rows):
        within(g, r, e, n, w)
