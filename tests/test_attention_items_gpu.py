"""GPU tests of the exact softmax attention where every CTA goes through several work items: the
carry-over from item to item (barrier phases, ring positions, the counter), against the fp64
oracle within its derived bounds, with the device status word read after each."""
import numpy as np
import pytest
import torch

import rank_linear_complexity_gb300.linformer as lf
from oracle import softmax_attention as orc

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF = torch.bfloat16


def make(b, hq, hk, nq, nk, d, seed, gain=1.5):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def rand(h, n, s):
        return (torch.randn(b, h, n, d, generator=g, device=DEV) * s).to(BF)

    return rand(hq, nq, gain), rand(hk, nk, gain), rand(hk, nk, 1), rand(hq, nq, 1)


def int32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV)


def status():
    torch.cuda.synchronize()
    assert lf.linformer_debug_read_device_status() == 0


def close(got, ref, bound, name):
    got, bad = orc.host64(got), np.isinf(ref)
    assert np.array_equal(got[bad], ref[bad]), name
    err = np.abs(np.where(bad, 0, got) - np.where(bad, 0, ref))
    assert (err <= bound).all(), f"{name}: worst {np.nanmax(err - bound)}"


def entries(t, at):
    return [x[at] for x in t]


# Valid lengths that put items of two query tiles before items of one (and of none) on a CTA: under
# the causal mask the second tile has a key block more, so the first runs ahead of it.
MIXED = [220, 150, 250, 30, 150, 150, 30, 220, 1, 255, 129, 0, 128, 200, 17, 256]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads,causal", [(3, True), (24, True), (24, False)],
                         ids=["in_turn", "counter", "counter_all_keys"])
def test_ragged_prompts_of_mixed_lengths(d, heads, causal):
    """heads 3: 192 items, more than the SMs but too few for the counter; 24: 1536, from it."""
    rng = np.random.default_rng(d + heads)
    ls = [MIXED[i] for j in range(4) for i in rng.permutation(len(MIXED))]
    b, n = len(ls), 256
    Q, K, V, dO = make(b, heads, heads, n, n, d, seed=heads + d)
    for i, l in enumerate(ls):
        for x in (Q, K, V, dO):
            x[i, :, l:] = float("nan")
    for _ in range(3):
        O, lse = lf.softmax_attention(Q, K, V, int32(ls), int32(ls), causal=causal)
        status()
        for i in rng.choice(b, 8, replace=False):
            at, one = slice(i, i + 1), slice(i % heads, i % heads + 1)
            q, k, v = (x[at, one] for x in (Q, K, V))
            ref, rl, bO, bl = orc.forward(q, k, v, [ls[i]], [ls[i]], causal=causal)
            close(O[at, one], ref, bO, f"O {i}")
            close(lse[at, one], rl, bl, f"lse {i}")
    # every row of every entry: an entry alone (one item a CTA) gives the same bits
    for i in range(0, b, 5):
        at = slice(i, i + 1)
        a = lf.softmax_attention(Q[at], K[at], V[at], int32(ls[at]), int32(ls[at]), causal=causal)
        assert torch.equal(a[0].view(torch.int16), O[at].view(torch.int16))
        assert torch.equal(a[1], lse[at])
    status()
