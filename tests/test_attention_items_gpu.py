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


# --- schedules: items in turn, in sets of heads, from the counter -----------------------------

def plan(b, hq, hk, nq, nk, d, causal=False, window=0, ragged=False):
    """(items, SMs, order) of the forward: the library's rules from sizes and the SM count."""
    sms = torch.cuda.get_device_properties(DEV).multi_processor_count
    box = 128
    while box > 1 and box // 2 >= nq:
        box //= 2
    heads = min(128 // box, hq // hk)
    tiles = -(-nq // box) * -(-(hq // hk) // heads)
    pairs, units = (tiles + 1) // 2, b * hk
    whole, window = units * pairs, 0 if window >= nk else window
    blocks = -(-(min(nk, window + 128) if window else nk) // 128)
    wanted = -(-6 * sms // whole) if box * heads <= 16 else sms // whole
    split = 1 if blocks < 12 else max(1, min(wanted, blocks // 4))
    return whole * split, sms, split


def gradient_error(got, ref, bound, name):
    """Elementwise within the bound, and 5e-3 in the 2-norm: three independent roundings of at
    most 2^-8 (P or dS, O within it, the result), rms 2^-8 / sqrt(3) each, are 3.9e-3, and the
    fp32 part is below 1e-3; delta's own rounding is no part of it, since the reference takes
    delta from the O that the kernel was given.

    Weights below the smallest normal fp32 number are zero in the kernels (in the 64-bit reference
    they are not): at most 2^-126 of a term each, over at most 2^12 rows, a term being at most
    2^14 (|dP - delta| with d = 128 products of values below 2^3) times 2^6 (|Q|, |K|): 2^-94."""
    close(got, ref, bound + 2.0 ** -94, name)
    if ref.size >= 4096 and np.linalg.norm(ref) > 0:
        rel = np.linalg.norm(orc.host64(got) - ref) / np.linalg.norm(ref)
        assert rel <= 5e-3, f"{name}: 2-norm {rel}"


def against_oracle(b, hq, hk, nq, nk, d, seed, q=None, k=None, scale=None, samples=6, gain=1.5, change=None, **kw):
    """Forward and backward of the whole call; sampled key/value heads (with their group) of sampled
    entries against the oracle."""
    Q, K, V, dO = make(b, hq, hk, nq, nk, d, seed, gain)
    if change:
        change(Q, K, V, dO)
    for i in range(b):
        for x, ls in ((Q, q), (dO, q), (K, k), (V, k)):
            if ls is not None:
                x[i, :, ls[i]:] = float("nan")
    O, lse = lf.softmax_attention(Q, K, V, int32(q), int32(k), scale=scale, **kw)
    grads = lf.softmax_attention_backward(Q, K, V, O, dO, lse, int32(q), int32(k), scale=scale, **kw)
    status()
    rng = np.random.default_rng(seed)
    g = hq // hk
    for n in rng.choice(b * hk, min(samples, b * hk), replace=False):
        i, h = int(n) // hk, int(n) % hk
        own, shared, at = slice(h * g, (h + 1) * g), slice(h, h + 1), slice(i, i + 1)
        x = (Q[at, own], K[at, shared], V[at, shared])
        ls = (None if q is None else q[at], None if k is None else k[at])
        ref, rl, bO, bl = orc.forward(*x, *ls, scale=scale, **kw)
        close(O[at, own], ref, bO, f"O {i} {h}")
        close(lse[at, own], rl, bl, f"lse {i} {h}")
        refs, bounds, _ = orc.backward(*x, dO[at, own], *ls, scale=scale, O=O[at, own], **kw)
        for name, y, hs, r, e in zip(("dQ", "dK", "dV"), grads, (own, shared, shared), refs, bounds):
            gradient_error(y[at, hs], r, e, f"{name} {i} {h}")
    return O, lse, grads


def mixed(b, n, seed, empty=True):
    rng = np.random.default_rng(seed)
    x = rng.integers(1, n + 1, b)
    if empty:
        x[::7] = 0
    x[1] = n
    return x.tolist()


FEW = {  # name: sizes, lengths of queries and keys, options, items a CTA from the counter
    "counter": ((32, 24, 12, 300, 300, 64), True, dict(causal=True), True),
    "counter_wide_window": ((40, 20, 10, 290, 290, 128), True, dict(causal=True, window=70), True),
    "counter_all_keys_wide": ((40, 9, 9, 129, 300, 96), True, {}, True),
    "in_turn": ((20, 32, 32, 200, 333, 64), False, {}, False),
    "in_turn_wide_group": ((60, 30, 10, 100, 270, 128), False, {}, False),
    "counter_no_lengths": ((20, 32, 16, 260, 260, 128), False, dict(causal=True), True),
}


@pytest.mark.parametrize("name", FEW)
def test_several_items_a_cta(name):
    (b, hq, hk, nq, nk, d), ragged, kw, counter = FEW[name]
    items, sms, split = plan(b, hq, hk, nq, nk, d, **kw)
    assert items > 2 * sms and split == 1
    assert counter == bool(ragged or kw.get("causal"))
    q, k = (mixed(b, nq, 1), mixed(b, nk, 2)) if ragged else (None, None)
    against_oracle(b, hq, hk, nq, nk, d, 3, q, k, samples=20, **kw)


SETS = {  # heads that stream more than L2 keeps (48 MB): forward in sets without a causal mask
    # (ragged ones from the counter, wide heads only), backward also with one (from 128 MB)
    "wide_all_keys": ((25, 8, 4, 2048, 1024, 128), False, {}),
    "wide_ragged": ((25, 8, 4, 2048, 1024, 128), True, {}),
    "all_keys": ((13, 16, 16, 4096, 1024, 64), False, {}),
    "ragged": ((13, 16, 16, 4096, 1024, 64), True, {}),
    "causal": ((17, 16, 16, 2048, 2048, 64), False, dict(causal=True)),
    "wide_causal": ((9, 16, 16, 2048, 2048, 128), True, dict(causal=True)),
}


@pytest.mark.parametrize("name", SETS)
def test_heads_in_sets_against_the_oracle(name):
    (b, hq, hk, nq, nk, d), ragged, kw = SETS[name]
    items, sms, split = plan(b, hq, hk, nq, nk, d, **kw)
    streamed = 4 * b * hk * nk * d
    assert items > 2 * sms and streamed > 48 << 20 and (kw or items // (b * hk) >= 16)
    q, k = (mixed(b, nq, 3), mixed(b, nk, 4)) if ragged else (None, None)
    against_oracle(b, hq, hk, nq, nk, d, 5, q, k, samples=4, **kw)


@pytest.mark.parametrize("d", [64, 128])
def test_tokens_split_within_a_window(d):
    """A window long enough for its keys to be split, ragged and with empty entries."""
    b, hq, hk, nq, nk, window = 3, 16, 2, 3, 4000, 1700
    assert plan(b, hq, hk, nq, nk, d, window=window)[2] > 1
    against_oracle(b, hq, hk, nq, nk, d, 7, [3, 2, 3], [4000, 3001, 0], causal=True, window=window)


# Shapes of a few items: parts of long sums, edges of tiles and steps, empty entries.
SHAPES = {
    "prompt": (2, 4, 2, 77, 77, 64, None, None, dict(causal=True)),
    "cross": (1, 3, 3, 130, 201, 40, None, None, {}),
    "token_split": (1, 2, 2, 1, 9000, 64, None, None, {}),
    "encoder": (2, 12, 12, 640, 640, 64, [640, 161], [640, 161], {}),
    "many_items": (6, 16, 8, 384, 384, 128, None, None, dict(causal=True)),
    "empty_rows": (3, 6, 3, 257, 129, 80, [257, 30, 129], [129, 77, 1], dict(causal=True)),
    "step_edges": (3, 4, 2, 192, 192, 128, [191, 63, 1], [191, 63, 1], dict(causal=True)),
    "few_keys": (2, 16, 2, 600, 46, 96, [600, 155], None, {}),
    "few_keys_causal": (1, 8, 1, 1100, 200, 64, [1090], [170], dict(causal=True)),
    "few_queries": (1, 4, 2, 40, 5000, 64, None, [4990], {}),
    "few_queries_window": (2, 2, 1, 300, 5000, 128, [300, 7], [5000, 200], dict(causal=True, window=3500)),
    "few_queries_none": (3, 2, 1, 30, 4500, 64, [0, 30, 29], [4500, 0, 4437], dict(causal=True)),
}


@pytest.mark.parametrize("name", SHAPES)
def test_gradients_with_the_forwards_own_result(name):
    """Every head, with delta from the O that the forward gave: no allowance for its rounding."""
    b, hq, hk, nq, nk, d, q, k, kw = SHAPES[name]
    against_oracle(b, hq, hk, nq, nk, d, 11, q, k, samples=b * hk, **kw)


# --- logits that outgrow the reference maximum ------------------------------------------------

@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("kw", [{}, dict(causal=True), dict(causal=True, window=200)],
                         ids=["all_keys", "causal", "window"])
def test_outgrown_maxima(d, kw):
    """Later blocks outgrow the first by more than 2^16 again and again, several items a CTA,
    forward and backward at scale 1."""
    b, hq, hk, n = 40, 8, 8, 520
    assert plan(b, hq, hk, n, n, d, **kw)[0] > 2 * plan(b, hq, hk, n, n, d, **kw)[1]

    def ramp(Q, K, V, dO):
        K.mul_(torch.linspace(0.01, 12 * 64 ** 0.5 / d ** 0.5, n, device=DEV)[:, None].to(BF))

    O, lse, _ = against_oracle(b, hq, hk, n, n, d, 9, scale=1.0, samples=8, gain=1.0, change=ramp, **kw)
    # the growth that the test is about happens: 128 keys against all that a row sees
    assert (lse[:, :, 400:].max() > 60).item()
