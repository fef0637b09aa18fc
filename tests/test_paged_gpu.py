"""GPU tests of the paged key/value cache against its fp64 oracle: rows appended and kept, trees, and
all of them together with the attention."""
import numpy as np
import pytest
import torch

import rank_linear_complexity_gb300.linformer as lf
from oracle import paged, rotary
from oracle.softmax_attention import host64
from tests.paged_cases import bits, cache, ints, random_tree

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF = torch.bfloat16


def status():
    torch.cuda.synchronize()
    assert lf.linformer_debug_read_device_status() == 0


def error_code():
    torch.cuda.synchronize()
    return lf.linformer_debug_read_device_status()


# --- append ---------------------------------------------------------------------------------

def check_append(b=3, hq=4, hk=2, n=5, d=64, page=16, starts=(0, 15, 33), counts=None, layout="rows",
                 dtype="bf16", rot=None, interleaved=False, amplitude=1.0, turn=True, queries=True,
                 placed=False, in_place=False, odd=False, seed=0, far=0):
    """Every element of the caches and of the turned queries against the oracle; whatever is not
    written keeps its bits (NaN among them)."""
    lengths = [s + n for s in starts]
    kc, vc, table = cache(b, hk, d, page, lengths, layout, dtype, seed, device=DEV)
    if odd:  # strides that are no multiples of 16 bytes
        wide = torch.full((*kc.shape[:3], d + 1), float("nan"), dtype=kc.dtype, device=DEV)
        wide[..., :d] = kc
        kc = wide[..., :d]
    g = torch.Generator(device=DEV).manual_seed(seed + 1)
    K, V, Q = (torch.randn(b, n, h, d, generator=g, device=DEV).to(kc.dtype).transpose(1, 2)
               for h in (hk, hk, hq))
    rot = d if rot is None else rot
    f = rotary.frequencies(rot)
    positions = None
    if placed:
        positions = torch.randint(far, far + 1000, (b, n), generator=g, device=DEV, dtype=torch.int32)
    before = kc.clone(), vc.clone()
    kw = {}
    if turn:
        kw = dict(phase=torch.from_numpy(rotary.phase_words(f)).to(DEV), rot=rot, positions=positions,
                  layout=lf.ROTARY_INTERLEAVED if interleaved else lf.ROTARY_HALVES,
                  amplitude=amplitude)
    want = paged.append(K, V, kc, vc, table.tolist(), starts, counts, f if turn else None,
                        None if positions is None else positions.cpu().numpy(), rot, interleaved,
                        amplitude, Q if turn and queries else None)
    if turn and queries:
        kw["Q"] = Q
        if in_place:
            kw["out"] = Q
    got = lf.cache_append(K, V, kc, vc, table, ints(starts, DEV),
                          counts=None if counts is None else ints(counts, DEV), **kw)
    status()
    # the turn in fp32 (angle and sines to 2^-22, two products and a sum), rounded once: half a step
    half = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24

    def near(x, y, turned):
        x = host64(x)
        assert np.array_equal(np.isnan(x), np.isnan(y))
        x, y = np.nan_to_num(x), np.nan_to_num(y)
        if not turned:
            assert np.array_equal(x, y)
            return
        # |x_a| + |x_z| < 10: sines off by 2^-23 each, a product rounded by 2^-24, so 15 2^-23; the
        # oracle's angle at position 2^31, a double, by 2 x 2^-22, so another 20 2^-22
        reach = amplitude * (24.0 if far else 8.0)
        assert (np.abs(x - y) <= half * np.abs(y) + 2.0 ** -21 * reach).all()
    near(kc, want[0], turn)
    near(vc, want[1], False)
    if turn and queries:
        assert got is (Q if in_place else got)
        near(got, want[2], True)
    else:
        assert got is None
    # rows that no sequence got keep their bits
    touched = np.zeros((kc.shape[0], page), dtype=bool)
    for bi in range(b):
        for i in range(n if counts is None else min(max(counts[bi], 0), n)):
            p, r = paged.place(kc, table.tolist()[bi], starts[bi] + i)
            touched[p, r] = True
    rest = torch.from_numpy(~touched).to(DEV)[:, None, :, None].expand(kc.shape)
    for x, y in zip((kc, vc), before):
        assert torch.equal(bits(x)[rest], bits(y)[rest])


@pytest.mark.parametrize("layout", ["rows", "heads", "fused"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(layout, dtype, interleaved):
    check_append(layout=layout, dtype=dtype, interleaved=interleaved)


@pytest.mark.parametrize("kw", [
    dict(n=1, starts=(0, 15, 16)), dict(n=40, starts=(0, 7, 130), page=8), dict(n=3, page=256),
    dict(rot=32), dict(d=40, rot=40), dict(d=40, rot=20, dtype="f32"), dict(d=5, rot=4), dict(d=80, rot=16),
    dict(d=128, hq=32, hk=8, n=7), dict(hq=1, hk=1), dict(b=1, starts=(3,)),
    dict(counts=(0, 5, 3)), dict(counts=(-2, 9, 1)), dict(turn=False), dict(queries=False),
    dict(placed=True), dict(placed=True, far=2 ** 31 - 2000), dict(amplitude=1.2), dict(in_place=True),
    dict(odd=True), dict(odd=True, dtype="f32", interleaved=True), dict(n=700, starts=(0, 1, 2), d=128),
    dict(b=70, starts=tuple(range(70)), n=1),
])
def test_append_shapes(kw):
    check_append(**kw)


def test_append_rows_without_a_page():
    """A table entry that names no page, a row behind the table, a start below zero: dropped and
    recorded, everything else written."""
    for starts, table_row, bad in (((14,), [0, 9], 0), ((14,), [0, -1], 0), ((30,), [0, 1], 1), ((-1,), [0, 1], 1)):
        kc = torch.full((2, 2, 16, 64), 7.0, dtype=BF, device=DEV)
        vc = kc.clone()
        K, V = torch.ones(2, 1, 2, 4, 64, dtype=BF, device=DEV)
        lf.cache_append(K, V, kc, vc, ints([table_row], DEV), ints(starts, DEV))
        assert error_code() != 0
        want = paged.append(K, V, torch.full_like(kc, 7.0), torch.full_like(kc, 7.0), [table_row], starts)
        assert np.array_equal(host64(kc), want[0]) and np.array_equal(host64(vc), want[1])
    status()


# --- keep -----------------------------------------------------------------------------------

@pytest.mark.parametrize("layout", ["rows", "heads", "fused"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kw", [dict(), dict(page=8, m=20, nodes=60), dict(d=40), dict(d=5, m=3), dict(m=1),
                                dict(counts=(0, 3, 9, -4))])
def test_keep(layout, dtype, kw):
    kw = dict(dict(page=16, m=7, nodes=30, d=64, counts=None), **kw)
    page, m, nodes, d, counts = (kw[x] for x in ("page", "m", "nodes", "d", "counts"))
    starts = (0, 5, 31, 100)
    kc, vc, table = cache(4, 3, d, page, [s + nodes for s in starts], layout, dtype, 3, device=DEV)
    rng = np.random.default_rng(5)
    # rising paths, one of them in place from its start to its end
    path = np.stack([np.sort(rng.choice(nodes, m, replace=False)) for _ in range(3)] + [np.arange(m)])
    want = paged.keep(kc, vc, table.tolist(), starts, path, counts)
    lf.cache_keep(kc, vc, table, ints(starts, DEV), ints(path.tolist(), DEV),
                  counts=None if counts is None else ints(counts, DEV))
    status()
    for x, y in zip((kc, vc), want):
        assert np.array_equal(host64(x), y, equal_nan=True)


def test_keep_the_same_node_twice_and_nodes_below_their_places():
    kc, vc, table = cache(1, 2, 64, 16, [40], device=DEV)
    for path, bad in (([3, 3, 3, 20, 20], False), ([0, 0, 5, 1, 9], True), ([4, 39, 40, 5, -1], True)):
        want = paged.keep(kc, vc, table.tolist(), (0,), np.array([path]))
        lf.cache_keep(kc, vc, table, ints([0], DEV), ints([path], DEV))
        assert (error_code() != 0) == bad
        for x, y in zip((kc, vc), want):
            assert np.array_equal(host64(x), y, equal_nan=True)


# --- trees ----------------------------------------------------------------------------------

@pytest.mark.parametrize("n", [1, 2, 31, 64, 65, 128, 200, 1024])
def test_tree_mask(n):
    for deep in (False, True):
        up = random_tree(3, n, seed=n, deep=deep)
        got = lf.tree_mask(up.to(DEV))
        status()
        assert np.array_equal(got.cpu().numpy(), paged.words(paged.ancestors(up.numpy())))


def test_tree_mask_of_a_chain_and_of_wrong_parents():
    chain = torch.arange(-1, 99, dtype=torch.int32)[None]
    assert np.array_equal(lf.tree_mask(chain.to(DEV)).cpu().numpy(),
                          paged.words(np.tril(np.ones((1, 100, 100), dtype=bool))))
    status()
    for wrong in (5, 6, -2, 2 ** 31 - 1):
        up = chain.clone()
        up[0, 5] = wrong
        got = lf.tree_mask(up.to(DEV))
        assert error_code() != 0
        assert np.array_equal(got.cpu().numpy(), paged.words(paged.ancestors(up.numpy())))


# --- together -------------------------------------------------------------------------------

def test_a_conversation():
    """Prompts, single tokens, a drafted tree and its accepted path, against one dense attention
    over the same tokens."""
    b, hq, hk, d, page, rot = 3, 8, 2, 64, 16, 64
    width, pages = 20, 70
    g = torch.Generator(device=DEV).manual_seed(11)
    kc, vc = (torch.full((pages, page, hk, d), float("nan"), dtype=BF, device=DEV).transpose(1, 2) for _ in range(2))
    table = torch.randperm(pages, generator=torch.Generator().manual_seed(1))[:b * width].view(b, width).to(torch.int32).to(DEV)
    phase = lf.rotary_phase(rot)
    total = 200

    def tokens(n):
        return [torch.randn(b, h, n, d, generator=g, device=DEV).to(BF) for h in (hq, hk, hk)]
    # the accepted tokens of every sequence, unturned
    kept = [[x[i:i + 1, :, :0] for x in tokens(1)] for i in range(b)]
    lengths = [0] * b

    def extend(i, x, rows):
        kept[i] = [torch.cat([a, y[i:i + 1, :, rows]], 2) for a, y in zip(kept[i], x)]

    def compare(O, i, queries, first):
        """Rows of O that stand at positions first.. of sequence i against the dense attention."""
        q, k, v = kept[i]
        tq, tk = lf.rotary(q, k, phase)
        want, _ = lf.softmax_attention(tq, tk, v, causal=True)
        got = O[i, :, queries].float()
        w = want[0, :, first:first + got.shape[1]].float()
        assert (got - w).norm() <= 6e-3 * w.norm()

    # prompts of differing lengths, in one padded call
    counts = [120, 1, 77]
    x = tokens(120)
    q = lf.cache_append(x[1], x[2], kc, vc, table, ints([0] * b, DEV), counts=ints(counts, DEV), Q=x[0],
                        phase=phase)
    O, _ = lf.paged_attention(q, kc, vc, table, ints(counts, DEV), q_lengths=ints(counts, DEV))
    for i in range(b):
        extend(i, x, slice(0, counts[i]))
        lengths[i] = counts[i]
        compare(O, i, slice(0, counts[i]), 0)
    for _ in range(3):  # tokens one by one
        x = tokens(1)
        q = lf.cache_append(x[1], x[2], kc, vc, table, ints(lengths, DEV), Q=x[0], phase=phase)
        lengths = [y + 1 for y in lengths]
        O, _ = lf.paged_attention(q, kc, vc, table, ints(lengths, DEV))
        for i in range(b):
            extend(i, x, slice(0, 1))
            compare(O, i, slice(0, 1), lengths[i] - 1)
    # a tree of drafted tokens, each at its depth behind the sequence
    n = 12
    up = random_tree(b, n, seed=5)
    depth = torch.zeros(b, n, dtype=torch.int32)
    for i in range(n):
        for s in range(b):
            depth[s, i] = 0 if up[s, i] < 0 else depth[s, up[s, i]] + 1
    x = tokens(n)
    q = lf.cache_append(x[1], x[2], kc, vc, table, ints(lengths, DEV), Q=x[0], phase=phase,
                        positions=(ints(lengths)[:, None] + depth).to(DEV))
    O, _ = lf.tree_attention(q, kc, vc, table, ints([y + n for y in lengths], DEV), lf.tree_mask(up.to(DEV)))
    paths = []
    for i in range(b):
        node = int(depth[i].argmax())  # the deepest branch is accepted
        path = []
        while node >= 0:
            path.insert(0, node)
            node = int(up[i, node])
        paths.append(path)
        extend(i, x, path)
        compare(O, i, path, lengths[i])
    m = max(len(p) for p in paths)
    lf.cache_keep(kc, vc, table, ints(lengths, DEV), ints([p + [0] * (m - len(p)) for p in paths], DEV),
                  counts=ints([len(p) for p in paths], DEV))
    lengths = [y + len(p) for y, p in zip(lengths, paths)]
    x = tokens(1)  # and on
    q = lf.cache_append(x[1], x[2], kc, vc, table, ints(lengths, DEV), Q=x[0], phase=phase)
    lengths = [y + 1 for y in lengths]
    O, _ = lf.paged_attention(q, kc, vc, table, ints(lengths, DEV))
    for i in range(b):
        extend(i, x, slice(0, 1))
        compare(O, i, slice(0, 1), lengths[i] - 1)
    status()
