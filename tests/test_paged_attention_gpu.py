"""GPU tests of the attention over pages against its fp64 oracle.  Every test runs with tables that
end with the sequences and with ones that reach far beyond: short tables' units of work stay whole,
others are cut anywhere and joined from their parts."""
import numpy as np
import pytest
import torch

import rank_linear_complexity_gb300.linformer as lf
from oracle import paged
from oracle.softmax_attention import host64
from tests.paged_cases import bits, cache, ints, random_tree

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF = torch.bfloat16
ROWS = 0  # of a table at least


@pytest.fixture(autouse=True, params=[0, 20000], ids=["short", "long"])
def table_rows(request):
    global ROWS
    ROWS = request.param
    yield
    ROWS = 0


def status():
    torch.cuda.synchronize()
    assert lf.linformer_debug_read_device_status() == 0


def error_code():
    torch.cuda.synchronize()
    return lf.linformer_debug_read_device_status()


def long_table(table, page):
    """The table with entries that name no page behind it."""
    more = max(0, ROWS // page - table.shape[1])
    return torch.nn.functional.pad(table, (0, more), value=-1).contiguous()


def check_attention(b=3, hq=4, hk=2, nq=1, d=64, page=16, k_lengths=(70, 1, 130), q_lengths=None,
                    causal=True, window=0, scale=None, layout="rows", tree=None, seed=0, gain=1.5,
                    width=None, clean=True):
    kc, vc, table = cache(b, hk, d, page, [max(0, x) for x in k_lengths], layout, "bf16", seed, device=DEV,
                          width=width, gain=gain)
    if width is None:
        table = long_table(table, page)
    g = torch.Generator(device=DEV).manual_seed(seed + 1)
    Q = (torch.randn(b, nq, hq, d, generator=g, device=DEV) * gain).to(BF).transpose(1, 2)
    if q_lengths is not None:
        for i, x in enumerate(q_lengths):
            Q[i, :, max(0, x):] = float("nan")
    kw = dict(q_lengths=None if q_lengths is None else ints(q_lengths, DEV), scale=scale)
    out = torch.full((b, hq, nq, d), 3.0, dtype=BF, device=DEV)
    lse = torch.full((b, hq, nq), 3.0, device=DEV)
    if tree is None:
        got = lf.paged_attention(Q, kc, vc, table, ints(k_lengths, DEV), causal=causal, window=window,
                                 out=out, lse=lse, **kw)
        want = paged.forward(Q, kc, vc, table.tolist(), k_lengths, q_lengths, causal, window, scale)
    else:
        got = lf.tree_attention(Q, kc, vc, table, ints(k_lengths, DEV),
                                torch.from_numpy(paged.words(tree)).to(DEV), out=out, lse=lse, **kw)
        want = paged.forward(Q, kc, vc, table.tolist(), k_lengths, q_lengths, scale=scale, tree=tree)
    if clean:
        status()
    assert got[0] is out and got[1] is lse
    O, l = host64(out), host64(lse)
    assert np.isfinite(O).all()
    assert (np.abs(O - want[0]) <= want[2]).all(), float((np.abs(O - want[0]) - want[2]).max())
    none = np.isneginf(want[1])
    assert np.array_equal(np.isneginf(l), none) and (O[none] == 0).all()
    assert (np.abs(l[~none] - want[1][~none]) <= want[3][~none]).all()
    # three independent roundings of rms 2^-8 / sqrt 3 (P, O, the reference's none) stay below 5e-3
    norm = np.linalg.norm(want[0])
    assert np.linalg.norm(O - want[0]) <= 5e-3 * norm
    return out, lse, (Q, kc, vc, table)


@pytest.mark.parametrize("layout", ["rows", "heads", "fused"])
@pytest.mark.parametrize("page", [8, 16, 32, 64, 128, 256])
def test_single_tokens(layout, page):
    check_attention(layout=layout, page=page)


@pytest.mark.parametrize("d", [8, 40, 64, 72, 80, 96, 120, 128])
def test_head_sizes(d):
    check_attention(d=d)
    check_attention(d=d, nq=70, k_lengths=(70, 200, 130))


@pytest.mark.parametrize("hq,hk", [(1, 1), (3, 3), (12, 12), (6, 2), (8, 1), (7, 1), (32, 8), (24, 3), (32, 1), (128, 1),
                                   (200, 1)])
@pytest.mark.parametrize("nq", [1, 5])
def test_heads(hq, hk, nq):
    check_attention(hq=hq, hk=hk, nq=nq, k_lengths=(70, 6, 140))


@pytest.mark.parametrize("k_lengths", [(1, 2, 3), (0, 0, 0), (127, 128, 129), (255, 256, 257), (0, 1000, 64),
                                       (5, -3, 2000), (4096, 100, 3333)])
@pytest.mark.parametrize("nq", [1, 3, 33])
def test_lengths(k_lengths, nq):
    """Sequences shorter than their new tokens among them: the first rows then see nothing."""
    check_attention(k_lengths=k_lengths, nq=nq)
    check_attention(k_lengths=k_lengths, nq=nq, causal=False, page=64, layout="heads")


def test_lengths_past_the_table_are_cut():
    check_attention(k_lengths=(64, 50, 64), width=4)
    kc, vc, table = cache(1, 2, 64, 16, [64], device=DEV)
    Q = torch.randn(1, 2, 1, 64, device=DEV).to(BF)
    got = [lf.paged_attention(Q, kc, vc, table, ints([x], DEV)) for x in (64, 65, 2 ** 31 - 1)]
    status()
    for x in got[1:]:
        assert torch.equal(bits(x[0]), bits(got[0][0])) and torch.equal(x[1], got[0][1])


@pytest.mark.parametrize("nq,q_lengths", [(1, (1, 0, 1)), (7, (7, 0, 3)), (40, (1, 40, -5)), (300, (300, 129, 0))])
def test_query_lengths(nq, q_lengths):
    for kw in (dict(), dict(causal=False), dict(window=11)):
        check_attention(nq=nq, q_lengths=q_lengths, k_lengths=(400, 130, 77), **kw)


@pytest.mark.parametrize("window", [1, 2, 16, 127, 128, 129, 1000])
@pytest.mark.parametrize("nq", [1, 9, 150])
def test_windows(window, nq):
    check_attention(nq=nq, window=window, k_lengths=(1111, 150, 333), page=32)


@pytest.mark.parametrize("nq", [16, 63, 64, 65, 127, 128, 129, 257, 600])
def test_chunks(nq):
    check_attention(nq=nq, k_lengths=(nq, nq + 1, 700), d=128, page=64)
    check_attention(nq=nq, k_lengths=(nq, nq + 77, 700), hq=8, hk=1)


@pytest.mark.parametrize("n", [1, 2, 25, 32, 64, 65, 100, 130])
@pytest.mark.parametrize("kw", [dict(), dict(hq=8, hk=1, d=128, page=64), dict(hq=3, hk=3, d=40, layout="fused")])
def test_trees(n, kw):
    tree = paged.ancestors(random_tree(3, n, seed=n).numpy())
    check_attention(nq=n, tree=tree, k_lengths=(n, n + 130, 600), **kw)
    check_attention(nq=n, tree=tree, k_lengths=(n, n + 130, 600), q_lengths=(n // 2, n, 0), **kw)


def test_any_mask_serves():
    """Masks that are no trees: random bits, none at all, every one, bits past the valid nodes; a
    tree longer than the rows of the cache."""
    r = np.random.default_rng(7)
    for n in (5, 70, 140):
        for m in (r.random((3, n, n)) < 0.3, np.zeros((3, n, n), bool), np.ones((3, n, n), bool)):
            check_attention(nq=n, tree=m, k_lengths=(n, 3 * n, n // 2))
            check_attention(nq=n, tree=m, k_lengths=(n, 3 * n, n // 2), q_lengths=(n, n - 2, 1), hq=8, hk=1)


def test_large_trees():
    n = 1024
    tree = paged.ancestors(random_tree(1, n, seed=1, deep=True).numpy())
    check_attention(b=1, nq=n, tree=tree, k_lengths=(n + 333,), page=128)


@pytest.mark.parametrize("scale", [0.01, 0.5, 3.0])
def test_scales(scale):
    check_attention(scale=scale, nq=4, k_lengths=(500, 90, 1300))
    check_attention(scale=scale, nq=200, k_lengths=(500, 200, 1300))


def test_growing_logits():
    """Maxima that rise from block to block, far past what an exponent holds unscaled."""
    for nq, hq in ((1, 4), (3, 16), (60, 8)):
        kc, vc, table = cache(1, 1, 64, 16, [1500], device=DEV, seed=4)
        table = long_table(table, 16)
        rise = torch.linspace(0.0, 60.0, 1500, device=DEV)
        k = kc.transpose(1, 2).clone()
        for j in range(1500):
            k[table[0, j // 16].long(), j % 16] *= rise[j] / 8
        kc = k.transpose(1, 2)
        Q = (torch.randn(1, hq, nq, 64, device=DEV, generator=torch.Generator(device=DEV).manual_seed(2)) * 2).to(BF)
        O, lse = lf.paged_attention(Q, kc, vc, table, ints([1500], DEV))
        status()
        want = paged.forward(Q, kc, vc, table.tolist(), (1500,), causal=True)
        assert (np.abs(host64(O) - want[0]) <= want[2]).all()
        assert (np.abs(host64(lse) - want[1]) <= want[3]).all()


@pytest.mark.parametrize("level", [-300.0, 0.0, 300.0])
def test_rows_whose_first_keys_come_late(level):
    """Blocks in which some rows of a tile see nothing, before blocks in which they do, at logits far
    from zero: windows that begin past a block's edge, trees whose nodes see no row before them."""
    for nq, hq, hk, lk, window in ((7, 4, 2, 400, 11), (60, 2, 2, 500, 20), (5, 8, 1, 1300, 9), (200, 4, 2, 900, 40)):
        kc, vc, table = cache(1, hk, 64, 16, [lk], device=DEV, seed=9)
        table = long_table(table, 16)
        kc[..., 0] = torch.where(kc[..., 0].isnan(), kc[..., 0], level / 4)
        Q = torch.randn(1, hq, nq, 64, device=DEV, generator=torch.Generator(device=DEV).manual_seed(2)).to(BF)
        Q[..., 0] = 32.0  # level logits on top of the others, scale 1 / 8
        O, lse = lf.paged_attention(Q, kc, vc, table, ints([lk], DEV), window=window)
        status()
        want = paged.forward(Q, kc, vc, table.tolist(), (lk,), causal=True, window=window)
        assert (np.abs(host64(O) - want[0]) <= want[2]).all() and (np.abs(host64(lse) - want[1]) <= want[3]).all()
        n = min(nq, 100)
        tree = paged.ancestors(random_tree(1, n, seed=3).numpy())
        Q = Q[:, :, :n].contiguous()
        for k in (n, n // 2):
            O, lse = lf.tree_attention(Q, kc, vc, table, ints([k], DEV), torch.from_numpy(paged.words(tree)).to(DEV))
            status()
            want = paged.forward(Q, kc, vc, table.tolist(), (k,), tree=tree)
            some = np.isfinite(want[1])
            assert np.array_equal(np.isneginf(host64(lse)), ~some)
            assert (np.abs(host64(O) - want[0]) <= want[2]).all() and (np.abs(host64(lse)[some] - want[1][some]) <= want[3][some]).all()


def test_many_sequences():
    r = np.random.default_rng(3)
    lengths = tuple(int(x) for x in r.integers(0, 300, 150))
    check_attention(b=150, k_lengths=lengths, hq=2, hk=1)
    check_attention(b=150, k_lengths=lengths, nq=3, hq=2, hk=2, page=8)


@pytest.mark.parametrize("kw", [dict(nq=1, hq=4, hk=4), dict(nq=1, hq=8, hk=4, d=128, layout="heads"),
                                dict(nq=12, hq=16, hk=4, d=40), dict(nq=40, hq=8, hk=4),
                                dict(nq=3, hq=4, hk=4, causal=False)])
def test_long_lists(kw):
    """Hundreds of blocks a CTA, units cut in the middle."""
    lengths = (40000, 1, 31234, 0, 36000, 29999, 33333, 35000, 38000, 12345)
    out = [check_attention(b=10, page=128, k_lengths=lengths, **kw) for _ in range(2)]
    assert torch.equal(bits(out[0][0]), bits(out[1][0])) and torch.equal(out[0][1], out[1][1])


def test_pages_that_are_not_there():
    """They count as rows of zeros, are recorded, and nothing outside the cache is read."""
    for nq, bad in ((1, 99), (1, -1), (40, 2 ** 31 - 1), (300, -7)):
        kc, vc, table = cache(2, 2, 64, 16, [400, 390], device=DEV, seed=6)
        table = long_table(table, 16)
        Q = torch.randn(2, 4, nq, 64, device=DEV, generator=torch.Generator(device=DEV).manual_seed(nq)).to(BF)
        table[1, 3] = bad
        O, lse = lf.paged_attention(Q, kc, vc, table, ints([400, 390], DEV))
        assert error_code() != 0
        want = paged.forward(Q, kc, vc, table.tolist(), (400, 390), causal=True)
        assert (np.abs(host64(O) - want[0]) <= want[2]).all()
        assert (np.abs(host64(lse) - want[1]) <= want[3]).all()


@pytest.mark.parametrize("nq", [1, 5, 70, 300])
@pytest.mark.parametrize("page", [8, 16, 64, 128])
@pytest.mark.parametrize("gone", [-1, 0, 10 ** 6])
def test_pages_before_the_window_may_be_gone(nq, page, gone):
    """Entries of pages that no query's window reaches are another sequence's by now, or nobody's."""
    for window, lengths in ((20, (1000, 333)), (129, (900, 1024)), (nq + 64, (1500, 700))):
        kc, vc, table = cache(2, 2, 64, page, lengths, device=DEV, seed=3)
        kc, vc = (torch.cat([x, torch.full_like(x[:1], float("nan"))]) for x in (kc, vc))
        for i, n in enumerate(lengths):
            first = max(0, n - nq + 1 - window)  # that the first query sees
            table[i, :first // page] = kc.shape[0] - 1 if gone == 0 else gone
        table = long_table(table, page)
        Q = torch.randn(2, 4, nq, 64, device=DEV, generator=torch.Generator(device=DEV).manual_seed(nq)).to(BF)
        O, lse = lf.paged_attention(Q, kc, vc, table, ints(list(lengths), DEV), window=window)
        status()
        # (hidden rows count as zeros in the oracle)
        clean = [torch.nan_to_num(x) for x in (kc, vc)]
        want = paged.forward(Q, *clean, table.tolist(), lengths, causal=True, window=window)
        assert (np.abs(host64(O) - want[0]) <= want[2]).all()
        assert (np.abs(host64(lse) - want[1]) <= want[3]).all()


def test_pages_shared_by_sequences():
    kc, vc, table = cache(1, 2, 64, 16, [200], device=DEV, seed=8)
    table = long_table(table, 16)
    Q = torch.randn(3, 4, 1, 64, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).to(BF)
    shared = table.expand(3, -1).contiguous()
    O, lse = lf.paged_attention(Q, kc, vc, shared, ints([200, 100, 17], DEV))
    status()
    want = paged.forward(Q, kc, vc, shared.tolist(), (200, 100, 17), causal=True)
    assert (np.abs(host64(O) - want[0]) <= want[2]).all()


def test_repeated_calls_agree():
    for nq in (1, 6, 64, 200):
        args = check_attention(nq=nq, hq=8, k_lengths=(3000, 700, 2050))[2]
        got = [lf.paged_attention(*args, ints((3000, 700, 2050), DEV)) for _ in range(3)]
        status()
        for x in got[1:]:
            assert torch.equal(bits(x[0]), bits(got[0][0])) and torch.equal(x[1], got[0][1])


def test_a_cache_past_32_bits():
    """Pages whose offsets pass 2^32 elements, and 2^31 rows."""
    pages, page, hk, d = 2 ** 17 + 8, 256, 1, 128  # 2^32 + elements, 8.6 GB each
    kc, vc = (torch.empty(pages, hk, page, d, dtype=BF, device=DEV) for _ in range(2))
    ids = [pages - 1, 5, pages - 3, 2 ** 17]
    g = torch.Generator(device=DEV).manual_seed(0)
    table = ints([ids], DEV)
    K, V = (torch.randn(1, hk, 1000, d, device=DEV, generator=g).to(BF) for _ in range(2))
    lf.cache_append(K, V, kc, vc, table, ints([0], DEV))
    for i, x in enumerate(ids):
        rows = min(page, 1000 - i * page)
        assert torch.equal(kc[x, 0, :rows], K[0, 0, i * page:i * page + rows])
        assert torch.equal(vc[x, 0, :rows], V[0, 0, i * page:i * page + rows])
    for nq in (1, 80):
        Q = torch.randn(1, 4, nq, d, device=DEV, generator=g).to(BF)
        O, lse = lf.paged_attention(Q, kc, vc, table, ints([1000], DEV))
        want, wl = lf.softmax_attention(Q, K, V, causal=True)
        status()
        # each side is within the rounding of P and of O of the same sums
        assert (O.float() - want.float()).norm() <= 6e-3 * want.float().norm()
        assert torch.allclose(lse, wl, atol=1e-4)
    lf.cache_keep(kc, vc, table, ints([0], DEV), ints([[900, 950, 999]], DEV))
    status()
    for i, j in enumerate((900, 950, 999)):
        assert torch.equal(kc[ids[0], 0, i], K[0, 0, j]) and torch.equal(vc[ids[0], 0, i], V[0, 0, j])


@pytest.mark.parametrize("nq", [1, 5, 70])
def test_nan_queries_and_keys(nq):
    """A row with NaN scores is NaN, whole or joined from parts; no other row is."""
    kw = dict(b=2, hq=4, hk=2, nq=nq, k_lengths=(3000, 900), d=64, page=64)
    _, _, (Q, kc, vc, table) = check_attention(**kw)
    want = paged.forward(Q, kc, vc, table.tolist(), (3000, 900), causal=True)
    bad = np.zeros((2, 4, nq), dtype=bool)

    def check():
        O, l = (host64(x) for x in lf.paged_attention(Q, kc, vc, table, ints((3000, 900), DEV)))
        assert np.array_equal(np.isnan(O), np.broadcast_to(bad[..., None], O.shape))
        assert np.array_equal(np.isnan(l), bad)
        assert (np.abs(O - want[0])[~bad] <= want[2][~bad]).all()
        assert (np.abs(l - want[1])[~bad] <= want[3][~bad]).all()
        status()

    Q = Q.clone()
    Q[0, 1, nq - 1, 3] = float("nan")
    bad[0, 1, nq - 1] = True
    check()
    # a key that the last query alone sees
    kc = kc.clone()
    kc[table[1, 899 // 64].long(), 1, 899 % 64, 5] = float("nan")
    bad[1, 2:, nq - 1] = True
    check()


@pytest.mark.parametrize("kw", [dict(nq=1, window=1500), dict(nq=9, window=2100), dict(nq=150, window=1300),
                                dict(nq=40, hq=8, window=1111, d=128)])
def test_wide_windows(kw):
    """Windows of more blocks than a unit keeps whole."""
    check_attention(k_lengths=(4000, 900, 2222), page=32, **kw)
    check_attention(k_lengths=(4000, 0, 2222), q_lengths=(kw["nq"], 1, max(1, kw["nq"] // 2)), page=64, layout="heads", **kw)


@pytest.mark.parametrize("kw", [dict(), dict(window=700), dict(causal=False)])
def test_whole_units_of_many_blocks(kw):
    """As many units as CTAs, so that each stays whole over more blocks than it otherwise would."""
    check_attention(b=1, hq=32, hk=8, d=40, nq=1100, k_lengths=(1777,), page=64, **kw)


def test_whole_trees_of_many_blocks():
    tree = paged.ancestors(random_tree(15, 64, seed=2).numpy())
    lengths = [64 + 130 * i for i in range(15)]
    check_attention(b=15, hq=32, hk=8, nq=64, tree=tree, k_lengths=lengths, d=40, page=32)
    check_attention(b=15, hq=32, hk=8, nq=64, tree=tree, k_lengths=lengths, q_lengths=[64, 0, 3] * 5, d=40, page=32)
