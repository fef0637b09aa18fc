"""GPU tests that the attention over pages gives the same bits whatever stands where no query does: in
the padding behind a sequence's queries, and in the shared memory that an earlier call left."""
import pytest
import torch

import rank_linear_complexity_gb300.linformer as lf
from tests.paged_cases import bits, cache, ints

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF = torch.bfloat16
LENGTHS = (9000, 5100, 2700)  # several blocks a CTA with eight key/value heads


def queries(hq, nq, d, seed, gain=1.5):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(len(LENGTHS), hq, nq, d, generator=g, device=DEV) * gain).to(BF)


def same(x, y):
    return torch.equal(bits(x[0]), bits(y[0])) and torch.equal(bits(x[1]), bits(y[1]))


# query heads on one key/value head and new tokens: 16, 32 and 64 columns, tiles of 128 rows
SHAPES = [(1, 9), (4, 7), (2, 30), (8, 12), (1, 200)]


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group,nq", SHAPES)
@pytest.mark.parametrize("tree", [False, True])
def test_padded_queries_change_no_bit(group, nq, d, tree):
    hk = 8
    kc, vc, table = cache(len(LENGTHS), hk, d, 16, LENGTHS, device=DEV, seed=nq)
    Q = queries(group * hk, nq, d, 1)
    valid = (nq // 2, 1, nq - 1)
    mask = torch.randint(-2 ** 62, 2 ** 62, (len(LENGTHS), nq, (nq + 63) // 64), device=DEV,
                         generator=torch.Generator(device=DEV).manual_seed(4))
    got = []
    for padding in (0.0, 1.0, 20.0, float("inf"), float("nan")):
        x = Q.clone()
        for i, n in enumerate(valid):
            x[i, :, n:] = queries(group * hk, nq, d, 2)[i, :, n:] * padding
        args = x, kc, vc, table, ints(LENGTHS, DEV)
        got.append(lf.tree_attention(*args, mask, q_lengths=ints(valid, DEV)) if tree
                   else lf.paged_attention(*args, q_lengths=ints(valid, DEV)))
    torch.cuda.synchronize()
    assert lf.linformer_debug_read_device_status() == 0
    for x in got[1:]:
        assert same(x, got[0])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group,nq", [(7, 12), (3, 32), (5, 30), (6, 16)])
def test_what_an_earlier_call_left_changes_no_bit(group, nq, d):
    """Tiles of 128 rows that heads and tokens do not fill, after calls that filled all of theirs."""
    hk = 8
    kc, vc, table = cache(len(LENGTHS), hk, d, 16, LENGTHS, device=DEV, seed=nq)
    Q = queries(group * hk, nq, d, 1)
    got = []
    for gain in (0.0, 2.0, 20.0, float("inf")):
        lf.paged_attention(queries(8 * hk, 64, d, 3, gain), kc, vc, table, ints(LENGTHS, DEV))
        got.append(lf.paged_attention(Q, kc, vc, table, ints(LENGTHS, DEV)))
    torch.cuda.synchronize()
    assert lf.linformer_debug_read_device_status() == 0
    for x in got[1:]:
        assert same(x, got[0])


@pytest.mark.parametrize("window", [0, 700])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group,nq", SHAPES)
def test_rows_past_the_lengths_change_no_bit(group, nq, d, window):
    hk = 8
    lengths = tuple(x - 37 for x in LENGTHS)  # that end inside a page and a block
    kc, vc, table = cache(len(LENGTHS), hk, d, 16, lengths, device=DEV, seed=nq)
    Q = queries(group * hk, nq, d, 1)
    got = []
    for x in (0.0, -30.0, 1e30, float("inf"), float("nan")):
        k, v = (torch.where(c.isnan(), torch.full_like(c, x), c) for c in (kc, vc))
        got.append(lf.paged_attention(Q, k, v, table, ints(lengths, DEV), window=window))
    torch.cuda.synchronize()
    assert lf.linformer_debug_read_device_status() == 0
    for x in got[1:]:
        assert same(x, got[0])
