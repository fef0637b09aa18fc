"""GPU tests of appends large enough for a thread to go through several heads: from the queries into the
keys and the values, a last thread with fewer heads, in place and not.  A row's result does not depend on how
many heads a thread takes, so the same rows appended a few at a time (one head a thread) have to give the
same bits; sampled rows are checked against the fp64 oracle (pairs, with A the sum of a pair's absolute
elements: 2^-21 A, and 2^-8 or 2^-24 of the result for its rounding)."""
import numpy as np
import pytest
import torch

import rank_linear_complexity_gb300.linformer as lf
from oracle import rotary
from oracle.softmax_attention import host64
from tests.paged_cases import bits, ints

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF = torch.bfloat16
PAGE = 16


def heads_a_thread(b, n, d, rot, heads, dtype, pieces=True):
    """The library's rule: as many heads as leave two full waves of threads, at most 16."""
    v = 4 if dtype == torch.float32 else 8
    if not pieces or rot % (2 * v) or d % v:
        v = 1
    sms = torch.cuda.get_device_properties(DEV).multi_processor_count
    return max(1, min(heads, 16, b * n * (rot // 2 // v + (d - rot) // v) * heads // (2 * sms * 2048)))


def check(hq, hk, b, n, d, rot, dtype, per, inter=False, ragged=False, in_place=False, placed=False, odd=False,
          step=1300):
    heads = hq + 2 * hk
    assert heads_a_thread(b, n, d, rot, heads, dtype, not odd) == per
    assert heads_a_thread(b, step, d, rot, heads, dtype, not odd) == 1
    g = torch.Generator(device=DEV).manual_seed(n)
    starts = [13 * i for i in range(b)]
    counts = [n - (n // 3) * i for i in range(b)] if ragged else [n] * b
    width = -(-(starts[-1] + n) // PAGE)
    table = torch.randperm(b * width, generator=g, device=DEV).to(torch.int32).view(b, width)
    room = d + 1 if odd else d  # (strides that are no multiples of 16 bytes: element by element)
    first = [torch.randn(b * width, PAGE, hk, room, generator=g, device=DEV).to(dtype) for _ in range(2)]
    K, V, Q = (torch.randn(b, n, h, d, generator=g, device=DEV).to(dtype).transpose(1, 2) for h in (hk, hk, hq))
    pos = torch.randint(0, 1 << 20, (b, n), generator=g, device=DEV, dtype=torch.int32) if placed else None
    f = rotary.frequencies(rot) if rot else None
    kw = dict(phase=torch.from_numpy(rotary.phase_words(f)).to(DEV), rot=rot, amplitude=1.25,
              layout=lf.ROTARY_INTERLEAVED if inter else lf.ROTARY_HALVES) if rot else {}

    def caches():
        both = [x.clone() for x in first]
        return both, [x[..., :d].transpose(1, 2) for x in both]
    whole, (kc, vc) = caches()
    asked = Q.clone() if hq else None
    got = lf.cache_append(K, V, kc, vc, table, ints(starts, DEV), counts=ints(counts, DEV) if ragged else None,
                          positions=pos, Q=asked, out=asked if in_place else None, **kw)
    parts, (kp, vp) = caches()
    turned = torch.empty_like(Q)
    for a in range(0, n, step):
        at = slice(a, min(a + step, n))
        at_pos = None if pos is None else pos[:, at].contiguous()
        x = Q[:, :, at].clone() if hq else None
        x = lf.cache_append(K[:, :, at], V[:, :, at], kp, vp, table, ints([s + a for s in starts], DEV),
                            counts=ints([c - a for c in counts], DEV) if ragged else None, positions=at_pos, Q=x, **kw)
        if hq:
            turned[:, :, at] = x
    torch.cuda.synchronize()
    assert lf.linformer_debug_read_device_status() == 0
    for x, y in zip(whole, parts):
        assert torch.equal(bits(x), bits(y))
    if hq:
        assert torch.equal(bits(got), bits(turned))
        if in_place:
            assert got is asked
        else:  # a tensor of its own, and the queries as they were
            assert got.untyped_storage().data_ptr() != asked.untyped_storage().data_ptr()
            assert torch.equal(bits(asked), bits(Q))
    half = 2.0 ** -8 if dtype == BF else 2.0 ** -24
    rng = np.random.default_rng(n)
    for i in range(b):
        # sampled rows, the last and those on either side of the count among them
        some = sorted({0, n - 1, counts[i] - 1, min(counts[i], n - 1), *rng.integers(0, n, 40).tolist()})
        at = torch.tensor(some, device=DEV)
        place = starts[i] + at
        pages, rows = table[i][place // PAGE].long(), place % PAGE
        held = [x[pages, :, rows].transpose(0, 1) for x in (kc, vc)]  # [hk][rows][d]
        before = [x[pages, rows, :, :d].transpose(0, 1) for x in first]
        k, v = K[i][:, at], V[i][:, at]
        here = (place if pos is None else pos[i][at]).cpu().numpy()[None]
        new = np.array(some) < counts[i]
        assert torch.equal(bits(held[1][:, new]), bits(v[:, new]))
        for x, y in zip(held, before):
            assert torch.equal(bits(x[:, ~new]), bits(y[:, ~new]))
        if not rot:
            assert torch.equal(bits(held[0][:, new]), bits(k[:, new]))
            continue
        for x, y, rows_of in ((held[0], k, new), (got[i][:, at] if hq else None, Q[i][:, at], slice(None))):
            if x is None:
                continue
            want = rotary.rotate(host64(y)[None], f, here, rot, inter, 1.25)[0][:, rows_of]
            # (the sum of all elements' pairs at most: the largest pair)
            bound = half * np.abs(want) + 2.0 ** -21 * 1.25 * 2 * np.abs(host64(y)).max()
            assert (np.abs(host64(x)[:, rows_of] - want) <= bound).all()


@pytest.mark.parametrize("inter", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("kw", [
    dict(hq=7, hk=3, b=1, n=26011, d=64, rot=64, dtype=BF, per=2),         # 13 heads in twos, one over
    dict(hq=7, hk=3, b=2, n=13003, d=64, rot=64, dtype=BF, per=2, ragged=True, in_place=True),
    dict(hq=7, hk=3, b=2, n=8209, d=128, rot=64, dtype=BF, per=4, ragged=True, placed=True),  # copied rests
    dict(hq=4, hk=5, b=1, n=9503, d=80, rot=40, dtype=torch.float32, per=3, in_place=True),    # 14 in threes
    dict(hq=1, hk=2, b=1, n=23003, d=64, rot=32, dtype=torch.float32, per=2, step=4000),         # 5 in twos
    dict(hq=2, hk=1, b=3, n=30011, d=128, rot=128, dtype=BF, per=4, ragged=True),              # one thread a row
    dict(hq=7, hk=3, b=1, n=6007, d=40, rot=40, dtype=BF, per=2, step=700, in_place=True),     # element by element
    dict(hq=7, hk=3, b=2, n=9001, d=64, rot=32, dtype=BF, per=13, step=300, odd=True, ragged=True),
    dict(hq=0, hk=7, b=1, n=26011, d=64, rot=64, dtype=BF, per=2),                             # keys alone
    dict(hq=13, hk=9, b=1, n=11003, d=96, rot=96, dtype=torch.float32, per=6, step=500, in_place=True),
])
def test_several_heads_a_thread(kw, inter):
    check(inter=inter, **kw)


def test_several_heads_a_thread_without_a_turn():
    check(hq=0, hk=7, b=2, n=28513, d=64, rot=0, dtype=BF, per=10, ragged=True, step=1000)
