"""CPU checks of the paged key/value cache: pins of its oracle, and every refusal of the library and
the binding, none of which touches a device."""
import math

import numpy as np
import pytest
import torch

import rank_linear_complexity_gb300.linformer as lf
from oracle import paged, rotary
from oracle import softmax_attention as att
from rank_linear_complexity_gb300 import build as libbuild
from tests.paged_cases import cache, ints, random_tree


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return lf.lib()


# --- refusals of the library (fake addresses: every call fails before anything is launched) ---

A = 1 << 20
NULL, SIZE, UNSUPPORTED, ENUM, ALIGN, VALUE = -1, -2, -3, -4, -5, -10


def strides(*x):
    import ctypes
    return (ctypes.c_int64 * 3)(*x)


def append(L, **kw):
    a = dict(K=A, sK=None, V=2 * A, sV=None, kc=3 * A, skc=None, vc=4 * A, svc=None, Q=5 * A, sQ=None,
             Y=6 * A, sY=None, table=A, starts=A, counts=None, phase=A, positions=None, b=2, hq=4, hk=2,
             n=3, d=64, pages=9, page=16, width=4, rot=64, layout=0, amplitude=1.0, dtype=1)
    assert set(kw) <= set(a)
    a.update(kw)
    return L.linformer_cache_append(*a.values(), 0)


@pytest.mark.parametrize("kw,want", [
    *[(dict([(x, None)]), NULL) for x in ("K", "V", "kc", "vc", "Q", "Y", "table", "starts", "phase")],
    (dict(b=0), SIZE), (dict(hq=-1), SIZE), (dict(hk=0), SIZE), (dict(n=0), SIZE), (dict(d=0), SIZE),
    (dict(pages=0), SIZE), (dict(width=0), SIZE), (dict(page=4), SIZE), (dict(page=24), SIZE),
    (dict(page=1 << 17), SIZE), (dict(page=0), SIZE), (dict(page=-16), SIZE), (dict(width=1 << 26), SIZE),
    (dict(b=1 << 29), SIZE), (dict(d=(1 << 20) + 2), SIZE),
    (dict(layout=2), ENUM), (dict(dtype=3), ENUM), (dict(dtype=2), UNSUPPORTED),
    (dict(rot=0), VALUE), (dict(rot=63), VALUE), (dict(rot=66), VALUE), (dict(amplitude=math.inf), VALUE),
    (dict(amplitude=math.nan), VALUE),
    (dict(phase=A + 4), ALIGN), (dict(positions=A + 2), ALIGN), (dict(starts=A + 1), ALIGN), (dict(counts=A + 2), ALIGN),
    (dict(table=A + 2), ALIGN), (dict(K=A + 8), ALIGN), (dict(V=A + 8), ALIGN), (dict(Q=A + 8), ALIGN), (dict(Y=A + 8), ALIGN),
    (dict(kc=A + 8), ALIGN), (dict(vc=A + 8), ALIGN),
    (dict(vc=3 * A), VALUE), (dict(K=3 * A), VALUE), (dict(V=3 * A), VALUE), (dict(Q=4 * A), VALUE), (dict(Y=A), VALUE),
    (dict(Y=2 * A), VALUE), (dict(Y=3 * A), VALUE), (dict(Y=4 * A), VALUE),
    (dict(Y=5 * A, sY=strides(768, 64, 256)), VALUE),  # in place, elsewhere
    (dict(sK=strides(0, 64, 64)), VALUE), (dict(sK=strides(-1, 64, 64)), VALUE), (dict(sV=strides(1 << 39, 64, 64)), VALUE),
    (dict(skc=strides(2048, 32, 64)), VALUE), (dict(svc=strides(2048, 1024, 0)), VALUE), (dict(sY=strides(768, 32, 64)), VALUE),
])
def test_append_refusals(L, kw, want):
    assert append(L, **kw) == want


def keep(L, **kw):
    a = dict(kc=A, skc=None, vc=2 * A, svc=None, table=A, starts=A, path=A, counts=None, b=2, hk=2, m=3, d=64,
             pages=9, page=16, width=4, dtype=1)
    a.update(kw)
    return L.linformer_cache_keep(*a.values(), 0)


@pytest.mark.parametrize("kw,want", [
    *[(dict([(x, None)]), NULL) for x in ("kc", "vc", "table", "starts", "path")],
    (dict(b=0), SIZE), (dict(hk=0), SIZE), (dict(m=0), SIZE), (dict(d=0), SIZE), (dict(pages=0), SIZE), (dict(page=12), SIZE),
    (dict(width=0), SIZE), (dict(b=1 << 28), SIZE), (dict(dtype=-1), ENUM), (dict(dtype=2), UNSUPPORTED),
    (dict(path=A + 2), ALIGN), (dict(starts=A + 2), ALIGN), (dict(counts=A + 3), ALIGN), (dict(kc=A + 4), ALIGN),
    (dict(vc=A), VALUE), (dict(skc=strides(64, 32, 64)), VALUE),
])
def test_keep_refusals(L, kw, want):
    assert keep(L, **kw) == want


def attend(L, tree, **kw):
    a = dict(Q=A, sQ=None, kc=2 * A, skc=None, vc=3 * A, svc=None, O=4 * A, sO=None, lse=A, table=A, k_lengths=A,
             q_lengths=None, mask=A, b=2, hq=4, hk=2, nq=3, d=64, pages=9, page=16, width=4, scale=0.1, causal=1,
             window=0, dtype=1)
    a.update(kw)
    if tree:
        del a["causal"], a["window"]
        return L.linformer_tree_attn_fwd(*a.values(), 0)
    del a["mask"]
    return L.linformer_paged_attn_fwd(*a.values(), 0)


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("kw,want", [
    *[(dict([(x, None)]), NULL) for x in ("Q", "kc", "vc", "O", "lse", "table", "k_lengths")],
    (dict(b=0), SIZE), (dict(hq=0), SIZE), (dict(hq=3), SIZE), (dict(hk=0), SIZE), (dict(nq=0), SIZE), (dict(d=0), SIZE),
    (dict(pages=0), SIZE), (dict(page=20), SIZE), (dict(page=1), SIZE), (dict(width=1 << 26), SIZE), (dict(b=1 << 28), SIZE),
    (dict(dtype=0), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(dtype=7), ENUM), (dict(d=136), UNSUPPORTED),
    (dict(d=60), UNSUPPORTED), (dict(scale=0.0), VALUE), (dict(scale=-1.0), VALUE), (dict(scale=math.inf), VALUE),
    (dict(scale=3e38), VALUE), (dict(scale=math.nan), VALUE),
    (dict(lse=A + 2), ALIGN), (dict(k_lengths=A + 1), ALIGN), (dict(q_lengths=A + 1), ALIGN), (dict(table=A + 1), ALIGN),
    (dict(Q=A + 8), ALIGN), (dict(O=A + 8), ALIGN), (dict(kc=A + 8), ALIGN), (dict(skc=strides(2052, 1024, 64)), ALIGN),
    (dict(sQ=strides(768, 196, 64)), ALIGN), (dict(O=A), VALUE), (dict(O=2 * A), VALUE), (dict(O=3 * A), VALUE),
    (dict(vc=2 * A), VALUE), (dict(sO=strides(768, 192, 32)), VALUE), (dict(sQ=strides(768, 0, 64)), VALUE),
])
def test_attention_refusals(L, tree, kw, want):
    assert attend(L, tree, **kw) == want


def test_refusals_of_one_of_the_two(L):
    for kw in (dict(window=-1), dict(window=4, causal=0), dict(causal=2), dict(causal=-1)):
        assert attend(L, False, **kw) == VALUE
    assert attend(L, True, mask=None) == NULL
    assert attend(L, True, mask=A + 4) == ALIGN
    assert attend(L, True, nq=1025) == SIZE
    for args, want in (((None, A, 1, 4), NULL), ((A, None, 1, 4), NULL), ((A, A, 0, 4), SIZE), ((A, A, 1, 0), SIZE),
                       ((A, A, 1, 1025), SIZE), ((A + 2, A, 1, 4), ALIGN), ((A, A + 4, 1, 4), ALIGN)):
        assert L.linformer_tree_mask(*args, 0) == want


def packed(L, call, words, count=None):
    import struct
    block = b"".join(struct.pack("=d" if isinstance(x, float) else "=q", x) for x in words)
    return L.linformer_cache_packed(call, block, len(words) if count is None else count)


def rows(address, *s):
    return [address, *(s or (6144, 1024, 64))]


PACKED = {
    "append": (0, rows(A) + rows(2 * A) + rows(3 * A) + rows(4 * A) + rows(5 * A) + rows(6 * A) + [A, A, 0, A, 0]
               + [2, 4, 2, 3, 64, 9, 16, 4, 64, 0, 1.0, 1, 0]),
    "keep": (1, rows(A) + rows(2 * A) + [A, A, A, 0] + [2, 2, 3, 64, 9, 16, 4, 1, 0]),
    "attend": (2, rows(A) + rows(2 * A) + rows(3 * A) + rows(4 * A) + [A, A, A, 0]
               + [2, 4, 2, 3, 64, 9, 16, 4, 0.1, 1, 0, 1, 0]),
    "tree": (3, rows(A) + rows(2 * A) + rows(3 * A) + rows(4 * A) + [A, A, A, 0, A]
             + [2, 4, 2, 3, 64, 9, 16, 4, 0.1, 1, 0]),
}


@pytest.mark.parametrize("name", PACKED)
def test_packed_refusals(L, name):
    """Every word is where the call's own argument is: a wrong value there gives that call's status."""
    call, words = PACKED[name]
    n = len(words)

    def wrong(at, value):
        return packed(L, call, [value if i == at else x for i, x in enumerate(words)])
    tensors = {"append": 6, "keep": 2}.get(name, 4)
    ints_from = next(i for i, x in enumerate(words) if i >= 4 * tensors and 0 < x < A)
    real = {"append": n - 3, "attend": n - 5, "tree": n - 3}.get(name)
    dtype = n - 2
    for t in range(tensors):
        assert wrong(4 * t, 0) == NULL and wrong(4 * t, words[4 * t] + 8) == ALIGN
        for k in range(3):
            assert wrong(4 * t + 1 + k, -64) == VALUE, (t, k)
    for at in range(4 * tensors, ints_from):
        assert wrong(at, A + 1) == ALIGN
        if words[at]:
            assert wrong(at, 0) == NULL
    for at in range(ints_from, n - 1):
        if at != real:
            for x in (1 << 31, -(1 << 31) - 1, 1 << 32, (1 << 32) + words[at]):
                assert wrong(at, x) == SIZE, at
    sizes = 8 if name != "keep" else 7
    for at in range(ints_from, ints_from + sizes):
        assert wrong(at, -1) == SIZE
    if real:
        assert wrong(real, math.nan) == VALUE
    assert wrong(dtype, 9) == ENUM
    for at, x in {"append": ((n - 5, 65), (n - 4, 2)), "attend": ((n - 4, 2), (n - 3, -1)), "tree": ((ints_from + 3, 1025),),
                  "keep": ()}[name]:
        assert wrong(at, x) in (VALUE, ENUM, SIZE)
    assert packed(L, call, words, n - 1) == VALUE and packed(L, call, words + [0]) == VALUE
    assert packed(L, 4, words) == ENUM and packed(L, -1, words) == ENUM
    assert L.linformer_cache_packed(call, None, n) == NULL


# --- refusals of the binding -----------------------------------------------------------------

def test_binding_refuses_host_tensors():
    kc, vc, table = cache(2, 2, 64, 16, [20, 30])
    x = torch.zeros(2, 2, 3, 64, dtype=torch.bfloat16)
    one = ints([1, 1])
    for call in (lambda: lf.cache_append(x, x, kc, vc, table, one), lambda: lf.cache_keep(kc, vc, table, one, ints([[0], [0]])),
                 lambda: lf.paged_attention(x, kc, vc, table, one), lambda: lf.tree_mask(ints([[-1, 0]])),
                 lambda: lf.tree_attention(x, kc, vc, table, one, torch.zeros(2, 3, 1, dtype=torch.int64)),
                 lambda: lf.tree_attention(x, kc, vc, table, one, None)):
        with pytest.raises(ValueError):
            call()


def on_a_device(monkeypatch):
    """Host tensors pass for a device's; a call that gets as far as the library fails the test."""
    monkeypatch.setattr(lf, "_stream_of", lambda device, *tensors: 0)

    def stop(*_):
        raise AssertionError("reached the library")
    monkeypatch.setattr(lf, "_call", stop)


@pytest.mark.parametrize("wrong", [
    dict(V="short"), dict(vc="f32"), dict(kc="heads"), dict(table="int64"), dict(table="rows"), dict(table="strided"),
    dict(starts="int64"), dict(counts="short"), dict(phase="short"), dict(positions="short"), dict(Q="short"),
    dict(out="short"), dict(out="alone"), dict(Q="unturned"), dict(rot="unturned"),
])
def test_append_binding(monkeypatch, wrong):
    on_a_device(monkeypatch)
    kc, vc, table = cache(2, 2, 64, 16, [20, 30])
    x, q = torch.zeros(2, 2, 3, 64, dtype=torch.bfloat16), torch.zeros(2, 4, 3, 64, dtype=torch.bfloat16)
    a = dict(K=x, V=x.clone(), k_cache=kc, v_cache=vc, table=table, starts=ints([1, 1]), counts=ints([1, 1]), Q=q,
             phase=torch.zeros(32, dtype=torch.int64), positions=ints([[0] * 3] * 2), out=q.clone())
    with pytest.raises(AssertionError, match="reached"):
        lf.cache_append(**a)
    (key, how), = wrong.items()
    key = {"kc": "k_cache", "vc": "v_cache"}.get(key, key)
    if how == "short":
        a[key] = a[key][:1] if a[key].dim() > 1 or key == "counts" else a[key][:-1]
    elif how == "f32":
        a[key] = a[key].float()
    elif how == "heads":
        a[key] = a[key][:, :1]
    elif how == "int64":
        a[key] = a[key].long()
    elif how == "rows":
        a[key] = a[key][:1]
    elif how == "strided":
        a[key] = a[key].repeat(1, 2)[:, ::2]
    elif how == "alone":
        a.update(Q=None)
    else:
        a.update(phase=None, positions=None, out=None)
        if key == "rot":
            a.update(Q=None, rot=64)
    with pytest.raises(ValueError):
        lf.cache_append(**a)


def test_other_bindings(monkeypatch):
    on_a_device(monkeypatch)
    kc, vc, table = cache(2, 2, 64, 16, [20, 30])
    q, one = torch.zeros(2, 4, 3, 64, dtype=torch.bfloat16), ints([1, 1])
    words = torch.zeros(2, 3, 1, dtype=torch.int64)
    good = [lambda **kw: lf.paged_attention(**{**dict(Q=q, k_cache=kc, v_cache=vc, table=table, k_lengths=one), **kw}),
            lambda **kw: lf.tree_attention(**{**dict(Q=q, k_cache=kc, v_cache=vc, table=table, k_lengths=one, mask=words), **kw})]
    for call in good:
        with pytest.raises(AssertionError, match="reached"):
            call()
        for kw in (dict(Q=q[:1]), dict(Q=q[..., :32]), dict(Q=q.float()), dict(k_lengths=one.long()), dict(k_lengths=one[:1]),
                   dict(q_lengths=one[:1]), dict(out=q[:, :2]), dict(lse=torch.zeros(2, 4, 2)), dict(v_cache=vc[:, :1]),
                   dict(table=table[:1]), dict(table=table.float())):
            with pytest.raises(ValueError):
                call(**kw)
    with pytest.raises(ValueError):
        good[0](window=2 ** 31)
    with pytest.raises(ValueError):
        good[1](mask=words[:, :2])
    for kw in (dict(path=ints([0])), dict(path=ints([[0]])), dict(starts=one.long()), dict(counts=one[:1])):
        with pytest.raises(ValueError):
            lf.cache_keep(**{**dict(k_cache=kc, v_cache=vc, table=table, starts=one, path=ints([[0], [0]])), **kw})
    for kw in (dict(parents=torch.zeros(2, 3)), dict(parents=ints([[0, 0]] * 2)[:, ::2]), dict(out=words[:1])):
        with pytest.raises(ValueError):
            lf.tree_mask(**{**dict(parents=ints([[-1] * 3] * 2)), **kw})


def test_sizes_past_32_bits():
    wide = torch.zeros(1, dtype=torch.bfloat16).expand(1, 2, 2 ** 32 + 3, 64)
    kc, vc, table = cache(1, 2, 64, 16, [20])
    with pytest.raises(ValueError, match="32-bit"):
        lf.cache_append(wide, wide, kc, vc, table, ints([0]))
    with pytest.raises(ValueError, match="32-bit"):
        lf.paged_attention(wide, kc, vc, table, ints([0]))
    with pytest.raises(ValueError, match="32-bit"):
        lf.tree_mask(ints([0]).expand(2 ** 32 + 1, 1))
    with pytest.raises(ValueError, match="32-bit"):
        lf.cache_keep(kc, vc, table, ints([0]), ints([0]).expand(1, 2 ** 32 + 1))


# --- pins of the oracle ----------------------------------------------------------------------

@pytest.mark.parametrize("layout", ["rows", "heads", "fused"])
def test_oracle_attention_is_the_dense_one(layout):
    lengths = [20, 0, 9]
    kc, vc, table = cache(3, 2, 8, 8, lengths, layout, "f32", 1)
    r = np.random.default_rng(0)
    Q = r.standard_normal((3, 4, 5, 8))
    dense = [np.zeros((3, 2, 20, 8)) for _ in range(2)]
    for i, n in enumerate(lengths):
        for j in range(n):
            for x, y in zip(dense, (kc, vc)):
                x[i, :, j] = y[table[i, j // 8].item(), :, j % 8].double().numpy()
    for kw in (dict(), dict(causal=True), dict(causal=True, window=3), dict(causal=True, q_lengths=[5, 2, 0])):
        got = paged.forward(Q, kc, vc, table.tolist(), lengths, scale=0.3, **kw)
        want = att.forward(Q, *dense, k_lengths=lengths, scale=0.3, **kw)
        assert np.allclose(got[0], want[0], atol=1e-13) and np.array_equal(np.isneginf(got[1]), np.isneginf(want[1]))
        assert np.allclose(got[1], want[1], atol=1e-12)


def test_oracle_trees():
    # a chain's tree is the causal mask
    kc, vc, table = cache(2, 2, 8, 8, [20, 9], "rows", "f32", 2)
    Q = np.random.default_rng(1).standard_normal((2, 4, 5, 8))
    chain = paged.ancestors(np.arange(-1, 4)[None].repeat(2, 0))
    assert np.array_equal(chain[0], np.tril(np.ones((5, 5), bool)))
    got = paged.forward(Q, kc, vc, table.tolist(), [20, 9], tree=chain)
    want = paged.forward(Q, kc, vc, table.tolist(), [20, 9], causal=True)
    assert np.allclose(got[0], want[0], atol=1e-13)
    # a node sees its path, one by one
    up = random_tree(2, 40, seed=3).numpy()
    see = paged.ancestors(up)
    for i in range(40):
        want = {i} | ({j for j in range(40) if see[0, up[0, i], j]} if up[0, i] >= 0 else set())
        assert set(np.flatnonzero(see[0, i])) == want
    w = paged.words(paged.ancestors(random_tree(1, 130, seed=4).numpy()))
    assert w.shape == (1, 130, 3) and w[0, 64, 1] & 1 == 1 and w[0, 63, 0] < 0 and w[0, 129, 2] & 2


def test_oracle_rows_appended_and_kept():
    kc, vc, table = cache(2, 2, 8, 8, [20, 9], "heads", "f32", 2)
    r = np.random.default_rng(2)
    K, V, Q = (r.standard_normal((2, h, 3, 8)) for h in (2, 2, 4))
    f = rotary.frequencies(8)
    k2, v2, q2 = paged.append(K, V, kc, vc, table.tolist(), [7, 4], [3, 1], f, rot=8, Q=Q)
    turned = rotary.rotate(K, f, np.array([[7, 8, 9], [4, 5, 6]]), 8)
    for bi, n in ((0, 3), (1, 1)):
        got = paged.rows(k2, table[bi].tolist(), 10 if bi == 0 else 5)
        assert np.array_equal(got[:, (7, 4)[bi]:], turned[bi, :, :n])
        assert np.array_equal(paged.rows(v2, table[bi].tolist(), 9)[:, (7, 4)[bi]:][:, :n], V[bi, :, :n][:, :2 if bi == 0 else 1])
    assert np.array_equal(q2, rotary.rotate(Q, f, np.array([[7, 8, 9], [4, 5, 6]]), 8))
    a, _ = paged.keep(kc, vc, table.tolist(), [2, 0], np.array([[0, 3, 7], [5, 8, 1]]), [3, 2])
    before, after = (paged.rows(x.astype(float) if isinstance(x, np.ndarray) else x.double().numpy(), table[0].tolist(), 20)
                     for x in (kc, a))
    assert np.array_equal(after[:, 2:5], before[:, [2, 5, 9]]) and np.array_equal(after[:, 5:], before[:, 5:])
    # a page that is not there, a row behind the table, a node below its place: left out
    assert paged.place(np.zeros((3, 1, 8, 1)), [0, 3, -1], 8) is None and paged.place(np.zeros((3, 1, 8, 1)), [0], 8) is None
    assert paged.place(np.zeros((3, 1, 8, 1)), [0], -1) is None and paged.place(np.zeros((3, 1, 8, 1)), [1], 7) == (1, 7)
    same, _ = paged.keep(kc, vc, table.tolist(), [2, 0], np.array([[0, 0, 1], [0, 0, 1]]))
    assert np.array_equal(same, kc.double().numpy(), equal_nan=True)


def test_every_wait_of_the_kernels_over_pages_has_a_code_of_its_own():
    """The code in the device status word names one place in the sources."""
    import os
    import re
    codes = []
    for name in ("paged_attn.cu", "paged_attn_wide.cu"):
        with open(os.path.join(libbuild.CSRC, name)) as f:
            src = f.read()
        codes += re.findall(r"spin\([^;]*?(1[2-5]\d)[,)]", src) + re.findall(r"product\([^;]*?(1[2-5]\d)\)", src)
        codes += re.findall(r"atomicExch\(p\.status, (\d+)\)", src)
    assert len(codes) >= 20
    assert sorted(codes) == sorted(set(codes))
    others = []
    for name in ("softmax_attn_fwd.cu", "softmax_attn_bwd.cu", "work_queue.cuh"):
        with open(os.path.join(libbuild.CSRC, name)) as f:
            others += re.findall(r"_spin\([^;]*?status, (\d+),", f.read())
    assert not set(codes) & set(others)
