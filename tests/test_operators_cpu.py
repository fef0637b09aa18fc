"""CPU checks of the softmax attention and the rotary positions: every refusal of the entry
points (nothing is launched, addresses are made up), the binding's own, and the pins of the two
fp64 oracles (scalar loops, autograd, differences, planted mistakes)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import rank_linear_complexity_gb300.linformer as lf
from oracle import rotary as rot_orc
from oracle import softmax_attention as att
from rank_linear_complexity_gb300 import build as libbuild

A = 1 << 20  # an aligned address that is never used: every call fails its checks


@pytest.fixture(scope="module")
def L():
    libbuild.build()
    return lf.lib()


def strides(*s):
    return (ctypes.c_int64 * 3)(*s)


FWD = [
    (dict(Q=None), -1), (dict(O=None), -1), (dict(lse=None), -1),
    (dict(b=0), -2), (dict(hq=0), -2), (dict(nq=0), -2), (dict(nk=0), -2), (dict(hq=3, hk=2), -2),
    (dict(nk=(1 << 29) + 1), -2),
    (dict(dtype=0), -3), (dict(dtype=2), -3), (dict(d=136), -3), (dict(d=20), -3),
    (dict(dtype=3), -4), (dict(dtype=-1), -4),
    (dict(Q=A + 8), -5), (dict(lse=A + 2), -5), (dict(ql=A + 2), -5),
    (dict(sK=(2 * 64 * 64, 64 * 64, 68)), -5),
    (dict(scale=0.0), -10), (dict(scale=-1.0), -10), (dict(scale=math.inf), -10),
    (dict(scale=math.nan), -10), (dict(causal=2), -10), (dict(window=4, causal=0), -10),
    (dict(window=-1), -10), (dict(sV=(0, 4096, 64)), -10), (dict(sV=(8192, -4096, 64)), -10),
    (dict(sO=(4 * 64 * 64, 64 * 64, 8)), -10), (dict(sQ=((1 << 38) + 8, 4096, 64)), -10),
]


def forward_args(**kw):
    a = dict(Q=A, sQ=None, K=A, sK=None, V=A, sV=None, O=A, sO=None, lse=A, ql=None, kl=None, b=2,
             hq=4, hk=2, nq=64, nk=64, d=64, scale=0.125, causal=1, window=0, dtype=1)
    a.update(kw)
    for k in ("sQ", "sK", "sV", "sO", "sdQ", "sdO"):
        if a.get(k) is not None:
            a[k] = strides(*a[k])
    return a


@pytest.mark.parametrize("kw,expected", FWD)
def test_forward_refusals(L, kw, expected):
    a = forward_args(**kw)
    st = L.linformer_softmax_attn_fwd(*(a[k] for k in (
        "Q", "sQ", "K", "sK", "V", "sV", "O", "sO", "lse", "ql", "kl", "b", "hq", "hk", "nq", "nk",
        "d", "scale", "causal", "window", "dtype")), 0)
    assert st == expected, lf.status_string(st)


@pytest.mark.parametrize("kw,expected", FWD + [
    (dict(dO=None), -1), (dict(dK=None), -1), (dict(dV=A + 4), -5), (dict(dO=A + 2), -5),
    (dict(sdQ=(4 * 64 * 64, 64 * 64, 32)), -10), (dict(sdO=(0, 1, 64)), -10)])
def test_backward_refusals(L, kw, expected):
    if kw == dict(sO=(4 * 64 * 64, 64 * 64, 8)):
        pytest.skip("O is an input here: its rows may overlap")
    a = forward_args(**kw)
    for k in ("dO", "dQ", "dK", "dV"):
        a.setdefault(k, A)
    st = L.linformer_softmax_attn_bwd(
        a["Q"], a["sQ"], a["K"], a["sK"], a["V"], a["sV"], a["O"], a["sO"], a["dO"], a.get("sdO"),
        a["lse"], a["dQ"], a.get("sdQ"), a["dK"], None, a["dV"], None, a["ql"], a["kl"], a["b"],
        a["hq"], a["hk"], a["nq"], a["nk"], a["d"], a["scale"], a["causal"], a["window"],
        a["dtype"], 0)
    assert st == expected, lf.status_string(st)


@pytest.mark.parametrize("kw,expected", [
    (dict(X=None), -1), (dict(Y=None), -1), (dict(phase=None), -1), (dict(hx2=1), -1),
    (dict(b=0), -2), (dict(hx=0), -2), (dict(hx2=-1), -2), (dict(n=0), -2), (dict(d=0), -2),
    (dict(b=1 << 16, hx=1 << 16), -2),
    (dict(dtype=2), -3), (dict(dtype=5), -4), (dict(layout=2), -4),
    (dict(X=A + 8), -5), (dict(phase=A + 4), -5), (dict(positions=A + 2), -5),
    (dict(rot=0), -10), (dict(rot=3), -10), (dict(rot=66), -10), (dict(inverse=2), -10),
    (dict(amplitude=math.nan), -10), (dict(start=2 ** 31 - 8), -10),
    (dict(sX=(64, 0, 64)), -10), (dict(sY=(4096, 4096, 32)), -10),
    (dict(Y=A, sY=(1 << 20, 1 << 13, 128)), -10),  # in place with other strides
])
def test_rotary_refusals(L, kw, expected):
    a = dict(X=A, sX=None, Y=A + 4096, sY=None, hx=4, X2=None, Y2=None, hx2=0, phase=A,
             positions=None, start=0, b=2, n=16, d=64, rot=64, layout=0, amplitude=1.0, inverse=0,
             dtype=0)
    a.update(kw)
    for k in ("sX", "sY"):
        if a[k] is not None:
            a[k] = strides(*a[k])
    st = L.linformer_rotary(a["X"], a["sX"], a["Y"], a["sY"], a["hx"], a["X2"], None, a["Y2"], None,
                            a["hx2"], a["phase"], a["positions"], a["start"], a["b"], a["n"],
                            a["d"], a["rot"], a["layout"], a["amplitude"], a["inverse"], a["dtype"],
                            0)
    assert st == expected, lf.status_string(st)


@pytest.mark.parametrize("kw,expected", [
    (dict(phase=None), -1), (dict(rot=0), -2), (dict(rot=7), -2), (dict(scaling=4), -4),
    (dict(phase=A + 4), -5), (dict(base=0.0), -10), (dict(base=math.inf), -10),
    (dict(factor=-1.0), -10), (dict(scaling=3, original=0), -10),
    (dict(scaling=3, original=8, fast=1.0, slow=1.0), -10)])
def test_phase_refusals(L, kw, expected):
    a = dict(phase=A, rot=64, base=1e4, scaling=0, factor=1.0, original=0, fast=32.0, slow=1.0)
    a.update(kw)
    assert L.linformer_rotary_phase(a["phase"], a["rot"], a["base"], a["scaling"], a["factor"],
                                    a["original"], a["fast"], a["slow"], 0) == expected


@pytest.mark.parametrize("kw", [dict(O=A), dict(O=A + 16), dict(O=A + 32), dict(scale=3e38)])
def test_forward_refuses_an_output_over_an_input(L, kw):
    a = forward_args(K=A + 16, V=A + 32, **kw)
    if "O" not in kw:
        a["O"] = A + 48
    st = L.linformer_softmax_attn_fwd(*(a[k] for k in (
        "Q", "sQ", "K", "sK", "V", "sV", "O", "sO", "lse", "ql", "kl", "b", "hq", "hk", "nq", "nk",
        "d", "scale", "causal", "window", "dtype")), 0)
    assert st == -10, lf.status_string(st)


@pytest.mark.parametrize("same", [("dQ", "Q"), ("dK", "K"), ("dV", "V"), ("dQ", "dO"), ("dK", "dV"),
                                  ("dV", "O")])
def test_backward_refuses_an_output_over_another_tensor(L, same):
    t = {k: A + 16 * i for i, k in enumerate(("Q", "K", "V", "O", "dO", "dQ", "dK", "dV"))}
    t[same[0]] = t[same[1]]
    st = L.linformer_softmax_attn_bwd(
        t["Q"], None, t["K"], None, t["V"], None, t["O"], None, t["dO"], None, A, t["dQ"], None,
        t["dK"], None, t["dV"], None, None, None, 2, 4, 2, 64, 64, 64, 0.125, 1, 0, 1, 0)
    assert st == -10, lf.status_string(st)


@pytest.mark.parametrize("y,x2,y2", [(A + 16, A + 32, A + 16), (A + 16, A + 16, A + 32),
                                     (A + 16, A + 32, A)])
def test_rotary_refuses_an_output_over_the_other_tensor(L, y, x2, y2):
    st = L.linformer_rotary(A, None, y, None, 4, x2, None, y2, None, 4, A, None, 0, 2, 16, 64, 64, 0,
                            1.0, 0, 1, 0)
    assert st == -10, lf.status_string(st)


def test_binding_refuses_rows_with_gaps_and_wide_integers():
    gaps = torch.zeros(2, 2, 3, 16)[..., ::2]
    for x in (gaps[..., :1], gaps):  # the same strides, the last dimension of size one first
        with pytest.raises(ValueError, match="contiguous"):
            lf._strides(x)
    assert lf._int32("start", -2 ** 31) == -2 ** 31
    for x in (2 ** 31, -2 ** 31 - 1, 2 ** 32):
        with pytest.raises(ValueError, match="32-bit"):
            lf._int32("start", x)


def test_binding_refuses_host_tensors_and_wrong_shapes():
    q = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        lf.softmax_attention(q, q, q)
    with pytest.raises(ValueError):
        lf.rotary(q, phase=torch.zeros(32, dtype=torch.int64))


def test_new_status_and_kernel_names(L):
    assert lf.status_string(-10) not in ("", "unknown status")
    names = {L.linformer_kernel_name(i) for i in range(lf.KERNEL_COUNT)}
    assert None not in names and len(names) == lf.KERNEL_COUNT
    assert L.linformer_kernel_name(lf.KERNEL_COUNT) is None


# --- pins of the attention oracle -----------------------------------------------------------

def inputs(b=2, hq=4, hk=2, nq=7, nk=9, d=8, seed=0):
    r = np.random.default_rng(seed)
    return (r.standard_normal((b, hq, nq, d)), r.standard_normal((b, hk, nk, d)),
            r.standard_normal((b, hk, nk, d)), r.standard_normal((b, hq, nq, d)))


OPTIONS = [dict(), dict(causal=True), dict(causal=True, window=3),
           dict(causal=True, q_lengths=[7, 3], k_lengths=[2, 9]),
           dict(q_lengths=[0, 5], k_lengths=[9, 0])]


@pytest.mark.parametrize("kw", OPTIONS)
def test_oracle_forward_against_scalar_loops(kw):
    Q, K, V, _ = inputs()
    O, lse, _, _ = att.forward(Q, K, V, scale=0.3, **kw)
    for b in range(2):
        lq = kw.get("q_lengths", [7, 7])[b]
        lk = kw.get("k_lengths", [9, 9])[b]
        for h in range(4):
            for i in range(7):
                seen = [j for j in range(lk) if i < lq and
                        (not kw.get("causal") or j <= i + lk - lq) and
                        (not kw.get("window") or j > i + lk - lq - kw["window"])]
                e = [math.exp(0.3 * sum(Q[b, h, i] * K[b, h // 2, j])) for j in seen]
                want = sum((x * V[b, h // 2, j] for x, j in zip(e, seen)), np.zeros(8))
                assert np.allclose(O[b, h, i], want / sum(e) if seen else 0, atol=1e-12)
                assert np.isclose(lse[b, h, i], math.log(sum(e)) if seen else -math.inf)


@pytest.mark.parametrize("kw", OPTIONS)
def test_oracle_backward_against_differences_and_autograd(kw):
    Q, K, V, dO = inputs(seed=1)
    grads, _, _ = att.backward(Q, K, V, dO, scale=0.3, **kw)
    rng = np.random.default_rng(2)
    for i, g in enumerate(grads):
        D = rng.standard_normal(g.shape)
        f = []
        for s in (1e-5, -1e-5):
            x = [Q, K, V]
            x[i] = x[i] + s * D
            f.append((att.forward(*x, scale=0.3, **kw)[0] * dO).sum())
        assert np.isclose((f[0] - f[1]) / 2e-5, (g * D).sum(), rtol=1e-7, atol=1e-8)
    t = [torch.tensor(x, requires_grad=True) for x in (Q, K, V)]
    s = torch.einsum("bhid,bhjd->bhij", t[0], t[1].repeat_interleave(2, 1)) * 0.3
    m = torch.stack([torch.from_numpy(att.visible(
        7, 9, kw.get("q_lengths", [7, 7])[b], kw.get("k_lengths", [9, 9])[b],
        kw.get("causal", False), kw.get("window", 0))) for b in range(2)])[:, None]
    e = torch.where(m, torch.exp(s), torch.zeros(()).double())
    p = e / e.sum(-1, keepdim=True).clamp_min(1e-300)
    (torch.einsum("bhij,bhjd->bhid", p, t[2].repeat_interleave(2, 1)) * torch.tensor(dO)).sum().backward()
    for g, x in zip(grads, t):
        assert np.allclose(g, x.grad.numpy(), atol=1e-12)


def test_oracle_padding_is_ignored_and_mistakes_are_caught():
    Q, K, V, dO = inputs(seed=3)
    kw = dict(q_lengths=[5, 7], k_lengths=[4, 9], causal=True)
    base = att.forward(Q, K, V, **kw)[0]
    Q2, K2, V2 = Q.copy(), K.copy(), V.copy()
    Q2[0, :, 5:], K2[0, :, 4:], V2[0, :, 4:] = np.nan, np.nan, np.nan
    assert np.array_equal(att.forward(Q2, K2, V2, **kw)[0], base)
    wrong = [att.forward(Q, K, V, scale=1.0, **kw)[0], att.forward(Q, K[:, ::-1], V, **kw)[0],
             att.forward(Q, K, V, q_lengths=[5, 7], k_lengths=[4, 9])[0]]
    for w in wrong:
        assert np.abs(w - base).max() > 1e-2


# --- pins of the rotary oracle --------------------------------------------------------------

def test_rotary_oracle():
    r = np.random.default_rng(4)
    x = r.standard_normal((1, 2, 5, 8))
    f = rot_orc.frequencies(6)
    assert np.allclose(f, [1.0, 1e4 ** (-1 / 3), 1e4 ** (-2 / 3)])
    pos = np.array([[0, 1, 2, 7, 100]])
    for inter in (False, True):
        y = rot_orc.rotate(x, f, pos, 6, inter)
        for i, p in enumerate(pos[0]):
            for k in range(3):
                a, z = (2 * k, 2 * k + 1) if inter else (k, k + 3)
                w = (x[0, :, i, a] + 1j * x[0, :, i, z]) * np.exp(1j * p * f[k])
                assert np.allclose(y[0, :, i, a], w.real) and np.allclose(y[0, :, i, z], w.imag)
        assert np.array_equal(y[..., 6:], x[..., 6:])
        back = rot_orc.rotate(y, f, pos, 6, inter, inverse=True)
        assert np.allclose(back, x)
    # scores depend on the distance alone
    q, k = x[:, :1], x[:, 1:]
    s = [(rot_orc.rotate(q, f, pos + o, 6)[0, 0, 3] * rot_orc.rotate(k, f, pos + o, 6)[0, 0, 1]).sum()
         for o in (0, 1000)]
    assert np.isclose(s[0], s[1])


def test_rotary_scalings():
    f = rot_orc.frequencies(64)
    assert np.allclose(rot_orc.frequencies(64, scaling=1, factor=4.0), f / 4)
    b = rot_orc.frequencies(64, scaling=2, factor=8.0)
    assert np.isclose(b[0], f[0]) and np.isclose(b[-1], f[-1] / 8)
    p = rot_orc.frequencies(64, scaling=3, factor=8.0, original=8192)
    turns = 8192 * f / (2 * math.pi)
    assert np.allclose(p[turns >= 32], f[turns >= 32]) and np.allclose(p[turns <= 1], f[turns <= 1] / 8)
    mid = (turns < 32) & (turns > 1)
    assert mid.any() and (p[mid] < f[mid]).all() and (p[mid] > f[mid] / 8).all()
    w = rot_orc.phase_words(np.array([math.pi, 2 * math.pi / 4]))
    assert w[0] == -(1 << 63) and w[1] == 1 << 62
