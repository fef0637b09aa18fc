"""GPU tests of the rotary positions (linformer_rotary, linformer_rotary_phase) against the fp64
oracle.  Bounds per element, with A = amplitude (|x_a| + |x_z|) the absolute terms:
  fp32: sine and cosine within 2^-22 (the phase as a float: at most pi 2^-25 of an angle; the
        functions: 2 ulp), three roundings of 2^-24: 2^-21 A;
  bf16: the same, and the result rounded once (half a step, 2^-8 of it)."""
import numpy as np
import pytest
import torch

import rank_linear_complexity_gb300.linformer as lf
from oracle import rotary as orc
from oracle.softmax_attention import host64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
SCALINGS = {"plain": {}, "linear": dict(scaling=1, factor=4.0), "base": dict(scaling=2, factor=8.0),
            "by_parts": dict(scaling=3, factor=8.0, original=8192)}


def make(b, h, n, d, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(b, h, n, d, generator=g).to(dtype).to(DEV)


def phase_of(rot, o):
    o = dict(o)
    return lf.rotary_phase(rot, scaling=o.get("scaling", 0), factor=o.get("factor", 1.0),
                           original_length=o.get("original", 0), device=DEV)


def status():
    torch.cuda.synchronize()
    assert lf.linformer_debug_read_device_status() == 0


def check(y, x, f, pos, rot, interleaved, amplitude=1.0, inverse=False):
    ref = orc.rotate(x, f, pos, rot, interleaved, amplitude, inverse)
    terms = orc.rotate(np.abs(host64(x)), np.zeros(rot // 2), np.zeros_like(pos), rot, interleaved)
    p = np.arange(rot // 2)
    a, z = (2 * p, 2 * p + 1) if interleaved else (p, p + rot // 2)
    both = terms[..., a] + terms[..., z]
    bound = np.zeros(ref.shape)
    bound[..., a] = bound[..., z] = abs(amplitude) * both * 2.0 ** -21
    if x.dtype == torch.bfloat16:
        bound[..., :rot] += 2.0 ** -8 * np.abs(ref[..., :rot]) * (1 + 2.0 ** -8)
    err = np.abs(host64(y) - ref)
    assert (err <= bound).all(), (err - bound).max()
    assert np.array_equal(host64(y)[..., rot:], host64(x)[..., rot:])


CASES = [
    # b, h, h2, n, d, rot, dtype, interleaved
    (1, 1, 0, 1, 2, 2, torch.float32, False),
    (2, 3, 1, 7, 64, 64, torch.bfloat16, False),
    (2, 3, 3, 33, 64, 32, torch.float32, True),
    (3, 2, 1, 5, 80, 40, torch.bfloat16, True),      # 20 pairs: element by element
    (1, 5, 2, 130, 128, 128, torch.bfloat16, True),
    (2, 4, 4, 9, 30, 10, torch.float32, False),      # odd sizes, part of the head
    (64, 32, 8, 1, 128, 128, torch.bfloat16, False),
    (1, 12, 12, 1000, 64, 48, torch.bfloat16, False),
]


@pytest.mark.parametrize("case", CASES, ids=[str(i) for i in range(len(CASES))])
@pytest.mark.parametrize("inverse", [False, True])
def test_matches_oracle(case, inverse):
    b, h, h2, n, d, rot, dtype, inter = case
    o = list(SCALINGS.values())[(b + h + n) % 4]
    x, x2 = make(b, h, n, d, dtype, 1), make(b, h2, n, d, dtype, 2) if h2 else None
    pos = torch.randint(0, 131072, (b, n), dtype=torch.int32, generator=torch.Generator().manual_seed(3))
    out = lf.rotary(x, x2, phase_of(rot, o), positions=pos.to(DEV), rot=rot,
                    layout=int(inter), amplitude=1.25, inverse=inverse)
    status()
    f = orc.frequencies(rot, **o)
    for y, src in zip(out if h2 else (out,), (x, x2)):
        check(y, src, f, pos.numpy(), rot, inter, 1.25, inverse)


@pytest.mark.parametrize("name", SCALINGS)
def test_phase_table(name):
    """The device's table against the oracle's frequencies: 2^-50 of a turn (the 64-bit power
    and its argument, a few roundings of 2^-53)."""
    for rot in (2, 64, 130):
        got = phase_of(rot, SCALINGS[name]).cpu().numpy()
        want = orc.phase_words(orc.frequencies(rot, **SCALINGS[name]))
        off = (got - want).astype(np.int64)  # wraps, as turns do
        assert np.abs(off.astype(np.float64)).max() <= 2.0 ** 14


def test_far_and_negative_positions():
    """Angles stay exact where fp32 products of position and frequency would be off by radians."""
    x = make(1, 2, 6, 64, torch.float32, 4)
    pos = torch.tensor([[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 16777217]], dtype=torch.int32)
    f = orc.frequencies(64)
    y = lf.rotary(x, phase=torch.from_numpy(orc.phase_words(f)).to(DEV), positions=pos.to(DEV))
    status()
    # the oracle's own angle, pos f in 64 bits, is off by up to 2^31 2^-53: 2^-22 more
    ref = orc.rotate(x, f, pos.numpy(), 64)
    terms = np.abs(host64(x))
    both = np.concatenate([terms[..., :32] + terms[..., 32:]] * 2, -1)
    assert (np.abs(host64(y) - ref) <= both * (2.0 ** -21 + 2.0 ** -21)).all()


def test_start_is_positions_from_start():
    x = make(2, 3, 50, 64, torch.bfloat16, 5)
    ph = lf.rotary_phase(64, device=DEV)
    pos = (torch.arange(50, dtype=torch.int32) + 4000).repeat(2, 1).to(DEV)
    a = lf.rotary(x, phase=ph, start=4000)
    assert torch.equal(a.view(torch.int16), lf.rotary(x, phase=ph, positions=pos).view(torch.int16))
    status()


def test_strided_in_place_and_one_tensor_or_two():
    b, h, h2, n, d = 2, 4, 2, 37, 64
    fused = torch.randn(b, n, (h + 2 * h2) * d, device=DEV, generator=torch.Generator(DEV).manual_seed(6))
    ph = lf.rotary_phase(d, device=DEV)
    for dtype in (torch.float32, torch.bfloat16):
        buf = fused.to(dtype)
        q = buf[..., :h * d].view(b, n, h, d).transpose(1, 2)
        k = buf[..., h * d:(h + h2) * d].view(b, n, h2, d).transpose(1, 2)
        keep = buf.clone()
        want = lf.rotary(q.contiguous(), k.contiguous(), ph)
        got = lf.rotary(q, k, ph)
        assert all(torch.equal(a, c) for a, c in zip(want, got))
        assert torch.equal(buf, keep)
        lf.rotary(q, k, ph, out=q, out2=k)
        assert torch.equal(q, want[0]) and torch.equal(k, want[1])
        assert torch.equal(buf[..., (h + h2) * d:], keep[..., (h + h2) * d:])
        # rows an odd number of elements apart: element by element
        odd = torch.zeros(b, h, n, d + 1, dtype=dtype, device=DEV)[..., :d]
        odd.copy_(want[0])
        back = lf.rotary(odd, phase=ph, inverse=True)
        assert torch.equal(back, lf.rotary(want[0].contiguous(), phase=ph, inverse=True))
    status()


def test_gradient_is_the_turn_backwards():
    """<rotary(x), g> = <x, rotary(g, inverse)> (the map is linear), and against differences:
    exact for a linear map."""
    x, g = make(2, 3, 11, 64, torch.float32, 7), make(2, 3, 11, 64, torch.float32, 8)
    ph = lf.rotary_phase(48, device=DEV)
    kw = dict(phase=ph, start=300, rot=48, layout=lf.ROTARY_INTERLEAVED, amplitude=1.5)
    dx = lf.rotary(g, inverse=True, **kw)
    left, right = (lf.rotary(x, **kw).double() * g).sum(), (x.double() * dx).sum()
    # 2^-21 of the absolute terms on each side
    allowed = 2 * 2.0 ** -21 * 2 * 1.5 * (x.double().abs().sum() * g.abs().max()).item()
    assert abs((left - right).item()) <= allowed
    e = make(2, 3, 11, 64, torch.float32, 9)
    diff = (host64(lf.rotary(x + e, **kw)) - host64(lf.rotary(x - e, **kw))) / 2
    slope = (diff * host64(g)).sum()
    assert abs(slope - (host64(e) * host64(dx)).sum()) <= 4 * allowed
    status()


def test_captured_and_other_stream():
    x = make(2, 3, 64, 64, torch.bfloat16, 10)
    ph = lf.rotary_phase(64, device=DEV)
    want = lf.rotary(x, phase=ph)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = lf.rotary(x, phase=ph)
    y.zero_()
    g.replay()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    z = lf.rotary(x, phase=ph, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(z, want)
    status()


def test_attention_layer_forward_and_backward():
    """The operators as a layer uses them: positions on a fused projection's queries and keys,
    causal attention, its gradients, and the positions' gradient, against the oracles run on
    the same intermediate tensors."""
    from oracle import softmax_attention as att
    b, hq, hk, n, d = 2, 8, 2, 200, 64
    bf = torch.bfloat16
    buf = torch.randn(b, n, (hq + 2 * hk) * d, device=DEV, generator=torch.Generator(DEV).manual_seed(12)).to(bf)
    q, k, v = (buf[..., s * d:e * d].view(b, n, e - s, d).transpose(1, 2)
               for s, e in ((0, hq), (hq, hq + hk), (hq + hk, hq + 2 * hk)))
    ph = lf.rotary_phase(d, device=DEV)
    Q, K = lf.rotary(q, k, ph)
    O, lse = lf.softmax_attention(Q, K, v, causal=True)
    dO = torch.randn(b, hq, n, d, device=DEV, generator=torch.Generator(DEV).manual_seed(13)).to(bf)
    dQ, dK, dV = lf.softmax_attention_backward(Q, K, v, O, dO, lse, causal=True)
    dq, dk = lf.rotary(dQ, dK, ph, inverse=True)
    status()
    pos = np.tile(np.arange(n), (b, 1))
    f = orc.frequencies(d)
    check(Q, q, f, pos, d, False)
    check(K, k, f, pos, d, False)
    ref, rl, bO, bl = att.forward(Q, K, v, causal=True)
    assert (np.abs(host64(O) - ref) <= bO).all() and (np.abs(host64(lse) - rl) <= bl).all()
    refs, bounds, rows = att.backward(Q, K, v, dO, causal=True)
    # O is the kernel's: its own error reaches delta as the rounding's does, once more
    for g, r, e, w in zip((dQ, dK, dV), refs, bounds, rows):
        assert (np.abs(host64(g) - r) <= e + 2 * w).all()
    check(dq, dQ, f, pos, d, False, inverse=True)
    check(dk, dK, f, pos, d, False, inverse=True)
