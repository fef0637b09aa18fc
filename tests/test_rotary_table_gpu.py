"""GPU tests of the rotary frequency table against 60-digit arithmetic: every word is the fraction
of a turn to its last bit (2^-64, one more for the rounding of the 64-bit pairs it is formed in),
so that the angles of far positions are right with the table that the library makes."""
from decimal import Decimal, localcontext

import numpy as np
import pytest
import torch

import rank_linear_complexity_gb300.linformer as lf

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
PI = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


def turns_of(rot, base=10000.0, scaling=0, factor=1.0, original=0, fast=32.0, slow=1.0):
    """The pairs' turns per position, as Decimals."""
    base, factor, fast, slow = (Decimal(x) for x in (base, factor, fast, slow))
    out = []
    with localcontext() as c:
        c.prec = 60
        if scaling == 2 and rot > 2:
            base *= factor ** (Decimal(rot) / (rot - 2))
        for i in range(rot // 2):
            t = base ** (Decimal(-2 * i) / rot) / (2 * PI)
            if scaling == 1:
                t /= factor
            if scaling == 3:
                keep = min(max((original * t - slow) / (fast - slow), Decimal(0)), Decimal(1))
                t *= keep + (1 - keep) / factor
            out.append(t)
    return out


CASES = [dict(rot=2), dict(rot=64), dict(rot=130), dict(rot=128, base=500000.0),
         dict(rot=64, base=0.5), dict(rot=96, scaling=1, factor=3.7), dict(rot=64, scaling=2, factor=8.0),
         dict(rot=2, scaling=2, factor=8.0), dict(rot=4, scaling=2, factor=0.3),
         dict(rot=128, scaling=3, factor=8.0, original=8192),
         dict(rot=80, scaling=3, factor=40.0, original=4096, fast=30.1, slow=1.3, base=1e6)]


def table(o):
    return lf.rotary_phase(o["rot"], o.get("base", 10000.0), o.get("scaling", 0), o.get("factor", 1.0),
                           o.get("original", 0), o.get("fast", 32.0), o.get("slow", 1.0), device=DEV)


def status():
    torch.cuda.synchronize()
    assert lf.linformer_debug_read_device_status() == 0


@pytest.mark.parametrize("o", CASES, ids=[str(i) for i in range(len(CASES))])
def test_every_word_to_its_last_bit(o):
    got = [w % (1 << 64) for w in table(o).tolist()]
    status()
    with localcontext() as c:
        c.prec = 60
        for i, (g, t) in enumerate(zip(got, turns_of(**o))):
            off = (g - int((t % 1 * 2 ** 64).to_integral_value())) % (1 << 64)
            assert min(off, (1 << 64) - off) <= 1, (i, g, off)


@pytest.mark.parametrize("o", [CASES[1], CASES[9]], ids=["plain", "by_parts"])
def test_angles_of_the_farthest_positions(o):
    """(1, 0) turned: within 2^-23 of the functions' values, 2^-25.3 for the argument as a float,
    and what the word (2^31 2^-64 turns) and its upper 32 bits leave out, 2 pi (2^-33 + 2^-32)."""
    pos = [2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, 2 ** 28 - 1, 99_999_999]
    h = o["rot"] // 2
    x = torch.zeros(1, 1, len(pos), o["rot"], device=DEV)
    x[..., :h] = 1
    y = lf.rotary(x, phase=table(o), positions=torch.tensor([pos], dtype=torch.int32, device=DEV))
    status()
    y = y[0, 0].double().cpu().numpy()
    with localcontext() as c:
        c.prec = 60
        t = np.array([[float(p * f % 1 * 2 * PI) for f in turns_of(**o)] for p in pos])
    for got, want in ((y[:, :h], np.cos(t)), (y[:, h:], np.sin(t))):
        bound = 2.0 ** -23 * np.abs(want) + 2.0 ** -25.3 + 2 * np.pi * 3 * 2.0 ** -33
        assert (np.abs(got - want) <= bound).all(), (np.abs(got - want) - bound).max()


def test_extreme_bases_stay_finite():
    """Frequencies past what the pairs resolve still give a table (as far as 64 bits go)."""
    for base in (1e-300, 1e300, 5e-324, 1.7e308):
        lf.rotary_phase(64, base, device=DEV)
    status()
