"""GPU tests of the rotary turn's accuracy: sines and cosines as they stand in the result (pairs
(1, 0))."""

import numpy as np
import pytest
import torch

import rank_linear_complexity_gb300.linformer as lf

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def status():
    torch.cuda.synchronize()
    assert lf.linformer_debug_read_device_status() == 0


def test_sines_and_cosines_of_every_part_of_a_turn():
    """x = (1, 0) gives (cos, sin) unrounded by products.  Each is off by at most 1 ulp of the
    function (2^-23 of its value), by the argument's rounding within an eighth of a turn (2^-27
    half turns: pi 2^-27 = 2^-25.3; times the function's slope, at most 1) and by the 32 bits of
    a turn that it keeps (2 pi 2^-32 = 2^-29.3)."""
    g = torch.Generator().manual_seed(1)
    near = torch.arange(8)[:, None] * (1 << 61) + torch.randint(-(1 << 40), 1 << 40, (8, 64), generator=g)
    words = torch.cat([torch.randint(-(1 << 63), (1 << 63) - 1, (512,), generator=g), near.flatten()])
    x = torch.zeros(1, 1, 1, 2, device=DEV)
    x[..., 0] = 1
    for w in words.tolist():
        w = (w + (1 << 63)) % (1 << 64) - (1 << 63)
        ph = torch.tensor([w], dtype=torch.int64, device=DEV)
        c, s = lf.rotary(x, phase=ph, start=1).flatten().double().tolist()
        t = 2 * np.pi * (w / 2.0 ** 64)
        for got, want in ((c, np.cos(t)), (s, np.sin(t))):
            assert abs(got - want) <= 2.0 ** -23 * abs(want) + 2.0 ** -25.3 + 2.0 ** -29.3, (w, got, want)
    status()
