"""GPU tests of the exact softmax attention at the ends of its range: large values beside logits
that grow along a row, against the fp64 oracle within its derived bounds."""
import numpy as np
import pytest
import torch

import rank_linear_complexity_gb300.linformer as lf
from oracle import softmax_attention as orc

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF = torch.bfloat16


def status():
    torch.cuda.synchronize()
    assert lf.linformer_debug_read_device_status() == 0


def close(got, ref, bound, name):
    err = np.abs(orc.host64(got) - ref)
    assert np.isfinite(err).all(), f"{name}: not finite"
    assert (err <= bound).all(), f"{name}: worst {(err - bound).max()}"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("growth", [6.0, 20.0, 38.0])
def test_large_values_behind_growing_logits(d, growth):
    """Logits whose maximum grows by 2^growth from the first block of keys to the last, over
    values of 2^105: the sums reach the largest weight times 640 times that."""
    n, nk = 150, 640
    g = torch.Generator().manual_seed(d)
    Q, K = torch.ones(1, 2, n, d), torch.randn(1, 2, nk, d, generator=g) * 0.1
    K[..., 0] += torch.linspace(0, growth * np.log(2), nk)
    V = torch.randn(1, 2, nk, d, generator=g) * 2.0 ** 105
    Q, K, V = (x.to(DEV, BF) for x in (Q, K, V))
    O, lse = lf.softmax_attention(Q, K, V, scale=1.0)
    status()
    ref, rl, bO, bl = orc.forward(Q, K, V, scale=1.0)
    close(O, ref, bO, "O")
    close(lse, rl, bl, "lse")
