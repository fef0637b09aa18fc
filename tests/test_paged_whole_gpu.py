"""GPU tests of which prompts' units of work stay whole (one kernel) and which are cut and joined (two): a
causal mask leaves the CTAs of a long prompt's first tokens idle while its last ones' work, unless units are
cut.  Either way the result is the dense call's."""
import pytest
import torch

import rank_linear_complexity_gb300.linformer as lf
from tests.paged_cases import ints

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF = torch.bfloat16


@pytest.mark.parametrize("hq,hk,nq,before,window,causal,kernels", [
    (1, 1, 38000, 0, 0, True, 2),        # 297 blocks a unit at most, 149 on average
    (2, 2, 19200, 0, 0, True, 2),
    (2, 1, 19200, 0, 0, True, 2),
    (3, 3, 12800, 12800, 0, True, 2),    # behind rows of the cache too
    (3, 3, 12800, 0, 12000, True, 2),    # a window that few queries fill
    (3, 3, 12800, 0, 3000, True, 1),     # and one that most do
    (3, 3, 12800, 12800, 12800, True, 1),
    (3, 3, 12800, 0, 0, False, 1),       # all units alike
    (3, 1, 12800, 0, 0, True, 1),        # two heads a unit
    (8, 8, 4608, 0, 0, True, 1),
])
def test_long_prompts(hq, hk, nq, before, window, causal, kernels):
    if torch.cuda.get_device_properties(DEV).multi_processor_count != 152:
        pytest.skip("the rule goes by the number of SMs")
    d, page = 64, 64
    g = torch.Generator(device=DEV).manual_seed(nq)
    n = before + nq
    pages = -(-n // page)
    kc, vc = (torch.randn(pages, page, hk, d, generator=g, device=DEV).to(BF).transpose(1, 2) for _ in range(2))
    table = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)[None]
    Q = torch.randn(1, nq, hq, d, generator=g, device=DEV).to(BF).transpose(1, 2)
    launches = lf.linformer_launch_count()
    O, lse = lf.paged_attention(Q, kc, vc, table, ints([n], DEV), causal=causal, window=window)
    assert lf.linformer_launch_count() - launches == kernels
    K, V = (x[table[0].long()].transpose(0, 1).reshape(1, hk, -1, d)[:, :, :n].contiguous() for x in (kc, vc))
    want, wl = lf.softmax_attention(Q, K, V, causal=causal, window=window)
    torch.cuda.synchronize()
    assert lf.linformer_debug_read_device_status() == 0
    # each side rounds P and O, three roundings of rms 2^-8 / sqrt 3 in all: as in the other tests of the paged
    # attention against the dense one
    assert (O.float() - want.float()).norm() <= 6e-3 * want.float().norm()
    assert torch.allclose(lse, wl, atol=1e-4)
