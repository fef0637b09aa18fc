"""GPU tests of rotary calls large enough for a thread to go through several heads: from the first
tensor into the second, a last thread with fewer heads, in place and not.  A row's result does not
depend on how many heads a thread takes, so parts of the call (one head a thread) have to give
the same bits; sampled rows are checked against the fp64 oracle (pairs, with A the sum of a
pair's absolute elements: 2^-21 A, and 2^-8 of the result where it is rounded to bf16)."""
import numpy as np
import pytest
import torch

import rank_linear_complexity_gb300.linformer as lf
from oracle import rotary as orc
from oracle.softmax_attention import host64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def heads_a_thread(b, n, d, rot, heads, dtype, in_place):
    """The library's rule: as many heads as leave two full waves of threads, at most 16."""
    v = 4 if dtype == torch.float32 else 8
    if rot % (2 * v) or d % v:
        v = 1
    chunks = rot // 2 // v + (0 if in_place else (d - rot) // v)
    sms = torch.cuda.get_device_properties(DEV).multi_processor_count
    return max(1, min(heads, 16, b * n * chunks * heads // (2 * sms * 2048)))


def bits(x):
    return x.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32)


@pytest.mark.parametrize("inter", [False, True], ids=["halves", "neighbours"])
@pytest.mark.parametrize("h,h2,n,d,rot,dtype,per", [
    (5, 2, 30001, 64, 64, torch.float32, 2),      # a thread crosses over
    (5, 2, 45007, 64, 64, torch.bfloat16, 2),
    (11, 8, 30011, 64, 48, torch.bfloat16, 4),    # 19 heads in fours
    (11, 8, 10007, 80, 40, torch.float32, 4),
    (3, 0, 130001, 64, 64, torch.bfloat16, 2),    # one tensor
    (20, 5, 60013, 40, 40, torch.bfloat16, 16),   # element by element, at most 16
])
def test_several_heads_a_thread(h, h2, n, d, rot, dtype, per, inter):
    b = 1
    assert heads_a_thread(b, n, d, rot, h + h2, dtype, False) == per
    g = torch.Generator(device=DEV).manual_seed(n)
    x = torch.randn(b, h, n, d, generator=g, device=DEV).to(dtype)
    x2 = torch.randn(b, h2, n, d, generator=g, device=DEV).to(dtype) if h2 else None
    ph = lf.rotary_phase(rot, device=DEV)
    pos = torch.randint(0, 1 << 20, (b, n), generator=g, device=DEV, dtype=torch.int32)
    kw = dict(phase=ph, rot=rot, layout=int(inter), amplitude=1.25)
    out = lf.rotary(x, x2, positions=pos, **kw)
    out, src = (out, (x, x2)) if h2 else ((out,), (x,))
    step = 1500
    assert heads_a_thread(b, step, d, rot, h + h2, dtype, False) == 1 or per == 16
    for a in range(0, n, step * 7):
        at = slice(a, min(a + step, n))
        for hh in range(max(h, h2)):
            for y, s in zip(out, src):
                if hh < s.shape[1]:
                    part = lf.rotary(s[:, hh:hh + 1, at], positions=pos[:, at].contiguous(), **kw)
                    assert torch.equal(bits(part), bits(y[:, hh:hh + 1, at]))
    rows = np.random.default_rng(n).choice(n, 64, replace=False)
    f = orc.frequencies(rot)
    p = np.arange(rot // 2)
    i, j = (2 * p, 2 * p + 1) if inter else (p, p + rot // 2)
    for y, s in zip(out, src):
        ref = orc.rotate(s[:, :, rows], f, pos[:, rows].cpu().numpy(), rot, inter, 1.25)
        both = np.abs(host64(s[:, :, rows]))
        bound = np.zeros(ref.shape)
        bound[..., i] = bound[..., j] = 1.25 * (both[..., i] + both[..., j]) * 2.0 ** -21
        if dtype == torch.bfloat16:
            bound[..., :rot] += 2.0 ** -8 * np.abs(ref[..., :rot]) * (1 + 2.0 ** -8)
        assert (np.abs(host64(y[:, :, rows]) - ref) <= bound).all()
    # in place, both tensors, the rest of a head left as it is
    want = [y.clone() for y in out]
    lf.rotary(x, x2, positions=pos, out=x, out2=x2, **kw)
    assert all(torch.equal(bits(a), bits(c)) for a, c in zip(src, want))
    torch.cuda.synchronize()
    assert lf.linformer_debug_read_device_status() == 0
