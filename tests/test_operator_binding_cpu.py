"""CPU checks of the softmax attention and rotary binding: integers that a C int would not hold are
refused before anything is allocated or launched."""
import pytest
import torch

import rank_linear_complexity_gb300.linformer as lf

WIDE = 2 ** 32 + 64  # 64 once it is cut to 32 bits


@pytest.mark.parametrize("kw", [dict(rot=WIDE), dict(original_length=2 ** 32 + 8192),
                                dict(scaling=2 ** 32 + 1), dict(rot=-WIDE)])
def test_wide_integers_of_the_table(kw):
    with pytest.raises(ValueError, match="32-bit"):
        lf.rotary_phase(**{**dict(rot=64), **kw, "device": "cpu"})


def long(shape):
    return torch.zeros(1, dtype=torch.bfloat16).expand(shape)


@pytest.mark.parametrize("shape", [(1, 2, WIDE, 64), (WIDE, 1, 1, 64)])
def test_sizes_past_32_bits(shape):
    x, small = long(shape), long((1, 2, 4, 64))
    phase = torch.zeros(32, dtype=torch.int64)
    for call in (lambda: lf.softmax_attention(x, x, x), lambda: lf.softmax_attention(small, x, x),
                 lambda: lf.softmax_attention_backward(x, x, x, x, x, None),
                 lambda: lf.softmax_attention_backward(small, x, x, small, small, None),
                 lambda: lf.rotary(x, phase=phase)):
        with pytest.raises(ValueError, match="32-bit"):
            call()


@pytest.mark.parametrize("kw", [dict(layout=2 ** 32), dict(rot=WIDE), dict(start=2 ** 31)])
def test_wide_integers_of_the_turn(kw):
    with pytest.raises(ValueError, match="32-bit"):
        lf.rotary(long((1, 2, 4, 64)), phase=torch.zeros(32, dtype=torch.int64), **kw)


def test_without_torchs_private_names(monkeypatch):
    """The quick names of the current stream and device are torch's own: without them the public
    ones serve."""
    class Stream:
        cuda_stream = 77

    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.delattr(torch._C, "_cuda_getDevice", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: Stream())
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    device = torch.device("cuda:0")
    assert lf._stream_of(device) == 77
    done = []
    lf._call(lambda x: done.append(x) or 0, device, (5,), "call")
    assert done == [5]


def test_every_wait_of_the_attention_kernels_has_a_code_of_its_own():
    """The code in the device status word names one wait in the sources."""
    import os
    import re
    from rank_linear_complexity_gb300 import build
    codes = []
    for name in ("softmax_attn_fwd.cu", "softmax_attn_bwd.cu", "work_queue.cuh"):
        with open(os.path.join(build.CSRC, name)) as f:
            codes += re.findall(r"_spin\([^;]*?status, (\d+),", f.read())
    assert len(codes) >= 40
    assert sorted(codes) == sorted(set(codes))
