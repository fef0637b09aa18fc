"""GPU tests of the softmax attention and rotary calls given a stream other than the current one:
outputs that a call makes belong to that stream, so neither side's queued work reaches the
other's memory."""
import pytest
import torch

import rank_linear_complexity_gb300.linformer as lf

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF = torch.bfloat16
LONG = 200_000_000  # cycles, about a tenth of a second


def status():
    torch.cuda.synchronize()
    assert lf.linformer_debug_read_device_status() == 0


def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == BF else torch.int32 if t.dtype == torch.float32
                               else torch.int64)


def calls():
    g = torch.Generator(device=DEV).manual_seed(1)
    Q, K, V, dO = (torch.randn(2, 8, 1024, 128, generator=g, device=DEV).to(BF) for _ in range(4))
    O, lse = lf.softmax_attention(Q, K, V)
    ph = lf.rotary_phase(128, device=DEV)
    torch.cuda.synchronize()
    return {
        "attention": lambda **kw: lf.softmax_attention(Q, K, V, **kw),
        "backward": lambda **kw: lf.softmax_attention_backward(Q, K, V, O, dO, lse, **kw),
        "rotary": lambda **kw: lf.rotary(Q, K, ph, **kw),
        "phase": lambda **kw: (lf.rotary_phase(1 << 19, device=DEV, **kw),),
    }


NAMES = ["attention", "backward", "rotary", "phase"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("as_int", [False, True])
def test_blocks_that_the_current_stream_still_writes(name, as_int):
    """Blocks freed on the current stream, whose queued work still writes them."""
    f = calls()[name]
    want = [x.clone() for x in f()]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    s = torch.cuda.Stream()
    old = [torch.empty_like(x) for x in want]
    torch.cuda.synchronize()
    torch.cuda._sleep(LONG)
    for x in old:
        x.zero_()
    del old, x
    got = f(stream=s.cuda_stream if as_int else s)
    torch.cuda.synchronize()
    assert all(torch.equal(bits(a), bits(b)) for a, b in zip(got, want))
    status()


@pytest.mark.parametrize("name", NAMES)
def test_results_dropped_while_the_stream_is_behind(name):
    """Results dropped before their stream has written them, the memory asked for again."""
    f = calls()[name]
    shapes = [(x.shape, x.dtype) for x in f()]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(LONG)
    got = f(stream=s)
    del got
    mine = [torch.zeros(sh, dtype=dt, device=DEV) for sh, dt in shapes]
    torch.cuda.synchronize()
    assert all((x == 0).all() for x in mine)
    status()


def test_outputs_given_by_the_caller_are_used():
    f = calls()["attention"]
    O, lse = f()
    mine = torch.empty_like(O), torch.empty_like(lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = f(stream=s, out=mine[0], lse=mine[1])
    s.synchronize()
    assert got[0] is mine[0] and got[1] is mine[1]
    assert torch.equal(bits(O), bits(mine[0])) and torch.equal(lse, mine[1])
    # the default stream by its handle
    got = f(stream=0)
    torch.cuda.synchronize()
    assert torch.equal(bits(O), bits(got[0]))
    status()
