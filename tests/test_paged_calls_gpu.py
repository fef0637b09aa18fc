"""GPU tests of how the cache calls are made: on other streams, in CUDA graphs, several at once, with
strided tensors, many sequences, guards around outputs and workspaces, no memory to be had."""
import numpy as np
import pytest
import torch

import rank_linear_complexity_gb300.linformer as lf
from oracle import paged
from oracle.softmax_attention import host64
from tests.paged_cases import bits, cache, ints, random_tree

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF = torch.bfloat16
LONG = 200_000_000  # cycles, about a tenth of a second


def status():
    torch.cuda.synchronize()
    assert lf.linformer_debug_read_device_status() == 0


def problem(b=3, hq=8, hk=2, nq=1, d=64, page=16, lengths=(700, 33, 1500), rows=20000, seed=0):
    """A batch over a table of `rows` rows: cut and joined (long ones), or whole (short ones)."""
    kc, vc, table = cache(b, hk, d, page, list(lengths), "rows", "bf16", seed, device=DEV)
    table = torch.nn.functional.pad(table, (0, max(0, rows // page - table.shape[1])), value=-1).contiguous()
    g = torch.Generator(device=DEV).manual_seed(seed)
    Q = torch.randn(b, hq, nq, d, generator=g, device=DEV).to(BF)
    return Q, kc, vc, table, ints(list(lengths), DEV)


def near(O, lse, Q, kc, vc, table, lengths, **kw):
    want = paged.forward(Q, kc, vc, table.tolist(), lengths.tolist(), **kw)
    assert (np.abs(host64(O) - want[0]) <= want[2]).all()
    some = np.isfinite(want[1])
    assert (np.abs(host64(lse)[some] - want[1][some]) <= want[3][some]).all()


def calls():
    """Name -> a call that makes its outputs, given a stream or none."""
    few, many = problem(), problem(nq=80)
    tree = paged.ancestors(random_tree(3, 80, seed=1).numpy())
    mask = torch.from_numpy(paged.words(tree)).to(DEV)
    up = random_tree(3, 80, seed=1).to(DEV)
    phase = lf.rotary_phase(64, device=DEV)
    K = torch.randn(3, 2, 5, 64, device=DEV).to(BF)
    rest = problem(seed=5)
    starts = ints([100, 3, 900], DEV)
    torch.cuda.synchronize()
    return {
        "few": lambda **kw: lf.paged_attention(*few, **kw),
        "many": lambda **kw: lf.paged_attention(*many, **kw),
        "tree": lambda **kw: lf.tree_attention(*many, mask, **kw),
        "mask": lambda **kw: (lf.tree_mask(up, **kw),),
        "append": lambda **kw: (lf.cache_append(K, K.clone(), *rest[1:4], starts, Q=K, phase=phase, **kw),),
    }


NAMES = ["few", "many", "tree", "mask", "append"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("as_int", [False, True])
def test_blocks_that_the_current_stream_still_writes(name, as_int):
    """A call given another stream: its outputs do not lie in memory that the current stream's queued
    work still writes."""
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


@pytest.mark.parametrize("rows", [1000, 20000])
@pytest.mark.parametrize("nq", [1, 6, 80])
def test_captured_in_a_graph(rows, nq):
    """Append and attend in one graph, replayed over inputs that change in place between replays."""
    lengths = (700, 33, 900)
    Q, kc, vc, table, total = problem(nq=nq, lengths=lengths, rows=rows, seed=3)
    starts = ints([x - nq if x >= nq else 0 for x in lengths], DEV)
    phase = lf.rotary_phase(64, device=DEV)
    K, V = (torch.randn(3, 2, nq, 64, device=DEV).to(BF) for _ in range(2))
    counts = ints([min(x, nq) for x in lengths], DEV)
    held = [x.clone() for x in (Q, K, V, kc, vc, total)]

    def step():
        q = lf.cache_append(K, V, kc, vc, table, starts, counts=counts, Q=Q, phase=phase)
        return lf.paged_attention(q, kc, vc, table, total, q_lengths=counts)
    want = [x.clone() for x in step()]
    status()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        O, lse = step()
    for change in (False, True, False):
        for x, y in zip((Q, K, V, kc, vc, total), held):
            x.copy_(y)
        if change:
            Q.mul_(0.5)
            total.sub_(20).clamp_(min=0)
        graph.replay()
        torch.cuda.synchronize()
        if change:
            again = step()
            assert torch.equal(bits(O), bits(again[0])) and torch.equal(lse, again[1])
            assert not torch.equal(bits(O), bits(want[0]))
        else:
            assert torch.equal(bits(O), bits(want[0])) and torch.equal(lse, want[1])
    status()


def test_two_graphs_and_eager_calls_at_once():
    """Workspaces are a call's own: graphs captured from the same calls, replayed on two streams while
    a third makes eager ones."""
    problems = [problem(nq=n, seed=i, lengths=(3000, 1700, 2500)) for i, n in enumerate((1, 40, 80))]
    want = [[x.clone() for x in lf.paged_attention(*p)] for p in problems]
    status()
    graphs = []
    for p in problems[:2] + problems[1:]:
        s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(g, stream=s):
            for _ in range(3):
                out = lf.paged_attention(*p)
        graphs.append((s, g, out))
    third = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        for s, g, out in graphs:
            with torch.cuda.stream(s):
                g.replay()
        eager = [lf.paged_attention(*problems[0], stream=third) for _ in range(2)]
        torch.cuda.synchronize()
        for (_, _, out), i in zip(graphs, (0, 1, 1, 2)):
            assert torch.equal(bits(out[0]), bits(want[i][0])) and torch.equal(out[1], want[i][1])
        for out in eager:
            assert torch.equal(bits(out[0]), bits(want[0][0]))
    status()


def test_calls_back_to_back_over_changing_inputs():
    """Kernels that are set up while the one before them runs still read what it wrote."""
    Q, kc, vc, table, lengths = problem(nq=1, lengths=(900, 33, 1000), rows=1024)
    phase = lf.rotary_phase(64, device=DEV)
    K = torch.randn(3, 2, 1, 64, device=DEV).to(BF)
    starts = lengths - 1
    steps = 30
    out = [lf.paged_attention(lf.cache_append(K * (i + 1), K, kc, vc, table, starts, Q=Q * (i + 1), phase=phase), kc, vc,
                              table, lengths) for i in range(steps)]
    torch.cuda.synchronize()
    for i in range(steps):
        q = lf.cache_append(K * (i + 1), K, kc, vc, table, starts, Q=Q * (i + 1), phase=phase)
        torch.cuda.synchronize()
        O, lse = lf.paged_attention(q, kc, vc, table, lengths)
        torch.cuda.synchronize()
        assert torch.equal(bits(O), bits(out[i][0])) and torch.equal(lse, out[i][1])
    status()


@pytest.mark.parametrize("rows", [64, 5000])
def test_more_sequences_than_a_launch_takes(rows):
    r = np.random.default_rng(1)
    lengths = [int(x) for x in r.integers(0, 60, 1100)]
    Q, kc, vc, table, k_lengths = problem(b=1100, hq=2, hk=1, d=40, page=8, lengths=lengths, rows=rows)
    tree = paged.ancestors(random_tree(1100, 3, seed=2).numpy())
    for nq in (1, 3):
        q = Q.expand(-1, -1, nq, -1).contiguous()
        q_lengths = ints([min(nq, x) if i % 7 else 0 for i, x in enumerate(lengths)], DEV)
        O, lse = lf.paged_attention(q, kc, vc, table, k_lengths, q_lengths=q_lengths)
        status()
        near(O, lse, q, kc, vc, table, k_lengths, causal=True, q_lengths=q_lengths.tolist())
    O, lse = lf.tree_attention(q, kc, vc, table, k_lengths, torch.from_numpy(paged.words(tree)).to(DEV), q_lengths=q_lengths)
    status()
    near(O, lse, q, kc, vc, table, k_lengths, tree=tree, q_lengths=q_lengths.tolist())


@pytest.mark.parametrize("nq", [1, 7, 130])
@pytest.mark.parametrize("rows", [1000, 20000])
def test_strided_queries_and_outputs_within_guards(nq, rows):
    """Queries that are a slice of a fused projection, an output that is one of a larger buffer: nothing
    beside it is written."""
    _, kc, vc, table, lengths = problem(nq=nq, lengths=(700, 0, 990), rows=rows)
    b, hq, d = 3, 8, 64
    fused = torch.randn(b, nq, (hq + 4) * d, device=DEV).to(BF)
    Q = fused[:, :, 2 * d:(2 + hq) * d].view(b, nq, hq, d).transpose(1, 2)
    around = torch.full((b, nq + 2, hq + 2, d), 5.0, dtype=BF, device=DEV)
    out = around[:, 1:nq + 1, 1:hq + 1].transpose(1, 2)
    lse_around = torch.full((b * hq * nq + 16,), 5.0, device=DEV)
    lse = lse_around[8:8 + b * hq * nq].view(b, hq, nq)
    got = lf.paged_attention(Q, kc, vc, table, lengths, out=out, lse=lse)
    status()
    assert got[0] is out
    near(out, lse, Q, kc, vc, table, lengths, causal=True)
    inner = torch.zeros_like(around, dtype=torch.bool)
    inner[:, 1:nq + 1, 1:hq + 1] = True
    assert (around[~inner] == 5.0).all() and (lse_around[:8] == 5.0).all() and (lse_around[8 + b * hq * nq:] == 5.0).all()


@pytest.mark.parametrize("nq,hq,d", [(1, 8, 64), (5, 8, 128), (16, 8, 40), (40, 4, 64), (80, 8, 64), (300, 4, 128)])
def test_workspace_guards(monkeypatch, nq, hq, d):
    monkeypatch.setenv("LINFORMER_WORKSPACE_GUARD", "1")
    for lengths in ((3000, 500, 4100), (9000, 0, 1), (100, 90, 128)):
        p = problem(nq=nq, hq=hq, d=d, lengths=lengths)
        O, lse = lf.paged_attention(*p)
        status()
        near(O, lse, *p, causal=True)


def test_no_memory_to_be_had(monkeypatch):
    monkeypatch.setenv("LINFORMER_FAIL_ALLOC", "1")
    for nq in (1, 80):
        p = problem(nq=nq)
        out, lse = torch.full_like(p[0], 3.0), torch.full(p[0].shape[:3], 3.0, device=DEV)
        launches = lf.linformer_launch_count()
        with pytest.raises(lf.LinformerError) as e:
            lf.paged_attention(*p, out=out, lse=lse)
        assert e.value.status == -7 and lf.linformer_launch_count() == launches
        torch.cuda.synchronize()
        assert (out == 3.0).all() and (lse == 3.0).all()
    status()


def test_kernels_are_counted():
    f = calls()
    torch.cuda.synchronize()
    lf.linformer_profile_enable(True)
    try:
        for name in NAMES:
            f[name]()
        torch.cuda.synchronize()
        seen = lf.linformer_profile_collect()
    finally:
        lf.linformer_profile_enable(False)
    assert seen["cache_kernels"][1] == 2 and seen["paged_attention_kernels"][1] == 6
    status()


@pytest.mark.parametrize("dense", [False, True])
def test_the_librarys_calls_one_argument_each(dense):
    """The entry points themselves, which the binding reaches with its arguments in one block."""
    import ctypes
    L = lf.lib()
    Q, kc, vc, table, lengths = problem(nq=20)
    if dense:
        kc, vc = kc.contiguous(), vc.contiguous()
    b, hq, hk, n, d, page, width = 3, 8, 2, 20, 64, 16, table.shape[1]
    K, V = (torch.randn(b, hk, n, d, device=DEV).to(BF) for _ in range(2))
    starts, counts, phase = ints([600, 3, 1400], DEV), ints([20, 0, 7], DEV), lf.rotary_phase(d, device=DEV)
    up = random_tree(3, n, seed=4)
    mask, path = lf.tree_mask(up.to(DEV)), ints([[0, 3, 9]] * 3, DEV)

    def strides(x):
        return None if dense else ctypes.addressof(keep_alive.setdefault(id(x), (ctypes.c_int64 * 3)(*x.stride()[:3])))
    keep_alive = {}

    def run(own):
        k, v = kc.clone(), vc.clone()
        out, lse, turned = torch.empty_like(Q), torch.empty(b, hq, n, device=DEV), torch.empty_like(Q)
        out2, lse2 = torch.empty_like(Q), torch.empty_like(lse)
        stream = torch.cuda.current_stream().cuda_stream
        pages = k.shape[0]
        if own:
            cache_args = [k.data_ptr(), strides(k), v.data_ptr(), strides(v)]
            assert L.linformer_cache_append(
                K.data_ptr(), None, V.data_ptr(), None, *cache_args, Q.data_ptr(), None, turned.data_ptr(), None,
                table.data_ptr(), starts.data_ptr(), counts.data_ptr(), phase.data_ptr(), None, b, hq, hk, n, d, pages,
                page, width, 32, 1, 1.25, 1, stream) == 0
            head = [turned.data_ptr(), None, *cache_args]
            tail = [b, hq, hk, n, d, pages, page, width, 0.2]
            assert L.linformer_paged_attn_fwd(
                *head, out.data_ptr(), None, lse.data_ptr(), table.data_ptr(), lengths.data_ptr(), counts.data_ptr(),
                *tail, 1, 50, 1, stream) == 0
            assert L.linformer_tree_attn_fwd(
                *head, out2.data_ptr(), None, lse2.data_ptr(), table.data_ptr(), lengths.data_ptr(), None,
                mask.data_ptr(), *tail, 1, stream) == 0
            assert L.linformer_cache_keep(
                *cache_args, table.data_ptr(), starts.data_ptr(), path.data_ptr(), counts.data_ptr(), b, hk, 3, d,
                pages, page, width, 1, stream) == 0
        else:
            lf.cache_append(K, V, k, v, table, starts, counts=counts, Q=Q, phase=phase_words(32), rot=32,
                            layout=lf.ROTARY_INTERLEAVED, amplitude=1.25, out=turned)
            lf.paged_attention(turned, k, v, table, lengths, q_lengths=counts, window=50, scale=0.2, out=out, lse=lse)
            lf.tree_attention(turned, k, v, table, lengths, mask, scale=0.2, out=out2, lse=lse2)
            lf.cache_keep(k, v, table, starts, path, counts=counts)
        status()
        return k, v, turned, out, out2, lse, lse2

    def phase_words(rot):
        return phase[:rot // 2].contiguous()
    for x, y in zip(run(True), run(False)):
        assert torch.equal(bits(x), bits(y))


@pytest.mark.parametrize("nq", [1, 80])
def test_dimensions_of_one_entry_may_have_any_stride(nq):
    """Their strides are never used: those that views leave there are no multiples of anything."""
    Q, kc, vc, table, lengths = problem(b=1, hq=4, hk=1, nq=nq, lengths=(500,))
    phase, K = lf.rotary_phase(64, device=DEV), torch.randn(1, 1, 1, 64, device=DEV).to(BF)

    def odd(x):
        return x.as_strided(x.shape, [s if n > 1 or i == 3 else 5 - 5 * (i == 1)
                                      for i, (n, s) in enumerate(zip(x.shape, x.stride()))])
    got = []
    for view in (lambda x: x, odd):
        k, v, q, x = kc.clone(), vc.clone(), Q.clone(), K.clone()
        turned = lf.cache_append(view(x), view(x), view(k), view(v), table, ints([499], DEV),
                                 Q=view(q[:, :, :1].contiguous()), phase=phase)
        out = lf.paged_attention(view(q), view(k), view(v), table, lengths, out=view(torch.empty_like(q)))
        lf.cache_keep(view(k), view(v), table, ints([490], DEV), ints([[0, 4]], DEV))
        status()
        got.append((turned, *out, k, v))
    for a, b in zip(*got):
        assert torch.equal(bits(a), bits(b))
