"""GPU tests of the exact softmax attention (linformer_softmax_attn_fwd / _bwd through the
Python binding) against the fp64 oracle, elementwise within the oracle's derived bounds, and
within 5e-3 in the 2-norm: three independent roundings of relative size at most 2^-8, rms
2^-8 / sqrt(3), give sqrt(3) x 2^-8 / sqrt(3) = 3.9e-3, and the fp32 part is below 1e-3.
The rounding of O that delta = dO.O takes over is one error for a whole row of dS, which sums
over the keys do not average out: its bound is allowed on top."""
import numpy as np
import pytest
import torch

import rank_linear_complexity_gb300.linformer as lf
from oracle import softmax_attention as orc

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF = torch.bfloat16


def tensors(b, hq, hk, nq, nk, d, seed=0, gain=1.5, packed=False):
    """Q, K, V, dO on the device; packed: Q, K and V as slices of one fused buffer."""
    g = torch.Generator().manual_seed(seed)

    def rand(h, n, s):
        return (torch.randn(b, h, n, d, generator=g) * s).to(BF)

    Q, K, V, dO = rand(hq, nq, gain), rand(hk, nk, gain), rand(hk, nk, 1), rand(hq, nq, 1)
    if packed:
        buf = torch.full((b, nq, (hq + 2 * hk) * d), float("nan"), dtype=BF, device=DEV)
        views, at = [], 0
        for x in (Q, K, V):
            h = x.shape[1]
            v = buf[:, :, at:at + h * d].view(b, nq, h, d).transpose(1, 2)
            v.copy_(x)
            views.append(v)
            at += h * d
        wide = torch.empty(b, nq, hq, d, dtype=BF, device=DEV).transpose(1, 2)
        return (*views, wide.copy_(dO))
    return tuple(x.to(DEV) for x in (Q, K, V, dO))


def lengths(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV)


def status():
    torch.cuda.synchronize()
    assert lf.linformer_debug_read_device_status() == 0


def within(got, ref, bound, name, rows=None):
    got, bad = orc.host64(got), np.isinf(ref)
    assert np.array_equal(got[bad], ref[bad]), name
    err = np.abs(np.where(bad, 0, got) - np.where(bad, 0, ref))
    assert np.isfinite(err).all(), f"{name}: not finite"
    over = err > bound
    assert not over.any(), f"{name}: {over.sum()} over, worst {(err - bound).max()} at " \
                           f"{np.unravel_index((err - bound).argmax(), err.shape)}"
    if ref.size >= 4096 and np.linalg.norm(ref[~bad]) > 0:
        rel = np.linalg.norm(err[~bad]) / np.linalg.norm(ref[~bad])
        extra = 0 if rows is None else np.linalg.norm(rows) / np.linalg.norm(ref)
        assert rel <= 5e-3 + extra, f"{name}: 2-norm {rel}"


CASES = {
    # name: b, hq, hk, nq, nk, d, options
    "one": (1, 1, 1, 1, 1, 64, {}),
    "prompt": (2, 4, 2, 77, 77, 64, dict(causal=True, packed=True)),
    "cross": (1, 3, 3, 130, 201, 40, {}),
    "token": (2, 8, 2, 1, 1000, 128, dict(k=[1000, 0])),
    "tokens_causal": (1, 8, 1, 5, 515, 96, dict(causal=True)),
    "window": (2, 2, 2, 300, 300, 128, dict(causal=True, window=100)),
    "ragged_empty_rows": (3, 6, 3, 257, 129, 80, dict(causal=True, q=[257, 30, 129],
                                                      k=[129, 77, 1])),
    "odd_group": (1, 5, 1, 200, 384, 64, {}),
    "token_split": (1, 2, 2, 1, 9000, 64, {}),
    "encoder": (2, 12, 12, 640, 640, 64, dict(q=[640, 161], k=[640, 161])),
    "tokens_window_split": (1, 16, 2, 3, 4000, 128, dict(causal=True, window=700)),
    "many_items": (6, 16, 8, 384, 384, 128, dict(causal=True, packed=True)),
    "many_short": (40, 6, 3, 100, 140, 64, dict(q=list(range(0, 100, 5)) * 2,
                                                k=list(range(7, 127, 3)))),
    "smallest_head": (2, 2, 1, 150, 150, 8, dict(causal=True)),
    "ends_in_tile": (2, 1, 1, 256, 256, 128, dict(q=[128, 129], k=[128, 129])),
}


def options(o):
    kw = dict(causal=o.get("causal", False), window=o.get("window", 0))
    return kw, o.get("q"), o.get("k")


def poison(Q, K, V, dO, q, k):
    """Rows past the lengths hold NaN."""
    for bi in range(Q.shape[0]):
        if q is not None:
            Q[bi, :, q[bi]:] = float("nan")
            dO[bi, :, q[bi]:] = float("nan")
        if k is not None:
            K[bi, :, k[bi]:] = float("nan")
            V[bi, :, k[bi]:] = float("nan")


@pytest.mark.parametrize("name", CASES)
def test_forward(name):
    b, hq, hk, nq, nk, d, o = CASES[name]
    kw, q, k = options(o)
    Q, K, V, dO = tensors(b, hq, hk, nq, nk, d, seed=nq + nk, packed=o.get("packed", False))
    poison(Q, K, V, dO, q, k)
    O, lse = lf.softmax_attention(Q, K, V, lengths(q), lengths(k), **kw)
    status()
    ref, rl, bO, bl = orc.forward(Q, K, V, q, k, **kw)
    within(O, ref, bO, "O")
    within(lse, rl, bl, "lse")


@pytest.mark.parametrize("name", CASES)
def test_backward(name):
    b, hq, hk, nq, nk, d, o = CASES[name]
    kw, q, k = options(o)
    Q, K, V, dO = tensors(b, hq, hk, nq, nk, d, seed=nq + nk + 1, packed=o.get("packed", False))
    poison(Q, K, V, dO, q, k)
    ref, rl, _, _ = orc.forward(Q, K, V, q, k, **kw)
    O = torch.from_numpy(ref).to(DEV, BF)
    lse = torch.from_numpy(rl).to(DEV, torch.float32)
    if q is not None:
        for bi in range(b):
            O[bi, :, q[bi]:] = float("nan")
    got = lf.softmax_attention_backward(Q, K, V, O, dO, lse, lengths(q), lengths(k), **kw)
    status()
    refs, bounds, rows = orc.backward(Q, K, V, dO, q, k, **kw)
    for n, g, r, e, w in zip(("dQ", "dK", "dV"), got, refs, bounds, rows):
        within(g, r, e, n, w)


MORE = {  # steps of 64: heads of one step, lengths that end in a step or on its edge, many of each
    "one_step_heads": (2, 24, 2, 40, 300, 64, dict(q=[33, 7], k=[300, 129])),
    "one_step_heads_wide": (2, 24, 2, 40, 300, 128, dict(q=[33, 7], k=[300, 129])),
    "two_step_heads": (3, 14, 2, 100, 70, 72, dict(q=[100, 64, 65], k=[70, 64, 65])),
    "step_edges": (3, 4, 2, 192, 192, 64, dict(causal=True, q=[192, 65, 64], k=[192, 65, 64])),
    "step_edges_wide": (3, 4, 2, 192, 192, 128, dict(causal=True, q=[191, 63, 1], k=[191, 63, 1])),
    "window_of_a_step": (1, 6, 3, 200, 330, 64, dict(causal=True, window=65, q=[131])),
    "long_ring": (1, 3, 1, 200, 2000, 128, dict(k=[1985])),
    # few items with many steps: split into parts
    "few_keys": (2, 16, 2, 600, 46, 96, dict(q=[600, 155])),
    "few_keys_causal": (1, 8, 1, 1100, 200, 64, dict(causal=True, q=[1090], k=[170])),
    "few_queries": (1, 4, 2, 40, 5000, 64, dict(k=[4990])),
    "few_queries_window": (2, 2, 1, 300, 5000, 128, dict(causal=True, window=3500, q=[300, 7], k=[5000, 200])),
    "few_keys_none": (3, 8, 2, 700, 40, 64, dict(q=[700, 0, 1], k=[0, 40, 40])),
    "few_queries_none": (3, 2, 1, 30, 4500, 64, dict(causal=True, q=[0, 30, 29], k=[4500, 0, 4437])),
    "long_ring_of_queries": (1, 12, 1, 700, 70, 64, dict(q=[650])),
}


@pytest.mark.parametrize("name", MORE)
def test_steps_and_their_edges(name):
    CASES[name] = MORE[name]
    test_forward(name)
    test_backward(name)


# --- ways of calling ----------------------------------------------------------------------

def same(a, b):
    return all(torch.equal(x.view(torch.int16), y.view(torch.int16)) if x.dtype == BF
               else torch.equal(x.view(torch.int32), y.view(torch.int32)) for x, y in zip(a, b))


def test_results_repeat_bit_for_bit():
    Q, K, V, dO = tensors(2, 8, 2, 500, 700, 128, seed=3)
    O, lse = lf.softmax_attention(Q, K, V)
    g = lf.softmax_attention_backward(Q, K, V, O, dO, lse)
    for _ in range(5):
        assert same(lf.softmax_attention(Q, K, V), (O, lse))
        assert same(lf.softmax_attention_backward(Q, K, V, O, dO, lse), g)
    status()


@pytest.mark.parametrize("nq,nk,causal", [(300, 2048, False), (2048, 300, False), (2048, 2048, True)])
def test_heads_in_sets(nq, nk, causal):
    """A batch that streams more than L2 holds (its heads are taken in sets) gives each entry what
    halves of it (which are not) give."""
    b, h, d = 17, 16, 64
    g = torch.Generator(device=DEV).manual_seed(nq)
    Q, K, V, dO = (torch.randn(b, h, n, d, generator=g, device=DEV).to(BF) for n in (nq, nk, nk, nq))
    q = torch.randint(1, nq + 1, (b,), generator=g, device=DEV, dtype=torch.int32)
    k = torch.randint(1, nk + 1, (b,), generator=g, device=DEV, dtype=torch.int32)

    def run(at):
        x = [t[at].contiguous() for t in (Q, K, V, dO, q, k)]
        O, lse = lf.softmax_attention(*x[:3], *x[4:], causal=causal)
        return (O, lse, *lf.softmax_attention_backward(*x[:3], O, x[3], lse, *x[4:], causal=causal))

    whole, halves = run(slice(0, b)), [run(slice(0, 8)), run(slice(8, b))]
    status()
    assert same(whole, [torch.cat(x) for x in zip(*halves)])


def test_wide_heads_in_sets_from_the_counter():
    """The same for heads of 128 under a causal mask with ragged lengths, twice."""
    b, h, n, d = 9, 16, 2048, 128
    g = torch.Generator(device=DEV).manual_seed(128)
    x = [torch.randn(b, h, n, d, generator=g, device=DEV).to(BF) for _ in range(4)]
    x += [torch.randint(1, n + 1, (b,), generator=g, device=DEV, dtype=torch.int32) for _ in range(2)]

    def run(at):
        Q, K, V, dO, q, k = (t[at].contiguous() for t in x)
        O, lse = lf.softmax_attention(Q, K, V, q, k, causal=True)
        return (O, lse, *lf.softmax_attention_backward(Q, K, V, O, dO, lse, q, k, causal=True))

    halves = [run(slice(0, 4)), run(slice(4, b))]
    for _ in range(2):
        assert same(run(slice(0, b)), [torch.cat(t) for t in zip(*halves)])
    status()


def test_outputs_only_where_they_belong():
    """Slices of wider buffers (rows, heads, columns around them untouched), lse in a longer one."""
    b, hq, hk, n, d = 2, 4, 2, 150, 64
    Q, K, V, dO = tensors(b, hq, hk, n, n, d, seed=5)
    kw = dict(causal=True, q_lengths=lengths([150, 77]), k_lengths=lengths([150, 77]))

    def room(h):
        return torch.full((b, h + 2, n + 3, d + 16), 7.0, dtype=BF, device=DEV)

    def inner(x):
        return x[:, 1:-1, 1:-2, 8:-8]

    O0, lse0 = lf.softmax_attention(Q, K, V, **kw)
    g0 = lf.softmax_attention_backward(Q, K, V, O0, dO, lse0, **kw)
    R = [room(hq), room(hq), room(hk), room(hk)]
    ends = torch.full((b * hq * n + 64,), 7.0, device=DEV)
    lse = ends[32:-32].view(b, hq, n)
    O, _ = lf.softmax_attention(Q, K, V, out=inner(R[0]), lse=lse, **kw)
    g = lf.softmax_attention_backward(Q, K, V, O, dO, lse, dQ=inner(R[1]), dK=inner(R[2]),
                                      dV=inner(R[3]), **kw)
    status()
    assert same((O, lse, *g), (O0, lse0, *g0))
    for x in R:
        inner(x).fill_(7.0)
        assert (x == 7.0).all()
    assert (ends[:32] == 7).all() and (ends[-32:] == 7).all()


def test_large_logits_after_small_ones():
    """A row's later blocks outgrow its first by more than fp32 holds; also the reverse."""
    for flip in (False, True):
        Q, K, V, dO = tensors(1, 2, 1, 200, 640, 64, seed=7, gain=1)
        ramp = torch.linspace(0.01, 40, 640, device=DEV)
        K.mul_((ramp.flip(0) if flip else ramp)[:, None].to(BF))
        O, lse = lf.softmax_attention(Q, K, V, scale=1.0)
        status()
        ref, rl, bO, bl = orc.forward(Q, K, V, scale=1.0)
        within(O, ref, bO, f"O {flip}")
        within(lse, rl, bl, f"lse {flip}")


def test_gradient_against_differences():
    """The kernel's gradients against central differences of the oracle's loss in a random
    direction.  With f = sum(O dO), |f' - difference| is below the gradients' own bounds times
    the direction, plus the difference's truncation: h^2 / 6 f''' with h = 1e-4, below 1e-6 of
    the gradient here."""
    b, hq, hk, n, d = 1, 4, 2, 90, 64
    Q, K, V, dO = tensors(b, hq, hk, n, n, d, seed=11, gain=1)
    kw = dict(causal=True)
    ref = orc.forward(Q, K, V, **kw)
    O, lse = torch.from_numpy(ref[0]).to(DEV, BF), torch.from_numpy(ref[1]).to(DEV, torch.float32)
    got = lf.softmax_attention_backward(Q, K, V, O, dO, lse, **kw)
    status()
    refs, bounds, _ = orc.backward(Q, K, V, dO, **kw)
    rng = np.random.default_rng(1)
    x = [orc.host64(t) for t in (Q, K, V)]
    g64 = orc.host64(dO)
    for i in range(3):
        D = rng.standard_normal(x[i].shape)
        h = 1e-4
        f = []
        for s in (h, -h):
            y = list(x)
            y[i] = x[i] + s * D
            f.append((orc.forward(*y, **kw)[0] * g64).sum())
        slope = (f[0] - f[1]) / (2 * h)
        mine = (orc.host64(got[i]) * D).sum()
        allowed = (bounds[i] * np.abs(D)).sum() + 1e-6 * np.abs(refs[i] * D).sum()
        assert abs(mine - slope) <= allowed, (i, mine, slope, allowed)


def test_two_streams_at_once():
    sets = [tensors(2, 8, 2, 300 + 7 * i, 500, 64, seed=20 + i) for i in range(2)]
    alone = []
    for Q, K, V, dO in sets:
        O, lse = lf.softmax_attention(Q, K, V)
        alone.append((O, lse, *lf.softmax_attention_backward(Q, K, V, O, dO, lse)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        got = []
        for (Q, K, V, dO), s in zip(sets, streams):
            with torch.cuda.stream(s):
                O, lse = lf.softmax_attention(Q, K, V)
                got.append((O, lse, *lf.softmax_attention_backward(Q, K, V, O, dO, lse)))
        torch.cuda.synchronize()
        assert all(same(x, y) for x, y in zip(got, alone))
    s = streams[0]   # a stream given as an argument, from another current one
    s.wait_stream(torch.cuda.current_stream())
    Q, K, V, _ = sets[0]
    got = lf.softmax_attention(Q, K, V, stream=s)
    s.synchronize()
    assert same(got, alone[0][:2])
    status()


@pytest.mark.parametrize("nq,nk", [(260, 260), (1, 5000)])
def test_captured_and_replayed(nq, nk):
    """Two graphs with forward and backward (and the split forward's workspace) replayed in
    turn, and once with inputs rewritten, give what eager calls give."""
    data = [tensors(2, 4, 2, nq, nk, 128, seed=30 + i) for i in range(2)]
    new = tensors(2, 4, 2, nq, nk, 128, seed=40)

    def step(Q, K, V, dO):
        O, lse = lf.softmax_attention(Q, K, V, causal=True)
        return (O, lse, *lf.softmax_attention_backward(Q, K, V, O, dO, lse, causal=True))

    eager = [step(*x) for x in data]
    eager_new = step(*new)
    torch.cuda.synchronize()
    graphs = []
    for x in data:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step(*x)
        graphs.append((g, out))
    for _ in range(3):
        for g, _ in graphs:
            g.replay()
    torch.cuda.synchronize()
    assert all(same(out, e) for (_, out), e in zip(graphs, eager))
    for dst, src in zip(data[0], new):
        dst.copy_(src)
    graphs[0][0].replay()
    torch.cuda.synchronize()
    assert same(graphs[0][1], eager_new)
    status()


def test_workspace_stays_in_its_bounds(monkeypatch):
    """Guard bytes behind the workspaces of a split forward and of a backward."""
    monkeypatch.setenv("LINFORMER_WORKSPACE_GUARD", "1")
    Q, K, V, dO = tensors(3, 4, 1, 3, 4000, 96, seed=50)
    O, lse = lf.softmax_attention(Q, K, V)
    lf.softmax_attention_backward(Q, K, V, O, dO, lse)
    status()


def test_failed_allocation_is_reported(monkeypatch):
    Q, K, V, dO = tensors(1, 2, 1, 64, 64, 64, seed=51)
    O, lse = lf.softmax_attention(Q, K, V)
    monkeypatch.setenv("LINFORMER_FAIL_ALLOC", "1")
    with pytest.raises(lf.LinformerError) as e:
        lf.softmax_attention_backward(Q, K, V, O, dO, lse)
    assert e.value.status == -7
    monkeypatch.delenv("LINFORMER_FAIL_ALLOC")
    lf.softmax_attention_backward(Q, K, V, O, dO, lse)
    status()


def test_long_cache_offsets():
    """One token over a cache whose last head starts beyond 2^31 elements (the other heads are
    a stride away, not memory that is read): 2.3 GB of K and of V, the head checked is real."""
    n, d, heads = 70000, 128, 2
    stride = (1 << 31) // 2 // d * d + d * 64
    buf = torch.empty(stride + n * d, dtype=BF, device=DEV)
    K = torch.as_strided(buf, (1, heads, n, d), (heads * stride, stride, d, 1))
    g = torch.Generator(device=DEV).manual_seed(9)
    for h in range(heads):
        K[0, h] = torch.randn(n, d, generator=g, device=DEV).to(BF)
    Q = torch.randn(1, heads, 1, d, generator=g, device=DEV).to(BF)
    O, lse = lf.softmax_attention(Q, K, K)
    status()
    ref, rl, bO, bl = orc.forward(Q, K, K)
    within(O, ref, bO, "O")
    within(lse, rl, bl, "lse")


def test_as_the_linformer_core():
    """Queries over the projected keys and values (nk = k): the attention step of the Linformer
    forward, with Kbar and Vbar from linformer_project_fwd rounded to bf16."""
    from rank_linear_complexity_gb300.workloads import BF16, HEADWISE, make_inputs
    b, h, n, d, k = 2, 3, 384, 64, 128
    x = make_inputs(b, h, n, d, k, HEADWISE, BF16, seed=60)
    g = {kk: (v.to(DEV) if v is not None else None) for kk, v in x.items()}
    Kb, Vb = lf.projection(g["K"], g["V"], g["E"], g["F"], None, HEADWISE)
    Kb, Vb = Kb.to(BF), Vb.to(BF)
    O, lse = lf.softmax_attention(g["Q"], Kb, Vb)
    status()
    ref, rl, bO, bl = orc.forward(g["Q"], Kb, Vb)
    within(O, ref, bO, "O")
    within(lse, rl, bl, "lse")
