"""Cases for measuring the transformer operators next to the Linformer attention: rotary
positions, exact softmax attention and its backward pass.

``own`` selects what ``run`` does: False computes each operator in a plain form
(elementary torch operations in 32 bits, angles in 64), True calls this package.

Ranges: head dimensions 8 to 128, 1 to 32 query heads on as many or fewer key/value heads,
1 to 16384 rows, dense [b][h][n][d] tensors and slices of one fused [b][n][(hq + 2 hk) d]
projection, full, causal, windowed and ragged batches.
"""
import math

import numpy as np
import torch

own = False

BASE = 10000.0       # rotary base
LONG_FACTOR = 8.0    # context extension of the scaled rotary cases
LONG_ORIGINAL = 8192
BETA_FAST, BETA_SLOW = 32.0, 1.0
QK_GAIN = 1.5        # sd of Q and K: logits of a trained model are wider than N(0, 1)


def _rotary(name, b, hq, hk, n, d, rot, **kw):
    c = dict(name=name, op="rotary", b=b, hq=hq, hk=hk, n=n, d=d, rot=rot, dtype="bf16",
             interleaved=False, scaled=False, inverse=False, packed=False, far=n)
    c.update(kw)
    return c


def _attention(name, op, b, hq, hk, nq, nk, d, **kw):
    c = dict(name=name, op=op, b=b, hq=hq, hk=hk, nq=nq, nk=nk, d=d, causal=False, window=0,
             ragged=False, packed=False)
    c.update(kw)
    return c


def listed():
    return [
        # one new token for each of 64 sequences, far into an extended context
        _rotary("rotary_token", 64, 32, 8, 1, 128, 128, scaled=True, far=65536),
        # fp32, neighbouring pairs, half of each head, an odd length
        _rotary("rotary_part_f32", 2, 12, 12, 4095, 64, 32, dtype="f32", interleaved=True),
        # the gradient through the positions of a long training batch, fused projection
        _rotary("rotary_back_long", 4, 16, 16, 16384, 64, 64, inverse=True, packed=True),
        # one new token against caches of differing lengths
        _attention("attend_token", "attend", 32, 32, 8, 1, 8192, 128, ragged=True),
        # a short prompt
        _attention("attend_short", "attend", 2, 4, 4, 77, 77, 64, causal=True, packed=True),
        # n = 4096 with 12 heads of 64, the sequence length and heads of the Linformer headline
        _attention("attend_4096", "attend", 16, 12, 12, 4096, 4096, 64),
        # a causal layer with shared key/value heads of 128
        _attention("attend_causal_8192", "attend", 2, 32, 8, 8192, 8192, 128, causal=True,
                   packed=True),
        # a sliding window over a long odd sequence
        _attention("attend_window", "attend", 1, 16, 2, 16383, 16383, 128, causal=True,
                   window=2048),
        # a small ragged cross-attention with an uncommon head size
        _attention("back_small", "backward", 3, 6, 3, 130, 201, 40, ragged=True),
        # n = 512 with 12 heads: the ragged encoder batch
        _attention("back_512", "backward", 32, 12, 12, 512, 512, 64, ragged=True),
        # n = 4096 with 12 heads of 64
        _attention("back_4096", "backward", 16, 12, 12, 4096, 4096, 64),
        # the causal layer's gradient, shared key/value heads, an odd length
        _attention("back_causal_8191", "backward", 1, 32, 8, 8191, 8191, 128, causal=True,
                   packed=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rotary", "attend", "backward"))
    limit = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        hk = rng.choice((1, 2, 3, 4, 8, 12))
        hq = hk * rng.choice((1, 1, 2, 4, 8))
        b = _log_int(rng, 1, 64)
        packed = rng.random() < 0.5
        if op == "rotary":
            n = 1 if rng.random() < 0.25 else _log_int(rng, 2, 16384)
            d = rng.choice((32, 64, 80, 96, 128))
            rot = rng.choice((d, d, d // 2))
            c = _rotary("", b, hq, hk, n, d, rot, dtype=rng.choice(("bf16", "bf16", "f32")),
                        interleaved=rng.random() < 0.4, scaled=rng.random() < 0.5,
                        inverse=rng.random() < 0.5, packed=packed,
                        far=max(n, _log_int(rng, 1024, 131072)))
        else:
            d = rng.choice((40, 64, 64, 80, 96, 128, 128))
            nk = _log_int(rng, 1 if op == "attend" else 32, 16384)
            kind = rng.random()
            if op == "attend" and kind < 0.3:
                nq = rng.choice((1, 1, 2, 5))      # new tokens over a cache
            elif kind < 0.5:
                nq = _log_int(rng, 1, 16384)       # cross-attention
            else:
                nq = nk
            causal = rng.random() < 0.5
            window = _log_int(rng, 16, 4096) if causal and rng.random() < 0.3 else 0
            c = _attention("", op, b, hq, hk, nq, nk, d, causal=causal, window=window,
                           ragged=rng.random() < 0.4, packed=packed and nq == nk)
        if _cost(c) <= limit and hq <= 32:
            del c["name"]
            return c


def _cost(c):
    w = work(c)
    if c["op"] == "rotary":
        return w["bytes"]
    # the plain form holds scores of every pair, masked or not
    return c["b"] * c["hq"] * c["nq"] * c["nk"] * max(c["d"], 64) + 64 * w["bytes"]


def _spread(n, b):
    """Lengths of a ragged batch: evenly spaced from n down to about a quarter of it."""
    return [max(1, n - (3 * n * i) // (4 * b)) for i in range(b)]


def _pairs(c):
    """Query/key pairs that the masks leave, over the batch (one head)."""
    total = 0
    b, nq, nk = c["b"], c["nq"], c["nk"]
    for lq, lk in zip(_spread(nq, b), _spread(nk, b)) if c["ragged"] else [(nq, nk)] * b:
        if not c["causal"]:
            total += lq * lk
            continue
        pos = np.arange(lq, dtype=np.int64) + (lk - lq)
        first = np.maximum(pos - c["window"] + 1, 0) if c["window"] else 0
        total += int(np.maximum(pos + 1 - first, 0).sum())
    return total


def work(case):
    c = case
    if c["op"] == "rotary":
        e = 4 if c["dtype"] == "f32" else 2
        x = c["b"] * (c["hq"] + c["hk"]) * c["n"] * c["d"]
        return {"bytes": 2.0 * e * x + 4 * c["b"] * c["n"],
                "flops": 3.0 * c["b"] * (c["hq"] + c["hk"]) * c["n"] * c["rot"]}
    b = c["b"]
    rows_q = sum(_spread(c["nq"], b)) if c["ragged"] else b * c["nq"]
    rows_k = sum(_spread(c["nk"], b)) if c["ragged"] else b * c["nk"]
    all_q, all_k = b * c["nq"] * c["hq"] * c["d"], b * c["nk"] * c["hk"] * c["d"]
    q, k = rows_q * c["hq"] * c["d"], rows_k * c["hk"] * c["d"]
    lse = 4 * b * c["nq"] * c["hq"]
    pairs = _pairs(c) * c["hq"]
    if c["op"] == "attend":
        return {"bytes": 2.0 * (q + 2 * k + all_q) + lse, "flops": 4.0 * pairs * c["d"]}
    # reads Q, K, V, O, dO and lse, writes dQ, dK, dV
    return {"bytes": 2.0 * (3 * q + 2 * k + all_q + 2 * all_k) + lse,
            "flops": 10.0 * pairs * c["d"]}


# --- inputs -----------------------------------------------------------------------------

def _heads(g, b, n, heads, d, dtype, packed, gains):
    """Tensors [b][h][n][d] for each entry of heads: dense, or slices of one fused buffer."""
    if packed:
        buf = torch.empty(b, n, sum(heads) * d, dtype=dtype, device="cuda")
        views, at = [], 0
        for h in heads:
            views.append(buf[:, :, at:at + h * d].view(b, n, h, d).transpose(1, 2))
            at += h * d
    else:
        views = [torch.empty(b, h, n, d, dtype=dtype, device="cuda") for h in heads]
    for v, gain in zip(views, gains):
        v.copy_(torch.randn(v.shape, generator=g, device="cuda", dtype=torch.float32) * gain)
    return views


def _like_output(c, n, h):
    """An output buffer as the surrounding program lays it out."""
    if c["packed"]:
        return torch.empty(c["b"], n, h, c["d"], dtype=torch.bfloat16,
                           device="cuda").transpose(1, 2)
    return torch.empty(c["b"], h, n, c["d"], dtype=torch.bfloat16, device="cuda")


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    if c["op"] == "rotary":
        dtype = torch.float32 if c["dtype"] == "f32" else torch.bfloat16
        q, k = _heads(g, c["b"], c["n"], (c["hq"], c["hk"]), c["d"], dtype, c["packed"], (1, 1))
        start = torch.randint(0, c["far"] - c["n"] + 1, (c["b"], 1), generator=g, device="cuda")
        pos = (start + torch.arange(c["n"], device="cuda")).to(torch.int32)
        freq = _frequencies(c)
        return dict(c=c, q=q, k=k, pos=pos, freq=freq.cuda(),
                    phase=_phase_steps(freq).cuda(), amplitude=_amplitude(c))
    same = c["nq"] == c["nk"] and c["packed"]
    gains = (QK_GAIN, QK_GAIN, 1.0)
    if same:
        q, k, v = _heads(g, c["b"], c["nq"], (c["hq"], c["hk"], c["hk"]), c["d"], torch.bfloat16,
                         True, gains)
    else:
        q, = _heads(g, c["b"], c["nq"], (c["hq"],), c["d"], torch.bfloat16, False, gains)
        k, v = _heads(g, c["b"], c["nk"], (c["hk"], c["hk"]), c["d"], torch.bfloat16, False,
                      gains[1:])
    s = dict(c=c, q=q, k=k, v=v, q_lengths=None, k_lengths=None, scale=1 / math.sqrt(c["d"]))
    if c["ragged"]:
        order = torch.randperm(c["b"], generator=g, device="cuda")
        for key, n in (("q_lengths", c["nq"]), ("k_lengths", c["nk"])):
            s[key] = torch.tensor(_spread(n, c["b"]), dtype=torch.int32, device="cuda")[order]
    s["out"] = _like_output(c, c["nq"], c["hq"])
    s["lse"] = torch.empty(c["b"], c["hq"], c["nq"], device="cuda")
    if c["op"] == "backward":
        # what the forward pass left, and the gradient that arrives
        o, lse = _attend(s)
        s["o"], s["lse"] = s["out"].copy_(o), lse
        s["do"] = _like_output(c, c["nq"], c["hq"])
        s["do"].copy_(torch.randn(o.shape, generator=g, device="cuda") * 0.05)
        s["dq"], s["dk"], s["dv"] = (torch.empty_like(x) for x in (q, k, v))
        del s["out"]
    return s


def _frequencies(c):
    """Angle per position of each pair, radians, 64 bits."""
    f = BASE ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])
    if c["scaled"]:
        # pairs that turn often within the original context keep their frequency, slow ones
        # are stretched by the factor, those between are blended
        turns = LONG_ORIGINAL * f / (2 * math.pi)
        keep = ((turns - BETA_SLOW) / (BETA_FAST - BETA_SLOW)).clamp(0, 1)
        f = f * (keep + (1 - keep) / LONG_FACTOR)
    return f


def _phase_steps(freq):
    """The table that the package's rotary takes: turns per position as 64-bit fractions."""
    steps = [int(round(f / (2 * math.pi) * 2.0 ** 64)) % (1 << 64) for f in freq.tolist()]
    return torch.tensor([s - (1 << 64) if s >= 1 << 63 else s for s in steps], dtype=torch.int64)


def _amplitude(c):
    return 0.1 * math.log(LONG_FACTOR) + 1 if c["scaled"] else 1.0


# --- the plain forms --------------------------------------------------------------------

def _rotate(x, cos, sin, c):
    y = x.float().clone()
    r = c["rot"]
    if c["interleaved"]:
        even, odd = y[..., 0:r:2].clone(), y[..., 1:r:2].clone()
        y[..., 0:r:2], y[..., 1:r:2] = even * cos - odd * sin, odd * cos + even * sin
    else:
        low, high = y[..., :r // 2].clone(), y[..., r // 2:r].clone()
        y[..., :r // 2], y[..., r // 2:r] = low * cos - high * sin, high * cos + low * sin
    return y.to(x.dtype)


def _rotary_plain(s):
    c = s["c"]
    angle = s["pos"].double()[:, None, :, None] * s["freq"]
    if c["inverse"]:
        angle = -angle
    cos, sin = ((f(angle) * s["amplitude"]).float() for f in (torch.cos, torch.sin))
    return _rotate(s["q"], cos, sin, c), _rotate(s["k"], cos, sin, c)


def _mask(s):
    """True where a query sees a key, [b or 1][1][1][nq][nk], or None."""
    c = s["c"]
    if not c["causal"] and not c["ragged"]:
        return None
    dev = s["q"].device
    lq = s["q_lengths"] if c["ragged"] else torch.tensor([c["nq"]], device=dev)
    lk = s["k_lengths"] if c["ragged"] else torch.tensor([c["nk"]], device=dev)
    lq, lk = lq.view(-1, 1, 1), lk.view(-1, 1, 1)
    i = torch.arange(c["nq"], device=dev).view(1, -1, 1)
    j = torch.arange(c["nk"], device=dev).view(1, 1, -1)
    m = (i < lq) & (j < lk)
    if c["causal"]:
        m = m & (j <= i + (lk - lq))
        if c["window"]:
            m = m & (j > i + (lk - lq) - c["window"])
    return m[:, None, None]


def _scores(s):
    """Masked scores [b][hk][g][nq][nk] in 32 bits."""
    c = s["c"]
    g = c["hq"] // c["hk"]
    q = s["q"].float().reshape(c["b"], c["hk"], g * c["nq"], c["d"])
    x = q @ s["k"].float().transpose(-1, -2) * s["scale"]
    x = x.view(c["b"], c["hk"], g, c["nq"], c["nk"])
    mask = _mask(s)
    return x if mask is None else x.masked_fill(~mask, float("-inf"))


def _attend(s):
    c = s["c"]
    b, hq, nq, nk, d = c["b"], c["hq"], c["nq"], c["nk"], c["d"]
    x = _scores(s)
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    o = (p.view(b, c["hk"], -1, nk) @ s["v"].float()).view(b, c["hk"], -1, nq, d)
    o = o / torch.where(total == 0, torch.ones_like(total), total)
    lse = (top + torch.log(total)).view(b, hq, nq)
    return o.view(b, hq, nq, d).to(torch.bfloat16), lse


def _backward(s):
    c = s["c"]
    b, hk, nk, d = c["b"], c["hk"], c["nk"], c["d"]
    lse = s["lse"].view(b, hk, -1, c["nq"], 1)
    p = torch.exp(_scores(s) - torch.where(lse == float("-inf"), torch.zeros_like(lse), lse))
    p = p.view(b, hk, -1, nk)
    do = s["do"].float().reshape(b, hk, -1, d)
    dv = p.transpose(-1, -2) @ do
    dp = do @ s["v"].float().transpose(-1, -2)
    ds = p * (dp - (p * dp).sum(-1, keepdim=True)) * s["scale"]
    dq = (ds @ s["k"].float()).view(b, c["hq"], c["nq"], d)
    dk = ds.transpose(-1, -2) @ s["q"].float().reshape(b, hk, -1, d)
    return tuple(x.to(torch.bfloat16) for x in (dq, dk, dv))


def run(state):
    s, c = state, state["c"]
    if own:
        import rank_linear_complexity_gb300.linformer as lf
        if c["op"] == "rotary":
            return lf.rotary(s["q"], s["k"], s["phase"], positions=s["pos"], rot=c["rot"],
                             layout=lf.ROTARY_INTERLEAVED if c["interleaved"] else lf.ROTARY_HALVES,
                             amplitude=s["amplitude"], inverse=c["inverse"])
        kw = dict(q_lengths=s["q_lengths"], k_lengths=s["k_lengths"], causal=c["causal"],
                  window=c["window"], scale=s["scale"])
        if c["op"] == "attend":
            return lf.softmax_attention(s["q"], s["k"], s["v"], out=s["out"], lse=s["lse"], **kw)
        return lf.softmax_attention_backward(s["q"], s["k"], s["v"], s["o"], s["do"], s["lse"],
                                             dQ=s["dq"], dK=s["dk"], dV=s["dv"], **kw)
    if c["op"] == "rotary":
        return _rotary_plain(s)
    if c["op"] == "attend":
        return _attend(s)
    return _backward(s)


# --- the definition in 64 bits ----------------------------------------------------------

def _exact_rotary(s):
    c = s["c"]
    r, out = c["rot"], []
    i = torch.arange(r // 2, device="cuda")
    first, second = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + r // 2)
    theta = s["pos"].double().unsqueeze(-1) * s["freq"]
    turn = torch.polar(torch.full_like(theta, s["amplitude"]), -theta if c["inverse"] else theta)
    for x in (s["q"], s["k"]):
        y = x.double().clone()
        z = torch.complex(y[..., first], y[..., second]) * turn.unsqueeze(1)
        y[..., first], y[..., second] = z.real, z.imag
        out.append(y)
    return tuple(out)


def _exact_unit(s, bi, h):
    """Probabilities and logsumexp of one sequence and query head over its valid part."""
    c = s["c"]
    lq = int(s["q_lengths"][bi]) if c["ragged"] else c["nq"]
    lk = int(s["k_lengths"][bi]) if c["ragged"] else c["nk"]
    kv = h // (c["hq"] // c["hk"])
    q, k, v = s["q"][bi, h, :lq].double(), s["k"][bi, kv, :lk].double(), s["v"][bi, kv, :lk].double()
    x = torch.einsum("id,jd->ij", q, k).mul_(s["scale"])
    if c["causal"]:
        ahead = torch.arange(lk, device="cuda")[None] - torch.arange(lq, device="cuda")[:, None]
        ahead -= lk - lq
        x[ahead > 0] = -math.inf
        if c["window"]:
            x[ahead <= -c["window"]] = -math.inf
    lse = torch.logsumexp(x, 1)
    seen = torch.isfinite(lse)
    p = x.sub_(torch.where(seen, lse, 0.0)[:, None]).exp_()
    return lq, lk, kv, q, k, v, p, lse


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "rotary":
        return _exact_rotary(s)
    b, hq, hk, nq, nk, d = (c[k] for k in ("b", "hq", "hk", "nq", "nk", "d"))
    f64 = dict(dtype=torch.float64, device="cuda")
    if c["op"] == "attend":
        o, lse = torch.zeros(b, hq, nq, d, **f64), torch.full((b, hq, nq), -math.inf, **f64)
        for bi in range(b):
            for h in range(hq):
                lq, lk, kv, q, k, v, p, l = _exact_unit(s, bi, h)
                o[bi, h, :lq], lse[bi, h, :lq] = p @ v, l
        return o, lse
    dq = torch.zeros(b, hq, nq, d, **f64)
    dk, dv = torch.zeros(b, hk, nk, d, **f64), torch.zeros(b, hk, nk, d, **f64)
    for bi in range(b):
        for h in range(hq):
            lq, lk, kv, q, k, v, p, _ = _exact_unit(s, bi, h)
            do = s["do"][bi, h, :lq].double()
            dv[bi, kv, :lk] += p.T @ do
            dp = do @ v.T
            g = p * (dp - torch.einsum("ij,ij->i", p, dp)[:, None]) * s["scale"]
            dq[bi, h, :lq] = g @ k
            dk[bi, kv, :lk] += g.T @ q
    return dq, dk, dv
