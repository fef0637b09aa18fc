"""Cases for measuring the operators of a paged key/value cache: appending keys and values with
the rotary turn on the way, attention of new tokens and of trees of drafted tokens over the
pages, and keeping the accepted tokens of a tree.

``own`` selects what ``run`` does: False computes each operator in a plain form (elementary
torch operations in 32 bits, angles in 64), True calls this package.

Ranges: pages of 8 to 256 rows in caches laid out [pages][heads][page][d], [pages][page][heads][d]
or with keys and values side by side, head dimensions 32 to 128, 1 to 32 query heads on as many or
fewer key/value heads, 1 to 64 sequences of 1 to 131072 tokens, idle ones among them, 1 to 4096 new
tokens, trees of 2 to 128 nodes.
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
SPARE = 1.125        # pages of the pool per page in use


def _append(name, b, hq, hk, n, past, d, page, **kw):
    c = dict(name=name, op="append", b=b, hq=hq, hk=hk, n=n, past=past, d=d, page=page, rot=d,
             dtype="bf16", layout="rows", interleaved=False, scaled=False, packed=False,
             ragged=False, placed=False)
    c.update(kw)
    return c


def _attend(name, b, hq, hk, nq, nk, d, page, **kw):
    c = dict(name=name, op="attend", b=b, hq=hq, hk=hk, nq=nq, nk=nk, d=d, page=page, causal=True,
             window=0, layout="rows", ragged=False, idle=0)
    c.update(kw)
    return c


def _tree(name, b, hq, hk, nq, nk, d, page, **kw):
    c = dict(name=name, op="tree", b=b, hq=hq, hk=hk, nq=nq, nk=nk, d=d, page=page, fresh=False,
             layout="rows", ragged=False, idle=0)
    c.update(kw)
    return c


def _keep(name, b, hk, nodes, most, past, d, page, **kw):
    c = dict(name=name, op="keep", b=b, hk=hk, nodes=nodes, most=most, past=past, d=d, page=page,
             dtype="bf16", layout="rows")
    c.update(kw)
    return c


def listed():
    return [
        # one new token of each of 64 sequences on its way into the cache, its queries turned too
        _append("append_token", 64, 32, 8, 1, 1024, 128, 16, packed=True, scaled=True),
        # fp32, neighbouring pairs, half of each head, drafted tokens at positions of their own
        _append("append_draft_f32", 6, 12, 12, 61, 333, 64, 32, rot=32, dtype="f32",
                interleaved=True, layout="heads", placed=True),
        # the prompts of a ragged batch
        _append("append_prompt", 8, 32, 8, 4096, 0, 128, 64, packed=True, ragged=True,
                layout="fused"),
        # one new token of two short conversations: latency counts
        _attend("attend_small", 2, 12, 12, 1, 500, 64, 16),
        # a serving batch: one new token over caches of differing lengths, two slots idle
        _attend("attend_token", 64, 32, 8, 1, 8192, 128, 16, ragged=True, idle=2),
        # one new token over a long document, many query heads on few key/value heads
        _attend("attend_long", 2, 16, 2, 1, 131072, 128, 128, layout="heads"),
        # five tokens at a time, a sliding window, an uncommon head size, an odd length
        _attend("attend_few_window", 16, 24, 3, 5, 6001, 96, 32, window=4095, layout="fused"),
        # the last chunk of a long prompt
        _attend("attend_chunk", 2, 32, 8, 2048, 16384, 128, 64, layout="heads"),
        # a small tree drafted for one conversation, its mask made on the way
        _tree("tree_small", 1, 12, 12, 25, 700, 64, 16, fresh=True),
        # trees of 64 drafted tokens over a serving batch
        _tree("tree_64", 16, 32, 8, 64, 8192, 128, 64, ragged=True, layout="heads"),
        # the accepted tokens of one tree
        _keep("keep_small", 1, 12, 25, 5, 675, 64, 16),
        # and of a serving batch's trees
        _keep("keep_64", 64, 8, 64, 16, 960, 128, 64, layout="heads"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("append", "attend", "attend", "tree", "keep"))
    limit = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        hk = rng.choice((1, 2, 3, 4, 8, 12))
        hq = hk * rng.choice((1, 1, 2, 4, 8))
        b = _log_int(rng, 1, 64)
        page = rng.choice((8, 16, 16, 32, 64, 128, 256))
        layout = rng.choice(("rows", "rows", "heads", "fused"))
        idle = rng.choice((0, 0, 1, 2)) if b > 4 else 0
        ragged = rng.random() < 0.5
        if op == "append":
            n = 1 if rng.random() < 0.4 else _log_int(rng, 2, 4096)
            d = rng.choice((32, 64, 80, 96, 128))
            c = _append("", b, hq, hk, n, _log_int(rng, 1, 4096) - 1, d, page,
                        rot=rng.choice((d, d, d // 2)), layout=layout,
                        dtype=rng.choice(("bf16", "bf16", "f32")), ragged=ragged,
                        interleaved=rng.random() < 0.4, scaled=rng.random() < 0.5,
                        packed=rng.random() < 0.5, placed=rng.random() < 0.3)
        elif op == "keep":
            most = rng.randint(2, 16)
            c = _keep("", b, hk, rng.randint(2 * most, 64), most, _log_int(rng, 1, 1024) - 1,
                      rng.choice((32, 64, 80, 96, 128)), page, layout=layout,
                      dtype=rng.choice(("bf16", "bf16", "f32")))
        else:
            d = rng.choice((40, 64, 64, 80, 96, 128, 128))
            if op == "tree":
                nq = _log_int(rng, 2, 128)
                c = _tree("", b, hq, hk, nq, _log_int(rng, nq, 16384), d, page, layout=layout,
                          ragged=ragged, idle=idle, fresh=rng.random() < 0.4)
            else:
                kind = rng.random()
                nq = (1 if kind < 0.5 else rng.randint(2, 8) if kind < 0.7
                      else _log_int(rng, 16, 2048))
                causal = rng.random() < 0.85
                c = _attend("", b, hq, hk, nq, _log_int(rng, nq, 131072), d, page, causal=causal,
                            window=_log_int(rng, 16, 8192) if causal and rng.random() < 0.3 else 0,
                            layout=layout, ragged=ragged, idle=idle)
        if _cost(c) <= limit and hq <= 32:
            del c["name"]
            return c


def _cost(c):
    if c["op"] in ("append", "keep"):
        new = c["n"] * (c["hq"] + 2 * c["hk"]) if c["op"] == "append" else 0
        # the rows that move and, as outputs, the whole pool
        return c["b"] * c["d"] * (4 * new + 2 * c["hk"] * (_rows(c) + c["page"]))
    # the plain form holds scores of every pair, masked or not
    return c["b"] * (c["hq"] * c["nq"] + 16 * c["hk"]) * (c["nk"] + c["page"]) * max(c["d"], 64)


def _rows(c):
    """Rows that a sequence takes in the cache at most."""
    return c["nk"] if "nk" in c else c["past"] + (c["n"] if c["op"] == "append" else c["nodes"])


def _spread(n, b):
    """Lengths of a ragged batch: evenly spaced from n down to about a quarter of it."""
    return [max(1, n - (3 * n * i) // (4 * b)) for i in range(b)]


def _lengths(c):
    """(queries, cache rows) of each sequence, in the order before they are shuffled."""
    b = c["b"]
    lk = _spread(c["nk"], b) if c["ragged"] else [c["nk"]] * b
    # chunks and trees differ too; the cache holds at least the new tokens
    lq = _spread(c["nq"], b) if c["ragged"] and c["nq"] > 1 else [c["nq"]] * b
    lk = [max(x, y) for x, y in zip(lk, lq)]
    for i in range(c["idle"]):
        lq[-1 - 2 * i] = lk[-1 - 2 * i] = 0
    return lq, lk


def _counts(c):
    """New rows of each sequence, in the order before they are shuffled."""
    return _spread(c["n"], c["b"]) if c["ragged"] else [c["n"]] * c["b"]


def work(case):
    c = case
    if c["op"] == "append":
        e = 4 if c["dtype"] == "f32" else 2
        rows, heads = sum(_counts(c)), c["hq"] + c["hk"]
        return {"bytes": 2.0 * e * (rows * 2 * c["hk"] + c["b"] * c["n"] * c["hq"]) * c["d"]
                + 4 * c["b"] * (c["n"] + 1),
                "flops": 3.0 * c["b"] * c["n"] * heads * c["rot"]}
    if c["op"] == "keep":
        e = 4 if c["dtype"] == "f32" else 2
        moved = sum(x - 1 for x in _accepted(c))
        return {"bytes": 4.0 * e * moved * c["hk"] * c["d"] + 8 * c["b"] * c["most"], "flops": 0.0}
    lq, lk = _lengths(c)
    pairs = rows = 0
    for q, k in zip(lq, lk):
        if not q:
            continue
        pos = np.arange(q, dtype=np.int64) + (k - q)
        if c["op"] == "tree":
            # every node sees what the cache held before, and a few of its tree
            pairs += q * (k - q) + int(q * (1 + math.log2(q)))
            rows += k
        elif not c["causal"]:
            pairs, rows = pairs + q * k, rows + k
        else:
            first = np.maximum(pos - c["window"] + 1, 0) if c["window"] else 0 * pos
            pairs += int((pos + 1 - first).sum())
            rows += k - int(first[0])
    q = c["b"] * c["nq"] * c["hq"]
    n = -(-c["nq"] // 64)
    mask = c["b"] * c["nq"] * (4 if c["fresh"] else 0) + 8 * c["b"] * c["nq"] * n if c["op"] == "tree" else 0
    return {"bytes": 4.0 * q * c["d"] + 4 * q + 4.0 * rows * c["hk"] * c["d"]
            + 4 * sum(-(-k // c["page"]) for k in lk) + mask,
            "flops": 4.0 * pairs * c["hq"] * c["d"]}


# --- inputs -----------------------------------------------------------------------------

def _shuffled(g, *lists):
    order = torch.randperm(len(lists[0]), generator=g, device="cuda")
    return tuple(torch.tensor(x, dtype=torch.int32, device="cuda")[order] for x in lists)


def _pool(c, g, dtype, rows):
    """(k_cache, v_cache, table) with pages in no order; rows: those that each sequence takes, by
    sequence.  Caches [pages][hk][page][d], by strides where the program lays them out otherwise."""
    b, hk, page, d = c["b"], c["hk"], c["page"], c["d"]
    width = max(1, -(-max(rows) // page))
    taken = [-(-r // page) for r in rows]
    pages = max(1, int(sum(taken) * SPARE))
    if c["layout"] == "heads":
        k, v = (torch.empty(pages, hk, page, d, dtype=dtype, device="cuda") for _ in range(2))
    elif c["layout"] == "rows":
        k, v = (torch.empty(pages, page, hk, d, dtype=dtype, device="cuda").transpose(1, 2)
                for _ in range(2))
    else:
        both = torch.empty(pages, 2, page, hk, d, dtype=dtype, device="cuda")
        k, v = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
    k.normal_(0, QK_GAIN, generator=g)
    v.normal_(0, 1, generator=g)
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((b, width), -1, dtype=torch.int32, device="cuda")
    used = torch.arange(width, device="cuda") < torch.tensor(taken, device="cuda")[:, None]
    table[used] = order[:sum(taken)]
    return k, v, table


def _heads(g, b, n, heads, d, dtype, packed):
    """Tensors [b][h][n][d] for each entry of heads: dense, or slices of one fused buffer."""
    if packed:
        buf = torch.empty(b, n, sum(heads) * d, dtype=dtype, device="cuda").normal_(generator=g)
        views, at = [], 0
        for h in heads:
            views.append(buf[:, :, at:at + h * d].view(b, n, h, d).transpose(1, 2))
            at += h * d
        return views
    return [torch.empty(b, h, n, d, dtype=dtype, device="cuda").normal_(generator=g) for h in heads]


def _parents(g, b, n):
    """A tree a sequence, int32 [b][n]: the parent of each node, before it, -1 of the root.  Nodes
    lean towards recent ones, so that branches get deep."""
    at = torch.arange(n, device="cuda")
    back = (torch.rand(b, n, generator=g, device="cuda") ** 2 * torch.clamp(at, max=12)).long()
    return (at - 1 - back).to(torch.int32)


def _accepted(c):
    """Tokens accepted of each sequence's tree, its root among them."""
    return [1 + (7 * i + c["most"] - 1) % c["most"] for i in range(c["b"])]


def _dtype(c):
    return torch.float32 if c["dtype"] == "f32" else torch.bfloat16


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    if c["op"] == "append":
        q, k, v = _heads(g, c["b"], c["n"], (c["hq"], c["hk"], c["hk"]), c["d"], _dtype(c), c["packed"])
        past = _spread(c["past"], c["b"]) if c["past"] else [0] * c["b"]
        starts, counts = _shuffled(g, past, _counts(c))
        kc, vc, table = _pool(c, g, _dtype(c), [_rows(c)] * c["b"])
        s = dict(c=c, q=q, k=k, v=v, kc=kc, vc=vc, table=table, starts=starts,
                 counts=counts if c["ragged"] else None, positions=None)
        if c["placed"]:
            # a tree's nodes stand at their depth behind the sequence
            depth = torch.randint(0, c["n"], (c["b"], c["n"]), generator=g, device="cuda").sort(1)[0]
            s["positions"] = (starts[:, None] + depth).to(torch.int32)
        freq = _frequencies(c)
        s.update(freq=freq.cuda(), phase=_phase_steps(freq).cuda(), amplitude=_amplitude(c),
                 out=torch.empty(c["b"], c["n"], c["hq"], c["d"], dtype=_dtype(c),
                                 device="cuda").transpose(1, 2))
        return s
    if c["op"] == "keep":
        b, m = c["b"], c["most"]
        kc, vc, table = _pool(c, g, _dtype(c), [_rows(c)] * b)
        starts, counts = _shuffled(g, _spread(c["past"], b) if c["past"] else [0] * b, _accepted(c))
        # the root, then nodes of later levels, behind the places that they move to
        later = torch.rand(b, c["nodes"] - m, generator=g, device="cuda").argsort(1)[:, :m - 1]
        path = torch.cat([torch.zeros(b, 1, dtype=torch.long, device="cuda"),
                          m + later.sort(1)[0]], 1).to(torch.int32)
        return dict(c=c, kc=kc, vc=vc, table=table, starts=starts, counts=counts, path=path)
    lq, lk = _shuffled(g, *_lengths(c))
    kc, vc, table = _pool(c, g, torch.bfloat16, lk.tolist())
    q = torch.empty(c["b"], c["nq"], c["hq"], c["d"], dtype=torch.bfloat16,
                    device="cuda").normal_(0, QK_GAIN, generator=g).transpose(1, 2)
    some = c["ragged"] and c["nq"] > 1 or c["idle"] > 0
    s = dict(c=c, q=q, kc=kc, vc=vc, table=table, q_lengths=lq if some else None, k_lengths=lk,
             scale=1 / math.sqrt(c["d"]), out=torch.empty_like(q),
             lse=torch.empty(c["b"], c["hq"], c["nq"], device="cuda"))
    if c["op"] == "tree":
        s["parents"] = _parents(g, c["b"], c["nq"])
        s["mask"] = _words_plain(s["parents"])
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


def _slots(s, first, offsets):
    """(page, row within it) of the cache rows first + offsets, [b][n] each."""
    at = (first[:, None] + offsets).long()
    page = torch.gather(s["table"].long(), 1, at // s["c"]["page"])
    return page, at % s["c"]["page"]


def _append_plain(s):
    c = s["c"]
    i = torch.arange(c["n"], device="cuda")[None]
    pos = s["starts"][:, None] + i if s["positions"] is None else s["positions"]
    angle = pos.double()[:, None, :, None] * s["freq"]
    cos, sin = ((f(angle) * s["amplitude"]).float() for f in (torch.cos, torch.sin))
    s["out"].copy_(_rotate(s["q"], cos, sin, c))
    page, row = _slots(s, s["starts"], i)
    valid = None if s["counts"] is None else (i < s["counts"][:, None])[:, :, None, None]
    for cache, x in ((s["kc"], _rotate(s["k"], cos, sin, c)), (s["vc"], s["v"])):
        new = x.transpose(1, 2)
        if valid is not None:  # rows behind a sequence's last keep what they held
            new = torch.where(valid, new, cache[page, :, row])
        cache[page, :, row] = new
    return s["kc"], s["vc"], s["out"]


def _keep_plain(s):
    c = s["c"]
    m = torch.arange(c["most"], device="cuda")[None]
    source, target = _slots(s, s["starts"], s["path"]), _slots(s, s["starts"], m)
    valid = (m < s["counts"][:, None])[:, :, None, None]
    for cache in (s["kc"], s["vc"]):
        new = torch.where(valid, cache[source[0], :, source[1]], cache[target[0], :, target[1]])
        cache[target[0], :, target[1]] = new
    return s["kc"], s["vc"]


def _words_plain(parents):
    """Which nodes each node sees, itself and its ancestors, int64 [b][n][ceil(n / 64)]."""
    b, n = parents.shape
    at = torch.arange(n, device="cuda")
    reach = ((parents[:, :, None] == at) | (at[:, None] == at)).float()
    for _ in range(max(1, (n - 1).bit_length())):  # paths of twice the length
        reach = ((reach @ reach) > 0).float()
    bits = torch.zeros(b, n, -(-n // 64) * 64, dtype=torch.int64, device="cuda")
    bits[:, :, :n] = reach.long()
    return (bits.view(b, n, -1, 64) << torch.arange(64, device="cuda")).sum(-1)


def _gathered(s, cache):
    """A cache's rows by sequence, [b][hk][width * page][d] in 32 bits."""
    c = s["c"]
    x = cache[s["table"].clamp(min=0).long()]  # [b][width][hk][page][d]
    return x.permute(0, 2, 1, 3, 4).reshape(c["b"], c["hk"], -1, c["d"]).float()


def _visible(s, words, nk):
    """True where a query sees a cache row, [b][1][1][nq][nk]."""
    c = s["c"]
    lk = s["k_lengths"].view(-1, 1, 1)
    lq = torch.full_like(lk, c["nq"]) if s["q_lengths"] is None else s["q_lengths"].view(-1, 1, 1)
    i = torch.arange(c["nq"], device="cuda").view(1, -1, 1)
    j = torch.arange(nk, device="cuda").view(1, 1, -1)
    m = (i < lq) & (j < lk)
    if words is not None:
        node = j - (lk - lq)
        inside = node.clamp(0, c["nq"] - 1).expand(c["b"], c["nq"], nk)
        bit = torch.gather(words, 2, inside // 64) >> (inside % 64) & 1
        m = m & ((node < 0) | (bit == 1))
    elif c["causal"]:
        m = m & (j <= i + (lk - lq))
        if c["window"]:
            m = m & (j > i + (lk - lq) - c["window"])
    return m[:, None, None]


def _attention_plain(s, words=None):
    c = s["c"]
    b, hq, hk, nq, d = c["b"], c["hq"], c["hk"], c["nq"], c["d"]
    k, v = _gathered(s, s["kc"]), _gathered(s, s["vc"])
    nk = k.shape[2]
    x = s["q"].float().reshape(b, hk, hq // hk * nq, d) @ k.transpose(-1, -2) * s["scale"]
    x = x.view(b, hk, hq // hk, nq, nk).masked_fill_(~_visible(s, words, nk), float("-inf"))
    top = x.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    p = x.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(b, hk, -1, nk) @ v).view(b, hk, -1, nq, d)
    o = o / torch.where(total == 0, torch.ones_like(total), total)
    s["out"].copy_(o.view(b, hq, nq, d))
    s["lse"].copy_((top + torch.log(total)).view(b, hq, nq))
    return s["out"], s["lse"]


def run(state):
    s, c = state, state["c"]
    if own:
        import rank_linear_complexity_gb300.linformer as lf
        if c["op"] == "append":
            lf.cache_append(s["k"], s["v"], s["kc"], s["vc"], s["table"], s["starts"],
                            counts=s["counts"], Q=s["q"], phase=s["phase"],
                            positions=s["positions"], rot=c["rot"], amplitude=s["amplitude"],
                            layout=lf.ROTARY_INTERLEAVED if c["interleaved"] else lf.ROTARY_HALVES,
                            out=s["out"])
            return s["kc"], s["vc"], s["out"]
        if c["op"] == "keep":
            lf.cache_keep(s["kc"], s["vc"], s["table"], s["starts"], s["path"], counts=s["counts"])
            return s["kc"], s["vc"]
        kw = dict(q_lengths=s["q_lengths"], scale=s["scale"], out=s["out"], lse=s["lse"])
        if c["op"] == "attend":
            return lf.paged_attention(s["q"], s["kc"], s["vc"], s["table"], s["k_lengths"],
                                      causal=c["causal"], window=c["window"], **kw)
        mask = lf.tree_mask(s["parents"]) if c["fresh"] else s["mask"]
        out = lf.tree_attention(s["q"], s["kc"], s["vc"], s["table"], s["k_lengths"], mask, **kw)
        return (*out, mask) if c["fresh"] else out
    if c["op"] == "append":
        return _append_plain(s)
    if c["op"] == "keep":
        return _keep_plain(s)
    if c["op"] == "attend":
        return _attention_plain(s)
    mask = _words_plain(s["parents"]) if c["fresh"] else s["mask"]
    out = _attention_plain(s, mask)
    return (*out, mask) if c["fresh"] else out


# --- the definition in 64 bits ----------------------------------------------------------

def _exact_append(s):
    c = s["c"]
    r = c["rot"]
    i = torch.arange(r // 2, device="cuda")
    first, second = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + r // 2)
    turned = []
    for x in (s["q"], s["k"]):
        y = x.double().clone()
        for bi in range(c["b"]):
            pos = (int(s["starts"][bi]) + torch.arange(c["n"], device="cuda") if s["positions"] is None
                   else s["positions"][bi])
            theta = torch.outer(pos.double(), s["freq"])
            turn = torch.polar(torch.full_like(theta, s["amplitude"]), theta)
            z = torch.complex(y[bi][..., first], y[bi][..., second]) * turn
            y[bi][..., first], y[bi][..., second] = z.real, z.imag
        turned.append(y)
    caches = [s["kc"].double(), s["vc"].double()]
    for bi in range(c["b"]):
        count = c["n"] if s["counts"] is None else int(s["counts"][bi])
        at = int(s["starts"][bi]) + np.arange(count)
        pages = s["table"][bi].cpu().numpy()[at // c["page"]]
        for cache, x in zip(caches, (turned[1], s["v"].double())):
            cache[pages, :, at % c["page"]] = x[bi, :, :count].transpose(0, 1)
    return caches[0], caches[1], turned[0]


def _exact_keep(s):
    c = s["c"]
    old = [s["kc"].double(), s["vc"].double()]
    new = [x.clone() for x in old]
    for bi in range(c["b"]):
        table, start = s["table"][bi].tolist(), int(s["starts"][bi])
        for t, node in enumerate(s["path"][bi].tolist()[:int(s["counts"][bi])]):
            (p, r), (p2, r2) = divmod(start + t, c["page"]), divmod(start + node, c["page"])
            for x, y in zip(new, old):
                x[table[p], :, r] = y[table[p2], :, r2]
    return tuple(new)


def _exact_words(parents):
    b, n = parents.shape
    out = np.zeros((b, n, -(-n // 64)), dtype=np.uint64)
    for bi, row in enumerate(parents.tolist()):
        for i in range(n):
            j = i
            while j >= 0:
                out[bi, i, j // 64] |= np.uint64(1 << (j % 64))
                j = row[j]
    return out


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "append":
        return _exact_append(s)
    if c["op"] == "keep":
        return _exact_keep(s)
    b, hq, hk, nq, page, d = (c[k] for k in ("b", "hq", "hk", "nq", "page", "d"))
    o = torch.zeros(b, hq, nq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((b, hq, nq), -math.inf, dtype=torch.float64, device="cuda")
    words = _exact_words(s["parents"]) if c["op"] == "tree" else None
    for bi in range(b):
        lk = int(s["k_lengths"][bi])
        lq = nq if s["q_lengths"] is None else int(s["q_lengths"][bi])
        if not lq or not lk:
            continue
        pages = s["table"][bi, :-(-lk // page)].long()
        hidden = None
        if words is not None:
            bits = np.unpackbits(words[bi].view(np.uint8), axis=1, bitorder="little")[:lq, :lq]
            hidden = torch.zeros(lq, lk, dtype=torch.bool, device="cuda")
            hidden[:, lk - lq:] = torch.from_numpy(bits == 0).cuda()
        elif c["causal"]:
            ahead = torch.arange(lk, device="cuda")[None] - torch.arange(lk - lq, lk, device="cuda")[:, None]
            hidden = ahead > 0
            if c["window"]:
                hidden |= ahead <= -c["window"]
        for kv in range(hk):
            k, v = (torch.cat(list(x[pages, kv]))[:lk].double() for x in (s["kc"], s["vc"]))
            for h in range(kv * (hq // hk), (kv + 1) * (hq // hk)):
                x = torch.einsum("id,jd->ij", s["q"][bi, h, :lq].double(), k).mul_(s["scale"])
                if hidden is not None:
                    x[hidden] = -math.inf
                l = torch.logsumexp(x, 1)
                p = x.sub_(torch.where(torch.isfinite(l), l, 0.0)[:, None]).exp_()
                o[bi, h, :lq], lse[bi, h, :lq] = p @ v, l
    if c["op"] == "tree" and c["fresh"]:
        return o, lse, torch.from_numpy(words.view(np.int64)).cuda()
    return o, lse
