"""Paged caches for the tests: pages in no order, NaN wherever no valid row stands."""
import torch

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def cache(b, hk, d, page, lengths, layout="rows", dtype="bf16", seed=0, spare=3, width=None,
          device="cpu", gain=1.0):
    """(k_cache, v_cache, table): lengths[i] valid rows of sequence i.  Unused table entries are
    -1, unused rows NaN."""
    g = torch.Generator().manual_seed(seed)
    dt = DTYPES[dtype]
    need = [-(-x // page) for x in lengths]
    pages = sum(need) + spare
    width = max(1, max(need)) if width is None else width
    order = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((b, width), -1, dtype=torch.int32)
    full = torch.full((2, pages, hk, page, d), float("nan"))
    at = 0
    for i, x in enumerate(lengths):
        table[i, :need[i]] = order[at:at + need[i]]
        at += need[i]
        for j in range(need[i]):
            rows = min(page, x - j * page)
            full[:, table[i, j].long(), :, :rows] = torch.randn(2, hk, rows, d, generator=g) * gain
    if layout == "heads":
        k, v = (full[i].to(dt).to(device).contiguous() for i in range(2))
    elif layout == "rows":
        k, v = (full[i].to(dt).to(device).transpose(1, 2).contiguous().transpose(1, 2)
                for i in range(2))
    else:  # keys and values side by side
        both = full.to(dt).to(device).permute(1, 0, 3, 2, 4).contiguous()
        k, v = both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2)
    return k, v, table.to(device)


def bits(t):
    return t.contiguous().view({2: torch.int16, 4: torch.int32, 8: torch.int64}[t.element_size()])


def ints(x, device="cpu"):
    return torch.tensor(x, dtype=torch.int32, device=device)


def random_tree(b, n, seed=0, deep=False):
    g = torch.Generator().manual_seed(seed)
    up = torch.zeros(b, n, dtype=torch.int32)
    for i in range(n):
        low = max(-1, i - 3) if deep else -1
        up[:, i] = torch.randint(low, max(i, low + 1), (b,), generator=g, dtype=torch.int32)
    up[:, 0] = -1
    return up
