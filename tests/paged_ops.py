"""Random operations on a PagedMemory against plain lists of rows, one per sequence:
what a stream appended last is what its memory holds, whatever was forked, freed,
trimmed, compacted or restored in between.  Used on the CPU (with fakes of the
device calls) and on the GPU."""

import random

import torch


def contents(mem, b, plane=0):
    """Sequence b's memory rows [fill, H, dh] of one plane, as the device holds them."""
    kv = mem.kv
    begin, fill = int(kv.begin[b]), int(kv.fill[b])
    assert (begin, fill) == (mem.begin[b], mem.fill[b])
    x = (begin + torch.arange(fill)) % kv.rows
    page = kv.table[b].cpu().long()[x // kv.page_rows]
    assert fill == 0 or int(page.min()) >= 0
    return kv.pool.cpu()[plane][page, :, x % kv.page_rows]


def check(mem, want):
    users = [0] * mem.kv.n_pages
    assert (mem._table == mem.kv.table.cpu().numpy()).all()
    for row in mem._table:
        for p in row:
            if p >= 0:
                users[p] += 1
    assert users == [mem.pages.users(p) for p in range(mem.kv.n_pages)]
    assert mem.pages.n_free == users.count(0)
    for b in range(mem.B):
        for plane in range(mem.kv.pool.shape[0]):
            assert torch.equal(contents(mem, b, plane), want[b][:, plane])


def run(make, device, seed, steps=120):
    """make() -> a PagedMemory; the operations and their order come from the seed."""
    rng = random.Random(seed)
    mem = make()
    planes, H, dh = mem.kv.pool.shape[0], mem.kv.H, mem.kv.pool.shape[-1]
    dtype = mem.kv.pool.dtype
    want = [torch.zeros(0, planes, H, dh, dtype=dtype) for _ in range(mem.B)]
    g = torch.Generator().manual_seed(seed)
    kept = None
    for _ in range(steps):
        what = rng.random()
        b, c = rng.randrange(mem.B), rng.randrange(mem.B)
        if what < 0.6:
            N = rng.randint(1, mem.max_new)
            new = torch.randn(planes // 2, mem.B, N, 2, H, dh, generator=g).to(dtype)
            k, v = (new[:, :, :, i].transpose(2, 3).to(device) for i in (0, 1))
            if rng.random() < 0.5:
                rows = [sorted(rng.sample(range(N), rng.randint(0, N))) for _ in range(mem.B)]
                mem.append(k, v, rows=rows)
            else:
                n = [rng.randint(0, N) for _ in range(mem.B)] if rng.random() < 0.7 else None
                rows = [range(N if n is None else n[i]) for i in range(mem.B)]
                mem.append(k, v, n)
            # [rows, planes, H, dh]
            flat = new.permute(1, 2, 0, 3, 4, 5).reshape(mem.B, N, planes, H, dh)
            for i in range(mem.B):
                rest = torch.cat([want[i], flat[i, list(rows[i])]])
                want[i] = rest[max(0, len(rest) - mem.M):]
        elif what < 0.75:
            mem.fork(b, c)
            want[c] = want[b].clone()
        elif what < 0.8:
            mem.free(b)
            want[b] = want[b][:0]
        elif what < 0.87:
            free = mem.pages.n_free
            assert mem.trim() == mem.pages.n_free - free
        elif what < 0.94:
            n = mem.compact()
            assert n == mem.kv.n_pages - mem.pages.n_free and mem._table.max() < max(n, 1)
        elif kept is None or rng.random() < 0.5:
            kept = mem.checkpoint(), [w.clone() for w in want]
        else:
            mem = make() if rng.random() < 0.5 else mem
            mem.restore(kept[0])
            want = [w.clone() for w in kept[1]]
        check(mem, want)
