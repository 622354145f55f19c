"""What is measured of the paged memory and of the attention for drafted trees.

Three operators of the library, in calls as a streaming program makes them:

  tree    relative-position attention of a tree of drafted tokens over a paged
          memory (the verification step of speculative decoding)
  append  rows of keys and values put behind the memory in its pages: a whole
          prompt, or the accepted path of a drafted tree, with the memory's
          begin and fill advanced
  copy    pages copied to other pages in every layer (a stream forked into
          several continuations)

``run`` computes each in elementary torch operations, or calls the library when
``own`` is set.  Sequence b's memory row t lies in table row
x = (begin[b] + t) mod (slots * page_rows): page table[b][x // page_rows], row
x % page_rows of it.
"""

import math

import numpy as np
import torch

own = False

DH = 64
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def _tree(name, B, H, N, lo, hi, P, shape, dtype="bf16", short=False):
    """N nodes per sequence against memories of lo..hi rows in pages of P rows."""
    return {"name": name, "op": "tree", "B": B, "H": H, "N": N, "lo": lo, "hi": hi, "P": P,
            "shape": shape, "dtype": dtype, "short": short}


def _append(name, layers, B, H, N, lo, hi, keep, P, accept, dtype="bf16"):
    return {"name": name, "op": "append", "layers": layers, "B": B, "H": H, "N": N, "lo": lo,
            "hi": hi, "keep": keep, "P": P, "accept": accept, "dtype": dtype}


def _copy(name, layers, H, P, pages, pairs, dtype="bf16"):
    return {"name": name, "op": "copy", "layers": layers, "H": H, "P": P, "pages": pages,
            "pairs": pairs, "dtype": dtype}


def listed():
    return [
        # one stream, one new token against the evaluation memory of 1600: a
        # plain decoding step, where latency counts
        _tree("tree_token_B1_M1600", 1, 16, 1, 1600, 1600, 64, "chain"),
        # eight streams of unlike lengths, a draft of eight tokens in a row
        _tree("tree_chain8_B8_M3800", 8, 16, 8, 1900, 3800, 64, "chain"),
        # a tree of 26 nodes for four short streams (odd sizes everywhere)
        _tree("tree_26_B4_M517", 4, 8, 26, 131, 517, 32, "branch", short=True),
        # a wide tree over long memories
        _tree("tree_64_B16_M3800", 16, 16, 64, 3800, 3800, 128, "branch"),
        # a served batch of 64 streams of unlike lengths, 16 nodes each
        _tree("tree_16_B64_M3800", 64, 16, 16, 950, 3800, 64, "branch", short=True),
        # the exact single-precision path
        _tree("tree_f32_13_B2_M777", 2, 8, 13, 401, 777, 64, "branch", dtype="f32"),
        # the accepted path of a drafted tree, one stream of the 12-layer stack
        _append("accept_12x_B1", 12, 1, 8, 26, 512, 512, 512, 64, True),
        # the same for a served batch of a 12-layer stack with 16 heads
        _append("accept_12x_B64_H16", 12, 64, 16, 64, 700, 3800, 3800, 64, True),
        # a prompt of 1600 rows for one layer of 16 streams, into empty memories
        _append("prompt_B16_L1600", 1, 16, 16, 1600, 0, 0, 1600, 128, False),
        # one fork in the 12-layer stack: the partly filled page of a stream
        _copy("fork_12x_1", 12, 8, 64, 64, 1),
        # 48 forks in a 12-layer stack with 16 heads
        _copy("fork_12x_48", 12, 16, 64, 160, 48),
        # a few pages of a single-precision cache, pages of odd length
        _copy("fork_f32_5", 3, 8, 96, 24, 5, dtype="f32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "append", "copy"])
    if op == "tree":
        f32 = rng.random() < 0.2
        B = _log(rng, 1, 6 if f32 else 64)
        hi = _log(rng, 1, 1500 if f32 else 3800)
        N = _log(rng, 1, 64)
        if not f32 and B * N > 1024:
            N = max(1, 1024 // B)
        lo = rng.choice([hi, rng.randint(0, hi)])
        return {"op": op, "B": B, "H": rng.choice([1, 8, 16]), "N": N, "lo": lo, "hi": hi,
                "P": rng.choice([32, 64, 96, 128]), "shape": rng.choice(["chain", "branch", "roots"]),
                "dtype": "f32" if f32 else "bf16", "short": rng.random() < 0.5}
    if op == "append":
        accept = rng.random() < 0.5
        dtype = rng.choice(["bf16", "bf16", "f32"])
        layers = rng.randint(1, 12) if accept else rng.randint(1, 2)
        B = _log(rng, 1, 16 if dtype == "f32" else 32)
        N = _log(rng, 1, 64 if accept else 700)
        hi = rng.randint(0, 900)
        return {"op": op, "layers": layers, "B": B, "H": rng.choice([1, 8, 16]), "N": N,
                "lo": rng.randint(0, hi), "hi": hi, "keep": hi + rng.randint(0, N),
                "P": rng.choice([32, 64, 96, 128]), "accept": accept, "dtype": dtype}
    pages = _log(rng, 2, 96)
    return {"op": op, "layers": rng.randint(1, 12), "H": rng.choice([1, 8, 16]),
            "P": rng.choice([32, 64, 96, 128]), "pages": pages, "pairs": rng.randint(1, pages // 2),
            "dtype": rng.choice(["bf16", "bf16", "f32"])}


# ---------------------------------------------------------------------------
# sizes that a case fixes (not its seed)
# ---------------------------------------------------------------------------

def _fills(case):
    B, lo, hi = case["B"], case["lo"], case["hi"]
    if B == 1:
        return [hi]
    return [lo + (hi - lo) * ((5 * b + 2) % B) // (B - 1) for b in range(B)]


def _counts(case):
    """Nodes, or new rows, of each sequence."""
    B, N = case["B"], case["N"]
    if case["op"] == "append":
        # accepted paths are short: one to eight nodes of the tree
        return [1 + (3 * b + 4) % min(8, N) if case["accept"] else N for b in range(B)]
    return [max(1, N - (7 * b) % (N // 2 + 1)) if case["short"] else N for b in range(B)]


def _esize(case):
    return 4 if case["dtype"] == "f32" else 2


def work(case):
    e = _esize(case)
    if case["op"] == "tree":
        fills, ns = _fills(case), _counts(case)
        H, row = case["H"], DH * e
        kv = sum(2 * (f + n) for f, n in zip(fills, ns)) * H * row
        qo = sum(2 * n for n in ns) * H * row + sum(ns) * H * 4
        table = H * (max(fills) + case["N"]) * row
        pairs = sum(n * (f + min(n, 8)) for f, n in zip(fills, ns)) * H
        return {"bytes": kv + qo + table, "flops": 6 * DH * pairs}
    if case["op"] == "append":
        rows = sum(_counts(case)) * case["H"] * 2 * case["layers"]
        return {"bytes": 2 * rows * DH * e, "flops": 0}
    rows = case["pairs"] * case["H"] * case["P"] * 2 * case["layers"]
    return {"bytes": 2 * rows * DH * e, "flops": 0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _parents(shape, B, N, g):
    """parents [B, N] int32: chains, trees grown below random earlier nodes (most
    of them recent), or several first tokens with short continuations."""
    par = torch.full((B, N), -1, dtype=torch.int32)
    for i in range(1, N):
        if shape == "chain":
            par[:, i] = i - 1
        elif shape == "branch":
            back = torch.randint(1, min(i, 6) + 1, (B,), generator=g)
            par[:, i] = (i - back).int()
        else:
            p = torch.randint(-1, i, (B,), generator=g)
            par[:, i] = torch.where(p < i // 2, torch.full_like(p, -1), p).int()
    return par


def _paths(B, N, counts, width, g):
    """Accepted nodes, ascending, [B, width] (the entries behind a sequence's
    count are -1)."""
    rows = torch.full((B, width), -1, dtype=torch.int32)
    for b, n in enumerate(counts):
        rows[b, :n] = torch.sort(torch.randperm(N, generator=g)[:n])[0].int()
    return rows


class _State:
    pass


def _memory(st, B, slots, P, H, layers, fills, dt, gc, gd, std):
    """A pool whose pages are handed out in random order, with a few pages that
    no sequence owns; memories begin at random table rows."""
    n_pages = B * slots + 3
    st.pool = (torch.randn(2 * layers, n_pages, H, P, DH, generator=gd, device="cuda") * std).to(dt)
    st.table = torch.randperm(n_pages, generator=gc)[:B * slots].view(B, slots).int().cuda()
    st.begin = torch.randint(0, slots * P, (B,), generator=gc).int().cuda()
    st.fill = torch.tensor(fills, dtype=torch.int32).cuda()


def prepare(case, seed):
    gc = torch.Generator().manual_seed(seed)
    gd = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    st = _State()
    st.case = case
    rand = lambda *s, std=1.0: (torch.randn(*s, generator=gd, device="cuda") * std).to(dt)
    if case["op"] == "copy":
        L, H, P, pages, n = case["layers"], case["H"], case["P"], case["pages"], case["pairs"]
        _memory(st, 1, pages, P, H, L, [0], dt, gc, gd, 0.64)
        ids = torch.randperm(pages, generator=gc)[:2 * n].int().cuda()
        st.src, st.dst = ids[:n].contiguous(), ids[n:].contiguous()
    elif case["op"] == "append":
        L, B, H, N, P = case["layers"], case["B"], case["H"], case["N"], case["P"]
        slots = -(-(max(case["hi"], case["keep"]) + N) // P) + 1
        _memory(st, B, slots, P, H, L, _fills(case), dt, gc, gd, 0.64)
        counts = _counts(case)
        # keys and values as the projection leaves them: [B, N, H, 64] per layer
        kv = rand(L, B, N, 2, H, DH, std=0.64)
        st.k = kv[:, :, :, 0].transpose(2, 3)
        st.v = kv[:, :, :, 1].transpose(2, 3)
        st.n = torch.tensor(counts, dtype=torch.int32).cuda()
        st.width = max(counts)
        st.rows = _paths(B, N, counts, st.width, gc).cuda() if case["accept"] else None
        st.begin_out, st.fill_out = torch.zeros_like(st.begin), torch.zeros_like(st.fill)
    else:
        B, H, N, P = case["B"], case["H"], case["N"], case["P"]
        fills = _fills(case)
        slots = -(-(max(fills) + N) // P) + 1
        _memory(st, B, slots, P, H, 2, fills, dt, gc, gd, 0.64)
        st.layer = 1
        # q, and k and v, as their projections leave them: [B, N, (2,) H, 64]
        st.q = rand(B, N, H, DH, std=0.64).transpose(1, 2)
        kv = rand(B, N, 2, H, DH, std=0.64)
        st.k, st.v = (kv[:, :, i].transpose(1, 2) for i in range(2))
        st.r_rows = max(fills) + N
        st.r = rand(H, st.r_rows, DH, std=0.45)
        st.u, st.v_bias = rand(H, DH, std=0.02), rand(H, DH, std=0.02)
        st.parents = _parents(case["shape"], B, N, gc).cuda()
        st.n = torch.tensor(_counts(case), dtype=torch.int32).cuda() if case["short"] else None
        st.out = torch.zeros(B, N, H, DH, dtype=dt, device="cuda").transpose(1, 2)
        st.lse = torch.zeros(B, H, N, dtype=torch.float32, device="cuda")
        st.scale = 1.0 / math.sqrt(DH)
    if own:
        import transformer_xl_relative_pos_gb300 as txl
        st.txl = txl
        st.mem = txl.PagedKV(st.pool, st.table, st.begin, st.fill)
    return st


# ---------------------------------------------------------------------------
# the operators
# ---------------------------------------------------------------------------

def run(st):
    op = st.case["op"]
    if own:
        if op == "copy":
            st.txl.paged_copy(st.mem, st.src, st.dst)
            return st.pool
        if op == "append":
            st.txl.paged_append(st.mem, st.k, st.v, n_new=st.n, rows=st.rows,
                                keep=st.case["keep"], state_out=(st.begin_out, st.fill_out))
            return [st.pool, st.begin_out, st.fill_out]
        out, lse = st.txl.relattn_tree_fwd(st.q, st.k, st.v, st.mem, st.layer, st.r, st.u,
                                           st.v_bias, st.parents, st.scale, n_nodes=st.n,
                                           out=st.out, lse=st.lse)
        return [out, lse]
    if op == "copy":
        st.pool[:, st.dst.long()] = st.pool[:, st.src.long()]
        return st.pool
    if op == "append":
        return _append_plain(st)
    return _tree_plain(st)


def _table_rows(st, t):
    """Page and row of the page of the memory rows t [B, T]."""
    P = st.case["P"]
    x = (st.begin[:, None].long() + t) % (st.table.shape[1] * P)
    return torch.gather(st.table.long(), 1, x // P), x % P


def _append_plain(st):
    case = st.case
    L, B, H = case["layers"], case["B"], case["H"]
    t = torch.arange(st.width, device="cuda").expand(B, -1)
    keep = t < st.n[:, None]
    page, row = _table_rows(st, st.fill[:, None].long() + t)
    b = torch.arange(B, device="cuda")[:, None].expand_as(t)[keep]
    src = (t if st.rows is None else st.rows.long())[keep]
    page, row = page[keep], row[keep]
    pool = st.pool.view(L, 2, *st.pool.shape[1:])
    # [L, rows, H, 64] with the indexed axes moved together
    pool[:, 0].transpose(2, 3)[:, page, row] = st.k.transpose(2, 3)[:, b, src]
    pool[:, 1].transpose(2, 3)[:, page, row] = st.v.transpose(2, 3)[:, b, src]
    total = st.fill + st.n
    st.fill_out = torch.clamp(total, max=case["keep"])
    st.begin_out = (st.begin + total - st.fill_out) % (st.table.shape[1] * case["P"])
    return [st.pool, st.begin_out, st.fill_out]


def _tree_plain(st):
    case = st.case
    B, H, N, P = case["B"], case["H"], case["N"], case["P"]
    F = st.table.shape[1] * P
    f32 = lambda x: x.float()
    # depth and ancestors (itself included) by doubling
    node = torch.arange(N, device="cuda")
    par = st.parents.long()
    anc = (node[None, :, None] == node).expand(B, N, N)      # anc[b, i, a]
    hop, depth = par, (par >= 0).long()
    for _ in range(max(1, (N - 1).bit_length())):
        safe = hop.clamp(min=0)
        live = hop >= 0
        up = torch.gather(anc, 1, safe[:, :, None].expand(B, N, N)) & live[:, :, None]
        anc = anc | up
        depth = depth + torch.where(live, torch.gather(depth, 1, safe), torch.zeros_like(depth))
        hop = torch.where(live, torch.gather(hop, 1, safe), hop)
    # keys and values: the memory's rows out of their pages, then the nodes
    t = torch.arange(F, device="cuda").expand(B, -1)
    page, row = _table_rows(st, t)
    kp, vp = st.pool[2 * st.layer], st.pool[2 * st.layer + 1]
    k = torch.cat([f32(kp[page, :, row]).transpose(1, 2), f32(st.k)], 2)   # [B, H, F + N, 64]
    v = torch.cat([f32(vp[page, :, row]).transpose(1, 2), f32(st.v)], 2)
    fill = st.fill.long()[:, None, None]
    dist = torch.cat([fill + depth[:, :, None] - t[:, None],
                      depth[:, :, None] - depth[:, None]], 2)             # [B, N, F + N]
    seen = torch.cat([(t < st.fill[:, None])[:, None].expand(B, N, F), anc], 2)
    seen = seen & (dist < st.r_rows)
    q = f32(st.q)
    u, vb = f32(st.u)[None, :, None], f32(st.v_bias)[None, :, None]
    a = (q + u) @ k.transpose(2, 3)
    pos = (q + vb) @ f32(st.r).transpose(1, 2)                            # [B, H, N, r_rows]
    idx = (st.r_rows - 1 - dist).clamp(0, st.r_rows - 1)
    a = (a + torch.gather(pos, 3, idx[:, None].expand(B, H, N, F + N))) * st.scale
    a = torch.where(seen[:, None], a, torch.full_like(a, -math.inf))
    m = a.amax(3, keepdim=True)
    e = torch.exp(a - m)
    s = e.sum(3, keepdim=True)
    v = torch.where(torch.cat([t < st.fill[:, None],
                               torch.ones(B, N, dtype=torch.bool, device="cuda")], 1)[:, None, :, None],
                    v, torch.zeros_like(v))
    out = (e @ v) / s
    lse = (m + torch.log(s))[..., 0]
    if st.n is not None:
        live = node[None] < st.n[:, None]
        out = torch.where(live[:, None, :, None], out, f32(st.out))
        lse = torch.where(live[:, None], lse, st.lse)
    return [out.to(st.out.dtype), lse]


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    """What ``run`` returns, from the definitions, row by row and node by node
    on the CPU; None where the outputs are too many for that."""
    if work(case)["bytes"] > 4e8 or work(case)["flops"] > 4e10:
        return None
    st = prepare(case, seed)
    host = lambda x: x.detach().cpu()
    table, begin, fill = (host(x).numpy().astype(np.int64) for x in (st.table, st.begin, st.fill))
    P = case["P"]
    R = table.shape[1] * P

    def place(b, row):
        x = (int(begin[b]) + row) % R
        return int(table[b, x // P]), x % P

    if case["op"] == "copy":
        pool = host(st.pool)
        res = pool.clone()
        for s, d in zip(host(st.src).tolist(), host(st.dst).tolist()):
            res[:, d] = pool[:, s]
        return res.double()
    if case["op"] == "append":
        pool, k, v = host(st.pool).clone(), host(st.k), host(st.v)
        begin_out, fill_out = [], []
        for b, n in enumerate(_counts(case)):
            for t in range(n):
                page, row = place(b, int(fill[b]) + t)
                src = int(st.rows[b, t]) if st.rows is not None else t
                pool[0::2, page, :, row] = k[:, b, :, src]
                pool[1::2, page, :, row] = v[:, b, :, src]
            total = int(fill[b]) + n
            left = min(total, case["keep"])
            fill_out.append(left)
            begin_out.append((int(begin[b]) + total - left) % R)
        return [pool.double(), np.array(begin_out), np.array(fill_out)]
    H, N = case["H"], case["N"]
    q, k, v, r, u, vb = (host(x).double().numpy() for x in (st.q, st.k, st.v, st.r, st.u, st.v_bias))
    kp, vp = host(st.pool[2 * st.layer]), host(st.pool[2 * st.layer + 1])
    par = host(st.parents).numpy()
    out = np.zeros((case["B"], H, N, DH))
    lse = np.zeros((case["B"], H, N))
    for b, n in enumerate(_counts(case)):
        where = np.array([place(b, t) for t in range(int(fill[b]))], dtype=np.int64).reshape(-1, 2)
        mk = kp[where[:, 0], :, where[:, 1]].double().numpy()   # [fill, H, 64]
        mv = vp[where[:, 0], :, where[:, 1]].double().numpy()
        for i in range(n):
            path = [i]
            while par[b, path[-1]] >= 0:
                path.append(int(par[b, path[-1]]))
            depth = len(path) - 1
            # distances: to the memory's rows, then to the node's ancestors
            dist = np.concatenate([fill[b] + depth - np.arange(int(fill[b])), np.arange(depth + 1)])
            on = dist < st.r_rows
            for h in range(H):
                keys = np.concatenate([mk[:, h], k[b, h, path]])[on]
                vals = np.concatenate([mv[:, h], v[b, h, path]])[on]
                pos = r[h, st.r_rows - 1 - dist[on]]
                a = st.scale * (keys @ (q[b, h, i] + u[h]) + pos @ (q[b, h, i] + vb[h]))
                top = a.max()
                e = np.exp(a - top)
                out[b, h, i] = (e @ vals) / e.sum()
                lse[b, h, i] = top + np.log(e.sum())
    return [out, lse]
