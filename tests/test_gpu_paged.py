"""The paged memory's kernels against a plain model of it: rows put behind a
memory, the state advanced, pages copied ("Transformer-XL: Attentive Language
Models Beyond a Fixed-Length Context", §3.2: the memory takes the newest states).
All of them move values, so everything is compared bit for bit, over the whole
pool: what a call must not write has to be as it was."""

import numpy as np
import pytest
import torch

import transformer_xl_relative_pos_gb300 as txl
from parity import dev

pytestmark = pytest.mark.gpu

INDEX = -8
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def make(B, H, P, slots, layers, dtype, seed, spare=2, begin=None, fill=None):
    """A memory with random contents, its pages dealt out in random order."""
    g = torch.Generator().manual_seed(seed)
    n_pages = B * slots + spare
    pool = torch.randn(2 * layers, n_pages, H, P, 64, generator=g).to(DTYPES[dtype]).to(dev())
    table = torch.randperm(n_pages, generator=g)[:B * slots].view(B, slots).int().to(dev())
    R = slots * P
    begin = torch.randint(0, R, (B,), generator=g) if begin is None else torch.tensor(begin)
    fill = torch.randint(0, R + 1, (B,), generator=g) if fill is None else torch.tensor(fill)
    return txl.PagedKV(pool, table, begin.int().to(dev()), fill.int().to(dev())), g


def model_append(mem, k, v, layer, n, rows, keep):
    """(pool, begin, fill) after the append, on the host."""
    pool, table = mem.pool.cpu().clone(), mem.table.cpu().numpy()
    begin, fill = mem.begin.cpu().numpy().copy(), mem.fill.cpu().numpy().copy()
    if k.dim() == 4:
        k, v = k[None], v[None]
    k, v = k.cpu(), v.cpu()
    P, R = mem.page_rows, mem.rows
    for b in range(mem.B):
        m = min(max(n[b], 0), R - fill[b])
        for t in range(m):
            x = (begin[b] + fill[b] + t) % R
            page, src = table[b, x // P], t if rows is None else rows[b][t]
            if 0 <= page < mem.n_pages and 0 <= src < k.shape[-2]:
                for i in range(k.shape[0]):
                    pool[2 * (layer + i), page, :, x % P] = k[i, b, :, src]
                    pool[2 * (layer + i) + 1, page, :, x % P] = v[i, b, :, src]
        if keep is not None:
            left = min(fill[b] + m, keep)
            begin[b] = (begin[b] + fill[b] + m - left) % R
            fill[b] = left
    return pool, begin, fill


def check(mem, want, status=0):
    torch.cuda.synchronize()
    assert txl.device_status() == status
    pool, begin, fill = want
    assert torch.equal(mem.pool.cpu(), pool)
    np.testing.assert_array_equal(mem.begin.cpu().numpy(), begin)
    np.testing.assert_array_equal(mem.fill.cpu().numpy(), fill)
    assert int(mem.ticket) == 0


def operand(layers, B, H, N, dtype, g, layout):
    """k or v [layers, B, H, N, 64]: dense, as a projection's [B, N, 2, H, 64], or
    with padded rows."""
    if layout == "dense":
        t = torch.randn(layers, B, H, N, 64, generator=g).to(DTYPES[dtype]).to(dev())
        return t, t.flip(0).contiguous() if layers > 1 else (t + 1).contiguous()
    if layout == "stacked":
        t = torch.randn(layers, B, N, 2, H, 64, generator=g).to(DTYPES[dtype]).to(dev())
        return t[:, :, :, 0].transpose(2, 3), t[:, :, :, 1].transpose(2, 3)
    t = torch.randn(layers, B, H, N, 2, 72, generator=g).to(DTYPES[dtype]).to(dev())
    return t[..., 0, :64], t[..., 1, 8:]


# B, H, P, slots, layers, N, layout, dtype, fills (None: anything), counts
APPENDS = [
    (1, 1, 32, 1, 1, 1, "dense", "bf16", [0], [1]),
    (1, 8, 64, 9, 12, 26, "stacked", "bf16", [512], [5]),
    (3, 2, 32, 4, 2, 40, "stacked", "bf16", [0, 31, 88], [40, 33, 40]),
    (3, 3, 96, 2, 1, 100, "padded", "f32", [92, 1, 50], [100, 0, 99]),
    (4, 5, 128, 3, 2, 7, "padded", "bf16", None, [7, 0, -3, 90]),
    (2, 16, 64, 30, 1, 1600, "stacked", "bf16", [0, 200], [1600, 1333]),
    (70, 1, 32, 2, 1, 3, "dense", "f32", [60] * 70, [3] * 70),
]


@pytest.mark.parametrize("B,H,P,slots,layers,N,layout,dtype,fills,counts", APPENDS)
@pytest.mark.parametrize("in_place", [True, False])
def test_append_a_segment(B, H, P, slots, layers, N, layout, dtype, fills, counts, in_place):
    mem, g = make(B, H, P, slots, layers, dtype, seed=B * 100 + N, fill=fills)
    k, v = operand(layers, B, H, N, dtype, g, layout)
    n = torch.tensor(counts, dtype=torch.int32)
    room = mem.rows - mem.fill.cpu().numpy()
    counts = np.clip(counts, 0, N)
    over = INDEX if (counts > room).any() else 0
    keep = min(mem.rows, max(1, int(mem.fill.max()) + 2))
    pool, begin, fill = model_append(mem, k, v, 0, counts, None, keep)
    if in_place:
        txl.paged_append(mem, k, v, n_new=n.to(dev()), keep=keep)
        check(mem, (pool, begin, fill), over)
    else:
        old = mem.begin.cpu().numpy(), mem.fill.cpu().numpy()
        outs = torch.zeros_like(mem.begin), torch.zeros_like(mem.fill)
        txl.paged_append(mem, k, v, n_new=n.to(dev()), keep=keep, state_out=outs)
        check(mem, (pool, *old), over)
        np.testing.assert_array_equal(outs[0].cpu().numpy(), begin)
        np.testing.assert_array_equal(outs[1].cpu().numpy(), fill)


@pytest.mark.parametrize("B,H,P,layers,N,dtype", [(1, 2, 32, 3, 26, "bf16"), (5, 3, 64, 2, 64, "f32")])
def test_append_the_accepted_path(B, H, P, layers, N, dtype):
    mem, g = make(B, H, P, 4, layers, dtype, seed=7 + B, fill=list(range(40, 40 + B)))
    k, v = operand(layers, B, H, N, dtype, g, "stacked")
    counts = [(3 * b + 5) % 9 for b in range(B)]
    rows = [sorted(torch.randperm(N, generator=g)[:9].tolist()) for _ in range(B)]
    rows[0][1] = rows[0][0]                                  # the same row twice
    want = model_append(mem, k, v, 0, counts, rows, 44)
    txl.paged_append(mem, k, v, n_new=torch.tensor(counts, dtype=torch.int32).to(dev()),
                     rows=torch.tensor(rows, dtype=torch.int32).to(dev()), keep=44)
    check(mem, want)


def test_append_to_one_layer_leaves_the_state():
    mem, g = make(2, 2, 32, 3, 4, "bf16", seed=3, fill=[10, 50])
    k, v = operand(1, 2, 2, 9, "bf16", g, "stacked")
    want = model_append(mem, k[0], v[0], 2, [9, 9], None, None)
    txl.paged_append(mem, k[0], v[0], layer=2)
    check(mem, want)
    # layer by layer, then the state on its own
    txl.paged_advance(mem, 9, keep=55)
    np.testing.assert_array_equal(mem.fill.cpu().numpy(), [19, 55])
    np.testing.assert_array_equal(mem.begin.cpu().numpy(), [want[1][0], (want[1][1] + 4) % 96])
    txl.paged_advance(mem, torch.tensor([0, 200], dtype=torch.int32).to(dev()), keep=96)
    np.testing.assert_array_equal(mem.fill.cpu().numpy(), [19, 96])
    assert txl.device_status() == INDEX                      # 200 rows do not fit
    txl.paged_append(mem, k[0][:, :, :0], v[0][:, :, :0], keep=7)   # no rows: a smaller memory
    np.testing.assert_array_equal(mem.fill.cpu().numpy(), [7, 7])


def test_append_with_bad_indices_writes_the_good_rows_only():
    mem, g = make(3, 2, 32, 3, 1, "bf16", seed=4, begin=[30, 0, 5], fill=[0, 3, 60])
    mem.table[0, 1] = mem.n_pages
    mem.table[1, 0] = -1
    mem.table[2, 2] = 2 ** 31 - 1
    k, v = operand(1, 3, 2, 40, "bf16", g, "dense")
    rows = torch.arange(40).repeat(3, 1)
    rows[2, 3], rows[2, 4], rows[2, 5] = -1, 40, 2 ** 31 - 1
    want = model_append(mem, k[0], v[0], 0, [40, 40, 36], rows.tolist(), 96)
    txl.paged_append(mem, k[0], v[0], rows=rows.int().to(dev()), keep=96)
    check(mem, want, INDEX)


def test_a_state_out_of_range_is_brought_back():
    mem, g = make(4, 1, 32, 2, 1, "bf16", seed=6, begin=[-1, 64, 2 ** 31 - 1, -2 ** 31],
                  fill=[5, 70, -4, 2 ** 31 - 1])
    txl.paged_advance(mem, 3, keep=64)
    torch.cuda.synchronize()
    assert txl.device_status() == INDEX
    np.testing.assert_array_equal(mem.begin.cpu().numpy(), [63, 0, (2 ** 31 - 1) % 64, 0])
    np.testing.assert_array_equal(mem.fill.cpu().numpy(), [8, 64, 3, 64])


def test_a_sliding_memory_goes_around_its_ring():
    # Many segments through a table of four pages: the memory is always the
    # newest rows of everything appended, and the state comes back into range.
    B, H, P, keep = 2, 2, 32, 70
    mem, g = make(B, H, P, 4, 1, "bf16", seed=8, begin=[3, 120], fill=[0, 0])
    seen = [torch.empty(H, 0, 64, dtype=torch.bfloat16) for _ in range(B)]
    for s in range(30):
        k = torch.randn(B, H, 11, 64, generator=g).bfloat16()
        n = torch.tensor([s % 12, 11 - s % 12], dtype=torch.int32)
        txl.paged_append(mem, k.to(dev()), -k.to(dev()), n_new=n.to(dev()), keep=keep)
        pool, table = mem.pool.cpu(), mem.table.cpu()
        begin, fill = mem.begin.tolist(), mem.fill.tolist()
        for b in range(B):
            seen[b] = torch.cat([seen[b], k[b, :, :n[b]]], 1)[:, -keep:]
            assert fill[b] == seen[b].shape[1] and 0 <= begin[b] < mem.rows
            x = (begin[b] + torch.arange(fill[b])) % mem.rows
            page = table[b, x // P].long()
            assert torch.equal(pool[0, page, :, x % P].transpose(0, 1), seen[b])
            assert torch.equal(pool[1, page, :, x % P].transpose(0, 1), -seen[b])
    assert txl.device_status() == 0


@pytest.mark.parametrize("layers,H,P,dtype", [(1, 1, 32, "bf16"), (12, 8, 64, "bf16"), (2, 3, 96, "f32")])
@pytest.mark.parametrize("n", [0, 1, 7])
def test_copy_pages(layers, H, P, dtype, n):
    mem, g = make(1, H, P, 20, layers, dtype, seed=9 + n)
    ids = torch.randperm(20, generator=g)[:2 * n].int()
    want = mem.pool.cpu().clone()
    want[:, ids[n:].long()] = want[:, ids[:n].long()]
    txl.paged_copy(mem, ids[:n].to(dev()), ids[n:].to(dev()))
    check(mem, (want, mem.begin.cpu().numpy(), mem.fill.cpu().numpy()))


def test_copy_skips_bad_pairs():
    mem, _ = make(1, 2, 32, 8, 2, "bf16", seed=11)
    want = mem.pool.cpu().clone()
    want[:, 3] = want[:, 1]
    src = torch.tensor([1, -1, 2, mem.n_pages, 5, 2 ** 31 - 1], dtype=torch.int32)
    dst = torch.tensor([3, 4, mem.n_pages, 6, 5, -2 ** 31], dtype=torch.int32)
    txl.paged_copy(mem, src.to(dev()), dst.to(dev()))
    check(mem, (want, mem.begin.cpu().numpy(), mem.fill.cpu().numpy()), INDEX)


def test_append_and_copy_in_a_graph_and_on_another_stream():
    # A captured append advances the state at every replay.
    mem, g = make(2, 2, 32, 4, 2, "bf16", seed=12, fill=[0, 5])
    k, v = operand(2, 2, 2, 6, "bf16", g, "stacked")
    n = torch.tensor([6, 2], dtype=torch.int32, device=dev())
    src, dst = (torch.tensor([x], dtype=torch.int32, device=dev()) for x in (8, 9))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        txl.paged_append(mem, k, v, n_new=n, keep=20)
        txl.paged_copy(mem, src, dst)
    for _ in range(5):
        pool, begin, fill = model_append(mem, k, v, 0, [6, 2], None, 20)
        pool[:, 9] = pool[:, 8]
        graph.replay()
        check(mem, (pool, begin, fill))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        want = model_append(mem, k, v, 0, [6, 2], None, 20)
        txl.paged_append(mem, k, v, n_new=n, keep=20)
    side.synchronize()
    check(mem, want)


def test_the_same_row_twice_and_one_page_copied_to_several():
    mem, g = make(2, 3, 32, 4, 2, "bf16", seed=31, fill=[10, 40])
    k, v = operand(2, 2, 3, 5, "bf16", g, "stacked")
    rows = [[4, 4, 0, 4], [1, 1, 1, 1]]
    want = model_append(mem, k, v, 0, [4, 3], rows, 60)
    txl.paged_append(mem, k, v, rows=torch.tensor(rows, dtype=torch.int32, device=dev()),
                     n_new=torch.tensor([4, 3], dtype=torch.int32, device=dev()), keep=60)
    check(mem, want)
    pool = mem.pool.cpu().clone()
    free = [p for p in range(mem.n_pages) if p not in mem.table.cpu()]
    page = int(mem.table[0, 0])
    pool[:, free] = pool[:, [page] * len(free)]
    ids = lambda x: torch.tensor(x, dtype=torch.int32, device=dev())
    txl.paged_copy(mem, ids([page] * len(free)), ids(free))
    check(mem, (pool, *want[1:]))


def test_layers_appended_at_once_on_streams():
    # Without a state to advance, calls for different layers of one memory may overlap.
    mem, g = make(3, 4, 64, 6, 4, "bf16", seed=32, fill=[0, 100, 250])
    k, v = operand(4, 3, 4, 100, "bf16", g, "stacked")
    want = model_append(mem, k, v, 0, [100] * 3, None, 200)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    for i, s in enumerate(streams):
        txl.paged_append(mem, k[i], v[i], layer=i, stream=s)
    torch.cuda.synchronize()
    txl.paged_advance(mem, 100, keep=200)
    check(mem, want)


def test_calls_for_different_memories_at_once():
    mems = [make(3, 4, 64, 8, 2, "bf16", seed=20 + i, fill=[7, 100, 300]) for i in range(2)]
    ops = [operand(2, 3, 4, 90, "bf16", g, "stacked") for _, g in mems]
    want = [model_append(m, *o, 0, [90] * 3, None, 350) for (m, _), o in zip(mems, ops)]
    streams = [torch.cuda.Stream() for _ in mems]
    torch.cuda.synchronize()
    for (m, _), o, s in zip(mems, ops, streams):
        txl.paged_append(m, *o, keep=350, stream=s)
    torch.cuda.synchronize()
    for (m, _), w in zip(mems, want):
        check(m, w)


def test_the_binding_refuses():
    mem, g = make(2, 2, 32, 3, 2, "bf16", seed=30)
    k, v = operand(2, 2, 2, 6, "bf16", g, "dense")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev())
    for bad in (lambda: txl.paged_append(mem, k.float(), v.float()),
                lambda: txl.paged_append(mem, k, v[0]),
                lambda: txl.paged_append(mem, k[:, :1], v[:, :1]),
                lambda: txl.paged_append(mem, k.transpose(3, 4), v.transpose(3, 4)),
                lambda: txl.paged_append(mem, k.cpu(), v.cpu()),
                lambda: txl.paged_append(mem, k, v, n_new=i32(1)),
                lambda: txl.paged_append(mem, k, v, n_new=torch.ones(2, device=dev())),
                lambda: txl.paged_append(mem, k, v, rows=i32(1, 2)),
                lambda: txl.paged_append(mem, k, v, state_out=(mem.begin, mem.fill)),
                lambda: txl.paged_copy(mem, i32(1, 2), i32(3)),
                lambda: txl.paged_advance(mem, i32(1), keep=3),
                lambda: txl.PagedKV(mem.pool, mem.table.long()),
                lambda: txl.PagedKV(mem.pool[..., ::2], mem.table)):
        with pytest.raises(ValueError):
            bad()
    for bad, status in ((lambda: txl.paged_append(mem, k, v, layer=1), -4),
                        (lambda: txl.paged_append(mem, k, v, keep=97), -4),
                        (lambda: txl.paged_append(mem, k, v, keep=-1), -1),
                        (lambda: txl.paged_append(mem, k.expand(2, 2, 2, 6, 64)[:, :, :1].expand(2, 2, 2, 6, 64),
                                                  v, keep=3), -1),
                        (lambda: txl.paged_advance(mem, -1, keep=3), -1)):
        with pytest.raises(txl.TxlError) as e:
            bad()
        assert e.value.status == status
    assert txl.device_status() == 0


def test_bench_tree_line():
    import json
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "bench.py", "--tree", "--shapes", "2,5,200", "--calls", "2"], cwd=root,
                       capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-2000:]
    line = json.loads(r.stdout.strip().splitlines()[-1])["tree"]
    # keys and values of 2 x 16 x 205 rows, the table, q and out, the log-sums
    assert line["algorithmic_bytes"] == 2 * 64 * 16 * (2 * 2 * 205 + 205 + 2 * 2 * 5) + 4 * 2 * 16 * 5
    assert line["us_per_call"] > 0 and line["append_us"] > 0 and 0 < line["hbm_frac"]
