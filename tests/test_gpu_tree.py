"""txl_relattn_tree_fwd (attention for trees of drafted tokens over a paged memory)
against the 64-bit model of tests/tree_model.py, within that model's bounds: node
counts from one to 64, memories from none to long ones that begin and end inside
a tile and go around their ring, tables shorter than the memory, NaN and infinities in
every place that must have no influence, key ranges, layouts, both types."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import transformer_xl_relative_pos_gb300 as txl
from parity import dev
from tree_model import depths_and_ancestors, tree_attention

pytestmark = pytest.mark.gpu

INDEX = -8
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
MARK = 7.0  # what the outputs hold before a call


def tree(kind, B, N, g):
    par = torch.full((B, N), -1, dtype=torch.int32)
    for i in range(1, N):
        if kind == "chain":
            par[:, i] = i - 1
        elif kind == "wide":
            par[:, i] = torch.randint(-1, min(i, 3), (B,), generator=g).int()
        else:
            par[:, i] = torch.randint(max(-1, i - 5), i, (B,), generator=g).int()
    return par.to(dev())


class Case:
    """A memory whose unused page rows hold NaN, and operands for one call."""

    def __init__(self, B, H, N, fills, P=64, slots=None, layers=1, layer=0, kind="near", dtype="bf16",
                 r_rows=None, counts=None, layout="stacked", begin=None, std=1.0, scale=0.125, seed=0):
        g = self.g = torch.Generator().manual_seed(seed + 1000 * N + B)
        dt = DT[dtype]
        fills = [fills] * B if isinstance(fills, int) else list(fills)
        slots = slots or max(fills) // P + 2
        n_pages = B * slots + 1
        pool = torch.full((2 * layers, n_pages, H, P, 64), float("nan"))
        table = torch.randperm(n_pages, generator=g)[:B * slots].view(B, slots)
        R = slots * P
        begin = torch.randint(0, R, (B,), generator=g) if begin is None else torch.tensor(begin)
        for b in range(B):
            x = (int(begin[b]) + torch.arange(fills[b])) % R
            pool[2 * layer, table[b, x // P], :, x % P] = torch.randn(fills[b], H, 64, generator=g) * std
            pool[2 * layer + 1, table[b, x // P], :, x % P] = torch.randn(fills[b], H, 64, generator=g)
        self.mem = txl.PagedKV(pool.to(dt).to(dev()), table.int().to(dev()), begin.int().to(dev()),
                               torch.tensor(fills, dtype=torch.int32).to(dev()))
        self.layer, self.B, self.H, self.N, self.dt = layer, B, H, N, dt
        self.counts = [N] * B if counts is None else counts
        self.scale = scale
        self.parents = tree(kind, B, N, g)
        rnd = lambda *s, std=std: (torch.randn(*s, generator=g) * std).to(dt).to(dev())
        self.r = rnd(H, r_rows or max(fills) + N, 64)
        self.u, self.vb = rnd(H, 64), rnd(H, 64)
        qkv = rnd(B, N, 3, H, 64)
        self.q, self.k, self.v = (qkv[:, :, i].transpose(1, 2) for i in range(3))
        if layout == "dense":
            self.q, self.k, self.v = (t.contiguous() for t in (self.q, self.k, self.v))
        for b, n in enumerate(self.counts):
            for t in (self.q, self.k, self.v):
                t[b, :, max(0, n):] = float("nan")
        self.out = torch.full((B, N, H, 64), MARK, dtype=dt, device=dev()).transpose(1, 2)
        self.lse = torch.full((B, H, N), MARK, device=dev())

    def call(self, n_splits=0, **kw):
        n = None
        if self.counts != [self.N] * self.B:
            n = torch.tensor(self.counts, dtype=torch.int32).to(dev())
        return txl.relattn_tree_fwd(self.q, self.k, self.v, self.mem, self.layer, self.r, self.u, self.vb,
                                    self.parents, self.scale, n_nodes=n, out=self.out, lse=self.lse,
                                    n_splits=n_splits, **kw)

    def want(self):
        return tree_attention(self.q, self.k, self.v, self.mem, self.layer, self.r, self.u, self.vb,
                              self.parents, self.scale, self.counts)

    def check(self, n_splits=0, status=0, want=None):
        self.call(n_splits)
        torch.cuda.synchronize()
        assert txl.device_status() == status
        out, lse, out_b, lse_b = want or self.want()
        got, got_lse = self.out.cpu().double().numpy(), self.lse.cpu().double().numpy()
        left = np.isnan(lse)
        assert (got_lse[left] == MARK).all() and (got[left] == MARK).all()
        with np.errstate(invalid="ignore"):
            err, err_lse = np.abs(got - out), np.abs(got_lse - lse)
        err_lse[got_lse == lse] = 0
        bad = ~(err <= out_b) & ~left[..., None]
        assert not bad.any(), (f"out: {bad.sum()} of {bad.size}, first at {np.argwhere(bad)[0]}, "
                               f"worst {np.nanmax(err / np.maximum(out_b, 1e-300)):.3g} bounds")
        bad = ~(err_lse <= lse_b) & ~left
        assert not bad.any(), f"lse: first at {np.argwhere(bad)[0]}, {np.nanmax(err_lse):.3g}"


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [1, 2, 7, 8, 9, 16, 17, 31, 32, 33, 48, 49, 64])
def test_node_counts(N, dtype):
    Case(2, 2, N, [70, 131], dtype=dtype, seed=1).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kind", ["chain", "wide", "near"])
@pytest.mark.parametrize("N", [16, 64])
def test_shapes_of_trees(kind, N, dtype):
    Case(3, 1, N, [0, 33, 200], kind=kind, dtype=dtype, P=32, seed=2).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [3, 20, 40])
@pytest.mark.parametrize("P,slots", [(32, 3), (64, 2), (96, 1), (128, 1)])
def test_memories_in_their_ring(P, slots, N, dtype):
    # every length from none to all rows of the table, from every kind of first row
    R = P * slots
    fills = [0, 1, 2, 31, 32, 33, 63, 64, 65, R - 1, R, R]
    begin = [5, 0, R - 1, 1, 0, 31, 17, 32, R - 64, R - 1, 0, 33]
    Case(12, 1, N, fills, P=P, slots=slots, begin=begin, dtype=dtype, seed=3).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,n_splits", [(1, 1), (5, 2), (16, 8), (26, 3), (30, 8), (64, 1), (50, 7)])
def test_key_ranges(N, n_splits, dtype):
    c = Case(2, 2, N, [901, 30], dtype=dtype, seed=4)
    want = c.want()
    c.check(n_splits, want=want)
    c.check(0, want=want)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("r_rows", [1, 2, 5, 31, 32, 40, 63, 64, 65, 100, 164, 400])
@pytest.mark.parametrize("N", [9, 30, 64])
def test_tables_shorter_and_longer_than_the_memory(N, r_rows, dtype):
    Case(2, 1, N, [100, 64], r_rows=r_rows, kind="chain", dtype=dtype, seed=5).check(2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,counts", [(12, [12, 0, 1, 5]), (32, [17, 32, 0, 16]), (64, [64, 3, 33, -2]),
                                      (4, [9, 4, 3, 1])])
def test_sequences_of_fewer_nodes(N, counts, dtype):
    c = Case(4, 2, N, [40, 500, 0, 77], counts=counts, dtype=dtype, seed=6)
    c.check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layouts_layers_and_one_tree_for_all(dtype):
    c = Case(3, 4, 11, [50, 60, 0], layers=3, layer=2, layout="dense", dtype=dtype, seed=7)
    c.check()
    c.parents = c.parents[1].contiguous()
    c.check()
    a = txl.relattn_tree_fwd(c.q, c.k, c.v, c.mem, 2, c.r, c.u, c.vb, c.parents, 0.125)
    b, lse = txl.relattn_tree_fwd(c.q, c.k, c.v, c.mem, 2, c.r, c.u, c.vb, c.parents, 0.125, lse=True)
    assert torch.equal(a, b) and torch.equal(a, c.out) and torch.equal(lse, c.lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_memories(dtype):
    Case(2, 2, 16, [3800, 2711], dtype=dtype, P=128, seed=8, std=0.6).check()
    Case(1, 1, 1, [12000], dtype=dtype, seed=9, std=0.6).check()
    Case(1, 2, 64, [3800], dtype=dtype, seed=10, std=0.6).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_sharp_scores(dtype):
    Case(2, 2, 26, [300, 77], dtype=dtype, seed=11, std=4.0).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("N", [6, 40])
def test_what_a_node_does_not_see_has_no_influence(N, value, dtype):
    # Node 1's key and value are not finite: only its descendants may notice.  A memory
    # row that the table reaches from some nodes only, likewise.
    c = Case(1, 2, N, [80], dtype=dtype, seed=12, r_rows=84)
    want = c.want()
    depth, anc = depths_and_ancestors(c.parents[0].cpu().numpy())
    free = ~anc[:, 1]
    assert 0 < free.sum() < N and depth.max() > 5 if N > 6 else True
    c.k[0, :, 1, 3] = value
    c.v[0, :, 1] = value
    c.call()
    torch.cuda.synchronize()
    got, out, bound = c.out.cpu().double().numpy()[0], want[0][0], want[2][0]
    assert (np.abs(got - out)[:, free] <= bound[:, free]).all()
    assert not np.isfinite(got[:, ~free]).any()
    assert np.isnan(c.lse.cpu().numpy()[0][:, ~free]).all() or np.isinf(value)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [8, 30, 64])
def test_rows_past_the_table_have_no_influence(N, dtype):
    # The oldest rows the table reaches from shallow nodes hold infinities that deep
    # nodes do not see, and rows older than the table's reach hold NaN.
    r_rows, F = 60, 100
    c = Case(1, 2, N, [F], kind="chain", dtype=dtype, seed=13, r_rows=r_rows, begin=[7])
    depth = np.arange(N)
    want = c.want()
    x = (7 + torch.arange(F)) % c.mem.rows
    page, row = c.mem.table[0].cpu()[x // 64].long(), x % 64
    for t in range(F):
        if F - t >= r_rows:           # seen by no node
            c.mem.pool[:, page[t], :, row[t]] = float("nan")
        elif F + 3 - t >= r_rows:     # seen by nodes of depth 0, 1 or 2 only
            c.mem.pool[1, page[t], :, row[t]] = float("inf")
    c.call(2)
    torch.cuda.synchronize()
    got = c.out.cpu().double().numpy()[0]
    assert not np.isfinite(got[:, depth < 3]).any()
    assert (np.abs(got - want[0][0]) <= want[2][0])[:, depth >= 3].all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_in_what_is_seen_shows(dtype):
    c = Case(2, 1, 20, [90, 90], dtype=dtype, seed=14)
    c.q[0, 0, 4, 9] = float("nan")
    c.call()
    torch.cuda.synchronize()
    out, lse = c.out.cpu(), c.lse.cpu()
    assert torch.isnan(out[0, 0, 4]).all() and torch.isnan(lse[0, 0, 4])
    ok = torch.ones(2, 1, 20, dtype=torch.bool)
    ok[0, 0, 4] = False
    assert torch.isfinite(out[ok]).all() and torch.isfinite(lse[ok]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [5, 33])
def test_bad_pages_and_parents(N, dtype):
    c = Case(3, 2, N, [200, 150, 64], dtype=dtype, seed=15, begin=[0, 100, 0], slots=4)
    c.mem.table[0, 1] = c.mem.n_pages
    c.mem.table[1, 2] = -5
    c.mem.table[2, 0] = 2 ** 31 - 1
    c.parents[0, 2] = 2                   # itself
    c.parents[1, 1] = 77                  # no such node
    c.parents[2, 3] = -2 ** 31
    c.check(2, status=INDEX)


@pytest.mark.parametrize("N,n_splits", [(1, 0), (4, 1), (8, 2)])
def test_a_chain_is_a_decoding_step(N, n_splits):
    # The same keys through txl_relattn_fwd's dense decode kernels: two kernels of one
    # formula, each within its own half step of it.
    c = Case(2, 3, N, [300, 300], kind="chain", seed=16, layout="dense")
    c.check(n_splits)
    x = (c.mem.begin[:, None].long() + torch.arange(300, device=dev())) % c.mem.rows
    page, row = torch.gather(c.mem.table.long(), 1, x // 64), x % 64
    kx, vx = (torch.cat([c.mem.pool[i][page, :, row].transpose(1, 2), t], 2).contiguous()
              for i, t in ((0, c.k), (1, c.v)))
    dense = txl.relattn_fwd(c.q, kx, vx, c.r, c.u, c.vb, 300, 0.125)
    err = (dense.double() - c.out.double()).abs()
    assert (err <= 2.0 ** -7 * c.out.double().abs() + 1e-3).all()


def test_results_repeat_bit_for_bit():
    for N in (3, 26, 64):
        c = Case(4, 4, N, [700, 10, 0, 333], seed=17)
        c.call()
        first = c.out.clone(), c.lse.clone()
        for _ in range(3):
            c.out.fill_(0), c.lse.fill_(0)
            c.call()
            assert torch.equal(c.out, first[0]) and torch.equal(c.lse, first[1])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_graphs_and_streams(dtype):
    # Captured once, replayed for other lengths, trees and contents: all of it lies on
    # the device.  Two graphs and an eager call at once share nothing.
    cs = [Case(2, 2, 12, [200, 64], P=32, slots=9, dtype=dtype, seed=18 + i) for i in range(2)]
    graphs = []
    for c in cs:
        c.call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.call()
        graphs.append(graph)
    for c in cs:
        c.mem.fill.copy_(torch.tensor([150, 3]))
        c.mem.begin.add_(torch.tensor([50, 61], device=dev())).remainder_(c.mem.rows)
        c.parents.copy_(tree("wide", 2, 12, c.g))
        c.q.neg_()
        c.out.fill_(0)
    third = Case(2, 2, 40, [300, 1], dtype=dtype, seed=20)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for graph, s in zip(graphs, streams):
        with torch.cuda.stream(s):
            graph.replay()
    third.call(stream=streams[2])
    torch.cuda.synchronize()
    for c in cs + [third]:
        out, lse, out_b, lse_b = c.want()
        assert (np.abs(c.out.cpu().double().numpy() - out) <= out_b).all()
        assert (np.abs(c.lse.cpu().double().numpy() - lse) <= lse_b).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.0, -0.125, 0.3, -1e-3])
@pytest.mark.parametrize("N", [5, 13, 30, 64])
def test_scales_of_either_sign(N, scale, dtype):
    Case(2, 2, N, [130, 33], scale=scale, r_rows=120, dtype=dtype, seed=23).check(2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,H,slots", [(40, 10, 64), (64, 5, 64), (33, 16, 64), (40, 10, 6), (65, 5, 64), (256, 2, 6)])
def test_many_sequences_of_unlike_lengths(B, H, slots, dtype):
    # more blocks than are resident at once: the longest memories come first (up to 64
    # sequences, with tables of 2048 rows and more); equal lengths and sequences without
    # nodes among them
    g = torch.Generator().manual_seed(B)
    fills = torch.randint(0, 130, (B,), generator=g).tolist()
    fills[1] = fills[7] = fills[B - 1]
    counts = [2] * B
    counts[3] = counts[B - 2] = 0
    Case(B, H, 2, fills, P=32, slots=slots, counts=counts, dtype=dtype, seed=24).check()


def test_outputs_made_by_the_call_belong_to_its_stream():
    # Work waits on the current stream; a call on another stream must not come to lie
    # before the filling of its own outputs.
    c = Case(2, 2, 12, [100, 40], counts=[12, 5], seed=25)
    n = torch.tensor(c.counts, dtype=torch.int32).to(dev())
    args = (c.q, c.k, c.v, c.mem, 0, c.r, c.u, c.vb, c.parents, 0.125)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    big = torch.randn(4096, 4096, device=dev())
    for stream in (side, side.cuda_stream):
        for _ in range(20):
            big = torch.mm(big, big).clamp_(-1, 1)
        out, lse = txl.relattn_tree_fwd(*args, n_nodes=n, lse=True, stream=stream)
        torch.cuda.synchronize()
        want, want_lse, out_b, lse_b = c.want()
        left = np.isnan(want_lse)
        assert (out.float().cpu().numpy()[left] == 0).all() and (lse.cpu().numpy()[left] == 0).all()
        assert (np.abs(out.cpu().double().numpy() - want) <= out_b)[~left].all()
        assert (np.abs(lse.cpu().double().numpy() - want_lse) <= lse_b)[~left].all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_offsets_past_32_bits(dtype):
    # Pages behind 2^33 bytes of a plane: rows appended to them, attended to and copied,
    # as in a small pool, bit for bit.
    dt, H, P, B, N = DT[dtype], 2, 128, 2, 20
    size = H * P * 64
    far = (2 ** 33) // (size * dt.itemsize)
    big = txl.PagedKV(torch.empty(2, far + 8, H, P, 64, dtype=dt, device=dev()),
                      torch.tensor([[far + 1, far + 4], [far + 6, far + 3]], dtype=torch.int32, device=dev()))
    small = txl.PagedKV(torch.empty(2, 8, H, P, 64, dtype=dt, device=dev()),
                        torch.tensor([[1, 4], [6, 3]], dtype=torch.int32, device=dev()))
    g = torch.Generator().manual_seed(26)
    rnd = lambda *s: torch.randn(*s, generator=g).to(dt).to(dev())
    k, v = rnd(B, H, 200, 64), rnd(B, H, 200, 64)
    q, kn, vn = rnd(B, H, N, 64), rnd(B, H, N, 64), rnd(B, H, N, 64)
    r, u, vb, parents = rnd(H, 200, 64), rnd(H, 64), rnd(H, 64), tree("near", B, N, g)
    got = []
    for mem, at in ((big, far), (small, 0)):
        txl.paged_append(mem, k, v, keep=200)
        out = [txl.relattn_tree_fwd(q, kn, vn, mem, 0, r, u, vb, parents, 0.125)]
        ids = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev()) + at
        txl.paged_copy(mem, ids(1, 6), ids(0, 7))
        mem.table.copy_(torch.stack([ids(0, 4), ids(7, 3)]))
        mem.pool[:, at + 1].zero_(), mem.pool[:, at + 6].zero_()
        out.append(txl.relattn_tree_fwd(q, kn, vn, mem, 0, r, u, vb, parents, 0.125))
        got.append(out)
    assert txl.device_status() == 0
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[0][0])
    assert torch.equal(got[1][1], got[1][0]) and torch.isfinite(got[0][0]).all()
    del big
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_first_call_of_a_process_may_be_captured(dtype):
    # (attributes and occupancy of the kernels are looked up during a capture then)
    code = ("import sys; sys.path[:0] = ['tests', '.']\n"
            "import torch, numpy as np\n"
            "from test_gpu_tree import Case\n"
            f"c = Case(2, 2, 12, [200, 64], dtype='{dtype}', seed=27)\n"
            "torch.cuda.synchronize()\n"
            "g = torch.cuda.CUDAGraph()\n"
            "with torch.cuda.graph(g):\n"
            "    c.call()\n"
            "g.replay()\n"
            "torch.cuda.synchronize()\n"
            "out, lse, out_b, lse_b = c.want()\n"
            "assert (np.abs(c.out.cpu().double().numpy() - out) <= out_b).all()\n"
            "print('ok')\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stderr[-3000:]


def test_drafting_together():
    # A stream as it runs: a prompt appended, then rounds of a drafted tree attended
    # to, its accepted path appended and the memory slid; against the model, and the memory's
    # contents against the accepted rows in order.
    B, H, N, keep = 2, 2, 12, 90
    g = torch.Generator().manual_seed(21)
    pool = torch.full((2, 9, H, 32, 64), float("nan"), dtype=torch.bfloat16, device=dev())
    table = torch.tensor([[3, 1, 7, 5], [0, 8, 2, 6]], dtype=torch.int32, device=dev())
    mem = txl.PagedKV(pool, table)
    rnd = lambda *s: torch.randn(*s, generator=g).bfloat16().to(dev())
    prompt = rnd(2, B, 40, H, 64)
    txl.paged_append(mem, prompt[0].transpose(1, 2), prompt[1].transpose(1, 2), keep=keep)
    history = [prompt[:, b].cpu() for b in range(B)]
    r, u, vb = rnd(H, keep + N, 64), rnd(H, 64), rnd(H, 64)
    for step in range(12):
        qkv = rnd(3, B, N, H, 64).transpose(2, 3)
        parents = tree("near", B, N, g)
        args = (qkv[0], qkv[1], qkv[2], mem, 0, r, u, vb, parents, 0.125)
        got, lse = txl.relattn_tree_fwd(*args, lse=True)
        out, want_lse, out_b, lse_b = tree_attention(*args, [N] * B)
        assert (np.abs(got.cpu().double().numpy() - out) <= out_b).all()
        assert (np.abs(lse.cpu().double().numpy() - want_lse) <= lse_b).all()
        path = torch.full((B, N), -1, dtype=torch.int32)
        n = torch.zeros(B, dtype=torch.int32)
        for b in range(B):
            i, chain = int(torch.randint(0, N, (1,), generator=g)), []
            while i >= 0:
                chain.insert(0, i)
                i = int(parents[b, i])
            path[b, :len(chain)] = torch.tensor(chain)
            n[b] = len(chain)
            rows = qkv[1:, b].cpu().transpose(1, 2)[:, chain]
            history[b] = torch.cat([history[b], rows], 1)[:, -keep:]
        txl.paged_append(mem, qkv[1], qkv[2], rows=path.to(dev()), n_new=n.to(dev()), keep=keep)
        for b in range(B):
            fill = int(mem.fill[b])
            assert fill == history[b].shape[1]
            x = (int(mem.begin[b]) + torch.arange(fill)) % mem.rows
            held = mem.pool.cpu()[:, table[b].cpu()[x // 32].long(), :, x % 32].transpose(0, 1)
            assert torch.equal(held, history[b])
    assert txl.device_status() == 0


def test_the_binding_refuses():
    c = Case(2, 2, 6, [10, 20], seed=22)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev())
    base = dict(q=c.q, k=c.k, v=c.v, r=c.r, u=c.u, vb=c.vb, parents=c.parents, out=None, lse=None, n=None)

    def call(**kw):
        a = dict(base, **kw)
        return txl.relattn_tree_fwd(a["q"], a["k"], a["v"], c.mem, a.get("layer", 0), a["r"], a["u"], a["vb"],
                                    a["parents"], a.get("scale", 0.125), n_nodes=a["n"], out=a["out"],
                                    lse=a["lse"], n_splits=a.get("n_splits", 0))
    for kw in (dict(q=c.q.float()), dict(q=c.q[:, :1]), dict(k=c.k[:, :, :5]), dict(q=c.q.cpu()),
               dict(r=c.r[:1]), dict(r=c.r.float()), dict(u=c.u[0]), dict(parents=c.parents[:, :5]),
               dict(parents=c.parents.long()), dict(n=i32(1)), dict(n=torch.ones(2, device=dev())),
               dict(lse=torch.zeros(2, 2, 6, dtype=torch.float64, device=dev())),
               dict(lse=torch.zeros(2, 6, 2, device=dev())), dict(out=torch.zeros_like(c.q, dtype=torch.float32)),
               dict(q=c.q.transpose(2, 3).contiguous().transpose(2, 3))):
        with pytest.raises((ValueError, TypeError)):
            call(**kw)
    wide = torch.zeros(2, 2, 65, 64, dtype=torch.bfloat16, device=dev())
    for kw, status in ((dict(layer=1), -4), (dict(layer=-1), -1), (dict(scale=float("nan")), -1),
                       (dict(n_splits=9), -2), (dict(n_splits=-1), -1),
                       (dict(q=wide, k=wide, v=wide, parents=torch.zeros(65, dtype=torch.int32, device=dev())), -2),
                       (dict(k=c.k[:1].expand(2, 2, 6, 64)), -1)):
        with pytest.raises(txl.TxlError) as e:
            call(**kw)
        assert e.value.status == status, kw
    call()
    assert txl.device_status() == 0
