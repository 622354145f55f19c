"""The paged stack's host side on the CPU: with fakes of the device calls (the attention of a draft
by the 64-bit model of tests/tree_model.py), restoring checkpoints,
what accept takes, and taps."""

import numpy as np
import pytest
import torch

import oracle
import txl_inputs
from test_paged_host import FakeKV, fake_append, fake_copy
from tree_model import tree_attention
from transformer_xl_relative_pos_gb300 import model, paged

W = txl_inputs.Workload("paged_host", B=2, H=2, dh=4, L=8, M=70, d_model=8, dtype="f32", seed=61,
                        d_ff=16, n_layer=2, n_seg=3, vocab=31)


def fake_tree(q, k_new, v_new, mem, layer, r, u, v_bias, parents, scale, *, n_nodes=None, out=None, **kw):
    B, N = q.shape[0], q.shape[2]
    counts = [N] * B if n_nodes is None else n_nodes.tolist()
    got = torch.from_numpy(tree_attention(q, k_new, v_new, mem, layer, r, u, v_bias, parents, scale, counts)[0])
    out.copy_(torch.where(torch.isnan(got), out.double(), got))
    return out


@pytest.fixture(autouse=True)
def on_the_cpu(monkeypatch):
    monkeypatch.setattr(paged.txl, "PagedKV", FakeKV)
    monkeypatch.setattr(paged.txl, "paged_copy", fake_copy)
    monkeypatch.setattr(paged.txl, "paged_append", fake_append)
    monkeypatch.setattr(model.txl, "relattn_tree_fwd", fake_tree)
    monkeypatch.setattr(model.txl, "rel_pos_emb", lambda K, d, dtype, device: torch.from_numpy(
        oracle.reversed_table(oracle.sinusoid_table(K, d))).to(dtype))


def stack(M=W.M, H=W.H):
    return model.XLStack(txl_inputs.draw_stack(W), H, M, "cpu", torch.float32, paged=True)


def tokens(B, N, seed=0):
    return torch.randint(0, W.vocab, (B, N), generator=torch.Generator().manual_seed(seed))


def memory(M, max_new, P=32, fill=0):
    mem = paged.PagedMemory(1, 2, 1, M, max_new, device="cpu", dtype=torch.float32, page_rows=P, dh=2)
    while mem.fill[0] < fill:
        k = torch.ones(1, 2, 1, min(max_new, fill - mem.fill[0]), 2)
        mem.append(k, k)
    return mem


@pytest.mark.parametrize("theirs,ours,P", [((150, 10), (60, 100), 32), ((60, 100), (150, 10), 32),
                                           ((128, 64), (70, 64), 64), ((70, 64), (128, 64), 64)])
def test_a_checkpoint_of_another_memory_length_is_refused(theirs, ours, P):
    # The tables have one shape, the lengths that the memories slide by do not.
    a, b = memory(*theirs, P, fill=theirs[0]), memory(*ours, P, fill=20)
    assert a.kv.table.shape == b.kv.table.shape
    before = b._table.copy(), list(b.begin), list(b.fill), b.pages.n_free, b.kv.pool.clone()
    with pytest.raises(ValueError):
        b.restore(a.checkpoint())
    assert (b._table == before[0]).all() and (b.begin, b.fill) == before[1:3]
    assert b.pages.n_free == before[3] and torch.equal(b.kv.pool, before[4])


def test_a_checkpoint_that_names_no_length_is_refused_by_its_fills():
    # (as an earlier version wrote them)
    a = memory(128, 64, 64, fill=100)
    ck = a.checkpoint()
    ck = {k: ck[k] for k in ("pool", "table", "begin", "fill", "users")}
    with pytest.raises(ValueError):
        memory(70, 64, 64).restore(ck)
    b = memory(128, 64, 64)
    b.restore(ck)
    assert b.fill == [100, 100]


def test_a_refused_checkpoint_leaves_the_stack_as_it_is():
    a, other = stack(), stack(M=40)
    for s in (a, other):
        s.segment(tokens(2, 8, seed=1))
    h = a.draft(tokens(2, 3, seed=2), torch.tensor([-1, 0, 0]))
    memory, ck = a.memory, other.checkpoint()
    for bad in (ck, {"paged": dict(a.checkpoint()["paged"], M=71)},
                {"paged": dict(a.checkpoint()["paged"], pool=ck["paged"]["pool"].double())}):
        with pytest.raises(ValueError):
            a.restore(bad)
        assert a.memory is memory and a.memory.fill == [8, 8]
    assert torch.equal(a.draft(tokens(2, 3, seed=2), torch.tensor([-1, 0, 0])), h)
    a.accept([[0, 2], [0]])
    assert a.memory.fill == [10, 9]


def test_a_checkpoint_resumes():
    a, b = stack(), stack()
    a.segment(tokens(2, 8, seed=1))
    ck = a.checkpoint()
    want = a.segment(tokens(2, 5, seed=2))
    b.segment(tokens(2, 9, seed=3))
    b.draft(tokens(2, 2, seed=4), torch.tensor([-1, 0]))
    b.restore(ck)
    with pytest.raises(RuntimeError):
        b.accept([[0], [0]])                 # (what was drafted before is of another memory)
    assert torch.equal(b.segment(tokens(2, 5, seed=2)), want)


@pytest.mark.parametrize("form", ["tensor", "list"])
def test_only_paths_of_drafted_nodes_are_accepted(form):
    # Sequence 0: 0 -> 1 -> 2, 0 -> 3 -> 4 -> 5; sequence 1: 0 -> 1, 2 -> 3 (4 and 5 are not drafted).
    parents, n_nodes = [[-1, 0, 1, 0, 3, 4], [-1, 0, -1, 2, 3, 4]], [6, 4]
    a = stack()
    a.segment(tokens(2, 8, seed=1))
    if form == "tensor":
        parents, n_nodes = torch.tensor(parents), torch.tensor(n_nodes)
    a.draft(tokens(2, 6, seed=2), parents, n_nodes)
    for bad in ([[0, 1, 3], []],             # 3 follows 0
                [[0, 2], []], [[1], []],     # an ancestor left out
                [[1, 0], []], [[0, 0], []],  # out of order, twice
                [[], [2, 3, 4]], [[], [4]],  # behind the sequence's nodes
                [[], [0, 1, 2]],             # another root's
                [[6], []], [[-1], []], [[0]], [[0], [0], [0]]):
        with pytest.raises(ValueError):
            a.accept(bad)
        assert a.memory.fill == [8, 8]
    if form == "tensor":                     # what the caller does with them afterwards is of no account
        parents.fill_(-1), n_nodes.zero_()
    a.accept([[0, 3, 4], (2, 3)])
    assert a.memory.fill == [11, 10]


def test_one_tree_for_all_and_parents_that_are_no_earlier_nodes():
    a = stack()
    a.draft(tokens(2, 4, seed=3), torch.tensor([9, 0, 2, -7]))   # node 0, 2 and 3 follow the memory
    with pytest.raises(ValueError):
        a.accept([[0, 1, 2], []])
    a.accept([[0, 1], np.array([3])])
    assert a.memory.fill == [2, 1]


def test_taps_of_a_draft_hold_every_layer():
    # Sequences of 8 and 10 rows, and a chain of 5: each layer's attention and output follow from
    # what its tap holds, and a tap keeps it when the memory goes on.
    a = stack()
    a.segment(tokens(2, 8, seed=1))
    a.draft(tokens(2, 2, seed=2), torch.tensor([-1, 0]))
    a.accept([[], [0, 1]])
    a.taps = []
    h = a.segment(tokens(2, 5, seed=3))
    assert len(a.taps) == W.n_layer and torch.equal(a.taps[-1]["h_out"], h)
    a.segment(tokens(2, 8, seed=4))
    for n, tap in enumerate(a.taps[:W.n_layer]):
        assert tap["M"] == [8, 10] and torch.equal(tap["h"], a.taps[n - 1]["h_out"] if n else tap["h"])
        for b, M in enumerate(tap["M"]):
            k, v = (torch.cat([m, x[b]], 1)[None].double().numpy() for m, x in zip(tap["mem"][b], (tap["k"], tap["v"])))
            rel = oracle.distance_table(tap["r"][:, -(M + 5):].double().numpy())
            want, _ = oracle.relattn(tap["q"][b:b + 1], k, v, rel, a.u, a.v_bias, M, 5, a.scale)
            # (the attention is exact here, its output rounded to fp32)
            assert np.allclose(tap["a"][b].numpy(), want[0], rtol=2.0 ** -23, atol=1e-12)
            lay = {x: w.numpy() for x, w in a.layers[n].items()}
            out = oracle.layer_post(tap["a"][b:b + 1].transpose(1, 2).reshape(1, 5, -1), tap["h"][b:b + 1], lay)
            assert np.abs(tap["h_out"][b].numpy() - out[0]).max() < 1e-5
