"""The paged stack in 32 bits against the 64-bit streams of tests/paged_stack_model.py, whose bound
wrong paths, orders, forks and masks exceed by far; and the pages of every layer against the drafted
rows, bit for bit, in both types."""

import numpy as np
import pytest
import torch

import paged_stack_model as m
import transformer_xl_relative_pos_gb300 as txl
from parity import dev
from transformer_xl_relative_pos_gb300.model import XLStack

pytestmark = pytest.mark.gpu


def stack(dtype=torch.float32):
    return XLStack(m.params(), m.W.H, m.W.M, dev(), dtype, paged=True)


def error(got, want):
    return np.abs(got.double().cpu().numpy() - want).max()


@pytest.mark.parametrize("where", ["cpu", "cuda"])
def test_streams_draft_accept_fork_and_go_on(where):
    a = stack()
    a.segment(m.PROMPT)
    h = a.draft(m.DRAFT, torch.tensor(m.PARENTS, device=where), torch.tensor(m.N_NODES, device=where))
    for b in range(m.W.B):
        for node in range(m.N_NODES[b]):
            if node not in m.PARENTS[b]:     # a leaf
                assert error(h[b, m.path_to(b, node)], m.drafted(b, node)) < m.BOUND, (b, node)
    with pytest.raises(ValueError):
        a.accept([[], [11], []])
    a.accept(m.ACCEPTED)
    assert a.memory.fill == [35, 30, 40]
    a.fork(*m.FORK)
    want = m.continued()
    assert error(a.segment(m.MORE), want) < m.BOUND
    assert a.memory.fill == [40, 40, 40] and txl.device_status() == 0


def test_memories_that_slide_while_one_stands_still():
    # Accepted paths of unlike lengths, round after round, past M rows: sequence 2 accepts nothing
    # after the prompt, sequence 0 everything.
    a = stack()
    a.segment(m.PROMPT)
    taken = [[m.PROMPT[b]] for b in range(m.W.B)]
    for step in range(9):
        toks = m.tokens(7, 10 + step)
        a.draft(toks, torch.arange(-1, 6))
        n = [7, step % 4, 0]
        a.accept([range(x) for x in n])
        for b in range(m.W.B):
            taken[b].append(toks[b, :n[b]])
    h = a.draft(m.MORE, torch.arange(-1, 19))
    for b in range(m.W.B):
        assert error(h[b], m.run(taken[b] + [m.MORE[b]])) < m.BOUND, b
    assert a.memory.fill == [40, 40, 30] and txl.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_pages_hold_the_accepted_rows(dtype):
    a = stack(dtype)
    layers, seqs = range(m.W.n_layer), range(m.W.B)
    held = lambda: [[a.memory.rows(n, b) for b in seqs] for n in layers]
    a.segment(m.PROMPT)
    before = held()
    a.taps = []
    a.draft(m.DRAFT, torch.tensor(m.PARENTS), torch.tensor(m.N_NODES))
    a.accept(m.ACCEPTED)
    after = held()
    for n in layers:
        for b in seqs:
            for i, name in enumerate("kv"):
                rows = torch.cat([before[n][b][i], a.taps[n][name][b][:, m.ACCEPTED[b]]], 1)
                assert torch.equal(after[n][b][i], rows[:, -m.W.M:])
    # a fork holds the same rows, and each of the two then its own
    src, dst = m.FORK
    a.fork(src, dst)
    forked = held()
    for n in layers:
        assert all(torch.equal(x, y) for x, y in zip(forked[n][dst], after[n][src]))
        assert all(torch.equal(x, y) for b in (0, src) for x, y in zip(forked[n][b], after[n][b]))
    a.taps = []
    a.draft(m.MORE[:, :5], torch.arange(-1, 4))
    paths = [[], [0, 1], [0, 1, 2, 3, 4]]
    a.accept(paths)
    last = held()
    for n in layers:
        for b in seqs:
            for i, name in enumerate("kv"):
                rows = torch.cat([forked[n][b][i], a.taps[n][name][b][:, paths[b]]], 1)
                assert torch.equal(last[n][b][i], rows[:, -m.W.M:])
    assert txl.device_status() == 0


def test_a_checkpoint_of_a_stack_of_another_memory_is_refused():
    # 40 and 60 rows of memory make tables of one shape
    a = stack()
    a.segment(m.PROMPT)
    want = a.draft(m.MORE, torch.arange(-1, 19)).clone()
    other = XLStack(m.params(), m.W.H, 60, dev(), torch.float32, paged=True)
    other.segment(m.PROMPT)
    assert other.memory.kv.table.shape == a.memory.kv.table.shape
    with pytest.raises(ValueError):
        a.restore(other.checkpoint())
    assert a.memory.fill == [30, 30, 30]
    assert torch.equal(a.draft(m.MORE, torch.arange(-1, 19)), want)


@pytest.mark.parametrize("M", [0, 1, 40])
def test_nothing_accepted_changes_nothing(M):
    a = XLStack(m.params(), m.W.H, M, dev(), torch.float32, paged=True)
    a.segment(m.PROMPT)
    before = [[x.clone() for b in range(m.W.B) for x in a.memory.rows(n, b)] for n in range(m.W.n_layer)]
    want = a.draft(m.MORE, torch.arange(-1, 19)).clone()
    a.accept([[], [], []])
    assert a.memory.fill == [min(M, 30)] * m.W.B
    assert torch.equal(a.draft(m.MORE, torch.arange(-1, 19)), want)
    for n in range(m.W.n_layer):
        after = [x for b in range(m.W.B) for x in a.memory.rows(n, b)]
        assert all(x.shape[1] == min(M, 30) and torch.equal(x, y) for x, y in zip(before[n], after))
    assert txl.device_status() == 0
