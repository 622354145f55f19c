"""The paged memory's accounting on the device, and the paged stack: segments as chains,
trees of drafted tokens, accepted paths, forks and checkpoints ("Transformer-XL:
Attentive Language Models Beyond a Fixed-Length Context", §3.2 recurrence, §3.3
N-layer summary)."""

import math

import numpy as np
import pytest
import torch

import oracle
import paged_ops
import transformer_xl_relative_pos_gb300 as txl
import txl_inputs
from parity import compare, dev
from transformer_xl_relative_pos_gb300.model import XLStack

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", range(4))
def test_paged_memory_against_lists_of_rows(seed):
    M, max_new, P, dtype = [(70, 40, 32, torch.bfloat16), (130, 64, 64, torch.float32),
                            (0, 7, 32, torch.bfloat16), (200, 64, 96, torch.bfloat16)][seed]
    make = lambda: txl.PagedMemory(2, 4, 3, M, max_new, device=dev(), dtype=dtype, page_rows=P)
    paged_ops.run(make, dev(), seed, steps=60)
    assert txl.device_status() == 0


W = txl_inputs.Workload("paged_stack", B=3, H=2, dh=64, L=48, M=100, d_model=128, dtype="bf16",
                        seed=51, d_ff=256, n_layer=3, n_seg=6, vocab=204)
# Bound of a whole stack of three layers against fp64: sqrt(3) times a layer's half an
# output ulp (2^-9 * 8 for LayerNorm outputs below 8) plus 1e-2 of its inner roundings is
# 4.5e-2; two stacks of one formula differ by at most twice that.
STACK_MAX, STACK_RMS = 6e-2, 1.5e-2


def stack(paged=True, dtype=torch.bfloat16, **kw):
    return XLStack(txl_inputs.draw_stack(W), W.H, W.M, dev(), dtype, paged=paged, **kw)


def tokens(*shape, seed=0):
    return torch.randint(0, W.vocab, shape, generator=torch.Generator().manual_seed(seed))


def close(a, b, what):
    compare(a.float().cpu().numpy(), b.double().cpu().numpy(), 2 * STACK_MAX, 2 * STACK_RMS, what=what)


def test_a_paged_stream_is_the_stream():
    # Segments as chains through the pages against the stack that re-projects its
    # hidden-state memory: the same contexts, so the same states up to rounding; the last
    # segment also against the oracle.
    a, b = stack(), stack(paged=False)
    toks = txl_inputs.draw_stack(W)["tokens"]
    for s in range(W.n_seg):
        mems = [m.double().cpu().numpy() for m in b.memories()] if s == W.n_seg - 1 else None
        got, want = a.segment(toks[s]), b.segment(toks[s])
        close(got, want, f"segment {s}")
    rounded = lambda t: t.to(torch.bfloat16).double().numpy()
    p = txl_inputs.draw_stack(W)
    layers = [{k: rounded(v) for k, v in lay.items()} for lay in p["layers"]]
    want, _ = oracle.segment_forward(toks[-1].numpy(), rounded(p["emb"]), layers, mems, rounded(p["u"]),
                                     rounded(p["v_bias"]), W.H, W.M, 1.0 / math.sqrt(W.dh))
    compare(got.double().cpu().numpy(), want, STACK_MAX, STACK_RMS, what="last segment")
    assert a.memory.fill == [W.M] * W.B and txl.device_status() == 0


def test_a_paged_stream_in_fp32():
    a, b = stack(dtype=torch.float32), stack(paged=False, dtype=torch.float32)
    toks = txl_inputs.draw_stack(W)["tokens"]
    for s in range(W.n_seg):
        got, want = a.segment(toks[s]), b.segment(toks[s])
    # fp32 arithmetic on O(1) states: 1e-5 per attention call, three layers, two stacks
    compare(got.cpu().numpy(), want.double().cpu().numpy(), 1e-4, what="fp32 stream")


def test_every_path_of_a_draft_is_a_chain():
    # A tree's states along a path are those of the path drafted on its own, and of the
    # stack that processes memory and path as segments.
    a = stack()
    a.segment(tokens(3, 40, seed=1))
    parents = torch.tensor([-1, 0, 0, 1, 3, 2, -1, 6, 7, 4, 4, 9])
    toks = tokens(3, len(parents), seed=2)
    tree = a.draft(toks, parents)
    for leaf in (5, 8, 10, 11):
        path = [leaf]
        while parents[path[0]] >= 0:
            path.insert(0, int(parents[path[0]]))
        chain = a.draft(toks[:, path], torch.arange(-1, len(path) - 1))
        close(chain, tree[:, path], f"path to {leaf}")
    b = stack(paged=False)
    b.segment(tokens(3, 40, seed=1))
    close(tree[:, [0, 1, 3, 4, 10]], b.segment(toks[:, [0, 1, 3, 4, 10]]), "as a segment")


def test_streams_accept_fork_and_end_apart():
    # Three sequences accept different paths; each then continues as a stack of its own
    # that saw only what it accepted.
    a = stack()
    prompt = tokens(3, 30, seed=3)
    a.segment(prompt)
    parents = torch.tensor([[-1, 0, 1, 0, 3], [-1, -1, 1, 2, 3], [-1, 0, 1, 2, 3]])
    toks = tokens(3, 5, seed=4)
    n_nodes = [5, 4, 5]
    a.draft(toks, parents, n_nodes)
    rows = [[0, 3, 4], [], [0, 1, 2, 3, 4]]
    a.accept(rows)
    assert a.memory.fill == [33, 30, 35]
    a.fork(2, 1)                             # sequence 1 goes on as sequence 2
    assert a.memory.fill == [33, 35, 35]
    more = tokens(3, 20, seed=5)
    got = a.segment(more)
    for b, (src, path) in enumerate([(0, rows[0]), (2, rows[2]), (2, rows[2])]):
        one = stack()
        one.segment(prompt[src:src + 1])
        one.segment(toks[src:src + 1, path])
        close(got[b:b + 1], one.segment(more[b:b + 1]), f"sequence {b}")
    a.memory.free(0)
    close(a.draft(more[:, :8], torch.arange(-1, 7))[:1], stack().segment(more[:1, :8]), "an empty memory")


def test_drafting_changes_nothing_and_checkpoints_resume():
    a = stack()
    a.segment(tokens(3, 64, seed=6))
    a.segment(tokens(3, 64, seed=7))
    ck = a.checkpoint()
    first = a.draft(tokens(3, 33, seed=8), torch.arange(-1, 32)).clone()
    again = a.draft(tokens(3, 33, seed=8), torch.arange(-1, 32))
    assert torch.equal(first, again)
    a.accept([range(33)] * 3)
    want = a.segment(tokens(3, 9, seed=9)).clone()
    b = stack()
    b.restore(ck)
    b.draft(tokens(3, 33, seed=8), torch.arange(-1, 32))
    b.accept([range(33)] * 3)
    assert torch.equal(b.segment(tokens(3, 9, seed=9)), want)


def test_the_paged_stack_refuses():
    for kw in (dict(cache_kv=True), dict(graphs=True)):
        with pytest.raises(ValueError):
            stack(**kw)
    a = stack()
    with pytest.raises(RuntimeError):
        a.accept([[0]])
    with pytest.raises(RuntimeError):
        a.fork(0, 1)
    with pytest.raises(RuntimeError):
        a.checkpoint()
    with pytest.raises(RuntimeError):
        a.memories()
    with pytest.raises(ValueError):
        a.segment(tokens(1, 65))
    with pytest.raises(RuntimeError):
        stack(paged=False).draft(tokens(1, 2), torch.tensor([-1, 0]))
    a.draft(tokens(2, 4), torch.tensor([-1, 0, 1, 2]))
    with pytest.raises(ValueError):
        a.accept([[0], [4]])
    a.accept([[0], []])
    with pytest.raises(RuntimeError):
        a.accept([[0], []])                  # nothing drafted any more
    with pytest.raises(ValueError):
        stack(paged=False).restore(a.checkpoint())
