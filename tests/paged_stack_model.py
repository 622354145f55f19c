"""What a paged stack's streams should give, in 64 bits by the oracle's recurrence ("Transformer-XL:
Attentive Language Models Beyond a Fixed-Length Context", §3.2 memory, §3.3 N-layer summary): every
sequence on its own, as segments of what it has accepted.

The weights of the attention are five times those of txl_inputs.draw_stack, so that queries,
keys and table rows are O(1) (0.1 * sqrt(128) = 1.1) and the context matters.

BOUND of a 32-bit stack of three layers: 1e-5 per attention call, the 32-bit path's
tolerance for operands of this size; a layer passes an error of its input on with a gain of about
three (the residual, and the queries and the keys through scores of standard deviation about one),
1e-5 * (1 + 3 + 9) = 1.3e-4, and its projections and feed-forward, sums of 128 and 256 products
of O(1), add as much again: 3e-4.  The mistakes of MISTAKES are at least ten times that
(test_oracle_paged_stack.py), so a stack that makes one of them fails.
"""

import math

import numpy as np
import torch

import oracle
import txl_inputs

W = txl_inputs.Workload("paged_streams", B=3, H=2, dh=64, L=48, M=40, d_model=128, dtype="f32", seed=52,
                        d_ff=256, n_layer=3, n_seg=2, vocab=204)
BOUND = 3e-4
PARENTS = [[-1, 0, 0, 1, 3, 2, -1, 6, 7, 4, 4, 9],     # several branches, two first tokens
           [-1, -1, 1, 2, 2, 1, 4, 6, 6, 0, 9, 10],
           list(range(-1, 11))]                        # a chain
N_NODES = [12, 11, 12]
ACCEPTED = [[0, 1, 3, 4, 10], [], list(range(12))]
FORK = 2, 1                                            # sequence 1 goes on as sequence 2


def params():
    p = txl_inputs.draw_stack(W)
    for lay in p["layers"]:
        for name in ("W_q", "W_kE", "W_kR", "W_v", "W_o"):
            lay[name] = lay[name] * 5
    return p


def tokens(N, seed):
    return torch.randint(0, W.vocab, (W.B, N), generator=torch.Generator().manual_seed(seed))


PROMPT, DRAFT, MORE = tokens(30, 1), tokens(12, 2), tokens(20, 3)


def path_to(b, node):
    path = [node]
    while PARENTS[b][path[0]] >= 0:
        path.insert(0, PARENTS[b][path[0]])
    return path


def run(segments):
    """The states [L, d] of the last of one sequence's segments (lists of tokens; empty ones
    are skipped)."""
    p = params()
    f64 = lambda t: t.double().numpy()
    layers = [{k: f64(w) for k, w in lay.items()} for lay in p["layers"]]
    mems = oracle.empty_memories(W.n_layer, 1, W.d_model)
    for s in segments:
        if len(s):
            h, mems = oracle.segment_forward(np.asarray(s)[None], f64(p["emb"]), layers, mems, f64(p["u"]),
                                             f64(p["v_bias"]), W.H, W.M, 1.0 / math.sqrt(W.dh))
    return h[0]


def drafted(b, node):
    """States along the path to a node of sequence b's tree."""
    return run([PROMPT[b], DRAFT[b][path_to(b, node)]])


def continued(accepted=ACCEPTED, fork=FORK):
    """States of MORE for every sequence, after the accepted nodes (in that order) and a fork."""
    src = list(range(W.B))
    if fork:
        src[fork[1]] = fork[0]
    return np.stack([run([PROMPT[s], DRAFT[s][accepted[s]], MORE[b]]) for b, s in enumerate(src)])


# what a wrong stack would compute instead of continued()[b]
MISTAKES = {
    "another path accepted": (0, dict(accepted=[[0, 1, 3, 4, 9], [], ACCEPTED[2]])),
    "an ancestor left out": (0, dict(accepted=[[0, 1, 3, 10], [], ACCEPTED[2]])),
    "in another order": (0, dict(accepted=[[10, 4, 3, 1, 0], [], ACCEPTED[2]])),
    "the drafted rows in place of the accepted": (0, dict(accepted=[[0, 1, 2, 3, 4], [], ACCEPTED[2]])),
    "nothing accepted": (0, dict(accepted=[[], [], ACCEPTED[2]])),
    "no fork": (1, dict(fork=None)),
    "a fork of another sequence": (1, dict(fork=(0, 1))),
}
