"""The stack's tokens on the host (CPU, with fakes of the device calls as in test_paged_stack_host): -1
is none there too, and ids outside the vocabulary are refused before the stream moves."""

import pytest
import torch

from test_paged_stack_host import W, on_the_cpu, stack, tokens  # noqa: F401 (a fixture for every test)


def test_minus_one_is_a_zero_embedding_on_the_host():
    s = stack()
    toks = tokens(2, 5, seed=1)
    toks[0, 2] = toks[1, 4] = -1
    got = s._embed(toks)
    assert bool((got[toks < 0] == 0).all())
    assert torch.equal(got[toks >= 0], s.emb[toks[toks >= 0]])


@pytest.mark.parametrize("bad,dtype", [(W.vocab, torch.int32), (-2, torch.int32), (W.vocab, torch.int64),
                                       (-2, torch.int64), (2 ** 40, torch.int64)])
def test_ids_outside_the_vocabulary_are_refused(bad, dtype):
    s = stack()
    s.segment(tokens(2, 6, seed=2))
    toks = tokens(2, 3, seed=3).to(dtype)
    h = s.draft(toks, torch.tensor([-1, 0, 1]))
    wrong = toks.clone()
    wrong[1, 2] = bad
    for call in (lambda: s.segment(wrong), lambda: s.draft(wrong, torch.tensor([-1, 0, 1])),
                 lambda: s.score(toks, wrong), lambda: s.log_probs(h, wrong)):
        with pytest.raises(IndexError):
            call()
        assert s.memory.fill == [6, 6]
    assert torch.equal(s.draft(toks, torch.tensor([-1, 0, 1])), h)
