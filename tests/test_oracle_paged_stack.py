"""The streams of tests/paged_stack_model.py tell a right paged stack from wrong ones: mistakes planted
in the 64-bit recurrence move its states by ten bounds and more; and the stack's host code, with
fakes of the device calls on the CPU, is within one."""

import numpy as np
import pytest
import torch

import paged_stack_model as m
from test_paged_stack_host import on_the_cpu  # noqa: F401  (a fixture)
from transformer_xl_relative_pos_gb300.model import XLStack


@pytest.fixture(scope="module")
def right():
    return m.continued()


@pytest.mark.parametrize("name", m.MISTAKES)
def test_a_mistake_shows(name, right):
    b, kw = m.MISTAKES[name]
    assert np.abs(m.continued(**kw)[b] - right[b]).max() > 10 * m.BOUND


def test_a_tree_without_its_mask_shows():
    # every earlier node seen, as in a chain of all nodes
    for b, node in ((0, 10), (0, 8), (1, 8)):
        path = m.path_to(b, node)
        chain = m.run([m.PROMPT[b], m.DRAFT[b][:node + 1]])[path]
        assert np.abs(chain - m.drafted(b, node)).max() > 10 * m.BOUND


def test_the_host_code_of_the_stack():
    stack = XLStack(m.params(), m.W.H, m.W.M, "cpu", torch.float32, paged=True)
    stack.segment(m.PROMPT)
    h = stack.draft(m.DRAFT, torch.tensor(m.PARENTS), m.N_NODES)
    for b, node in ((0, 10), (1, 8), (2, 11)):
        assert np.abs(h[b, m.path_to(b, node)].numpy() - m.drafted(b, node)).max() < m.BOUND
    stack.accept(m.ACCEPTED)
    stack.fork(*m.FORK)
    assert np.abs(stack.segment(m.MORE).numpy() - m.continued()).max() < m.BOUND
