"""The limits that fp32 operands are held to on the GPU find a lost bf16 term (CPU only): with the
inputs of vocab_terms, every product or term that a three-term product has shows."""

import pytest
import torch

import vocab_terms as vt


@pytest.mark.parametrize("N,V,d", vt.UNIFORM)
def test_a_lost_term_of_the_products_shows(N, V, d):
    case = vt.Uniform(N, V, d)
    assert torch.equal(case.h.float().double(), case.h) and torch.equal(case.w.float().double(), case.w)
    dh, dw = case.exact()
    whole = case.grads()
    assert vt.rel(whole[0], dh) < vt.GRAD_LIMIT / 10 and vt.rel(whole[1], dw) < vt.GRAD_LIMIT / 10
    for lost in vt.PRODUCTS:
        got = case.grads((lost,), (lost,))
        assert vt.rel(got[0], dh) > 1.25 * vt.GRAD_LIMIT, lost
        assert vt.rel(got[1], dw) > 1.25 * vt.GRAD_LIMIT, lost
    for n in (1, 2):    # operands of one and of two terms
        few = tuple((i, j) for i, j in vt.PRODUCTS if i >= n or j >= n)
        got = case.grads(few, few)
        assert vt.rel(got[0], dh) > 2 * vt.GRAD_LIMIT and vt.rel(got[1], dw) > 2 * vt.GRAD_LIMIT


@pytest.mark.parametrize("N,V,d", vt.STEEP)
def test_a_lost_term_of_the_logits_shows(N, V, d):
    case = vt.Steep(N, V, d)
    dw, lse = case.dw(), torch.logsumexp(case.z, 1)
    for lost in ((),) + tuple((p,) for p in vt.PRODUCTS):
        z = case.scale * vt.product(case.h, case.w.t().contiguous(), lost)
        errors = vt.rel(case.dw(z), dw) / vt.STEEP_LIMIT, vt.rel(torch.logsumexp(z, 1), lse) / vt.LSE_LIMIT
        if lost:
            assert min(errors) > 1.25, (lost, errors)
        else:
            assert max(errors) < 0.1, errors
