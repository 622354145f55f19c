"""The log probabilities' outputs on the GPU, held in the norm: errors relative to the whole
output's norm against 64 bits, where the element-wise worst cases of vocab_model leave room for a
lost term."""

import pytest
import torch

import transformer_xl_relative_pos_gb300 as txl
from parity import dev

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _ok():
    torch.cuda.synchronize()
    assert txl.device_status() == 0


def _inputs(N, V, d, dtype, seed, spread=2.0):
    g = torch.Generator(device=dev()).manual_seed(seed)
    h = torch.randn(N, d, generator=g, device=dev()).to(dtype)
    w = (torch.randn(V, d, generator=g, device=dev()) * (spread / d ** 0.5)).to(dtype)
    t = torch.randint(0, V, (N,), generator=g, device=dev())
    t[torch.rand(N, generator=g, device=dev()) < 0.1] = -1
    return h, w, t, torch.randn(N, generator=g, device=dev())


def _grads64(h, w, t, lse, dlogp, scale=1.0):
    """dh and dw in 64 bits, from the statistics that the call is given."""
    h, w, live = h.double(), w.double(), t >= 0
    g = torch.where(live, dlogp.double(), torch.zeros_like(dlogp, dtype=torch.float64))
    G = torch.exp(scale * (h @ w.t()) - lse.double()[:, None]).mul_(-g[:, None])
    G[live, t[live]] += g[live]
    return scale * (G @ w), scale * (G.t() @ h)


def _rel(x, want):
    return float((x.double() - want).norm() / want.norm())


# fp32 gradients, off in the norm by at most:
#   the logits' sums of d / 16 additions, each cut by 0 to 1 units of 2^-23 and scaled by the mean of that,
#   so off by 0.29 sqrt(d / 16) 2^-23 of |z| (2 here; d = 1032: 5e-7), which G takes as a relative error;
#   the products' sums of at most 256 additions: 0.29 * 16 * 2^-23 = 5.5e-7 at random and, with the mean between
#   0.2 and 0.3 of 2^-24 an addition and 0.27 taken for it, 0.07 * 256 * 2^-24 = 1.1e-6;
#   the terms beyond the third and the products left out: 3 * 2^-24.
# Together below 2e-6; half as much again is allowed.
F32_NORM = 3e-6


@pytest.mark.parametrize("N,V,d", [(1100, 25001, 1032), (700, 50257, 1032), (300, 28000, 520)])
def test_gradients_of_long_sums_over_several_tiles(N, V, d):
    # vocabularies whose least number of parts (7, 13) is none of the usual ones
    h, w, t, dlogp = _inputs(N, V, d, F32, N + V)
    lse = torch.logsumexp(h.double() @ w.double().t(), 1).float()
    dh, dw = txl.logprob_bwd(h, w, t, lse, dlogp)
    only_h, _ = txl.logprob_bwd(h, w, t, lse, dlogp, grads=(torch.empty_like(h), None))
    _, only_w = txl.logprob_bwd(h, w, t, lse, dlogp, grads=(None, torch.empty_like(w)))
    _ok()
    want_h, want_w = _grads64(h, w, t, lse, dlogp)
    assert _rel(dh, want_h) <= F32_NORM and _rel(dw, want_w) <= F32_NORM
    assert torch.equal(dh, only_h) and torch.equal(dw, only_w)
