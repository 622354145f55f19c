"""txl_relattn_tree_fwd where its result is known without a tolerance for rounding: a node's result
does not depend on its neighbours' queries, infinite values show as the formula has them, and
nodes whose every score is -infinity."""

import numpy as np
import pytest
import torch

import transformer_xl_relative_pos_gb300 as txl
from parity import dev
from test_gpu_tree import Case

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [2, 8, 9, 16, 26, 40, 64])
def test_a_node_does_not_depend_on_its_neighbours_queries(N, dtype):
    # The running maxima of a tile's nodes rise in other chunks than their neighbours': a
    # node's own sums are not touched then.  Node i with all other queries zero, bit for bit.
    c = Case(1, 2, N, [1500], kind="chain", dtype=dtype, std=4.0, seed=31)
    c.call(1)
    out, lse, q = c.out.clone(), c.lse.clone(), c.q.clone()
    for i in (0, N // 2, N - 1):
        c.q.zero_()
        c.q[:, :, i] = q[:, :, i]
        c.call(1)
        assert torch.equal(c.lse[:, :, i], lse[:, :, i]), i
        assert torch.equal(c.out[:, :, i], out[:, :, i]), i
    assert txl.device_status() == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N", [8, 16, 32, 64])
def test_lse_of_a_constant_beside_rising_scores(N, dtype):
    # Even nodes: every score is a (one exact product), so lse = scale * a + log(keys), whatever
    # the odd nodes' maxima do in every chunk.  Roundings on the way: log2(e), its product with
    # the scale, the score in log2 units, the last sum, ln(2) and its product: six half steps of
    # lse; the sum of K equal terms (K / 16 + 64) * 2 u, exp2 2^-22.
    F, a = 3200, 11520.0
    c = Case(1, 1, N, [F], dtype=dtype, P=64, begin=[0], seed=32, kind="wide")
    page = c.mem.table[0].long()
    keys = torch.zeros(c.mem.slots * 64, 64, dtype=torch.float32)
    t = torch.arange(F)
    keys[:F, 0], keys[:F, 1] = 1.0, (t // 32).float()
    c.mem.pool[0, page, 0] = keys.view(-1, 64, 64).to(c.dt).to(dev())
    c.r.zero_(), c.u.zero_(), c.vb.zero_(), c.q.zero_(), c.k.zero_()
    c.k[..., 0] = 1.0
    c.q[:, :, 0::2, 0] = a
    c.q[:, :, 1::2, 1] = 16.0
    c.parents.fill_(-1)
    c.call(1)
    K = F + 1
    want = 0.125 * a + np.log(K)
    bound = 6 * U * want + (K / 16 + 64) * 2 * U + 2.0 ** -22
    got = c.lse[0, 0, 0::2].cpu().double().numpy()
    assert (np.abs(got - want) <= bound).all(), (np.abs(got - want).max(), bound)
    assert txl.device_status() == 0


def check_infinite_values(N, n_splits, dtype):
    # Rows that every node sees: an infinity is the sum's, infinities of either sign and NaN
    # give NaN, and the other dimensions are as without them.
    c = Case(1, 2, N, [300], dtype=dtype, seed=33, begin=[11])
    out, lse, out_b, lse_b = c.want()
    x = (11 + torch.arange(300)) % c.mem.rows
    page, row = c.mem.table[0].cpu().long()[x // 64], x % 64
    inf, nan = float("inf"), float("nan")
    for t, dim, value in ((3, 5, inf), (130, 5, inf), (40, 6, -inf), (299, 20, inf), (0, 21, -inf),
                          (100, 7, inf), (250, 7, -inf), (77, 8, nan)):
        c.mem.pool[1, page[t], :, row[t], dim] = value
    c.call(n_splits)
    torch.cuda.synchronize()
    assert txl.device_status() == 0
    got = c.out.cpu().double().numpy()
    for dim, value in ((5, inf), (6, -inf), (20, inf), (21, -inf)):
        assert (got[..., dim] == value).all(), (dim, got[..., dim])
    assert np.isnan(got[..., [7, 8]]).all()
    rest = [d for d in range(64) if d not in (5, 6, 7, 8, 20, 21)]
    assert (np.abs(got - out) <= out_b)[..., rest].all()
    assert (np.abs(c.lse.cpu().double().numpy() - lse) <= lse_b).all()


@pytest.mark.parametrize("N,dtype,n_splits", [(N, "f32", s) for N in (1, 5, 8, 13, 17, 64) for s in (0, 1, 3, 7)] +
                         [(N, "bf16", s) for N in (17, 32, 40, 64) for s in (0, 1, 2, 5)])
def test_infinite_values_in_key_ranges(N, n_splits, dtype):
    check_infinite_values(N, n_splits, dtype)


@pytest.mark.parametrize("n_splits", [0, 1, 2, 5])
@pytest.mark.parametrize("N", [1, 5, 7, 8, 9, 13, 16])
def test_infinite_values_with_probabilities_in_two_parts(N, n_splits):
    check_infinite_values(N, n_splits, "bf16")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("F,n_splits", [(0, 1), (90, 1), (90, 4)])
@pytest.mark.parametrize("N", [1, 8, 12, 30, 64])
def test_nodes_whose_every_score_is_minus_infinity(N, F, n_splits, dtype):
    # softmax of nothing but -infinity is 0 / 0: out NaN, lse -infinity.  The other half of the
    # heads is as ever.
    c = Case(2, 2, N, [F, F], kind="chain", dtype=dtype, seed=34)
    out, lse, out_b, lse_b = c.want()
    c.q[:, 0, :, 3], c.u[0, 3] = 1.0, 0.5
    c.k[:, 0, :, 3] = -float("inf")
    c.mem.pool[0, :, 0, :, 3] = -float("inf")
    c.call(n_splits)
    torch.cuda.synchronize()
    assert txl.device_status() == 0
    got, got_lse = c.out.cpu().double().numpy(), c.lse.cpu().double().numpy()
    assert np.isnan(got[:, 0]).all() and (got_lse[:, 0] == -np.inf).all()
    assert (np.abs(got - out) <= out_b)[:, 1].all() and (np.abs(got_lse - lse) <= lse_b)[:, 1].all()
