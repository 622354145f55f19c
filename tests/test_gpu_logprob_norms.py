"""The log probabilities' outputs on the GPU, held in the norm: errors relative to the whole
output's norm against 64 bits, where the element-wise worst cases of vocab_model leave room for a
lost term (vocab_terms has inputs on which one shows)."""

import pytest
import torch

import transformer_xl_relative_pos_gb300 as txl
import vocab_terms as vt
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


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,top", [(1, 8), (3, 0), (40, 8), (150, 3), (300, 0), (300, 8)])
def test_nearly_certain_tokens_to_their_own_size(N, top, dtype):
    # log p = -sum of the others' exp(z - z_t), 1e-12 to 6, to a relative error.  Whole numbers, so the
    # accumulators' sums are exact; a logit beside the target's is then off by the factor to log2 units (its
    # rounding, the product's, and the mean cut of 4 additions: 3 of 2^-24 of at most 17, 3.0e-6), by the
    # rounding of its distance from the largest (half of 2^-18, below 64 log2 units, times ln 2: 1.3e-6) and by the
    # exponential (2^-22): its term by 4.6e-6 of itself.  Sums of positive terms, 50 roundings of 2^-24 at most
    # on a term's way: 3e-6.  Together below 2^-16.
    # Beneath that stands what the largest logit's own rounding leaves: its exact value lies up to x = 2^-19
    # log2 units above the rounded one that the sums are taken from, and log of the sum and logit, both of x ln 2
    # = 2^-19.5, are subtracted.  In units of 2^-42: the factor's 49 bits of 64 (0.35), x rounded (0.35), its
    # exponential less 1, argument and function (three of 2^-24: 1.1), the logarithm (one of 2^-23: 0.7), its sum
    # with the low part's (0.35): 2.9, below 2^-40.  The entropy subtracts the weighted mean of the logits, x once
    # more through five roundings (1.8): 4.7, below 2^-39.
    V, d, scale = 3000, 64, 0.125
    g = torch.Generator().manual_seed(60 + N)
    h = torch.randint(-2, 3, (N, d), generator=g).double()
    w = torch.randint(-1, 2, (V, d), generator=g).double()
    t = torch.randperm(V, generator=g)[:N]
    # (targets' rows along their states: logits of 9 to 38, where the others have 8.6 and more in all)
    for i in range(N):
        goal, at = 8.0 * (9.0 + 20.0 * ((i * 7) % max(N, 2)) / max(N - 1, 1)), h[i].abs().sum()
        w[t[i]] = torch.sign(h[i]) * torch.ceil(goal / at)
    z = scale * (h @ w.t())
    others = z.clone()
    others[torch.arange(N), t] = -float("inf")
    logp = -torch.log1p(torch.exp(torch.logsumexp(others, 1) - z[torch.arange(N), t]))
    D = lambda x: x.to(dtype).cuda()
    res = txl.logprob_fwd(D(h), D(w), t.cuda(), scale=scale, top=top)
    _ok()
    lp = z - z[torch.arange(N), t][:, None] + logp[:, None]
    lp[torch.arange(N), t] = logp
    entropy = -(torch.exp(lp) * lp).sum(1)
    rel = lambda x, want, floor=2.0 ** -40: (((x.cpu().double() - want).abs() - floor) / want.abs()).max().item()
    got = rel(res.logp, logp)
    print(f"{N} {top} {dtype}: log p {float(logp.min()):.1e} to {float(logp.max()):.1e}, off by {got:.1e}, "
          f"entropy by {rel(res.entropy, entropy, 2.0 ** -39):.1e}")
    assert float(logp.max()) > -1e-4 or N == 1
    assert got <= 2.0 ** -16
    # (terms p log p: the same error, and that of log p)
    assert rel(res.entropy, entropy, 2.0 ** -39) <= 2.0 ** -15
    if top:
        best = torch.argmax(z, 1)
        ours = best == t
        assert torch.equal(res.top_ids[:, 0].cpu().long(), best) and bool(ours.any())
        assert rel(res.top_logp[:, 0].cpu()[ours], logp[ours]) <= 2.0 ** -16


@pytest.mark.parametrize("case,kind", [("one term of many rows", "bf16_f32"), ("one term of many rows", "f32"),
                                       ("most rows padded", "bf16_f32"), ("one row of many words", "f32")])
def test_fp32_gradients_of_sparse_sums(case, kind):
    # a sum of one term, or a few, among many that are zero or tiny: nothing of it is cut, so the mean that the
    # results are scaled by (0.27 of 2^-24 for each addition of a part's chain) is itself the error.  A chain has 256
    # additions, of a bf16 pair's two terms 512: 8.2e-6.  The pair's own residual is 2^-18 of G at most, fp32's three
    # terms are exact here, and the result's rounding 2^-24.  Together below 2^-16.
    # (Sizes with more tiles than SMs, where no sum is split for their sake.)
    dtype = F32 if kind == "f32" else BF
    N, V, d = (20000, 12000, 1024) if case != "one row of many words" else (300, 400000, 1024)
    g = torch.Generator(device=dev()).manual_seed(8)
    # logits: 0 for most words, -60 for the words from 200 on (probability e^-65: as good as none)
    h = torch.randint(1, 200, (N, d), generator=g, device=dev()).double() / 128
    h[:, 0] = 1.0
    w = torch.zeros(V, d, dtype=torch.float64, device=dev())
    w[200:, 0] = -60.0
    t = torch.full((N,), -1, device=dev())
    dlogp = torch.ones(N, dtype=torch.float64, device=dev())
    if case == "one term of many rows":
        t[:] = torch.randint(0, 200, (N,), generator=g, device=dev())
        t[::200] = 200 + torch.arange(N // 200, device=dev())      # each of a hundred words once
        some = torch.arange(200, 200 + N // 200, device=dev())
        want = h[::200]                                              # dw: G is 1 for its row, e^-65 for others
    elif case == "most rows padded":
        t[-7:] = torch.arange(207, 214, device=dev())
        some = torch.arange(207, 214, device=dev())
        want = h[-7:]
    else:
        # the words from 200 on with their own rows: dh of a row is its word's, less the mean of the first 200
        w[200:, 1:] = torch.randint(1, 200, (V - 200, d - 1), generator=g, device=dev()).double() / 128
        h[:, 1:] = 0.0
        t[:] = 200 + torch.randint(0, V - 200, (N,), generator=g, device=dev())
        want = w[t]                                                  # (the first 200 words' rows are zero)
    D = lambda x: x.to(dtype)
    lse = torch.logsumexp(h @ w.t(), 1).float()
    dh, dw = txl.logprob_bwd(D(h), D(w), t, lse, dlogp.float(), grad_dtype=F32)
    _ok()
    got = dh if case == "one row of many words" else dw[some]
    off = ((got.double() - want).abs() / want.abs()).max().item()
    print(f"{case}, {kind}: off by {off:.2e}")
    assert off <= 2.0 ** -16


@pytest.mark.parametrize("kind", ["bf16", "bf16_f32", "f32"])
def test_dh_over_chunks_of_the_vocabulary(kind):
    # G is past the workspace's limit: the chunks' sums of dh, added in their order.  bf16 results: G's rounding and
    # the result's, 2^-8 each at most; fp32: F32_NORM above.
    N, V, d = 20000, 60000, 16
    dtype, grad = F32 if kind == "f32" else BF, BF if kind == "bf16" else F32
    h, w, t, dlogp = _inputs(N, V, d, dtype, 9)
    lse = torch.cat([torch.logsumexp(x.double() @ w.double().t(), 1) for x in h.split(4000)]).float()
    ws = torch.full((txl.logprob_bwd_workspace_size(N, V, d, dtype, grad_dtype=grad),), 255, dtype=torch.uint8,
                    device=dev())
    dh, dw = txl.logprob_bwd(h, w, t, lse, dlogp, grad_dtype=grad, workspace=ws)
    again = txl.logprob_bwd(h, w, t, lse, dlogp, grad_dtype=grad, workspace=ws.fill_(255))
    _ok()
    want_h, want_w = torch.empty(N, d, dtype=torch.float64, device=dev()), 0.0
    for i in range(0, N, 4000):
        a = slice(i, i + 4000)
        want_h[a], part = _grads64(h[a], w, t[a], lse[a], dlogp[a])
        want_w = want_w + part
    limit = lambda x: F32_NORM if kind == "f32" else 2 * 2.0 ** -8
    assert _rel(dh, want_h) <= limit(dh) and _rel(dw, want_w) <= limit(dw)
    assert torch.equal(dh, again[0]) and torch.equal(dw, again[1])
    if kind != "bf16_f32":   # (where dw's type, that of w when it is not asked for, is the same)
        only_h, _ = txl.logprob_bwd(h, w, t, lse, dlogp, grads=(torch.empty_like(h), None), workspace=ws.fill_(255))
        _, only_w = txl.logprob_bwd(h, w, t, lse, dlogp, grads=(None, torch.empty_like(w)), workspace=ws)
        assert torch.equal(dh, only_h) and torch.equal(dw, only_w)
    # replays of a captured call follow its inputs
    graph, out = torch.cuda.CUDAGraph(), (torch.empty_like(dh), torch.empty_like(dw))
    with torch.cuda.graph(graph):
        txl.logprob_bwd(h, w, t, lse, dlogp, grads=out, workspace=ws)
    dlogp.neg_()
    for _ in range(2):
        graph.replay()
    _ok()
    assert torch.equal(out[0], -dh) and torch.equal(out[1], -dw)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("where", ["first words", "every other range", "all but one"])
@pytest.mark.parametrize("N,top", [(3, 4), (100, 0), (300, 0), (300, 4)])
def test_words_masked_by_the_lowest_value(N, top, where, dtype):
    # logits of -1.7e38 (the type's lowest times 0.5) have no part in anything, whole chunks and ranges of them
    # either; and a gradient of the entropies of 2^30 times their probability of zero is zero
    V, d, scale = 6000, 64, 0.5
    g = torch.Generator().manual_seed(N)
    h = torch.randn(N, d, generator=g).to(dtype).double()
    w = (torch.randn(V, d, generator=g) * 0.5).to(dtype).double()
    h[:, 0] = 1.0
    w[:, 0] = 0.0
    at = torch.arange(V)
    off = {"first words": at < 4000, "every other range": at // 640 % 2 == 0, "all but one": at != 4321}[where]
    keep = at[~off]
    w[off, 0] = float(torch.finfo(torch.bfloat16).min)
    t = keep[torch.randint(0, len(keep), (N,), generator=g)]
    D = lambda x: x.to(dtype).to(dev())
    res = txl.logprob_fwd(D(h), D(w), t.to(dev()), scale=scale, top=top)
    lp = torch.log_softmax(scale * h @ w[keep].t(), 1)
    place = torch.searchsorted(keep, t)
    entropy = -(torch.exp(lp) * lp).sum(1)
    # (fp32 sums: 2^-20 of numbers of size 10)
    close = lambda x, want: float((x.cpu().double() - want).abs().max()) <= 1e-5
    assert close(res.logp, lp[torch.arange(N), place]) and close(res.entropy, entropy)
    assert close(res.lse, torch.logsumexp(scale * h @ w[keep].t(), 1))
    if top:
        some = min(top, len(keep))
        assert torch.equal(res.top_ids[:, :some].cpu().long(), keep[torch.sort(lp, 1, descending=True)[1][:, :some]])
    factor = 2.0 ** 30
    dlogp, dent = torch.randn(N, generator=g) * factor, torch.randn(N, generator=g) * factor
    dh, dw = txl.logprob_bwd(D(h), D(w), t.to(dev()), res.lse, dlogp.to(dev()), entropy=res.entropy,
                             dentropy=dent.to(dev()), scale=scale, grad_dtype=F32)
    _ok()
    assert bool(torch.isfinite(dh).all()) and bool(torch.isfinite(dw).all()) and bool((dw.cpu()[off] == 0).all())
    lp = scale * h @ w[keep].t() - res.lse.cpu().double()[:, None]
    p = torch.exp(lp)
    G = -dlogp.double()[:, None] * p - dent.double()[:, None] * p * (lp + res.entropy.cpu().double()[:, None])
    G[torch.arange(N), place] += dlogp.double()
    want = scale * G.t() @ h
    if where == "all but one":
        return   # (one word is certain: its gradient is what is left of equal numbers)
    # G: a bf16 pair, or terms, from statistics of 2^-20
    assert _rel(dw.cpu()[keep], want) <= 2.0 ** -16
    if N > 3:
        # G rounded to bf16 once (in fp32: not), and the result
        assert _rel(dh.cpu()[:, 1:], (scale * G @ w[keep])[:, 1:]) <= (2 * 2.0 ** -8 if dtype == BF else 2.0 ** -16)


@pytest.mark.parametrize("N,V,d", vt.UNIFORM)
def test_every_term_of_fp32_operands_is_in_the_products(N, V, d):
    # off by F32_NORM's arithmetic, with G = dlogp exp(-log V): the exponent in log2 units rounded (2^-21, times ln
    # 2: 3.3e-7) and the exponential (2^-22).  Below 3e-6; a lost term is more (test_vocab_terms).
    case = vt.Uniform(N, V, d)
    D = lambda x: x.float().to(dev())
    dh, dw = txl.logprob_bwd(D(case.h), D(case.w), case.t.to(dev()), case.lse.to(dev()), D(case.dlogp))
    _ok()
    want_h, want_w = case.exact()
    print(f"dh {vt.rel(dh.cpu(), want_h):.1e}, dw {vt.rel(dw.cpu()[1:], want_w):.1e}")
    assert vt.rel(dh.cpu(), want_h) <= vt.GRAD_LIMIT and vt.rel(dw.cpu()[1:], want_w) <= vt.GRAD_LIMIT


@pytest.mark.parametrize("N,V,d", vt.STEEP)
def test_every_term_of_fp32_operands_is_in_the_logits(N, V, d):
    # logits of 30: 33 additions of d / 16 at most, each cut by 0 to 1 units of 2^-23 of up to 30 (0.29 of that at
    # random, 6e-6, and 0.05 of 2^-24 each beside the mean: 3e-6), three roundings of up to 37 (2^-24 each: 6e-6):
    # 1.5e-5 of a probability, 5e-7 of a log-sum-exp.
    case = vt.Steep(N, V, d)
    D = lambda x: x.float().to(dev())
    res = txl.logprob_fwd(D(case.h), D(case.w), case.t.to(dev()), scale=case.scale)
    _, dw = txl.logprob_bwd(D(case.h), D(case.w), case.t.to(dev()), case.lse.to(dev()), D(case.dlogp), scale=case.scale)
    _ok()
    off = vt.rel(dw.cpu()[1:], case.dw()), vt.rel(res.lse.cpu(), torch.logsumexp(case.z, 1))
    print("dw %.1e, lse %.1e" % off)
    assert off[0] <= vt.STEEP_LIMIT and off[1] <= vt.LSE_LIMIT


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,V,d,top", [(1, 5000, 512, 8), (17, 1204, 512, 5), (200, 9001, 200, 3), (100, 700, 40, 0),
                                       (515, 9001, 128, 9), (300, 1000, 1024, 0), (2000, 5003, 264, 0)])
def test_log_probabilities_in_the_norm(N, V, d, top, dtype):
    # logits of some 2: d / 16 additions, 0.29 sqrt(64) 2^-23 at random and 0.07 * 64 * 2^-24 beside the mean, of 2:
    # 1.1e-6 of a term of the sums; half a rounding or two of a result of 5 to 12.  Below 1e-6 of that.
    h, w, t, _ = _inputs(N, V, d, dtype, 7 * N + V)
    res = txl.logprob_fwd(h, w, t, top=top)
    _ok()
    lp = torch.log_softmax(h.double() @ w.double().t(), 1)
    want = {"lse": torch.logsumexp(h.double() @ w.double().t(), 1), "entropy": -(torch.exp(lp) * lp).sum(1)}
    live = t >= 0
    want["logp"] = torch.where(live, lp.gather(1, t.clamp(min=0)[:, None])[:, 0], torch.zeros_like(lp[:, 0]))
    if top:
        want["top_logp"] = torch.sort(lp, 1, descending=True)[0][:, :top]
    off = {k: _rel(getattr(res, k), x) for k, x in want.items() if float(x.norm())}
    print(" ".join(f"{k} {x:.1e}" for k, x in off.items()))
    assert all(x <= 1e-6 for x in off.values()), off


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,d", [(3, 4096), (3, 65536), (300, 4096)])
def test_logits_of_sparse_states(N, d, dtype):
    # states of one element: nothing of a logit is cut, and the mean cut that it is scaled by, d 2^-30, is its
    # error; beside it three roundings of logits of up to 24 and one of the result, and the sums' 2^-20
    V = 700
    g = torch.Generator().manual_seed(d + N)
    h = torch.zeros(N, d, dtype=torch.float64)
    at = torch.randint(0, d, (N,), generator=g)
    h[torch.arange(N), at] = 4.0
    w = (torch.randn(V, d, generator=g) * 1.5).to(dtype)
    z = h @ w.double().t()
    res = txl.logprob_fwd(h.to(dtype).to(dev()), w.to(dev()), top=2)
    _ok()
    most = float(z.abs().max())
    off = (d * 2.0 ** -30 + 4 * 2.0 ** -24) * most + 2.0 ** -20
    want = torch.logsumexp(z, 1)
    assert most < 32 and float((res.lse.cpu().double() - want).abs().max()) <= off
    best = torch.sort(z, dim=1, descending=True, stable=True)   # (bf16 words have equal elements)
    assert torch.equal(res.top_ids.cpu().long(), best[1][:, :2])
    assert float((res.top_logp.cpu().double() - (best[0][:, :2] - want[:, None])).abs().max()) <= 2 * off
