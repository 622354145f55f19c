"""txl_logprob_fwd and txl_logprob_bwd on the GPU against the 64-bit softmax of
vocab_model, with that module's bounds: both types, one row to several tiles, odd
vocabularies, padding, ties, infinities, strides, id types, other streams, captured
graphs, vocabulary chunks; gradients against the formula and against differences; and
what they refuse."""

import math

import pytest
import torch

import transformer_xl_relative_pos_gb300 as txl
import vocab_model as model
from parity import dev

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def _ok():
    torch.cuda.synchronize()
    assert txl.device_status() == 0


def _inputs(N, V, d, dtype, seed, spread=2.0):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(N, d, generator=g).to(dtype)
    w = (torch.randn(V, d, generator=g) * (spread / d ** 0.5)).to(dtype)
    t = model.tokens_with_padding(N, V, g, dtype=torch.int32 if N % 2 else torch.int64)
    return h, w, t


def _products(dtype):
    return 2 if dtype == F32 else 1


def _close(got, want, off, what):
    diff = (got.detach().cpu().double().reshape(want.shape) - want).abs()
    assert bool((diff <= off).all()), (what, float(diff.max()), float((diff - off).max()))


def _check_fwd(res, ref, top):
    _close(res.lse, ref.lse, ref.lse_off, "lse")
    _close(res.entropy, ref.entropy, ref.ent_off, "entropy")
    if ref.t is not None:
        _close(res.logp, ref.logp, ref.logp_off, "logp")
    if top:
        ids, logp = (x.cpu().reshape(-1, top) for x in (res.top_ids.long(), res.top_logp))
        some = ref.top_ids.shape[1]    # (a vocabulary may have fewer)
        assert torch.equal(ids[:, :some], ref.top_ids) and bool((ids[:, some:] == -1).all())
        _close(logp[:, :some], ref.top_logp, ref.logp_off[:, None], "top_logp")
        assert bool(logp[:, some:].isnan().all())


# (rows, vocabulary, width, alternatives, scale): one row; less than a tile of rows and columns;
# ends inside tiles, 32-column groups and 64-wide steps; several row tiles; as many
# alternatives as the vocabulary has
FWD = [(1, 1, 8, 1, 1.0), (1, 5000, 512, 8, 1.0), (3, 16, 24, 16, -0.7), (17, 204, 512, 5, 1.0),
       (130, 333, 72, 3, 0.5), (129, 2049, 200, 16, 1.3), (256, 700, 64, 2, 1.0), (64, 9001, 128, 9, 1.0),
       # without alternatives: either form, by the vocabulary
       (100, 700, 40, 0, 1.0), (200, 1000, 64, 0, -0.8), (256, 20001, 64, 0, 1.0), (65, 128, 512, 0, 2.0),
       # more than 256 rows: the rows in the tiles' rows
       (300, 1000, 64, 0, 1.0), (300, 333, 72, 3, -0.5), (257, 5, 16, 16, 1.0), (700, 2049, 200, 16, 1.3),
       (515, 9001, 128, 9, 1.0), (1000, 130, 520, 8, 0.0), (400, 40000, 24, 1, 1.0)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,V,d,top,scale", FWD)
def test_logprob_fwd(N, V, d, top, scale, dtype):
    h, w, t = _inputs(N, V, d, dtype, N + V)
    ws = torch.full((max(1, txl.logprob_fwd_workspace_size(N, V, d, dtype, top=top)),), 255,
                    dtype=torch.uint8, device=dev())
    res = txl.logprob_fwd(h.to(dev()), w.to(dev()), t.to(dev()), scale=scale, top=top, workspace=ws)
    _ok()
    _check_fwd(res, model.LogProb(h, w, t, scale, top, _products(dtype)), top)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [40, 300])
def test_logprob_ties_go_to_the_lowest_index(N, dtype):
    # small whole numbers: every product and sum is exact, and many logits are equal
    g = torch.Generator().manual_seed(3)
    h = torch.randint(-2, 3, (N, 16), generator=g).to(dtype)
    w = torch.randint(-1, 2, (700, 16), generator=g).to(dtype)
    h[7] = 0      # every logit equal
    res = txl.logprob_fwd(h.to(dev()), w.to(dev()), top=16)
    _ok()
    ref = model.LogProb(h, w, None, 1.0, 16)
    assert res.logp is None
    assert torch.equal(res.top_ids.cpu().long(), ref.top_ids)
    assert res.top_ids[7].tolist() == list(range(16))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [2, 300])
def test_logprob_order_beyond_single_precision(N, dtype):
    # six logits that are all 2^24 in fp32 sums, told apart by the exact ones; two are equal
    d, V = 64, 600
    h = torch.zeros(N, d, dtype=dtype)
    h[:, 0], h[:, 1] = 4096.0, 1.0
    w = torch.zeros(V, d, dtype=dtype)
    best = torch.tensor([5, 590, 17, 256, 300, 31])
    w[best, 0] = 4096.0
    w[best, 1] = torch.tensor([1.0, 4.0, 2.0, 4.0, 7.0, 3.0]).to(dtype) * 0.03125
    res = txl.logprob_fwd(h.to(dev()), w.to(dev()), top=6)
    _ok()
    assert res.top_ids.tolist() == [[300, 256, 590, 31, 17, 5]] * N
    assert torch.equal(res.top_ids.cpu().long(), model.LogProb(h, w, None, 1.0, 6).top_ids)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,top", [(3, 0), (3, 8), (40, 8), (300, 0), (300, 8)])
def test_logprob_of_nearly_certain_tokens(N, top, dtype):
    # log p = -sum of the others' exp(z - z_t), here 1e-8 to 1e-4: a sum of the others and the 1 keeps a few
    # units of 2^-24 of it.  The 1 enters once in its thread's sum (N <= 256: two tiles at most, so three
    # additions that may round by 2^-24 each; else one for 32 columns of at most 3000 / 4: 24, of a random
    # walk's 5 within six deviations 15 half units) and is rounded once more where the ranges are joined;
    # the others are off by their logits' errors (2^-20 of the value at the sizes here).
    V, d = 3000, 128
    g = torch.Generator().manual_seed(40 + N)
    w = (torch.randn(V, d, generator=g) * 0.2).to(dtype)
    t = torch.randint(0, V, (N,), generator=g)
    lift = torch.linspace(4.5, 6.5, N)[:, None]
    h = (torch.randn(N, d, generator=g) * 0.3 + w[t].double() * lift).to(dtype)
    res = txl.logprob_fwd(h.to(dev()), w.to(dev()), t.to(dev()), top=top)
    _ok()
    ref = model.LogProb(h, w, t, 1.0, 0)
    assert float(ref.logp.max()) > -1e-6
    units = 4 if N <= 256 else 16
    _close(res.logp, ref.logp, units * 2.0 ** -24 + 2.0 ** -20 * ref.logp.abs() + ref.logp.abs() * ref.logp_off, "logp")


@pytest.mark.parametrize("repeat", [1, 60])
def test_logprob_infinite_logits(repeat):
    d, V = 64, 300
    g = torch.Generator().manual_seed(4)
    h = torch.randn(5, d, generator=g).to(BF)
    w = torch.randn(V, d, generator=g).to(BF)
    h[:, 0] = 1.0
    w[:, 0] = 0.0
    w[::3, 0] = float("-inf")           # a third of the vocabulary has probability zero
    h[3, 0] = -1.0                      # ... and makes this row's logits +inf
    h[4] = float("nan")
    t = torch.tensor([1, 3, -1, 4, 5])
    # (300 rows: the kernel of many)
    res = txl.logprob_fwd(h.repeat(repeat, 1).to(dev()), w.to(dev()), t.repeat(repeat).to(dev()), top=5)
    _ok()
    res = txl.LogProbs(*(x.view(repeat, 5, *x.shape[1:]) for x in res))
    same = lambda x: all(torch.equal(x[0].nan_to_num(7, 8, 9), y.nan_to_num(7, 8, 9)) for y in x)
    assert all(same(x) for x in res)
    res = txl.LogProbs(*(x[0] for x in res))
    keep = torch.ones(V, dtype=torch.bool)
    keep[::3] = False
    ref = model.LogProb(h[:3], w[keep], None, 1.0, 5)
    _close(res.lse[:3], ref.lse, ref.lse_off, "lse")
    _close(res.entropy[:3], ref.entropy, ref.ent_off, "entropy")
    back = torch.arange(V)[keep]
    assert torch.equal(res.top_ids[:3].cpu().long(), back[ref.top_ids])
    assert float(res.logp[1]) == -math.inf and float(res.logp[2]) == 0.0
    for x in (res.lse, res.entropy, res.logp):
        assert bool(x[3:].isnan().all())
    assert res.top_ids[4].tolist() == [-1] * 5


@pytest.mark.parametrize("N", [2, 300])
def test_logprob_fewer_numbers_than_places_and_all_minus_infinity(N):
    h = torch.ones(N, 8, dtype=BF)
    w = torch.zeros(3, 8, dtype=BF)
    w[1] = float("nan")
    res = txl.logprob_fwd(h.to(dev()), w.to(dev()), top=4)
    assert res.top_ids[0].tolist() == [0, 2, -1, -1] and bool(res.lse.isnan().all())
    w = torch.full((3, 8), float("-inf"), dtype=BF)
    res = txl.logprob_fwd(h.to(dev()), w.to(dev()), torch.zeros(N, dtype=torch.int64, device=dev()), top=3)
    _ok()
    assert res.lse.tolist() == [-math.inf] * N and bool(res.logp.isnan().all())
    assert res.top_ids[1].tolist() == [0, 1, 2]


def test_logprob_strided_states_and_table_streams_and_graph():
    # the last position of every segment, a table inside a wider one
    g = torch.Generator().manual_seed(6)
    states = torch.randn(9, 7, 128, generator=g).to(BF).to(dev())
    wide = (torch.randn(501, 192, generator=g) * 0.2).to(BF).to(dev())
    h, w = states[:, -1], wide[:, 32:160]
    t = torch.randint(0, 501, (9,), generator=g).to(dev())
    ref = model.LogProb(h.cpu(), w.cpu(), t.cpu(), 1.0, 4)
    side = [torch.cuda.Stream() for _ in range(2)]
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
    both = [txl.logprob_fwd(h, w, t, top=4, stream=s) for s in side]
    _ok()
    for res in both:
        _check_fwd(res, ref, 4)
    whole = txl.logprob_fwd(states, w, top=2)
    assert whole.lse.shape == (9, 7) and whole.top_ids.shape == (9, 7, 2)
    assert torch.equal(whole.lse[:, -1], both[0].lse)
    # replays of a captured call follow its inputs
    ws = torch.empty(txl.logprob_fwd_workspace_size(9, 501, 128, top=4), dtype=torch.uint8, device=dev())
    graph = torch.cuda.CUDAGraph()
    out = txl.logprob_fwd(h, w, t, top=4)
    with torch.cuda.graph(graph):
        txl.logprob_fwd(h, w, t, top=4, out=out, workspace=ws)
    states.mul_(-0.5)
    t.copy_((t + 100) % 501)
    graph.replay()
    _ok()
    _check_fwd(out, model.LogProb(h.cpu(), w.cpu(), t.cpu(), 1.0, 4), 4)


def test_logprob_targets_out_of_range_are_recorded():
    h, w, _ = _inputs(4, 20, 16, BF, 1)
    t = torch.tensor([3, 20, -7, -1])
    res = txl.logprob_fwd(h.to(dev()), w.to(dev()), t.to(dev()))
    assert txl.device_status() == -8
    assert res.logp[1:].tolist() == [0, 0, 0] and float(res.logp[0]) < 0


def test_logprob_empty_batch():
    w = torch.randn(20, 16, device=dev())
    h = torch.empty(0, 16, device=dev())
    t = torch.empty(0, dtype=torch.int64, device=dev())
    res = txl.logprob_fwd(h, w, t, top=2)
    assert res.lse.shape == (0,) and res.top_ids.shape == (0, 2)
    dh, dw = txl.logprob_bwd(h, w, t, res.lse, res.logp)
    _ok()
    assert dh.shape == (0, 16) and bool((dw == 0).all())


# ---------------------------------------------------------------------------
# gradients
# ---------------------------------------------------------------------------

def _check_grads(got, ref, N, V, dtype, dw_dtype, dlogp, dent, lse, ent):
    dh, dw, dh_size, dw_size, dh_full, dw_full = ref.grads(dlogp, dent, ent, lse)
    # G before its rounding: the logit's error and the statistics' conversion, of the terms
    # that make it up
    g_off = float((2 * ref.z_off + 2.0 ** -20 + 4 * model.F32_CUT * ref.lse.abs()).max())
    out = lambda dt: model.BF16_HALF if dt == BF else 2.0 ** -24
    # G's rounding: bf16, a bf16 pair (the square of it), three terms (2^-24)
    g_h = model.BF16_HALF if dtype == BF else 2.0 ** -24
    g_w = g_h if dtype == dw_dtype else model.BF16_HALF ** 2
    products = _products(dtype)
    tol_h = (g_h + products * V * model.F32_CUT) * dh_size + g_off * dh_full + out(dtype) * dh.abs() + 1e-40
    tol_w = (g_w + products * N * model.F32_CUT) * dw_size + g_off * dw_full + out(dw_dtype) * dw.abs() + 1e-40
    for name, x, want, tol in (("dh", got[0], dh, tol_h), ("dw", got[1], dw, tol_w)):
        if x is not None:
            _close(x, want, tol, name)


BWD = [(1, 1, 8, 1.0), (5, 204, 512, 1.0), (130, 333, 72, -0.5), (129, 2049, 200, 1.3),
       (700, 100, 264, 1.0), (33, 5003, 64, 0.7), (257, 7000, 640, 1.0),
       # few rows over many words: both terms of G apart, sums of many parts
       (5, 9001, 200, 1.0), (100, 9001, 72, -0.8), (127, 30001, 264, 1.0)]


@pytest.mark.parametrize("kind", ["bf16", "bf16_f32", "f32"])
@pytest.mark.parametrize("entropy", [False, True])
@pytest.mark.parametrize("N,V,d,scale", BWD)
def test_logprob_bwd(N, V, d, scale, entropy, kind):
    dtype = F32 if kind == "f32" else BF
    dw_dtype = BF if kind == "bf16" else F32
    h, w, t = _inputs(N, V, d, dtype, 3 * N + V)
    g = torch.Generator().manual_seed(11)
    dlogp = torch.randn(N, generator=g)
    dent = torch.randn(N, generator=g) * (torch.rand(N, generator=g) < 0.7) if entropy else None
    D = lambda x: None if x is None else x.to(dev())
    res = txl.logprob_fwd(D(h), D(w), D(t), scale=scale)
    ws = torch.full((txl.logprob_bwd_workspace_size(N, V, d, dtype, grad_dtype=dw_dtype),), 255,
                    dtype=torch.uint8, device=dev())
    args = (D(h), D(w), D(t), res.lse, D(dlogp))
    kw = dict(entropy=res.entropy if entropy else None, dentropy=D(dent), scale=scale)
    got = txl.logprob_bwd(*args, **kw, grad_dtype=dw_dtype, workspace=ws)
    _ok()
    assert got[0].dtype == dtype and got[1].dtype == dw_dtype
    ref = model.LogProb(h, w, t, scale, 0, _products(dtype))
    _check_grads(got, ref, N, V, dtype, dw_dtype, dlogp, dent, res.lse.cpu(), res.entropy.cpu())
    again = txl.logprob_bwd(*args, **kw, grad_dtype=dw_dtype)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


def test_logprob_bwd_one_of_the_gradients_and_entropy_alone():
    N, V, d = 40, 300, 128
    h, w, t = _inputs(N, V, d, BF, 2)
    h, w, t = h.to(dev()), w.to(dev()), t.to(dev())
    res = txl.logprob_fwd(h, w, t)
    dlogp = torch.randn(N, device=dev())
    both = txl.logprob_bwd(h, w, t, res.lse, dlogp)
    only_h = txl.logprob_bwd(h, w, t, res.lse, dlogp, grads=(torch.empty_like(h), None))
    only_w = txl.logprob_bwd(h, w, t, res.lse, dlogp, grads=(None, torch.empty_like(w)))
    assert torch.equal(both[0], only_h[0]) and torch.equal(both[1], only_w[1])
    dent = torch.randn(N, device=dev())
    got = txl.logprob_bwd(h, w, None, res.lse, None, entropy=res.entropy, dentropy=dent)
    _ok()
    ref = model.LogProb(h.cpu(), w.cpu(), None, 1.0, 0)
    _check_grads(got, ref, N, V, BF, BF, None, dent.cpu(), res.lse.cpu(), res.entropy.cpu())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_logprob_bwd_rows_without_a_part_hold_anything(dtype):
    N, V, d = 150, 100, 64
    h, w, t = _inputs(N, V, d, dtype, 5)
    h, w, t = h.to(dev()), w.to(dev()), t.to(dev())
    dead = t < 0
    assert bool(dead.any())
    res = txl.logprob_fwd(h, w, t)
    dlogp = torch.randn(N, device=dev())
    want = txl.logprob_bwd(h, w, t, res.lse, dlogp)
    h2, lse2, dlogp2 = h.clone(), res.lse.clone(), dlogp.clone()
    h2[dead] = float("nan")
    h2[dead.nonzero()[0]] = float("inf")
    lse2[dead] = float("nan")
    dlogp2[dead] = float("inf")
    got = txl.logprob_bwd(h2, w, t, lse2, dlogp2)
    _ok()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool((got[0][dead] == 0).all())


def test_logprob_bwd_in_vocabulary_chunks():
    # G of all logits (2.4 GB) is past the workspace's limit
    N, V, d = 20000, 60000, 16
    g = torch.Generator(device=dev()).manual_seed(1)
    h = torch.randn(N, d, generator=g, device=dev()).to(BF)
    w = torch.randn(V, d, generator=g, device=dev()).to(BF) * 0.5
    t = torch.randint(0, V, (N,), generator=g, device=dev())
    assert txl.logprob_bwd_workspace_size(N, V, d) < 2 * N * V
    lse = txl.logprob_fwd(h, w, t).lse
    dlogp = torch.randn(N, generator=g, device=dev())
    dh, dw = txl.logprob_bwd(h, w, t, lse, dlogp)
    _ok()
    # the same rows by themselves, in one chunk, and columns by the formula in 64 bits
    some = slice(5000, 5200)
    part, _ = txl.logprob_bwd(h[some], w, t[some], lse[some], dlogp[some])
    lp = h.double() @ w.double()[59000:59200].t() - lse.double()[:, None]
    G = -dlogp.double()[:, None] * torch.exp(lp)
    col = torch.arange(59000, 59200, device=dev())
    G += dlogp.double()[:, None] * (t[:, None] == col)
    want = G.t() @ h.double()
    size = G.abs().t() @ h.double().abs()
    # (sums in another order and grouping: of terms of size |G| |w|)
    ref = model.LogProb(h[some].cpu(), w.cpu(), t[some].cpu(), 1.0, 0)
    _, _, dh_size, _, _, _ = ref.grads(dlogp[some].cpu(), None, None, lse[some].cpu())
    tol = 2 * V * model.F32_CUT * dh_size + 2 * model.BF16_HALF * part.cpu().double().abs() + 1e-30
    assert bool(((dh[some].cpu().double() - part.cpu().double()).abs() <= tol).all())
    tol = (model.BF16_HALF + N * model.F32_CUT + 1e-4) * size + model.BF16_HALF * want.abs()
    assert bool(((dw[59000:59200].double() - want).abs() <= tol).all())


def test_logprob_bwd_of_few_rows_in_vocabulary_chunks():
    # G of all logits, a pair, is past the workspace's limit
    N, V, d = 128, 2200000, 8
    g = torch.Generator(device=dev()).manual_seed(4)
    h = torch.randn(N, d, generator=g, device=dev()).to(BF)
    w = torch.randn(V, d, generator=g, device=dev()).to(BF) * 0.5
    t = torch.randint(0, V, (N,), generator=g, device=dev())
    t[::5] = -1
    assert txl.logprob_bwd_workspace_size(N, V, d) < 4 * N * V
    lse = txl.logprob_fwd(h, w, t).lse
    dlogp = torch.randn(N, generator=g, device=dev())
    dh, dw = txl.logprob_bwd(h, w, t, lse, dlogp)
    _ok()
    live = (t >= 0).double() * dlogp.double()
    want_h, size = torch.zeros(N, d, dtype=torch.float64, device=dev()), torch.zeros(N, d, dtype=torch.float64, device=dev())
    lse64 = torch.logsumexp(torch.cat([torch.logsumexp(h.double() @ w[i:i + 275000].double().t(), 1, keepdim=True)
                                       for i in range(0, V, 275000)], 1), 1)
    for i in range(0, V, 275000):
        W = w[i:i + 275000].double()
        G = -live[:, None] * torch.exp(h.double() @ W.t() - lse64[:, None])
        at = t - i
        here = (at >= 0) & (at < 275000) & (t >= 0)
        G[here, at[here]] += live[here]
        want_h += G @ W
        size += G.abs() @ W.abs()
        # G a pair (2^-16), its logits' sums of 8 and the log-sum-exp's error (V 2^-23 at most, of its terms),
        # sums of N; one rounding of the result
        tol = (2.0 ** -16 + V * model.F32_CUT + N * model.F32_CUT) * (G.abs().t() @ h.double().abs())
        got = dw[i:i + 275000].double()
        want = G.t() @ h.double()
        assert bool(((got - want).abs() <= tol + model.BF16_HALF * want.abs() + 1e-30).all())
    tol = (2.0 ** -16 + 2 * V * model.F32_CUT) * size + model.BF16_HALF * want_h.abs() + 1e-30
    assert bool(((dh.double() - want_h).abs() <= tol).all())


def test_logprob_bwd_against_differences():
    # a directional derivative of sum g logp + e H: central differences of the fp32 path in 64-bit
    # sums.  The third derivative of a log-softmax along a direction of logit changes at most D is at
    # most 2 D^3; the values' errors enter over the step.
    N, V, d = 6, 50, 32
    h, w, t = _inputs(N, V, d, F32, 21)
    t[0] = 3
    g = torch.Generator().manual_seed(5)
    dlogp, dent = torch.randn(N, generator=g), torch.randn(N, generator=g)
    eh, ew = torch.randn(N, d, generator=g), torch.randn(V, d, generator=g) * 0.3
    D = lambda x: x.to(dev())
    res = txl.logprob_fwd(D(h), D(w), D(t))
    dh, dw = txl.logprob_bwd(D(h), D(w), D(t), res.lse, D(dlogp), entropy=res.entropy, dentropy=D(dent))
    step = 2.0 ** -7

    def value(s):
        ref = model.LogProb(h.double() + s * eh.double(), w.double() + s * ew.double(), t, 1.0, 0)
        return float((ref.logp * dlogp.double()).sum() + (ref.entropy * dent.double()).sum())

    slope = (value(step) - value(-step)) / (2 * step)
    fine = (value(step / 2) - value(-step / 2)) / step
    got = float((dh.cpu().double() * eh).sum() + (dw.cpu().double() * ew).sum())
    # the step's error falls to a quarter when it is halved: three quarters of it is what the two
    # slopes differ by, and the finer one is off by a third of that; fp32 gradients by 1e-4 of
    # their terms
    size = float((dh.cpu().double() * eh).abs().sum() + (dw.cpu().double() * ew).abs().sum())
    assert abs(got - fine) <= abs(slope - fine) + 1e-4 * size


def test_logprob_bwd_captured_beside_an_eager_call():
    N, V, d = 70, 400, 128
    h, w, t = (x.to(dev()) for x in _inputs(N, V, d, BF, 13))
    res = txl.logprob_fwd(h, w, t)
    dlogp = torch.randn(N, device=dev())
    eager = txl.logprob_bwd(h, w, t, res.lse, dlogp)
    size = txl.logprob_bwd_workspace_size(N, V, d)
    graphs = []
    for _ in range(2):
        ws = torch.empty(size, dtype=torch.uint8, device=dev())
        grads = torch.zeros_like(h), torch.zeros_like(w)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            txl.logprob_bwd(h, w, t, res.lse, dlogp, grads=grads, workspace=ws)
        graphs.append((graph, grads, ws))
    for graph, _, _ in graphs:
        graph.replay()
    _ok()
    for _, grads, _ in graphs:
        assert all(torch.equal(a, b) for a, b in zip(grads, eager))


def test_logprob_refusals():
    h, w = torch.zeros(3, 16, device=dev()), torch.zeros(5, 16, device=dev())
    t = torch.zeros(3, dtype=torch.int64, device=dev())
    f = torch.zeros(3, device=dev())
    for bad in (lambda: txl.logprob_fwd(h.to(BF), w), lambda: txl.logprob_fwd(h[:, :8], w),
                lambda: txl.logprob_fwd(h, w, t[:2]), lambda: txl.logprob_fwd(h, w, t.float()),
                lambda: txl.logprob_fwd(h, w.t()), lambda: txl.logprob_fwd(h.cpu(), w),
                lambda: txl.logprob_bwd(h, w, t, f[:2], f),
                lambda: txl.logprob_bwd(h, w, t, f.double(), f)):
        with pytest.raises(ValueError):
            bad()
    for status, bad in (
            (-2, lambda: txl.logprob_fwd(h, w, top=17)), (-1, lambda: txl.logprob_fwd(h, w, top=-1,
                                                          out=txl.LogProbs(None, f, None))),
            (-1, lambda: txl.logprob_fwd(h, w, out=txl.LogProbs(None, None, None))),
            (-1, lambda: txl.logprob_fwd(h, w, scale=float("nan"))),
            (-7, lambda: txl.logprob_fwd(h, w, workspace=torch.zeros(256, dtype=torch.uint8, device=dev()))),
            (-1, lambda: txl.logprob_bwd(h, w, t, f, None)), (-1, lambda: txl.logprob_bwd(h, w, None, f, None)),
            (-1, lambda: txl.logprob_bwd(h, w, None, f, None, dentropy=f)),
            (-1, lambda: txl.logprob_bwd(h, w, t, f, f, grads=(None, None))),
            (-2, lambda: txl.logprob_bwd(h, w, t, f, f, grad_dtype=BF))):
        with pytest.raises(txl.TxlError) as e:
            bad()
        assert e.value.status == status
    assert txl.device_status() == 0


def test_lone_rows_with_any_stride():
    # (a stride that leads nowhere: C callers pass what their array has)
    for N, V in ((1, 50), (5, 1), (1, 1)):
        d = 64
        h, w, t = (x.to(dev()) for x in _inputs(N, V, d, BF, N + V))
        lse, dlogp = torch.zeros(N, device=dev()), torch.ones(N, device=dev())
        dh, dw = torch.zeros_like(h), torch.zeros_like(w)
        hs, ws = 8 if N == 1 else d, 8 if V == 1 else d
        kind = 4 if t.dtype == torch.int32 else 8
        room = torch.empty(max(txl.logprob_fwd_workspace_size(N, V, d), txl.logprob_bwd_workspace_size(N, V, d)),
                           dtype=torch.uint8, device=dev())
        stream = torch.cuda.current_stream().cuda_stream
        ptr = lambda *x: [y.data_ptr() for y in x]
        assert txl.lib().txl_logprob_fwd(h.data_ptr(), hs, w.data_ptr(), ws, t.data_ptr(), kind, None,
                                         lse.data_ptr(), None, None, None, N, V, d, 0, 1.0, txl.BF16,
                                         room.data_ptr(), room.numel(), stream) == 0
        assert txl.lib().txl_logprob_bwd(h.data_ptr(), hs, w.data_ptr(), ws, t.data_ptr(), kind, lse.data_ptr(),
                                         None, dlogp.data_ptr(), None, dh.data_ptr(), dw.data_ptr(), N, V, d, 1.0,
                                         txl.BF16, txl.BF16, room.data_ptr(), room.numel(), stream) == 0
        _ok()
        assert torch.equal(lse, txl.logprob_fwd(h, w, t).lse)
        want = txl.logprob_bwd(h, w, t, lse, dlogp)
        assert torch.equal(dh, want[0]) and torch.equal(dw, want[1])


def test_tables_past_two_to_the_31_elements():
    V, d = 33000, 65536
    g = torch.Generator(device=dev()).manual_seed(9)
    w = torch.empty(V, d, dtype=BF, device=dev())
    w.normal_(0.0, 0.02, generator=g)
    ids = torch.tensor([V - 1, 3, V - 2, V - 1, -1], device=dev())
    x = txl.embed_fwd(ids, w)
    assert torch.equal(x[:4], w[ids[:4]]) and bool((x[4] == 0).all())
    dtab = txl.embed_bwd(x, ids, V, dtype=BF)
    # (two equal rows of bf16 sum exactly, but for a doubled largest value)
    assert torch.equal(dtab[V - 1], 2 * w[V - 1]) and torch.equal(dtab[V - 2], w[V - 2]) and torch.equal(dtab[3], w[3])
    assert int((dtab.abs().amax(1) > 0).sum()) == 3
    del dtab
    h = torch.randn(5, d, generator=g, device=dev()).to(BF)
    t = torch.tensor([V - 1, V - 2, 0, -1, 32768], device=dev(), dtype=torch.int32)
    res = txl.logprob_fwd(h, w, t, scale=0.25, top=4)
    dlogp = torch.tensor([1.0, -0.5, 0.3, 7.0, 2.0], device=dev())
    dh, dw = txl.logprob_bwd(h, w, t, res.lse, dlogp, scale=0.25)
    _ok()
    z = torch.cat([0.25 * (h.double() @ w[i:i + 4096].double().t()) for i in range(0, V, 4096)], 1).cpu()
    lse = torch.logsumexp(z, 1)
    off = d * model.F32_CUT * 0.25 * (h.double().abs() @ w[:4096].double().abs().t()).max().item() * 1.1
    assert float((res.lse.cpu().double() - lse).abs().max()) <= off
    lp = z - lse[:, None]
    live = t.cpu() >= 0
    want = lp.gather(1, t.cpu().long().clamp(min=0)[:, None])[:, 0] * live
    assert float((res.logp.cpu().double() - want).abs().max()) <= 2 * off
    assert torch.equal(res.top_ids.cpu().long(), torch.sort(z, dim=1, descending=True, stable=True)[1][:, :4])
    # the last rows of dW: G a bf16 pair (residuals of 2^-16), one rounding of the result, probabilities
    # off by the logits' bound
    some = torch.arange(V - 200, V)
    hit = (some[None, :] == t.cpu()[:, None]).double()
    G = 0.25 * (dlogp.cpu().double() * live)[:, None] * (hit - torch.exp(lp[:, some]))
    p_off = 0.25 * (dlogp.cpu().double().abs() * live)[:, None] * torch.exp(lp[:, some]) * 2 * off
    h64 = h.cpu().double()
    tol = ((G.abs() * 2.0 ** -16 + p_off).t() @ h64.abs()) * 1.1 + model.BF16_HALF * (G.t() @ h64).abs() + 1e-30
    assert bool(((dw[V - 200:].cpu().double() - G.t() @ h64).abs() <= tol).all())
    # dh along some columns, over all of the table
    cols = slice(d - 64, d)
    G = 0.25 * (dlogp.cpu().double() * live)[:, None] * (torch.nn.functional.one_hot(t.cpu().long().clamp(min=0), V)
                                                        * live[:, None] - torch.exp(lp))
    W = w[:, cols].cpu().double()
    size = G.abs() @ W.abs()
    tol = (2.0 ** -16 + V * model.F32_CUT + 2 * off) * size * 1.1 + model.BF16_HALF * (G @ W).abs() + 1e-30
    assert bool(((dh[:, cols].cpu().double() - G @ W).abs() <= tol).all())


def test_two_host_threads_on_their_own_streams():
    import threading

    cases = []
    for seed, (N, V, d, top) in enumerate(((5, 3000, 256, 4), (300, 1000, 64, 0))):
        h, w, t = (x.to(dev()) for x in _inputs(N, V, d, BF, seed))
        dlogp = torch.randn(N, device=dev())
        res = txl.logprob_fwd(h, w, t, top=top)
        cases.append((h, w, t, dlogp, top, res, txl.logprob_bwd(h, w, t, res.lse, dlogp)))
    _ok()
    failures = []

    def run(h, w, t, dlogp, top, res, grads):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(30):
                    got = txl.logprob_fwd(h, w, t, top=top)
                    back = txl.logprob_bwd(h, w, t, got.lse, dlogp)
                    same = [torch.equal(a, b) for a, b in zip((*got, *back), (*res, *grads)) if a is not None]
                    assert all(same), same
        except BaseException as e:
            failures.append(e)

    threads = [threading.Thread(target=run, args=c) for c in cases]
    for x in threads:
        x.start()
    for x in threads:
        x.join(120)
    assert not failures, failures
    _ok()
