"""The model's two ends in use: the stack's embeddings and log probabilities (evaluation,
drafts chosen and accepted by them), graphs, and a training step of one layer whose
gradients run from the log probabilities through the attention to the tied table.

"Transformer-XL: Attentive Language Models Beyond a Fixed-Length Context", §3.3 N-layer
summary."""

import math

import pytest
import torch

import transformer_xl_relative_pos_gb300 as txl
import txl_inputs
import vocab_model as model
from parity import dev
from transformer_xl_relative_pos_gb300.model import XLStack, rel_table_heads

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

W = txl_inputs.Workload("vocab_stack", B=3, H=2, dh=64, L=24, M=40, d_model=128, dtype="bf16", seed=71,
                        d_ff=256, n_layer=2, n_seg=4, vocab=205)


def stack(**kw):
    return XLStack(txl_inputs.draw_stack(W), W.H, W.M, dev(), kw.pop("dtype", BF), **kw)


def tokens(*shape, seed=0):
    return torch.randint(0, W.vocab, shape, generator=torch.Generator().manual_seed(seed))


def _ok():
    torch.cuda.synchronize()
    assert txl.device_status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_the_embedding_is_the_tables_rows(dtype):
    s = stack(dtype=dtype)
    toks = tokens(W.B, W.L).to(dev())
    assert torch.equal(s._embed(toks), s.emb[toks])
    assert torch.equal(s._embed(toks.int()), s.emb[toks])
    assert torch.equal(s._embed(toks.t()), s.emb[toks.t()])      # (not contiguous)
    scaled = stack(dtype=dtype, emb_scale=math.sqrt(W.d_model))
    factor = torch.tensor(math.sqrt(W.d_model))
    assert torch.equal(scaled._embed(toks).cpu(), (s.emb[toks].float().cpu() * factor).to(dtype))
    _ok()


@pytest.mark.parametrize("kw", [dict(), dict(cache_kv=True), dict(cache_kv=True, graphs=True), dict(paged=True)])
def test_scores_of_a_stream(kw):
    # perplexity of a stream, segment by segment, against the 64-bit softmax of the same states
    s = stack(**kw)
    text = tokens(W.B, 5 * W.L + 1, seed=3)
    text[0, -3:] = -1                                             # a stream that ends early
    for i in range(5):
        seg, nxt = text[:, i * W.L:(i + 1) * W.L], text[:, i * W.L + 1:(i + 1) * W.L + 1]
        h = s.segment(seg.clamp(min=0))
        got = s.log_probs(h, nxt, top=3)
        _ok()
        ref = model.LogProb(h.cpu(), s.emb.cpu(), nxt, 1.0, 3)
        assert got.logp.shape == (W.B, W.L) and got.top_ids.shape == (W.B, W.L, 3)
        assert torch.equal(got.top_ids.cpu().long().view(-1, 3), ref.top_ids)
        for x, want, off in ((got.logp, ref.logp, ref.logp_off), (got.lse, ref.lse, ref.lse_off),
                             (got.entropy, ref.entropy, ref.ent_off)):
            assert bool(((x.cpu().double().view(-1) - want).abs() <= off).all())
    a, b = stack(**kw), stack(**kw)
    seg, nxt = tokens(W.B, W.L, seed=5), tokens(W.B, W.L, seed=6)
    one, two = a.score(seg, nxt, top=2), b.log_probs(b.segment(seg), nxt, top=2)
    assert all(torch.equal(x, y) for x, y in zip(one, two))


def test_drafts_grow_from_the_alternatives_and_are_accepted_by_them():
    # greedy decoding by drafted trees gives the tokens that greedy decoding one by one does
    plain, drafted = stack(paged=True), stack(paged=True)
    prompt = tokens(W.B, 9, seed=8)
    first = [s.log_probs(s.segment(prompt)[:, -1], top=2).top_ids.cpu() for s in (plain, drafted)]
    assert torch.equal(*first)
    want, tok = [], first[0][:, :1]
    for _ in range(3):
        want.append(tok)
        tok = plain.log_probs(plain.segment(tok)[:, -1], top=1).top_ids.cpu()
    # the two best first tokens, each followed by the third's and first's best of the text so far
    guess = torch.cat([first[1], torch.stack([want[1][:, 0], want[1][:, 0]], 1), want[2]], 1)
    parents = torch.tensor([-1, -1, 0, 1, 2])
    h = drafted.draft(guess, parents)
    best = drafted.log_probs(h, top=1).top_ids[..., 0].cpu()
    paths = []
    for b in range(W.B):
        path, node = [0], 0                                       # (the first token is the best)
        while True:
            child = [i for i in range(5) if int(parents[i]) == node and int(guess[b, i]) == int(best[b, node])]
            if not child:
                break
            node = child[0]
            path.append(node)
        paths.append(path)
    _ok()
    assert all(p == [0, 2, 4] for p in paths), paths
    drafted.accept(paths)
    assert torch.equal(best[:, 4:], tok)


def test_a_training_step_of_one_tied_layer():
    # loss = mean -log p(next) - 0.01 mean H of one attention layer with a residual; the table is both
    # ends, so its gradient is the log probabilities' plus the embedding's
    B, L, V, H, dh = 3, 20, 150, 2, 64
    d, M, scale = H * dh, 0, 1 / math.sqrt(64)
    g = torch.Generator().manual_seed(31)
    E = (torch.randn(V, d, generator=g) * 0.3).to(BF)
    Wq, Wk, Wv, Wo = ((torch.randn(d, d, generator=g) * d ** -0.5).to(BF) for _ in range(4))
    u, vb = ((torch.randn(H, dh, generator=g) * 0.2).to(BF) for _ in range(2))
    toks = torch.randint(0, V, (B, L), generator=g)
    nxt = torch.randint(0, V, (B, L), generator=g)
    nxt[1, -4:] = -1
    emb_scale = 2.0
    n = int((nxt >= 0).sum())
    dlogp = torch.full((B, L), -1.0 / n)
    dent = torch.full((B, L), -0.01 / (B * L))

    D = lambda t: t.to(dev())
    Ed = D(E)
    R = txl.rel_pos_emb(L, d, dtype=F32, device=dev())
    r = rel_table_heads(R, torch.eye(d, device=dev()), H).to(BF)
    h0 = txl.embed_fwd(D(toks), Ed, scale=emb_scale)
    heads = lambda x: x.view(B, L, H, dh).transpose(1, 2).contiguous()
    q, k, v = (heads(h0 @ D(w).t()) for w in (Wq, Wk, Wv))
    a = txl.relattn_fwd(q, k, v, r, D(u), D(vb), M, scale)
    flat = a.transpose(1, 2).reshape(B, L, d)
    h = (h0.float() + (flat @ D(Wo).t()).float()).to(BF)
    res = txl.logprob_fwd(h, Ed, D(nxt), top=1)
    gh, dE = txl.logprob_bwd(h, Ed, D(nxt), res.lse, D(dlogp), entropy=res.entropy, dentropy=D(dent),
                             grad_dtype=F32)
    da = heads(gh @ D(Wo))
    dq, dk, dv, *_ = txl.relattn_bwd(q, k, v, r, D(u), D(vb), da, M, scale)
    unhead = lambda x: x.transpose(1, 2).reshape(B, L, d)
    dh0 = gh.float() + sum(unhead(x) @ D(w).float() for x, w in ((dq, Wq), (dk, Wk), (dv, Wv)))
    txl.embed_bwd(dh0, D(toks), V, scale=emb_scale, out=dE, accumulate=True)
    _ok()

    # the same in 64 bits by automatic differentiation
    P = {name: t.double().requires_grad_() for name, t in dict(E=E).items()}
    x0 = P["E"][toks] * emb_scale
    h64 = lambda x: x.view(B, L, H, dh).transpose(1, 2)
    q64, k64, v64 = (h64(x0 @ w.double().t()) for w in (Wq, Wk, Wv))
    rel = r.cpu().double().flip(1)                                # row = distance
    dist = torch.arange(L)[:, None] - torch.arange(L)[None]
    pos = torch.einsum("bhid,hijd->bhij", q64 + vb.double()[None, :, None], rel[:, dist.clamp(min=0)])
    A = scale * ((q64 + u.double()[None, :, None]) @ k64.transpose(2, 3) + pos)
    A = A.masked_fill(dist < 0, -math.inf)
    y = x0 + (torch.softmax(A, -1) @ v64).transpose(1, 2).reshape(B, L, d) @ Wo.double().t()
    lp = torch.log_softmax(y @ P["E"].t(), -1)
    logp = lp.gather(2, nxt.clamp(min=0)[..., None])[..., 0] * (nxt >= 0)
    ent = -(lp.exp() * lp).sum(-1)
    ((logp * dlogp.double()).sum() + (ent * dent.double()).sum()).backward()
    want = P["E"].grad
    # the states differ by the bf16 roundings of h0, q, k, v, the scores' operands, a and h: seven
    # of 2^-8 of their size, which reach a gradient through a few products of norms near one; the
    # gradient's own five (dh, G, da, dq..., dout) as many.  Twelve of 2^-8 in the norm.
    err = float((dE.cpu().double() - want).norm() / want.norm())
    assert err <= 12 * model.BF16_HALF, err
    # (both ends are in it: without either the error is far above that)
    only = txl.logprob_bwd(h, Ed, D(nxt), res.lse, D(dlogp), entropy=res.entropy, dentropy=D(dent),
                           grad_dtype=F32)[1]
    assert float((only.cpu().double() - want).norm() / want.norm()) > 0.2


def test_captured_behind_copies_and_other_streams():
    # calls in one graph behind a copy, behind torch kernels, behind one another and behind a second
    # stream that joins: replays follow what those leave
    V, d, n = 300, 64, 500
    g = torch.Generator().manual_seed(4)
    E = (torch.randn(V, d, generator=g) * 0.3).to(BF).to(dev())
    src = torch.randint(0, V, (n,), generator=g).to(dev())
    toks, h = torch.zeros_like(src), torch.zeros(n, d, dtype=BF, device=dev())
    dlogp = torch.randn(n, generator=g).to(dev())
    other = torch.cuda.Stream()

    def step(stream=None):
        toks.copy_(src)                                    # a copy, then our kernel
        h.copy_(txl.embed_fwd(toks, E, scale=2.0))
        if stream is not None:                             # a second stream in between
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                h.mul_(1.5)
            torch.cuda.current_stream().wait_stream(stream)
        else:
            h.mul_(1.5)
        res = txl.logprob_fwd(h, E, toks, top=3)
        few = txl.logprob_fwd(h[:20], E, toks[:20], top=3)
        dh, dE = txl.logprob_bwd(h, E, toks, res.lse, dlogp, grad_dtype=F32)
        txl.embed_bwd(dh, toks, V, out=dE, accumulate=True)
        return [*res, *few, dh, dE]

    want = [t.clone() for t in step()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(other)
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        _ok()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    src.copy_(torch.flip(src, (0,)))
    want = [t.clone() for t in step()]
    graph.replay()
    _ok()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("kw", [dict(), dict(cache_kv=True), dict(cache_kv=True, graphs=True), dict(paged=True)])
def test_ids_outside_the_vocabulary(kw):
    # on the host they are refused before anything moves; on the device they count as none, and are recorded
    s, other = stack(**kw), stack(**kw)
    for i in range(3):
        seg = tokens(W.B, W.L, seed=40 + i)
        assert torch.equal(s.segment(seg), other.segment(seg))
        wrong = seg.clone()
        wrong[1, 5] = W.vocab
        with pytest.raises(IndexError):
            s.segment(wrong)
        with pytest.raises(IndexError):
            s.score(seg, wrong)
    _ok()
    none = wrong.clone()
    none[1, 5] = -1
    got, want = s.segment(wrong.to(dev())).clone(), other.segment(none)
    assert torch.equal(got, want)
    torch.cuda.synchronize()
    assert txl.device_status() == -8
