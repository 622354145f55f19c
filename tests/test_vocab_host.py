"""What the token embedding and the log probabilities refuse on the host (CPU only, nothing
launches), the sizes of their workspaces, and the binding's checks of operands."""

import pytest
import torch

import transformer_xl_relative_pos_gb300 as txl

OK, INVALID, UNSUPPORTED, MISALIGNED, SHAPE, WORKSPACE = 0, -1, -2, -3, -4, -7
NAN = float("nan")
MB = 1 << 20   # (operands a megabyte apart: none overlap)


def embed(tokens=MB, kind=8, emb=2 * MB, stride=16, out=3 * MB, n=4, V=10, d=16, scale=1.0, dtype=txl.F32):
    return txl.lib().txl_embed_fwd(tokens, kind, emb, stride, out, n, V, d, scale, dtype, None)


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=None), INVALID), (dict(emb=None), INVALID), (dict(out=None), INVALID),
    (dict(kind=2), INVALID), (dict(n=-1), INVALID), (dict(V=0), INVALID), (dict(d=0), INVALID),
    (dict(scale=NAN), INVALID), (dict(dtype=5), INVALID), (dict(stride=0), INVALID),
    (dict(stride=15), SHAPE), (dict(d=70000, stride=70000), UNSUPPORTED),
    (dict(tokens=MB + 4), MISALIGNED), (dict(emb=2 * MB + 2), MISALIGNED), (dict(out=3 * MB + 1), MISALIGNED),
    (dict(out=2 * MB + 64), INVALID), (dict(out=MB), INVALID),     # over the table, over the tokens
    (dict(n=0, tokens=None, out=None), OK),
])
def test_embed_fwd_refuses(kw, want):
    assert embed(**kw) == want


def embed_bwd(tokens=MB, kind=4, dout=2 * MB, stride=16, demb=3 * MB, n=4, V=10, d=16, scale=1.0, dtype=txl.F32,
              grad=txl.F32, acc=0, ws=4 * MB, ws_bytes=MB):
    return txl.lib().txl_embed_bwd(tokens, kind, dout, stride, demb, n, V, d, scale, dtype, grad, acc, ws,
                                   ws_bytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(tokens=None), INVALID), (dict(dout=None), INVALID), (dict(demb=None), INVALID),
    (dict(grad=9), INVALID), (dict(scale=NAN), INVALID), (dict(kind=1), INVALID),
    (dict(acc=1, grad=txl.BF16), UNSUPPORTED), (dict(d=12, stride=16, dtype=txl.BF16), UNSUPPORTED),
    (dict(d=12, stride=16, grad=txl.BF16), UNSUPPORTED), (dict(d=6, stride=8), UNSUPPORTED),
    (dict(stride=18), MISALIGNED), (dict(dout=2 * MB + 8), MISALIGNED), (dict(demb=3 * MB + 4), MISALIGNED),
    (dict(ws=4 * MB + 16), MISALIGNED), (dict(stride=12), SHAPE),
    (dict(ws=None), WORKSPACE), (dict(ws_bytes=100), WORKSPACE),
    (dict(demb=2 * MB + 32), INVALID), (dict(ws=3 * MB + 256), INVALID), (dict(n=0, acc=1), OK),
])
def test_embed_bwd_refuses(kw, want):
    assert embed_bwd(**kw) == want


def fwd(h=MB, hs=16, w=2 * MB, ws_=16, t=3 * MB, kind=8, logp=4 * MB, lse=5 * MB, ent=6 * MB, tl=None, ti=None,
        N=4, V=10, d=16, top=0, scale=1.0, dtype=txl.F32, ws=8 * MB, ws_bytes=MB):
    return txl.lib().txl_logprob_fwd(h, hs, w, ws_, t, kind, logp, lse, ent, tl, ti, N, V, d, top, scale, dtype,
                                     ws, ws_bytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(h=None), INVALID), (dict(w=None), INVALID), (dict(top=-1), INVALID), (dict(top=2), INVALID),
    (dict(logp=None, lse=None, ent=None), INVALID), (dict(scale=NAN), INVALID), (dict(dtype=2), INVALID),
    (dict(kind=3), INVALID), (dict(N=-1), INVALID), (dict(V=0), INVALID), (dict(hs=0), INVALID),
    (dict(top=17, tl=9 * MB, ti=10 * MB), UNSUPPORTED), (dict(d=12, hs=16, ws_=16), UNSUPPORTED),
    (dict(h=MB + 4), MISALIGNED), (dict(hs=18), MISALIGNED), (dict(w=2 * MB + 8), MISALIGNED),
    (dict(t=3 * MB + 4), MISALIGNED), (dict(lse=5 * MB + 2), MISALIGNED), (dict(ws=8 * MB + 64), MISALIGNED),
    (dict(hs=8), SHAPE), (dict(ws_=12), SHAPE), (dict(ws=None), WORKSPACE), (dict(ws_bytes=16), WORKSPACE),
    (dict(lse=4 * MB + 8), INVALID), (dict(logp=MB + 32), INVALID), (dict(ent=3 * MB + 28), INVALID),
    (dict(ws=2 * MB + 256), INVALID), (dict(top=1, tl=9 * MB, ti=9 * MB + 12), INVALID),
    (dict(N=0, h=None, t=None, logp=None, lse=None, ent=None, ws=None, ws_bytes=0), OK),
])
def test_logprob_fwd_refuses(kw, want):
    assert fwd(**kw) == want


def bwd(h=MB, hs=16, w=2 * MB, ws_=16, t=3 * MB, kind=8, lse=4 * MB, ent=None, g=5 * MB, e=None, dh=6 * MB,
        dw=7 * MB, N=4, V=10, d=16, scale=1.0, dtype=txl.F32, grad=txl.F32, ws=8 * MB, ws_bytes=MB):
    return txl.lib().txl_logprob_bwd(h, hs, w, ws_, t, kind, lse, ent, g, e, dh, dw, N, V, d, scale, dtype, grad,
                                     ws, ws_bytes, None)


@pytest.mark.parametrize("kw,want", [
    (dict(h=None), INVALID), (dict(w=None), INVALID), (dict(lse=None), INVALID),
    (dict(dh=None, dw=None), INVALID), (dict(t=None), INVALID), (dict(g=None), INVALID),
    (dict(t=None, g=None), INVALID), (dict(e=9 * MB), INVALID), (dict(scale=NAN), INVALID),
    (dict(grad=4), INVALID), (dict(grad=txl.BF16), UNSUPPORTED), (dict(d=20, hs=32, ws_=32), UNSUPPORTED),
    (dict(dh=6 * MB + 8), MISALIGNED), (dict(dw=7 * MB + 4), MISALIGNED), (dict(g=5 * MB + 2), MISALIGNED),
    (dict(hs=8), SHAPE), (dict(ws=None), WORKSPACE), (dict(ws_bytes=256), WORKSPACE),
    (dict(dh=MB), INVALID), (dict(dw=2 * MB), INVALID), (dict(dw=6 * MB + 64), INVALID),
    (dict(ws=4 * MB - 256), INVALID), (dict(N=0, dw=None, h=None, lse=None, t=None, g=None), OK),
])
def test_logprob_bwd_refuses(kw, want):
    assert bwd(**kw) == want


@pytest.mark.parametrize("call", [embed, embed_bwd, fwd, bwd])
@pytest.mark.parametrize("scale", [float("inf"), -float("inf")])
def test_infinite_scales_are_refused(call, scale):
    # (times the zeros of an absent token it would be NaN)
    assert call(scale=scale) == INVALID


def test_workspace_sizes():
    assert txl.embed_bwd_workspace_size(0, 10, 16) == 0
    assert txl.embed_bwd_workspace_size(100, 10, 6) == 0       # refused sizes need none
    assert txl.embed_bwd_workspace_size(1000, 10, 16) > 2 * 1000 * 8
    assert txl.logprob_fwd_workspace_size(4, 100, 64, top=17) == 0
    assert txl.logprob_fwd_workspace_size(4, 1000, 64, top=8) > txl.logprob_fwd_workspace_size(4, 1000, 64)
    assert (txl.logprob_fwd_workspace_size(500, 1000, 64, torch.float32) >=
            txl.logprob_fwd_workspace_size(500, 1000, 64) + 1500 * 64 * 6)
    N, V, d = 512, 4096, 64
    assert txl.logprob_bwd_workspace_size(N, V, d) >= N * V * 2
    assert txl.logprob_bwd_workspace_size(N, V, d, grad_dtype=torch.float32) >= N * V * 4
    # G in chunks of the vocabulary past 1 GiB
    assert txl.logprob_bwd_workspace_size(1 << 16, 1 << 18, 8) < 2 * (1 << 30)
    with pytest.raises(ValueError):
        txl.logprob_fwd_workspace_size(4, 10, 16, torch.float16)


def test_binding_refuses_host_tensors_and_other_kinds():
    x, ids = torch.zeros(3, 16), torch.zeros(3, dtype=torch.int64)
    for bad in (lambda: txl.embed_fwd(ids, x), lambda: txl.logprob_fwd(x, x),
                lambda: txl.logprob_bwd(x, x, ids, x[:, 0], x[:, 0]), lambda: txl.embed_bwd(x, ids, 4)):
        with pytest.raises((ValueError, RuntimeError)):
            bad()
    with pytest.raises(TypeError):
        txl.embed_fwd(ids, [[0.0]])
    with pytest.raises(TypeError):
        txl.logprob_fwd([[0.0]], [[0.0]])


@pytest.mark.parametrize("N,V,d", [(2048, 50257, 1024), (1024, 50257, 768), (2048, 50001, 512), (2048, 28000, 1024),
                                   (1024, 33000, 1024), (4096, 42000, 512), (1100, 25001, 1032), (700, 50257, 1032),
                                   (2048, 32000, 512), (1, 40000, 8), (5, 57344, 1272), (333, 5003, 520)])
def test_every_size_of_the_gradient_has_tiles_and_parts(N, V, d):
    # fp32: three bf16 terms of h, w and G in rows of whole lines, and the parts of dh that sums of at most
    # 64 steps of 64 words leave
    line, up128 = (d + 63) // 64 * 64, (V + 127) // 128 * 128
    steps = (V + 63) // 64
    parts = (steps + 63) // 64
    least = 6 * ((N + V) * line + N * up128) + (4 * parts * N * d if parts > 1 else 0)
    assert txl.logprob_bwd_workspace_size(N, V, d, torch.float32) >= least


def test_gradient_workspaces_over_many_sizes():
    # (no size divides by nothing; rows of G are there whatever the type)
    import random

    rng = random.Random(17)
    for _ in range(3000):
        N, V, d = (int(2 ** rng.uniform(0, b)) for b in (14, 18, 9))
        d *= 8
        for dtype, grad in ((torch.bfloat16,) * 2, (torch.bfloat16, torch.float32), (torch.float32,) * 2):
            assert txl.logprob_bwd_workspace_size(N, V, d, dtype, grad_dtype=grad) >= N * min(V, 128) * 2
            assert txl.logprob_fwd_workspace_size(N, V, d, dtype, top=rng.choice([0, 4])) >= N * 16


@pytest.mark.parametrize("N", [65536, 262144, 1 << 20])
@pytest.mark.parametrize("dtype,grad", [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32),
                                        (torch.float32, torch.float32)])
def test_the_gradients_workspace_grows_with_the_rows_not_their_square(N, dtype, grad):
    # V x d = 131072 x 1024: chunks of G of 1 GiB (or 128 columns of three terms), h in bf16 or three terms of it, w in
    # three terms, two fp32 dh, parts of a chunk's dw for chains of 64 steps (a quarter GiB) and of its dh (another)
    V, d = 131072, 1024
    terms = 3 if dtype == torch.float32 else 1
    g = max(1 << 30, N * 128 * 2 * 3)
    most = g + terms * N * d * 2 + (6 * V * d if terms == 3 else 0) + 2 * N * d * 4 + (1 << 29) + (1 << 28)
    assert txl.logprob_bwd_workspace_size(N, V, d, dtype, grad_dtype=grad) <= most


@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32 + 5, 2 ** 40 + 100])
def test_counts_past_an_int_are_refused_not_cut(big):
    # (2^32 + 5 rows are not 5)
    for size in (txl.embed_bwd_workspace_size(big, 10, 16), txl.embed_bwd_workspace_size(10, big, 16),
                 txl.logprob_fwd_workspace_size(big, 10, 16), txl.logprob_fwd_workspace_size(10, big, 16),
                 txl.logprob_fwd_workspace_size(10, 10, 16, top=big), txl.logprob_bwd_workspace_size(big, 10, 16),
                 txl.logprob_bwd_workspace_size(10, big, 16), txl.logprob_bwd_workspace_size(10, 10, big * 8)):
        assert size == 0
    assert txl.embed_bwd_workspace_size(-big, 10, 16) == 0
