"""txl_embed_fwd and txl_embed_bwd on the GPU against the 64-bit sums of
vocab_model: both types, odd sizes, padding, tokens that occur once, often (runs
across many chunks) or not at all, strided operands, id types, accumulation, other
streams, captured graphs; and what they refuse."""

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


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,V,d,scale,ids", [
    (1, 1, 8, 1.0, torch.int64), (7, 204, 512, 1.0, torch.int64), (33, 5, 264, 16.25, torch.int32),
    (1000, 3001, 1032, 22.627, torch.int32), (0, 9, 64, 1.0, torch.int64),
    (50, 11, 1, 1.5, torch.int64), (129, 40, 13, 1.0, torch.int32), (300, 7, 100, 0.3, torch.int64)])
def test_embed_fwd(n, V, d, scale, ids, dtype):
    g = torch.Generator().manual_seed(n + V)
    emb = torch.randn(V, d, generator=g).to(dtype)
    tok = model.tokens_with_padding(n, V, g, dtype=ids)
    out = txl.embed_fwd(tok.to(dev()), emb.to(dev()), scale=scale)
    _ok()
    # one rounding of the exact product
    want = (model.embed(tok, emb, 1.0).float() * torch.tensor(scale)).to(dtype)
    assert out.shape == (n, d) and torch.equal(out.cpu(), want)


def test_embed_fwd_strided_table_shape_stream_and_graph():
    g = torch.Generator().manual_seed(5)
    wide = torch.randn(40, 96, generator=g).to(BF).to(dev())
    emb = wide[:, 16:80]
    tok = torch.randint(0, 40, (3, 11), generator=g).to(dev())
    out = torch.full((3, 11, 64), 7.0, dtype=BF, device=dev())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    txl.embed_fwd(tok, emb, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, emb[tok])
    # a captured call reads the tokens of the replay
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        txl.embed_fwd(tok, emb, scale=2.0, out=out)
    tok.copy_((tok + 13) % 40)
    graph.replay()
    _ok()
    assert torch.equal(out, emb[tok] * 2)


def test_embed_ids_out_of_range_are_recorded_and_count_as_none():
    emb = torch.ones(4, 16, dtype=F32, device=dev())
    tok = torch.tensor([0, 4, -2, 3, 2 ** 40, -1], device=dev())
    out = txl.embed_fwd(tok, emb)
    assert txl.device_status() == -8
    assert out[:, 0].tolist() == [1, 0, 0, 1, 0, 0]
    grad = txl.embed_bwd(torch.ones(6, 16, device=dev()), tok, 4)
    assert txl.device_status() == -8
    assert grad[:, 3].tolist() == [1, 0, 0, 1]


def _check_grad(dout, tok, V, scale, grad, dtype_out):
    want, size = model.embed_grad(dout.cpu(), tok.cpu(), V, model.f32(scale))
    n = tok.numel()
    half = model.BF16_HALF if dtype_out == BF else 2.0 ** -24
    tol = (n + 2) * model.F32_CUT * size + half * want.abs() * 1.01 + 1e-45
    off = (grad.cpu().double() - want).abs()
    assert bool((off <= tol).all()), float((off - tol).max())
    absent = torch.ones(V, dtype=torch.bool)
    absent[tok.cpu().long().reshape(-1)[tok.cpu().reshape(-1) >= 0]] = False
    assert bool((grad.cpu()[absent] == 0).all())


# (tokens, vocabulary, width): one token; a few; every token often; hardly any twice; more than one
# chunk of positions each; wider than a column slice; vocabularies of two and three digits'
# passes; ends inside words and chunks
GRADS = [(1, 1, 8), (31, 3, 64), (2049, 40, 24), (70000, 1000, 8), (20000, 7, 264), (33, 204, 520), (257, 7, 264), (2000, 3, 72), (1025, 5003, 256),
         (700, 300001, 8), (5000, 512, 40), (40000, 513, 16)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,V,d", GRADS)
def test_embed_bwd(n, V, d, dtype):
    g = torch.Generator().manual_seed(n * 3 + V)
    tok = model.tokens_with_padding(n, V, g, dtype=torch.int32 if n % 2 else torch.int64).to(dev())
    dout = torch.randn(n, d, generator=g).to(dtype).to(dev())
    # what earlier calls left in the buffers has no influence
    ws = torch.full((txl.embed_bwd_workspace_size(n, V, d),), 255, dtype=torch.uint8, device=dev())
    out = torch.full((V, d), float("nan"), device=dev())
    grad = txl.embed_bwd(dout, tok, V, scale=1.7, out=out, workspace=ws)
    _ok()
    _check_grad(dout, tok, V, 1.7, grad, F32)
    again = txl.embed_bwd(dout, tok, V, scale=1.7)
    assert torch.equal(grad, again)


@pytest.mark.parametrize("n", [0, 1, 32, 64, 96, 97, 4096])
@pytest.mark.parametrize("kind", ["same", "none", "halves"])
def test_embed_bwd_runs_at_chunk_borders(n, kind):
    V, d = 6, 24
    tok = {"same": torch.full((n,), 4), "none": torch.full((n,), -1),
           "halves": torch.arange(n) // max(1, n // 2)}[kind].to(dev())
    g = torch.Generator().manual_seed(n)
    dout = torch.randn(n, d, generator=g).to(dev())
    grad = txl.embed_bwd(dout, tok, V)
    _ok()
    _check_grad(dout, tok, V, 1.0, grad, F32)


def test_embed_bwd_fp32_rows_of_four():
    g = torch.Generator().manual_seed(77)
    tok = model.tokens_with_padding(900, 33, g).to(dev())
    dout = torch.randn(900, 132, generator=g).to(dev())
    grad = txl.embed_bwd(dout, tok, 33)
    _ok()
    _check_grad(dout, tok, 33, 1.0, grad, F32)


def test_embed_bwd_bf16_output_strides_and_masked_garbage():
    g = torch.Generator().manual_seed(2)
    n, V, d = 300, 50, 72
    tok = model.tokens_with_padding(n, V, g).to(dev())
    wide = torch.randn(n, 3 * d, generator=g).to(BF).to(dev())
    dout = wide[:, d:2 * d]
    dout[tok < 0] = float("nan")   # positions without a token
    grad = txl.embed_bwd(dout, tok, V, dtype=BF)
    _ok()
    assert grad.dtype == BF
    clean = torch.where((tok < 0)[:, None], torch.zeros_like(dout), dout)
    _check_grad(clean, tok, V, 1.0, grad, BF)


def test_embed_bwd_accumulates_only_where_tokens_occur():
    g = torch.Generator().manual_seed(8)
    n, V, d = 130, 40, 40
    tok = torch.randint(0, 20, (n,), generator=g).to(dev())
    dout = torch.randn(n, d, generator=g).to(dev())
    base = torch.randn(V, d, generator=g).to(dev())
    base[30] = float("nan")        # a row that no token names
    out = base.clone()
    grad = txl.embed_bwd(dout, tok, V, out=out, accumulate=True)
    fresh = txl.embed_bwd(dout, tok, V)
    _ok()
    assert grad is out
    assert torch.equal(out[20:].isnan(), base[20:].isnan())
    assert torch.equal(out[:20], base[:20] + fresh[:20])


def test_embed_bwd_captured_and_on_two_streams():
    g = torch.Generator().manual_seed(9)
    n, V, d = 600, 97, 128
    tok = torch.randint(0, V, (n,), generator=g).to(dev())
    dout = torch.randn(n, d, generator=g).to(BF).to(dev())
    ws = torch.empty(txl.embed_bwd_workspace_size(n, V, d), dtype=torch.uint8, device=dev())
    out = torch.zeros(V, d, device=dev())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        txl.embed_bwd(dout, tok, V, out=out, workspace=ws)
    tok.copy_(torch.flip(tok, (0,)) // 2)
    graph.replay()
    _ok()
    _check_grad(dout, tok, V, 1.0, out, F32)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = [txl.embed_bwd(dout, tok, V, stream=s) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, out) for o in outs)


def test_embed_refusals():
    emb = torch.zeros(4, 16, device=dev())
    tok = torch.zeros(3, dtype=torch.int64, device=dev())
    for bad in (tok.cpu(), tok.float(), torch.zeros(6, dtype=torch.int64, device=dev())[::2]):
        with pytest.raises(ValueError):
            txl.embed_fwd(bad, emb)
    with pytest.raises(ValueError):
        txl.embed_fwd(tok, emb.half())
    with pytest.raises(ValueError):
        txl.embed_fwd(tok, emb, out=torch.zeros(3, 8, device=dev()))
    with pytest.raises(txl.TxlError):
        txl.embed_bwd(torch.zeros(3, 6, device=dev()), tok, 4)
    with pytest.raises(txl.TxlError):
        txl.embed_fwd(tok, emb, out=emb[:3])
    with pytest.raises(ValueError):
        txl.embed_bwd(torch.zeros(2, 16, device=dev()), tok, 4)
    with pytest.raises(ValueError):
        txl.embed_bwd(torch.zeros(3, 16, device=dev()), tok, 4, accumulate=True)
    with pytest.raises(txl.TxlError) as e:
        txl.embed_bwd(torch.zeros(3, 16, device=dev()), tok, 4, accumulate=True,
                      out=torch.zeros(4, 16, dtype=BF, device=dev()))
    assert e.value.status == -2
    with pytest.raises(txl.TxlError) as e:
        txl.embed_bwd(torch.zeros(3, 16, device=dev()), tok, 4,
                      workspace=torch.zeros(256, dtype=torch.uint8, device=dev()))
    assert e.value.status == -7
