"""The model's two ends directly behind one another: what one call writes, the next reads, with
nothing between them that would wait (each launch may begin beside its predecessor's end)."""

import re
from pathlib import Path

import pytest
import torch

import transformer_xl_relative_pos_gb300 as txl
from transformer_xl_relative_pos_gb300 import build

BF, F32 = torch.bfloat16, torch.float32
VOCAB_SOURCES = ["vocab.h", "embed.cu", "logprob.cu", "logprob_few.cu", "logprob_merge.cu"]


@pytest.mark.parametrize("name", VOCAB_SOURCES)
def test_no_load_takes_the_path_for_memory_that_nothing_writes(name):
    # a launch that may begin early is resident while its operands may still be written
    text = (Path(build.CSRC) / name).read_text()
    code = re.sub(r"//[^\n]*", "", text)
    assert not re.search(r"__ldg\s*\(|ld\.global\.nc|__restrict__|tex[12]D", code)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [3, 300])
def test_alternatives_are_the_next_tokens(n, dtype):
    # greedy decoding: the best words of one call are the tokens of the next, whose rows are the next
    # states, sixty times without a synchronisation; the same step by step with one after each call
    V, d = 5003, 264
    g = torch.Generator(device="cuda").manual_seed(5)
    E = torch.randn(V, d, generator=g, device="cuda").to(dtype)
    mix = (torch.randn(d, d, generator=g, device="cuda") / d ** 0.5).to(dtype)
    first = torch.randint(0, V, (n,), generator=g, device="cuda", dtype=torch.int32)

    def chain(wait):
        ids, h = first.clone(), torch.empty(n, d, dtype=dtype, device="cuda")
        outs = [txl.LogProbs(*(torch.empty(n, device="cuda") for _ in range(3)), torch.empty(n, 1, device="cuda"),
                             torch.empty(n, 1, dtype=torch.int32, device="cuda")) for _ in range(2)]
        ws = torch.empty(max(txl.logprob_fwd_workspace_size(n, V, d, dtype, top=1),
                             txl.logprob_bwd_workspace_size(n, V, d, dtype),
                             txl.embed_bwd_workspace_size(n, V, d)), dtype=torch.uint8, device="cuda")
        ones, dE = torch.ones(n, device="cuda"), torch.empty(V, d, device="cuda")
        grads, seen = (torch.empty_like(h), torch.empty_like(E)), []
        sync = torch.cuda.synchronize if wait else lambda: None
        for k in range(60):
            table, out = (E, mixed)[k % 2], outs[k % 2]
            txl.embed_fwd(ids.view(n), table, out=h)
            sync()
            txl.logprob_fwd(h, table, ids.view(n), scale=-0.1, top=1, out=out, workspace=ws)
            sync()
            ids = out.top_ids
            txl.logprob_bwd(h, table, ids.view(n), out.lse, ones, scale=-0.1, grads=grads, workspace=ws)
            sync()
            txl.embed_bwd(grads[0], ids.view(n), V, out=dE, workspace=ws)
            sync()
            if k % 10 == 9:
                seen += [t.clone() for t in (ids, h, out.logp, *grads, dE)]
        torch.cuda.synchronize()
        return seen

    mixed = (E.float() @ mix.float()).to(dtype)
    got, want = chain(False), chain(True)
    assert txl.device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert len(torch.unique(torch.stack([t.view(-1) for t in want[::6]]))) > 1   # (the words differ)
