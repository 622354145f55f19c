"""The state advanced apart from the rows: layers appended one by one and then advanced are what one
append of all layers is, whatever the counts on the device say."""

import pytest
import torch

import transformer_xl_relative_pos_gb300 as txl
from parity import dev
from test_gpu_paged import check, make, model_append, operand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("width", [None, 4])
def test_counts_past_the_rows_given_advance_by_what_was_appended(width, dtype):
    layers, B, H, N, keep = 3, 4, 2, 9, 60
    mem, g = make(B, H, 32, 3, layers, dtype, 71, fill=[40, 55, 0, 60])
    k, v = operand(layers, B, H, N, dtype, g, "stacked")
    counts = [N + 50, 3, -2, 2 ** 31 - 1]
    rows = None if width is None else torch.randint(0, N, (B, width), generator=g).int()
    most = N if width is None else width
    n = [min(max(c, 0), most) for c in counts]
    want = model_append(mem, k, v, 0, n, None if rows is None else rows.tolist(), keep)
    n_new = torch.tensor(counts, dtype=torch.int32, device=dev())
    for i in range(layers):
        txl.paged_append(mem, k[i], v[i], layer=i, n_new=n_new, rows=None if rows is None else rows.to(dev()))
    txl.paged_advance(mem, n_new, keep=keep, max_rows=most)
    check(mem, want)


def test_counts_that_are_the_state_itself():
    # every memory doubled: n_new is fill, which the call writes
    layers, B, H, N = 2, 3, 2, 40
    mem, g = make(B, H, 32, 4, layers, "bf16", 72, fill=[33, 1, 0])
    k, v = operand(layers, B, H, N, "bf16", g, "dense")
    want = model_append(mem, k, v, 0, [33, 1, 0], None, 50)
    txl.paged_append(mem, k, v, n_new=mem.fill, keep=50)
    check(mem, want)
    want = model_append(mem, k[:, :, :, :0], v[:, :, :, :0], 0, [0] * B, None, None)
    fill, begin = mem.fill.cpu(), mem.begin.cpu()
    txl.paged_advance(mem, mem.fill, keep=128)
    assert torch.equal(mem.fill.cpu(), torch.minimum(2 * fill, torch.tensor(128)))
    assert torch.equal(mem.begin.cpu(), begin) and torch.equal(mem.pool.cpu(), want[0])
    assert txl.device_status() == 0


def test_a_number_of_rows_past_max_rows_is_refused():
    mem, _ = make(2, 1, 32, 2, 1, "bf16", 73, fill=[0, 0])
    with pytest.raises(ValueError):
        txl.paged_advance(mem, 5, keep=10, max_rows=4)
    with pytest.raises(txl.TxlError):
        txl.paged_advance(mem, torch.ones(2, dtype=torch.int32, device=dev()), keep=10, max_rows=-1)
    assert mem.fill.tolist() == [0, 0]
