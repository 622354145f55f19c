"""Outputs of the paged memory's calls that would be written while other blocks still read them as
inputs are refused (CPU only, nothing launches)."""

import ctypes

import pytest

import transformer_xl_relative_pos_gb300 as txl
from test_paged_host import INVALID, SHAPE, append, kv

# (B = 3, slots = 3: begin at 8192, fill at 12288, 12 bytes each, table at 4096, 36 bytes.)  A
# keep past the table is refused after the overlaps: SHAPE says that no overlap was found.
PAST = 97


@pytest.mark.parametrize("kw,want", [
    (dict(n_new=20480), INVALID), (dict(n_new=24576), INVALID), (dict(n_new=20484), INVALID),
    (dict(n_new=20472), INVALID), (dict(n_new=20492), SHAPE), (dict(n_new=20468), SHAPE),
    (dict(n_new=8192), SHAPE),                               # the state is only read
    (dict(idx=20400, idx_stride=8), INVALID), (dict(idx=24584, idx_stride=8), INVALID),
    (dict(idx=20384, idx_stride=8), SHAPE), (dict(idx=20492, idx_stride=8), SHAPE),
    (dict(begin_out=4128), INVALID), (dict(fill_out=4088), INVALID), (dict(begin_out=4132), SHAPE),
    # in place: the same array, read last by who writes it, but no part of it
    (dict(n_new=12288, begin_out=8192, fill_out=12288), SHAPE),
    (dict(n_new=8192, begin_out=8192, fill_out=12288), SHAPE),
    (dict(n_new=12292, begin_out=8192, fill_out=12288), INVALID),
    (dict(idx=8188, idx_stride=8, begin_out=8192, fill_out=12288), INVALID),
])
def test_append_refuses_outputs_over_its_inputs(kw, want):
    a = dict(begin_out=20480, fill_out=24576, keep=PAST)
    a.update(kw)
    assert append(**a) == want


@pytest.mark.parametrize("n,b,f,want", [
    (20480, 20480, 24576, SHAPE), (24576, 20480, 24576, SHAPE), (20484, 20480, 24576, INVALID),
    (24568, 20480, 24576, INVALID), (12288, 8192, 12288, SHAPE), (8188, 8192, 12288, INVALID),
    (None, 4096, 24576, INVALID), (None, 20480, 4130 + 2, SHAPE), (None, 20480, 24576, SHAPE),
])
def test_advance_refuses_outputs_over_its_inputs(n, b, f, want):
    assert txl.lib().txl_paged_advance(ctypes.byref(kv()), n, 4, PAST, b, f, None) == want
