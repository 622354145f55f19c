"""The paged memory's host side (CPU only, nothing launches): the refusals of its
entry points, and the page pool's accounting against a model of it."""

import ctypes
import random

import pytest
import torch

import transformer_xl_relative_pos_gb300 as txl
from transformer_xl_relative_pos_gb300 import _lib

OK, INVALID, UNSUPPORTED, MISALIGNED, SHAPE = 0, -1, -2, -3, -4


def kv(**kw):
    """A txl_paged_kv of made-up, aligned addresses that are never read."""
    a = dict(pool=1 << 20, table=4096, begin=8192, fill=12288, ticket=16384, layers=2, n_pages=10,
             H=2, page_rows=32, dh=64, B=3, slots=3, dtype=txl.BF16)
    a.update(kw)
    return _lib._PagedKV(*(a[f] for f, _ in _lib._PagedKV._fields_))


class Rows(ctypes.Structure):
    """txl_rows."""

    _fields_ = [("ptr", ctypes.c_void_p), ("stride_b", ctypes.c_longlong),
                ("stride_h", ctypes.c_longlong), ("stride_row", ctypes.c_longlong)]


def rows(ptr=1 << 16, sb=2048, sh=64, sr=128):
    return Rows(ptr, sb, sh, sr)


BAD_KV = [(dict(pool=None), INVALID), (dict(table=None), INVALID), (dict(begin=None), INVALID),
          (dict(fill=None), INVALID), (dict(layers=0), INVALID), (dict(n_pages=0), INVALID),
          (dict(H=0), INVALID), (dict(B=0), INVALID), (dict(slots=0), INVALID),
          (dict(page_rows=0), INVALID), (dict(dtype=5), INVALID), (dict(dh=128), UNSUPPORTED),
          (dict(page_rows=48), UNSUPPORTED), (dict(page_rows=16), UNSUPPORTED),
          (dict(B=65536), UNSUPPORTED), (dict(slots=1 << 26), UNSUPPORTED),
          (dict(n_pages=1 << 30, H=2), UNSUPPORTED), (dict(pool=(1 << 20) + 8), MISALIGNED),
          (dict(table=4098), MISALIGNED), (dict(fill=12290), MISALIGNED)]


def append(mem=None, layer0=0, n_layers=1, k=None, v=None, layer_stride=0, N=8, idx=None,
           idx_stride=0, n_new=None, max_rows=8, keep=0, begin_out=None, fill_out=None):
    ref = ctypes.byref
    return txl.lib().txl_paged_append(ref(mem or kv()), layer0, n_layers, ref(k or rows()),
                                      ref(v or rows()), layer_stride, N, idx, idx_stride, n_new,
                                      max_rows, keep, begin_out, fill_out, None)


@pytest.mark.parametrize("kw,want", BAD_KV)
def test_a_bad_memory_is_refused(kw, want):
    m, L = kv(**kw), txl.lib()
    assert append(mem=m) == want
    assert L.txl_paged_advance(ctypes.byref(m), None, 1, 4, 20480, 24576, None) == want
    assert L.txl_paged_copy(ctypes.byref(m), 4096, 8192, 1, None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(layer0=-1), INVALID), (dict(n_layers=0), INVALID), (dict(N=-1), INVALID),
    (dict(max_rows=-1), INVALID), (dict(layer0=1, n_layers=2, layer_stride=64), SHAPE),
    (dict(max_rows=9), SHAPE),                               # more rows than k has
    (dict(idx=4096, idx_stride=7), SHAPE), (dict(idx=4098, idx_stride=8), MISALIGNED),
    (dict(idx=4096, idx_stride=8, N=0), SHAPE),
    (dict(n_new=4097), MISALIGNED),
    (dict(k=rows(ptr=None)), INVALID), (dict(v=rows(ptr=None)), INVALID),
    (dict(k=rows(ptr=65544)), MISALIGNED), (dict(v=rows(sr=4)), MISALIGNED),
    (dict(k=rows(sb=0)), INVALID), (dict(k=rows(sh=-64)), INVALID),
    (dict(n_layers=2, layer_stride=0), INVALID), (dict(n_layers=2, layer_stride=12), MISALIGNED),
    (dict(begin_out=20480), INVALID), (dict(fill_out=20480), INVALID),
    (dict(begin_out=20480, fill_out=20484), INVALID),        # overlap each other
    (dict(begin_out=8196, fill_out=24576), INVALID),         # overlap the state in part
    (dict(begin_out=20480, fill_out=24576, keep=97), SHAPE), # more than the table holds
    (dict(begin_out=20480, fill_out=24576, keep=-1), INVALID),
    (dict(begin_out=20482, fill_out=24576), MISALIGNED),
    (dict(mem=kv(ticket=None), begin_out=8192, fill_out=12288), INVALID),
    (dict(max_rows=0), OK),                                  # nothing to do
])
def test_append_refusals(kw, want):
    assert append(**kw) == want


def test_advance_and_copy_refusals():
    L, m = txl.lib(), kv()
    adv = lambda n, keep, b, f, rows=4: L.txl_paged_advance(ctypes.byref(m), n, rows, keep, b, f, None)
    assert adv(None, 4, None, 24576) == INVALID and adv(None, 4, 20480, None) == INVALID
    assert adv(None, -1, 20480, 24576) == INVALID and adv(None, 97, 20480, 24576) == SHAPE
    assert adv(4097, 4, 20480, 24576) == MISALIGNED and adv(None, 4, 20480, 24576, -1) == INVALID
    assert adv(None, 4, 8200, 24576) == INVALID
    copy = lambda s, d, n: L.txl_paged_copy(ctypes.byref(m), s, d, n, None)
    assert copy(None, 4096, 1) == INVALID and copy(4096, None, 1) == INVALID
    assert copy(4096, 8192, -1) == INVALID and copy(4098, 8192, 1) == MISALIGNED
    assert copy(None, None, 0) == OK


def test_the_binding_refuses_host_tensors_and_bad_shapes():
    pool = torch.zeros(2, 4, 1, 32, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        txl.PagedKV(pool, torch.zeros(1, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="pool must be"):
        txl.PagedKV(pool[:1], torch.zeros(1, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="table must be"):
        txl.PagedKV(pool, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="begin must be"):
        txl.PagedKV(pool, torch.zeros(1, 2, dtype=torch.int32), begin=torch.zeros(2, dtype=torch.int32))


def test_page_pool_against_a_model():
    rng = random.Random(5)
    pool, n = txl.PagePool(37), 37
    users = [0] * n
    held = []
    for _ in range(3000):
        what = rng.random()
        if what < 0.4:
            want = rng.randint(0, 9)
            free = users.count(0)
            if want > free:
                with pytest.raises(txl.TxlError) as e:
                    pool.alloc(want)
                assert e.value.status == SHAPE
            else:
                got = pool.alloc(want)
                assert len(set(got)) == want and all(users[p] == 0 for p in got)
                for p in got:
                    users[p] = 1
                held.append(got)
        elif what < 0.6 and held:
            pages = rng.choice(held)
            pool.retain(pages)
            for p in pages:
                users[p] += 1
            held.append(list(pages))
        elif held:
            pages = held.pop(rng.randrange(len(held)))
            freed = pool.release(pages)
            for p in pages:
                users[p] -= 1
            assert freed == sum(users[p] == 0 for p in pages)
        assert pool.n_free == users.count(0)
        assert [pool.users(p) for p in range(n)] == users


def test_page_pool_refusals_change_nothing():
    pool = txl.PagePool(4)
    a = pool.alloc(2)
    for bad in ([a[0], 9], [a[0], -1], [a[0], 3]):           # 3 has no user
        for call in (pool.retain, pool.release):
            with pytest.raises(txl.TxlError) as e:
                call(bad)
            assert e.value.status == INVALID
    with pytest.raises(txl.TxlError):
        pool.release([a[0], a[0]])                           # one user, named twice
    assert [pool.users(p) for p in a] == [1, 1] and pool.n_free == 2
    pool.retain([a[0]])
    assert pool.release([a[0], a[0], a[1]]) == 2             # two users, named twice
    assert pool.n_free == 4 and sorted(pool.alloc(4)) == [0, 1, 2, 3]
    assert txl.PagePool(0).alloc(0) == []
    L = txl.lib()
    assert L.txl_page_pool_init(None, 1, None, None) == INVALID
    assert L.txl_page_pool_alloc(None, None, 0) == INVALID


def tree_call(mem=None, q=None, k=None, v=None, out=None, layer=0, r=1 << 16, r_rows=8, u=1 << 16,
              vb=1 << 16, parents=4096, stride=8, n=None, lse=None, N=8, scale=0.125, n_splits=0):
    ref = ctypes.byref
    return txl.lib().txl_relattn_tree_fwd(ref(q or rows()), ref(k or rows()), ref(v or rows()),
                                          ref(mem or kv()), layer, r, r_rows, u, vb, parents, stride, n,
                                          ref(out or rows()), lse, N, scale, n_splits, None)


@pytest.mark.parametrize("kw,want", BAD_KV)
def test_tree_refuses_a_bad_memory(kw, want):
    assert tree_call(mem=kv(**kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(r=None), INVALID), (dict(u=None), INVALID), (dict(vb=None), INVALID),
    (dict(parents=None), INVALID), (dict(N=0), INVALID), (dict(layer=-1), INVALID),
    (dict(n_splits=-1), INVALID), (dict(stride=-1), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(layer=2), SHAPE), (dict(r_rows=0), SHAPE), (dict(stride=7), SHAPE),
    (dict(N=65, stride=65), UNSUPPORTED), (dict(n_splits=9), UNSUPPORTED),
    (dict(r_rows=1 << 30), UNSUPPORTED),
    (dict(r=(1 << 16) + 8), MISALIGNED), (dict(u=(1 << 16) + 2), MISALIGNED),
    (dict(parents=4098), MISALIGNED), (dict(n=4098), MISALIGNED), (dict(lse=4098), MISALIGNED),
    (dict(q=rows(ptr=None)), INVALID), (dict(out=rows(ptr=None)), INVALID),
    (dict(k=rows(ptr=8)), MISALIGNED), (dict(v=rows(sr=4)), MISALIGNED), (dict(out=rows(sh=0)), INVALID),
])
def test_tree_refusals(kw, want):
    assert tree_call(**kw) == want


class FakeKV:
    """What PagedMemory uses of PagedKV, with tensors on the CPU."""

    def __init__(self, pool, table):
        self.pool, self.table = pool, table
        self.begin = torch.zeros(table.shape[0], dtype=torch.int32)
        self.fill = torch.zeros(table.shape[0], dtype=torch.int32)
        self.n_pages, self.H, self.page_rows = pool.shape[1:4]
        self.slots = table.shape[1]
        self.rows = self.slots * self.page_rows


def fake_copy(kv, src, dst):
    assert len(set(dst.tolist())) == len(dst) and not set(dst.tolist()) & set(src.tolist())
    kv.pool[:, dst.long()] = kv.pool[:, src.long()]


def fake_append(kv, k, v, *, layer=0, n_new=None, rows=None, keep=None):
    written = set()
    for b in range(kv.table.shape[0]):
        n = k.shape[-2] if n_new is None else int(n_new[b])
        begin, fill = int(kv.begin[b]), int(kv.fill[b])
        assert fill + n <= kv.rows
        for t in range(n):
            x = (begin + fill + t) % kv.rows
            page = int(kv.table[b, x // kv.page_rows])
            src = t if rows is None else int(rows[b, t])
            assert page >= 0
            written.add((b, page))
            kv.pool[0::2, page, :, x % kv.page_rows] = k[:, b, :, src]
            kv.pool[1::2, page, :, x % kv.page_rows] = v[:, b, :, src]
        left = min(fill + n, keep)
        kv.begin[b], kv.fill[b] = (begin + fill + n - left) % kv.rows, left
    pages = [p for _, p in written]
    assert len(pages) == len(set(pages)), "two sequences wrote one page"


@pytest.mark.parametrize("seed", range(12))
def test_paged_memory_against_lists_of_rows(monkeypatch, seed):
    import paged_ops
    from transformer_xl_relative_pos_gb300 import paged
    monkeypatch.setattr(paged.txl, "PagedKV", FakeKV)
    monkeypatch.setattr(paged.txl, "paged_copy", fake_copy)
    monkeypatch.setattr(paged.txl, "paged_append", fake_append)
    M, max_new, P = [(70, 40, 32), (0, 7, 32), (100, 9, 64), (33, 64, 96)][seed % 4]
    make = lambda: paged.PagedMemory(2, 4, 1, M, max_new, device="cpu", dtype=torch.float32,
                                     page_rows=P, dh=2)
    paged_ops.run(make, "cpu", seed)


def test_paged_memory_refusals_change_nothing(monkeypatch):
    from transformer_xl_relative_pos_gb300 import paged
    monkeypatch.setattr(paged.txl, "PagedKV", FakeKV)
    monkeypatch.setattr(paged.txl, "paged_copy", fake_copy)
    monkeypatch.setattr(paged.txl, "paged_append", fake_append)
    mem = paged.PagedMemory(1, 2, 1, 64, 40, device="cpu", dtype=torch.float32, page_rows=32, dh=2,
                            n_pages=3)
    k = torch.ones(2, 1, 40, 2)
    mem.append(k[None], k[None], [40, 10])                   # three pages of three
    table = mem._table.copy()
    with pytest.raises(txl.TxlError) as e:
        mem.append(k[None], k[None], [0, 30])
    assert e.value.status == SHAPE
    for bad in (lambda: mem.append(k[None], k[None], [1]), lambda: mem.append(k[None], k[None], [1, -1]),
                lambda: mem.append(k[None], k[None], rows=[[0], [40]]),
                lambda: mem.append(k[None], k[None], rows=[[0]]),
                lambda: mem.append(k[None], k[None], [2, 2], rows=[[0], [0, 1]]),
                lambda: mem.reserve(41), lambda: paged.PagedMemory(1, 1, 1, 4, 0, device="cpu")):
        with pytest.raises(ValueError):
            bad()
    assert (mem._table == table).all() and mem.fill == [40, 10] and mem.pages.n_free == 0
    mem.free(0)
    mem.append(k[None], k[None], [0, 30])
    assert mem.fill == [0, 40]


def test_paged_memory_refuses_sequences_layers_and_checkpoints_of_others(monkeypatch):
    from transformer_xl_relative_pos_gb300 import paged
    monkeypatch.setattr(paged.txl, "PagedKV", FakeKV)
    monkeypatch.setattr(paged.txl, "paged_copy", fake_copy)
    monkeypatch.setattr(paged.txl, "paged_append", fake_append)
    make = lambda layers=2, H=1, dtype=torch.float32: paged.PagedMemory(
        layers, 2, H, 64, 40, device="cpu", dtype=dtype, page_rows=32, dh=2)
    mem = make()
    k = torch.ones(2, 2, 1, 8, 2)
    mem.append(k, k)
    table, ck = mem._table.copy(), mem.checkpoint()
    for bad in (lambda: mem.free(-1), lambda: mem.free(2), lambda: mem.fork(0, -1), lambda: mem.fork(-2, 1),
                lambda: mem.fork(0, 2)):
        with pytest.raises(IndexError):
            bad()
    for bad in (lambda: mem.append(k[0], k[0]), lambda: mem.append(k[:1], k[:1])):
        with pytest.raises(ValueError):
            bad()
    for other in (make(layers=1), make(H=2), make(dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            other.restore(ck)
        assert other.fill == [0, 0] and other.pages.n_free == other.kv.n_pages
    assert (mem._table == table).all() and mem.fill == [8, 8]


def test_the_tensors_of_a_memory_are_not_replaced():
    for name in ("pool", "table", "begin", "fill", "ticket"):
        with pytest.raises(AttributeError):
            setattr(txl.PagedKV.__new__(txl.PagedKV), name, None)
